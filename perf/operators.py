"""Cases for timing and checking the layer operators around the routed experts:

* ``norm``   a block output added to the residual stream, RMS-normalised and written as 8-bit rows
             (e4m3 codes with one fp32 scale a row, or one power-of-two scale per 32 columns);
* ``linear`` rows times a matrix of 4-bit codes with fp16 scale and bias per group of inputs, the rows
             bf16 or 8-bit;
* ``gated``  silu(x Wg^T) * (x Wu^T) on two such matrices, written as bf16 or as 8-bit rows for the
             down projection.

With ``own`` false ``run`` computes them from elementary torch operations in 32 bits; with ``own`` true it
calls this package's entry points.  Matrices are held in both forms: codes, scales and biases row by row
for the plain form, and the tiled record of ``include/moe.h`` (32 x 64 code tiles, scale/bias pairs in
tile order), which is laid out once when weights are loaded.
"""
import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decode step through a layer's norm, 8-bit rows for the next projection
        dict(name="norm t1 h4096 block", op="norm", t=1, h=4096, x="bf16", res="bf16", scale="block", rows=False),
        # a ragged batch in fp32 (the residual copies' type), the bf16 rows wanted beside the codes
        dict(name="norm t333 h2080 row", op="norm", t=333, h=2080, x="f32", res="f32", scale="row", rows=True),
        # a full prefill chunk at a wide hidden size
        dict(name="norm t4096 h8192 row", op="norm", t=4096, h=8192, x="bf16", res="bf16", scale="row", rows=False),
        # an attention output projection at one token
        dict(name="linear t1 4096x4096", op="linear", t=1, n=4096, k=4096, group=64, x="bf16", scale="none", out="bf16"),
        # a vocabulary head at one token, an odd number of outputs, fp32 logits
        dict(name="linear t1 100003x2048", op="linear", t=1, n=100003, k=2048, group=64, x="bf16", scale="none", out="f32"),
        # eight sequences decoded together on 8-bit rows
        dict(name="linear t8 6144x4096 q8", op="linear", t=8, n=6144, k=4096, group=64, x="e4m3", scale="block", out="bf16"),
        # a short ragged batch, small groups, a width that ends inside a tile
        dict(name="linear t77 1000x1536 g32", op="linear", t=77, n=1000, k=1536, group=32, x="bf16", scale="none", out="f32"),
        # a mid chunk on bf16 rows, long sums
        dict(name="linear t512 2048x8192", op="linear", t=512, n=2048, k=8192, group=64, x="bf16", scale="none", out="bf16"),
        # a full prefill chunk on 8-bit rows with one scale a row
        dict(name="linear t4096 4096x4096 q8", op="linear", t=4096, n=4096, k=4096, group=64, x="e4m3", scale="row",
             out="bf16"),
        # a dense feed-forward block at one token, 8-bit in and out
        dict(name="gated t1 1536x4096 q8", op="gated", t=1, n=1536, k=4096, group=64, x="e4m3", scale="block", out="e4m3"),
        # a prompt of odd length through a narrow gated block, 8-bit in, bf16 out
        dict(name="gated t201 1504x2048 q8", op="gated", t=201, n=1504, k=2048, group=64, x="e4m3", scale="row", out="bf16"),
        # a full prefill chunk through a wide gated block on bf16 rows
        dict(name="gated t4096 8192x4096", op="gated", t=4096, n=8192, k=4096, group=64, x="bf16", scale="none", out="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "gated"])
    t = _log(rng, 1, 4096)
    if op == "norm":
        return dict(op=op, t=t, h=32 * _log(rng, 4, 256), x=rng.choice(["bf16", "f32"]), res=rng.choice(["bf16", "f32"]),
                    scale=rng.choice(["row", "block"]), rows=rng.random() < 0.5)
    k = 64 * _log(rng, 4, 128)
    x, scale = rng.choice([("bf16", "none"), ("e4m3", "row"), ("e4m3", "block")])
    group = rng.choice([32, 64, 64])
    if op == "linear":
        n = _log(rng, 100, 100000)
        n = max(100, min(n, 4096 * 8192 * 4096 // (t * k)))
        return dict(op=op, t=t, n=n, k=k, group=group, x=x, scale=scale, out=rng.choice(["bf16", "f32"]))
    n = 32 * _log(rng, 4, 256)
    n = max(128, min(n, 4096 * 8192 * 4096 // (t * k) // 32 * 32))
    return dict(op=op, t=t, n=n, k=k, group=group, x=x, scale=scale, out=rng.choice(["bf16", "e4m3"]))


# ------------------------------------------------------------------ inputs

def _e4m3(v):
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _row_scale(v):
    """One fp32 scale a row: the largest magnitude over the largest code."""
    return (v.abs().amax(-1) / E4M3_MAX).clamp_min(2.0 ** -126)


def _block_exponent(v):
    """Per 32 columns the smallest E with the block's largest magnitude <= 448 * 2^E."""
    m, e = torch.frexp(v.abs().unflatten(-1, (-1, 32)).amax(-1))
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(m == 0, torch.full_like(e, -127), e).clamp(-127, 127)


def _quant(v, scale):
    """Rows v (fp32) as (codes, scales)."""
    if scale == "row":
        s = _row_scale(v)
        return _e4m3(v / s[:, None]), s
    e = _block_exponent(v)
    q = torch.ldexp(v.unflatten(-1, (-1, 32)), -e[..., None]).flatten(-2)
    return _e4m3(q), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _values(codes, s):
    """The fp32 values of 8-bit rows."""
    v = codes.float()
    if s.dtype == torch.float32:
        return v * s[:, None]
    return torch.ldexp(v.unflatten(-1, (-1, 32)), (s.view(torch.uint8).int() - 127)[..., None]).flatten(-2)


def _matrix(n, k, group, gen):
    """Codes uniform in 0..15, scale ~ U(0.005, 0.02), bias about -7.5 scales, so weights are roughly
    zero-mean; and the same matrix as the tiled record."""
    q = torch.randint(0, 16, (n, k), generator=gen, device="cuda", dtype=torch.uint8)
    s = (torch.rand((n, k // group), generator=gen, device="cuda") * 0.015 + 0.005).half()
    b = (torch.randn((n, k // group), generator=gen, device="cuda") * 0.01 - 7.5 * s.float()).half()
    pad = -n % 32
    qp = torch.nn.functional.pad(q, (0, 0, 0, pad)) if pad else q
    rows = n + pad
    v = qp.view(rows // 32, 32, k // 64, 2, 4, 8)
    word = v[..., 0].int()
    for j in range(1, 8):
        word |= v[..., j].int() << (4 * (j // 2) + 16 * (j % 2))
    codes = word.permute(0, 2, 3, 1, 4).contiguous().view(torch.uint8).view(-1)
    sb = torch.stack([s, b], -1)
    sb = torch.nn.functional.pad(sb, (0, 0, 0, 0, 0, pad)) if pad else sb
    sb = sb.view(rows // 32, 32, k // 64, 64 // group, 2).permute(0, 2, 3, 1, 4).contiguous().view(torch.uint8).view(-1)
    at = -(-codes.numel() // 256) * 256
    record = torch.zeros(-(-(at + sb.numel()) // 256) * 256, dtype=torch.uint8, device="cuda")
    record[: codes.numel()] = codes
    record[at: at + sb.numel()] = sb
    return dict(q=q, s=s, b=b, record=record)


def _rows(c, gen):
    """Rows of roughly unit variance with a few strong channels, as layers see them."""
    width = c["h"] if c["op"] == "norm" else c["k"]
    strong = 1 + 8 * (torch.rand(width, generator=gen, device="cuda") < 0.01).float()
    return torch.randn((c["t"], width), generator=gen, device="cuda") * strong


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(c=c)
    v = _rows(c, gen)
    t = c["t"]
    if c["op"] == "norm":
        h = c["h"]
        st["x"] = v.to(TYPES[c["x"]])
        st["residual"] = (2 * torch.randn((t, h), generator=gen, device="cuda")).to(TYPES[c["res"]])
        st["gamma"] = 1 + 0.1 * torch.randn(h, generator=gen, device="cuda")
        # the buffers that a program keeps for the call's outputs
        st["residual_out"] = torch.empty_like(st["residual"])
        st["rows"] = torch.empty((t, h), dtype=torch.bfloat16, device="cuda") if c["rows"] else None
        st["codes"] = torch.empty((t, h), dtype=torch.float8_e4m3fn, device="cuda")
        st["scale"] = (torch.empty(t, device="cuda") if c["scale"] == "row"
                       else torch.empty((t, h // 32), dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu))
    else:
        n, k = c["n"], c["k"]
        if c["x"] == "bf16":
            st["x"], st["x_scale"] = v.to(torch.bfloat16), None
        else:
            st["x"], st["x_scale"] = _quant(v, c["scale"])
        st["m"] = [_matrix(n, k, c["group"], gen) for _ in range(2 if c["op"] == "gated" else 1)]
        st["out_scale"] = None
        if c["out"] == "e4m3":
            st["out"] = torch.empty((t, n), dtype=torch.float8_e4m3fn, device="cuda")
            st["out_scale"] = torch.empty((t, n // 32), dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
        else:
            st["out"] = torch.empty((t, n), dtype=TYPES[c["out"]], device="cuda")
    if own:
        import mixture_experts_prefill_amd as mep

        st["mep"] = mep
        if c["op"] != "norm":
            st["layout"] = mep.moe_matrix_layout_make(c["n"], c["k"], c["group"])
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    c, mep = st["c"], st["mep"]
    if c["op"] == "norm":
        mep.moe_residual_norm(st["x"], st["gamma"], EPS, residual=st["residual"], residual_out=st["residual_out"],
                              out=st["rows"], codes=st["codes"], scale=st["scale"])
        return dict(residual=st["residual_out"], rows=st["rows"], codes=st["codes"], scale=st["scale"])
    if c["op"] == "linear":
        mep.moe_linear(st["x"], st["layout"], st["m"][0]["record"], st["out"], x_scale=st["x_scale"])
    else:
        mep.moe_linear_gated(st["x"], st["layout"], st["m"][0]["record"], st["m"][1]["record"], st["out"],
                             x_scale=st["x_scale"], out_scale=st["out_scale"])
    return dict(out=st["out"], scale=st["out_scale"])


def _weights(m, group):
    q = m["q"].float().unflatten(-1, (-1, group))
    return (q * m["s"].float()[..., None] + m["b"].float()[..., None]).flatten(-2)


def _run_plain(st):
    c = st["c"]
    if c["op"] == "norm":
        res = (st["x"].float() + st["residual"].float()).to(st["residual"].dtype)
        z = res.float()
        y = z * (1 / torch.sqrt(z.square().mean(-1, keepdim=True) + EPS)) * st["gamma"]
        codes, scale = _quant(y, c["scale"])
        return dict(residual=res, rows=y.to(torch.bfloat16) if c["rows"] else None, codes=codes, scale=scale)
    x = st["x"].float() if st["x_scale"] is None else _values(st["x"], st["x_scale"])
    y = torch.matmul(x, _weights(st["m"][0], c["group"]).t())
    if c["op"] == "linear":
        return dict(out=y.to(st["out"].dtype), scale=None)
    y = y / (1 + torch.exp(-y)) * torch.matmul(x, _weights(st["m"][1], c["group"]).t())
    if c["out"] == "e4m3":
        codes, scale = _quant(y, "block")
        return dict(out=codes, scale=scale)
    return dict(out=y.to(st["out"].dtype), scale=None)


# ------------------------------------------------------------------ what a pass cannot do without

def _size(name):
    return {"bf16": 2, "f32": 4, "e4m3": 1}[name]


def _scale_bytes(kind, t, width):
    return {"none": 0, "row": 4 * t, "block": t * (width // 32)}[kind]


def work(case):
    c = case
    t = c["t"]
    if c["op"] == "norm":
        h = c["h"]
        values = _size(c["x"]) + 2 * _size(c["res"]) + 1 + (2 if c["rows"] else 0)
        return {"bytes": t * h * values + 4 * h + _scale_bytes(c["scale"], t, h), "flops": 8 * t * h}
    n, k = c["n"], c["k"]
    mats = 2 if c["op"] == "gated" else 1
    nbytes = mats * (n * k // 2 + 4 * n * (k // c["group"])) + t * k * _size(c["x"]) + _scale_bytes(c["scale"], t, k)
    nbytes += t * n * _size(c["out"]) + (t * n // 32 if c["out"] == "e4m3" else 0)
    return {"bytes": nbytes, "flops": 2 * mats * t * n * k}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_e4m3(v):
    """v rounded to the nearest e4m3 value, ties to even: steps of 2^-3 of the leading power of two,
    2^-9 below 2^-6, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_quant(y, kind):
    t, width = y.shape
    if kind == "row":
        s = y.abs().max(dim=1).values.div(E4M3_MAX)
        s[s < 2.0 ** -126] = 2.0 ** -126
        return _exact_e4m3(y / s.view(t, 1)), s
    blocks = y.view(t, width // 32, 32)
    s = torch.exp2(torch.ceil(torch.log2(blocks.abs().max(dim=2).values / E4M3_MAX)).clamp(-127, 127))
    return _exact_e4m3(blocks / s.view(t, width // 32, 1)).view(t, width), s


def _exact_rows(st):
    x = st["x"].double()
    if st["x_scale"] is None:
        return x
    s = st["x_scale"].double() if st["x_scale"].dtype == torch.float32 else torch.exp2(
        st["x_scale"].view(torch.uint8).double() - 127)
    return x * s.view(x.shape[0], -1).repeat_interleave(x.shape[1] // max(1, s.numel() // x.shape[0]), dim=1)


def _exact_product(x, m, group):
    w = m["s"].double().repeat_interleave(group, dim=1) * m["q"].double()
    w += m["b"].double().repeat_interleave(group, dim=1)
    return x @ w.t()


def exact(case, seed):
    st = prepare(case, seed)
    c = st["c"]
    if c["op"] == "norm":
        z = st["x"].double() + st["residual"].double()
        stored = z.to(st["residual"].dtype).double()  # the stream as it is stored is what is normalised
        y = stored / torch.sqrt((stored * stored).sum(1, keepdim=True) / c["h"] + EPS) * st["gamma"].double()
        codes, scale = _exact_quant(y, c["scale"])
        return dict(residual=z, rows=y if c["rows"] else None, codes=codes, scale=scale)
    x = _exact_rows(st)
    y = _exact_product(x, st["m"][0], c["group"])
    if c["op"] == "linear":
        return dict(out=y, scale=None)
    y = y * torch.sigmoid(y) * _exact_product(x, st["m"][1], c["group"])
    if c["out"] == "e4m3":
        codes, scale = _exact_quant(y, "block")
        return dict(out=codes, scale=scale)
    return dict(out=y, scale=None)
