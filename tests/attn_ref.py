"""64-bit references of the paged key-value cache and the attention over it,
and error bounds for their fp32 kernels.  CPU, numpy and torch float64; shares
no code with the package: every element of a cache is found by its own index.
"""
import numpy as np
import torch

U32 = 2.0 ** -24                       # half a step of fp32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


class Cache:
    """The bytes of a cache, on the CPU, with the sections' places from the header's description."""

    def __init__(self, pages, page, heads, head, dtype, fill=None):
        self.pages, self.page, self.heads, self.head, self.dtype = pages, page, heads, head, dtype
        self.size = 2 if dtype == BF16 else 1
        self.cell = 16 // self.size
        up = lambda v: -(-v // 256) * 256
        self.values = up(pages * page * heads * head * self.size)
        self.scales = 0 if dtype == BF16 else up(pages * page * heads)
        self.bytes = torch.zeros(2 * self.values + 2 * self.scales, dtype=torch.uint8)
        if fill is not None:
            self.bytes.fill_(fill)

    def section(self, which):
        """The section's values as a flat view: k, v, ks, vs."""
        at, n = {"k": (0, self.values), "v": (self.values, self.values), "ks": (2 * self.values, self.scales),
                 "vs": (2 * self.values + self.scales, self.scales)}[which]
        b = self.bytes[at:at + n]
        return b if which in ("ks", "vs") else b.view(self.dtype)

    def index(self, which, slots):
        """Flat indices [len(slots), heads, head] (scales: [len(slots), heads]) of the tokens at these slots."""
        s = torch.as_tensor(slots, dtype=torch.int64)
        page, tok = (s // self.page)[:, None], (s % self.page)[:, None]
        block = (page * self.heads + torch.arange(self.heads)) * self.page
        if which in ("ks", "vs"):
            return block + tok
        d = torch.arange(self.head)
        block, tok = (block * self.head)[..., None], tok[..., None]
        if which == "k":
            return block + tok // 16 * 16 * self.head + d // self.cell * 16 * self.cell + tok % 16 * self.cell + d % self.cell
        return block + tok // self.cell * self.cell * self.head + d * self.cell + tok % self.cell

    def read(self, which, slots):
        """float64 values [len(slots), heads, head]."""
        flat = self.section(which)
        i = self.index(which, slots)
        v = (flat if self.size == 2 else flat.view(torch.uint8))[i].view(self.dtype).double()
        if self.size == 1:
            v = v * torch.exp2(self.section(which + "s")[self.index(which + "s", slots)].double() - 127)[..., None]
        return v

    def write(self, which, slots, x, scale=None):
        """Values of the cache's type [len(slots), heads, head], and their scale bytes."""
        flat = self.section(which)
        if self.size == 2:
            flat[self.index(which, slots)] = x
        else:
            flat.view(torch.uint8)[self.index(which, slots)] = x.view(torch.uint8)
            self.section(which + "s")[self.index(which + "s", slots)] = scale


def quantise(x):
    """float64 [.., head] -> (e4m3 codes of float32 values, scale bytes) with the smallest 2^E, max|x| <= 448 * 2^E;
    what is not finite becomes NaN and does not count."""
    fin = torch.isfinite(x)
    m = torch.where(fin, x.abs(), 0.0).amax(-1)
    mant, e = np.frexp((m / 448.0).numpy())
    e = np.where(m.numpy() == 0, -127, np.clip(np.where(mant == 0.5, e - 1, e), -127, 127))
    e = torch.from_numpy(e.astype(np.int64))
    c = (x * torch.exp2(-e.double())[..., None]).clamp(-448, 448)
    c = torch.where(fin, c, torch.nan).float().to(E4M3)
    return c, (e + 127).to(torch.uint8)


def rotate(x, angles):
    """x float64 [t, heads, head], angles float32 [t, rot] (cosines, sines)."""
    half = angles.shape[1] // 2
    c, s = angles[:, None, :half].double(), angles[:, None, half:].double()
    a, b = x[..., :half], x[..., half:2 * half]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., 2 * half:]], -1)


def attention(q, k, v, positions, scale, weight_half):
    """One sequence: q [rows, heads_q, head], k and v [tokens, heads, head] (float64), row i reads tokens 0 ..
    positions[i].  Returns the output [rows, heads_q, head], a bound on the kernel's error before its last rounding,
    and the square of what rounding the weights may add, summed as independent errors.

    Bound.  A score is a sum of `head` exact products in fp32, off by at most head * 2^-23 of the sum of their
    magnitudes, and the weight's exponent adds the roundings of scale * log2 e, of the product and of the largest
    score's (each half a step of at most the largest |score|) and two of exp2's result: delta in all, relative to the
    weight.  The weights' and the outputs' sums over n tokens are fp32: at most n + 64 steps (parts and their joining
    included) of half a step of their magnitude, twice that in the matrix core.  Weights are rounded by factors
    1 + e_j, |e_j| <= weight_half, before they are summed and meet v, which moves the output w.v to
    sum w_j (1 + e_j) v_j / sum w_j (1 + e_j) = w.v + sum w_j e_j (v_j - w.v) / (1 + sum w_j e_j): by at most
    weight_half (sum w_j |v_j| + |w.v|) (1 + 2 weight_half)."""
    rows, hq, d = q.shape
    n, hk, _ = k.shape
    g = hq // hk
    out = torch.zeros(rows, hq, d, dtype=torch.float64)
    err, var = torch.zeros_like(out), torch.zeros_like(out)
    if n == 0:
        return out, err, var
    pos = torch.as_tensor(positions)
    seen = torch.arange(n)[None, :] <= pos[:, None]
    for h in range(hq):
        kh, vh = k[:, h // g], v[:, h // g]
        s = (q[:, h] @ kh.t()) * scale
        mag = (q[:, h].abs() @ kh.abs().t()) * scale
        s = torch.where(seen, s, -torch.inf)
        top = s.amax(1, keepdim=True)
        p = torch.where(seen, torch.exp(s - torch.where(torch.isfinite(top), top, 0.0)), 0.0)
        l = p.sum(1, keepdim=True)
        w = torch.where(l > 0, p / l.clamp_min(1e-300), 0.0)
        out[:, h] = w @ vh
        big = torch.where(seen, mag, 0.0).amax(1, keepdim=True)
        delta = (2 * d + 8) * U32 * big + 8 * U32 + 2 * (n + 64) * U32
        vw = w @ vh.abs()
        o = out[:, h]
        err[:, h] = 2 * delta * vw * 1.01 + weight_half * (1 + 2 * weight_half) * (vw + o.abs())
        w2 = w ** 2
        var[:, h] = (weight_half ** 2) * (w2 @ vh ** 2 - 2 * o * (w2 @ vh) + o ** 2 * w2.sum(1, keepdim=True)).clamp_min(0)
    return out, err, var


def check_attention(got, ref, err, var, what):
    """got bf16 [rows, heads_q * head] against the reference: each value within its bound and half a step of bf16;
    and all of them together: roundings are independent and within +-half a step, so the sum of their squares is
    expected below a third of that of the half steps."""
    g = got.double().cpu().reshape(ref.shape)
    assert torch.isfinite(g).all(), f"{what}: not finite"
    e = (g - ref).abs()
    tol = err + HALF[BF16] * (ref.abs() + err) + 2.0 ** -134
    bad = e > tol
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((e / tol).max()):.3g} of the bound"
    if g.numel() >= 512:
        rms = float((e ** 2).sum()), float(((HALF[BF16] * ref) ** 2 + var).sum())
        assert rms[0] <= rms[1] + 1e-30, f"{what}: squared error {rms[0]:.3g} above {rms[1]:.3g}"


def plan(length, grow, page, pages, table, free, free_n, t):
    """moe_kv_plan row by row.  Lists in (table and free are changed), a dict out."""
    width = len(table[0])
    limit = width * page
    length = [min(max(x, 0), limit) for x in length]
    top = min(max(free_n, 0), pages)
    for s, g in enumerate(grow):
        if g < 0:
            for i in range(-(-length[s] // page)):
                if top < pages:
                    free[top] = table[s][i]
                    top += 1
    lacking, out_len, starts, positions, slots = 0, [], [0], [], []
    for s, g in enumerate(grow):
        old = 0 if g < 0 else length[s]
        held = old
        for i in range(max(g, 0)):
            if len(slots) == t:
                lacking += g - i
                break
            at = old + i
            positions.append(at)
            new = at >= -(-old // page) * page
            ok = at == held and at < limit
            if ok and new and at % page == 0:
                ok = top > 0
                if ok:
                    top -= 1
                    table[s][at // page] = free[top]
            if not ok:
                slots.append(-1)
                lacking += 1
                continue
            held += 1
            p = table[s][at // page]
            slots.append(p * page + at % page if 0 <= p < pages else -1)
            lacking += not 0 <= p < pages
        out_len.append(held)
        starts.append(len(slots))
    pad = t - len(slots)
    lacking = min(lacking, 2 ** 31 - 1)
    return dict(length_out=out_len, free_n_out=[top], starts=starts, positions=positions + [0] * pad,
                slots=slots + [-1] * pad, lacking=[lacking])
