"""What the layer operators' sums keep: every row of a long chunk against 64
bits, to the bounds of fp32 sums, and inputs made so that sums held in fewer
bits show.
"""
import pytest
import torch

import layer_ref as ref
from test_gpu_layer_ops import BF16, E4M3, F32, device_matrix, norm_inputs, rows

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("group", [64, 32])
@pytest.mark.parametrize("kind", ["none", "row", "block"])
@pytest.mark.parametrize("t,n,k", [(128, 51200, 128), (700, 9000, 320), (3000, 2304, 192)])
def test_a_strong_channel_leaves_the_others_sums(t, n, k, kind, group):
    """One channel of every group is up to 448 and its weight is exactly 0 (code 8, scale s, bias -8 s), the
    others are below 0.11: what is left is the others' sum, in products 2^12 and more below the largest one.
    A sum held to 16 bits of its largest product is off by about 64 * 2^-16 * 448 * 8 s; the bound here is
    that of fp32 sums, with the one rounding to bf16."""
    m = ref.Matrix(n, k, group, 21)
    m.b = (-8 * m.s.float()).half()                          # exact in fp16
    g = torch.Generator().manual_seed(t)
    strong = torch.arange(0, k, group) + 5
    m.q[:, strong] = 8
    v = torch.randn(t, k, generator=g).clamp(-3, 3) * 0.035
    v[:, strong] = 448.0 * (0.5 + torch.rand(t, strong.numel(), generator=g) / 2)
    c, s, d = ref.e4m3_rows(v, kind)
    cols = torch.randint(0, n, (64,), generator=g)
    part = ref.Matrix.__new__(ref.Matrix)                    # the same matrix, 64 of its rows
    part.n, part.k, part.group, part.q, part.s, part.b = 64, k, group, m.q[cols], m.s[cols], m.b[cols]
    y, err = part.product(d)
    dm = device_matrix(m)
    dc, ds = c.cuda(), None if s is None else s.cuda()
    for dtype in (F32, BF16):
        got = dm.linear(dc, ds, out_dtype=dtype)[:, cols.cuda()]
        ref.check_rounded(got, y, err, dtype, (t, n, k, kind, group, dtype))


@pytest.mark.parametrize("t,n", [(3, 64), (16, 64), (40, 64), (150, 25600)])
def test_silu_keeps_fp32(t, n):
    """Exact gates -100 .. 100 (one product each) and exact up values: what is off is the activation's alone.
    exp within one step (two half steps), then a product, a sum, a quotient and the product with up, half a step
    each: six half steps; where exp leaves fp32's normal range, half a step of 2^-149 times the gate."""
    k = 64
    a = torch.linspace(-6.66, 6.66, t).to(BF16)
    x = torch.zeros(t, k, dtype=BF16)
    x[:, 0], x[:, 1] = a, 2.0 ** 20
    mats = []
    for first, second in ((torch.arange(n) % 16, 0), (0, torch.arange(n) % 13 + 1)):
        m = ref.Matrix(n, k, 64)
        m.q[:], m.s[:], m.b[:] = 0, 1.0, 0.0
        m.q[:, 0], m.q[:, 1] = first, second
        mats.append(m)
    g, u = (x.double() @ m.values().t() for m in mats)
    y = g / (1 + torch.exp(-g)) * u
    tol = 6 * ref.U32 * y.abs() + (g.abs() + 1) * u.abs() * 2.0 ** -149 + 2.0 ** -149
    out = device_matrix(mats[0]).gated(device_matrix(mats[1]), x.cuda(), out_dtype=F32).double().cpu()
    bad = ~((out - y).abs() <= tol)
    worst = (out - y).abs() / (ref.U32 * y.abs()).clamp_min(2.0 ** -149)
    assert not bad.any(), (t, n, int(bad.sum()), float(worst.max()), float(g.flatten()[worst.argmax()]))


# every row and column of long chunks (at least 200 tiles of 128 rows x 256 outputs, 128 when gated), to the bounds
# of fp32 sums; rows and columns that end inside a tile, parts of a 16-group chunk and more than one
LONG = [(65, 51200, 64), (700, 9000, 576), (1300, 4600, 320), (4096, 1700, 192)]


@pytest.mark.parametrize("group", [64, 32])
@pytest.mark.parametrize("kind", ["bf16", "none", "row", "block"])
@pytest.mark.parametrize("t,n,k", LONG)
def test_long_chunk_every_output(t, n, k, kind, group):
    m = ref.Matrix(n, k, group, 31)
    dm = device_matrix(m)
    x, s, d = rows(t, k, 31, kind)
    y, err = m.product(d)
    for dtype in (F32, BF16):
        ref.check_rounded(dm.linear(x, s, out_dtype=dtype), y, err, dtype, (t, n, k, kind, group, dtype))


def check_unbiased(got, y, what):
    """The part of got along y is y's own.  Each code is off by at most half a step, 2^-4 |y|, either way as
    often: its part along y has at most the standard deviation 2^-4 / sqrt 3 * sqrt(sum y^4) / sum y^2, six of
    which are allowed, and 2^-8 for the values' density not being level inside a step (a step of at most |y| / 8
    shifts a mean by its square / 24 times the density's relative slope, at most 6 / |y|)."""
    part = float((got * y).sum() / (y * y).sum()) - 1
    bound = 6 * 2.0 ** -4 / 3 ** 0.5 * float((y ** 4).sum().sqrt() / (y * y).sum()) + 2.0 ** -8
    assert bound < 0.012, bound                       # else the test has too few values to show anything
    assert abs(part) <= bound, (what, part, bound)


@pytest.mark.parametrize("group", [64, 32])
@pytest.mark.parametrize("kind", ["bf16", "row", "block"])
@pytest.mark.parametrize("t,n,k", [(70, 25600, 64), (700, 4512, 704), (4096, 896, 320)])
def test_long_chunk_gated_every_output(t, n, k, kind, group):
    g, u = ref.Matrix(n, k, group, 1), ref.Matrix(n, k, group, 2)
    dg, du = device_matrix(g), device_matrix(u)
    x, s, d = rows(t, k, 32, kind)
    y, err = ref.gated(g.product(d), u.product(d))
    what = (t, n, k, kind, group)
    for dtype in (F32, BF16):
        ref.check_rounded(dg.gated(du, x, s, out_dtype=dtype), y, err, dtype, (what, dtype))
    codes, scale = dg.gated(du, x, s, out_dtype=E4M3)
    ref.check_codes(codes, scale, y, err, what)
    check_unbiased(codes.cpu().double() * ref.scale_values(scale).repeat_interleave(32, 1), y, what)


def test_unbiased_check_sees_two_percent():
    """The check above on its own: exact codes pass, codes of values 2% larger do not."""
    y, _ = ref.gated(*[(torch.randn(512, 512, generator=torch.Generator().manual_seed(i)).double() * 3, 0) for i in (1, 2)])
    for factor, good in ((1.0, True), (1.02, False), (0.98, False)):
        c, s, values = ref.e4m3_rows((y * factor).float(), "block")
        if good:
            check_unbiased(values, y, factor)
        else:
            with pytest.raises(AssertionError):
                check_unbiased(values, y, factor)


# ------------------------------------------------------------------ the ends of the ranges

def wide_matrix(n, k, group, seed):
    """A matrix too large for the CPU: (MoeMatrix, its rows j as a ref.Matrix)."""
    import mixture_experts_prefill_amd as mep

    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0, 16, (n, k), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand((n, k // group), generator=g, device="cuda") * 0.015 + 0.005).half()
    b = (torch.randn((n, k // group), generator=g, device="cuda") * 0.01 - 7.5 * s.float()).half()

    def part(j):
        m = ref.Matrix.__new__(ref.Matrix)
        m.n, m.k, m.group = len(j), k, group
        m.q, m.s, m.b = (v[j].cpu() for v in (q, s, b))
        return m

    return mep.MoeMatrix.from_codes(q, s, b, group), part


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("group", [64, 32])
@pytest.mark.parametrize("t,n", [(1, 100), (4, 100), (16, 100), (20, 100), (300, 17000)])
def test_longest_rows(t, n, group, kind):
    """k = 65536, through every kernel."""
    k = 65536
    dm, part = wide_matrix(n, k, group, 5)
    x, s, d = rows(t, k, 33, kind)
    j = [0, 1, 31, 32, n // 2, n - 2, n - 1]
    y, err = part(j).product(d)
    for dtype in (F32, BF16):
        ref.check_rounded(dm.linear(x, s, out_dtype=dtype)[:, j], y, err, dtype, (t, n, group, kind, dtype))


@pytest.mark.parametrize("t", [1, 20, 65])
def test_most_outputs(t):
    """n = 2^24, through every kernel."""
    n, k = 1 << 24, 64
    dm, part = wide_matrix(n, k, 64, 6)
    x, s, d = rows(t, k, 34, "block")
    j = [0, 31, 32, 255, 256, 12345, n // 2 - 1, n // 2, n // 2 + 1, n - 257, n - 256, n - 33, n - 32, n - 1]
    y, err = part(j).product(d)
    out = torch.full((t, n), float("nan"), device="cuda")
    dm.linear(x, s, out=out)
    ref.check_rounded(out[:, j], y, err, F32, t)
    assert not bool(torch.isnan(out).any())


@pytest.mark.parametrize("kind", ["bf16", "row"])
@pytest.mark.parametrize("t,n", [(16, 70), (60, 70), (1100, 6000)])
def test_widest_row_strides(t, n, kind):
    """Input rows 2^22 elements apart and output rows 2^25: places past 2^32 bytes and elements."""
    k = 128
    m = ref.Matrix(n, k, 64, 7)
    x, s, d = rows(t, k, 35, kind)
    wide = torch.empty((t, 1 << 22), dtype=x.dtype, device="cuda")
    wide[:, 64:64 + k].copy_(x)
    y, err = m.product(d)
    step = 1 << 25 if t <= 60 else 1 << 22
    for dtype in (F32, BF16):
        out = torch.empty((t, step), dtype=dtype, device="cuda")[:, 5:5 + n]
        device_matrix(m).linear(wide[:, 64:64 + k], s, out=out)
        ref.check_rounded(out, y, err, dtype, (t, n, kind, dtype))


def test_residual_norm_widest_row_strides():
    import mixture_experts_prefill_amd as mep

    t, h = 1100, 96
    x, r, gamma = norm_inputs(t, h, BF16, F32, 8)
    s, y, err = ref.norm(x, r, gamma, 1e-6)
    wx, wr, wo, wc = (torch.empty((t, 1 << 22), dtype=v, device="cuda")[:, 32:32 + h] for v in (BF16, F32, BF16, E4M3))
    wx.copy_(x)
    wr.copy_(r)
    sc = torch.empty((t, h // 32), dtype=torch.uint8, device="cuda")
    mep.moe_residual_norm(wx, gamma.cuda(), 1e-6, wr, wr, wo, wc, sc)
    assert torch.equal(wr.cpu(), s)
    ref.check_rounded(wo, y, err, BF16, "strides")
    ref.check_codes(wc, sc, y, err, "strides")
