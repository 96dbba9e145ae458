"""moe_linear, moe_linear_gated and moe_residual_norm against 64-bit
references: types, scales, groups, one row to many, widths that end inside a
tile, strides, rows that hold NaN or zeros, streams and captured graphs, and
the three together as a layer runs them.
"""
import pytest
import torch

import layer_ref as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
GUARD = 77.0


def device_matrix(m):
    import mixture_experts_prefill_amd as mep

    return mep.MoeMatrix.from_codes(m.q.cuda(), m.s.cuda(), m.b.cuda(), m.group)


def rows(t, k, seed, kind):
    """(device rows, device scale, float64 values) of a kind: bf16, none, row, block."""
    g = torch.Generator().manual_seed(seed + 17 * t + k)
    v = torch.randn(t, k, generator=g) * (1 + 8 * (torch.rand(k, generator=g) < 0.02).float())
    if kind == "bf16":
        x = v.to(BF16)
        return x.cuda(), None, x.double()
    c, s, d = ref.e4m3_rows(v, kind)
    return c.cuda(), None if s is None else s.cuda(), d


KINDS = ["bf16", "none", "row", "block"]
# one row to several row blocks, widths inside and across tiles, one step of K and odd step counts
SHAPES = [(1, 32, 64), (1, 100, 4096), (2, 1, 128), (7, 33, 192), (8, 64, 576), (9, 95, 1088), (16, 32, 2048),
          (17, 257, 320), (31, 31, 64), (32, 96, 1024), (33, 65, 640), (64, 128, 512), (65, 40, 256), (128, 300, 448),
          (129, 513, 1024), (257, 64, 2112), (300, 1000, 704)]


@pytest.mark.parametrize("group", [64, 32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t,n,k", SHAPES)
def test_linear(t, n, k, kind, group):
    m = ref.Matrix(n, k, group)
    dm = device_matrix(m)
    x, s, d = rows(t, k, 1, kind)
    y, err = m.product(d)
    for dtype in (F32, BF16):
        # a guard column and guard rows around the output
        buf = torch.full((t + 2, n + 1), GUARD, dtype=dtype, device="cuda")
        out = buf[1:t + 1, :n]
        dm.linear(x, s, out=out)
        ref.check_rounded(out, y, err, dtype, (t, n, k, kind, group, dtype))
        assert bool((buf[0] == GUARD).all() and (buf[-1] == GUARD).all() and (buf[:, n] == GUARD).all())
        # accumulate adds in fp32 with one rounding more
        base = torch.randn(t, n, generator=torch.Generator().manual_seed(3)).to(dtype)
        out.copy_(base)
        dm.linear(x, s, out=out, accumulate=1)
        ref.check_rounded(out, y + base.double(), err + ref.U32 * (y.abs() + base.double().abs()), dtype, "accumulate")
        assert bool((buf[0] == GUARD).all() and (buf[-1] == GUARD).all() and (buf[:, n] == GUARD).all())


@pytest.mark.parametrize("group", [64, 32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t,n,k", [(1, 64, 256), (5, 32, 64), (12, 96, 1088), (30, 160, 512), (48, 64, 320),
                                   (130, 224, 640), (260, 32, 1024)])
def test_gated(t, n, k, kind, group):
    g, u = ref.Matrix(n, k, group, 1), ref.Matrix(n, k, group, 2)
    dg, du = device_matrix(g), device_matrix(u)
    x, s, d = rows(t, k, 2, kind)
    y, err = ref.gated(g.product(d), u.product(d))
    for dtype in (F32, BF16):
        buf = torch.full((t + 2, n + 3), GUARD, dtype=dtype, device="cuda")
        dg.gated(du, x, s, out=buf[1:t + 1, 1:n + 1])
        ref.check_rounded(buf[1:t + 1, 1:n + 1], y, err, dtype, (t, n, k, kind, group, dtype))
        assert bool((buf[0] == GUARD).all() and (buf[-1] == GUARD).all() and (buf[:, 0] == GUARD).all()
                    and (buf[:, n + 1:] == GUARD).all())
    codes, scale = dg.gated(du, x, s, out_dtype=E4M3)
    ref.check_codes(codes, scale, y, err, (t, n, k, kind, group))


def test_gated_width_inside_a_tile():
    n, k, t = 50, 128, 3
    g, u = ref.Matrix(n, k, 64, 1), ref.Matrix(n, k, 64, 2)
    x, _, d = rows(t, k, 2, "bf16")
    y, err = ref.gated(g.product(d), u.product(d))
    ref.check_rounded(device_matrix(g).gated(device_matrix(u), x), y, err, BF16, "n = 50")


def test_gated_saturates_smoothly():
    """Gate values far below zero (exp overflows) and far above it."""
    n, k = 32, 64
    g = ref.Matrix(n, k, 64, 3)
    g.s[:] = 0.0
    g.b[:] = torch.linspace(-8, 8, n)[:, None].half()
    u = ref.Matrix(n, k, 64, 4)
    x = torch.full((2, k), 4.0).to(BF16)
    y, err = ref.gated(g.product(x.double()), u.product(x.double()))
    out = device_matrix(g).gated(device_matrix(u), x.cuda(), out_dtype=F32)
    assert bool(torch.isfinite(out).all())
    ref.check_rounded(out, y, err + 1e-36, F32, "saturated gates")


@pytest.mark.parametrize("t", [3, 40, 150])
@pytest.mark.parametrize("kind", ["bf16", "row"])
def test_every_code_value_is_exact(kind, t):
    """Integer data: every sum is exact in fp32, so the result is too."""
    n, k = 64, 512
    m = ref.Matrix(n, k, 64)
    m.s[:] = 1.0
    m.b[:] = -8.0
    v = torch.randint(-8, 9, (t, k), generator=torch.Generator().manual_seed(t)).float()
    y = v.double() @ m.values().t()
    if kind == "bf16":
        out = device_matrix(m).linear(v.to(BF16).cuda(), out_dtype=F32)
    else:
        out = device_matrix(m).linear(v.to(E4M3).cuda(), torch.full((t,), 2.0).cuda(), out_dtype=F32)
        y = 2 * y
    assert torch.equal(out.cpu().double(), y)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t", [4, 70])
def test_strided_rows(t, kind):
    """x a column slice of a wider buffer, out a column slice too."""
    n, k = 70, 256
    m = ref.Matrix(n, k, 64)
    x, s, d = rows(t, k, 5, kind)
    wide = torch.zeros((t, k + 64), dtype=torch.uint8, device="cuda").view(E4M3) if kind != "bf16" else torch.zeros(
        (t, k + 64), dtype=BF16, device="cuda")
    wide[:, 32:32 + k].copy_(x)
    y, err = m.product(d)
    out = torch.full((t, 2 * n), GUARD, device="cuda")
    device_matrix(m).linear(wide[:, 32:32 + k], s, out=out[:, n:])
    ref.check_rounded(out[:, n:], y, err, F32, kind)
    assert bool((out[:, :n] == GUARD).all())


@pytest.mark.parametrize("t", [6, 100])
@pytest.mark.parametrize("kind", ["bf16", "row", "block"])
def test_bad_rows_stay_alone(kind, t):
    """A row with a NaN (or an infinity) gives non-finite outputs; the others keep theirs."""
    n, k = 64, 256
    m = ref.Matrix(n, k, 64)
    dm = device_matrix(m)
    x, s, d = rows(t, k, 6, kind)
    want = dm.linear(x, s, out_dtype=F32)
    bad = x.clone()
    if kind == "bf16":
        bad[2, 5], bad[4, 70] = float("nan"), float("inf")
    else:
        bad.view(torch.uint8)[2, 5] = 0x7F
        bad.view(torch.uint8)[4, 70] = 0xFF
    got = dm.linear(bad, s, out_dtype=F32)
    good = [r for r in range(t) if r not in (2, 4)]
    assert torch.equal(got[good], want[good])
    assert not bool(torch.isfinite(got[[2, 4]]).any())


def test_block_scales_span_the_range():
    """Blocks of very different magnitude in one row."""
    n, k, t = 40, 512, 5
    m = ref.Matrix(n, k, 64)
    v = torch.randn(t, k, generator=torch.Generator().manual_seed(8))
    v *= torch.exp2(torch.linspace(-60, 30, k // 32)).repeat_interleave(32)
    v[3, :64] = 0
    c, s, d = ref.e4m3_rows(v, "block")
    y, err = m.product(d)
    ref.check_rounded(device_matrix(m).linear(c.cuda(), s.cuda(), out_dtype=F32), y, err, F32, "blocks")
    assert torch.equal(device_matrix(m).linear(c.cuda(), s.cuda().view(torch.float8_e8m0fnu), out_dtype=F32),
                       device_matrix(m).linear(c.cuda(), s.cuda(), out_dtype=F32))


@pytest.mark.parametrize("group", [64, 32])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("t,n", [(3, 70), (7, 70), (40, 70), (100, 51200)])
def test_smallest_block_scales(t, n, dtype, group):
    """Scale bytes from 0 (2^-127) on.  A row value below 2^-126 may count as 0,
    and so may a sum: at most k + k / group + 16 sums of each output."""
    k = 192
    m = ref.Matrix(n, k, group, seed=3)
    g = torch.Generator().manual_seed(77)
    c = torch.randint(0, 256, (t, k), generator=g, dtype=torch.uint8)
    c[(c & 0x7f) == 0x7f] = 0x3a                                      # no NaN
    c = c.view(torch.float8_e4m3fn)
    s = torch.randint(0, 13, (t, k // 32), generator=g, dtype=torch.uint8)
    s[0] = 0
    d = c.double() * torch.exp2(s.double() - 127).repeat_interleave(32, 1)
    y, err = m.product(d)
    reach = (15 * m.s.double() + m.b.double().abs()).repeat_interleave(group, 1).sum(1)
    err = err + 2.0 ** -126 * (reach + k + k // group + 16)[None, :]
    if n == 51200 and dtype == BF16:
        err = err + ref.e4m3_product_error(m, d)
    ref.check_rounded(device_matrix(m).linear(c.cuda(), s.cuda(), out_dtype=dtype), y, err, dtype, "small scales")


@pytest.mark.parametrize("centred", [True, False])
def test_linear_large(centred):
    """A full chunk, checked on rows at both ends and in between (row sums against a 64-bit product)."""
    t, n, k = 4096, 1000, 1024
    m = ref.Matrix(n, k, 64, 9, centred)
    dm = device_matrix(m)
    pick = [0, 1, 31, 32, 127, 128, 255, 1023, 2048, 3001, 4000, 4094, 4095]
    for kind in ("bf16", "block", "row"):
        x, s, d = rows(t, k, 9, kind)
        out = dm.linear(x, s, out_dtype=F32)
        y, err = m.product(d[pick])
        ref.check_rounded(out[pick], y, err, F32, kind)
        # the same rows alone, in a call of few rows, within both calls' bounds
        sp = None if s is None else s[pick].contiguous()
        alone = dm.linear(x.view(torch.uint8 if kind != "bf16" else BF16)[pick].view(x.dtype), sp, out_dtype=F32)
        assert bool(((alone - out[pick]).double().cpu().abs() <= 2 * err).all())


# at least 200 tiles of 128 rows x 256 outputs (128 when gated), the long chunks' kernel: row counts and widths
# that end inside a tile, one step of K, part of a 16-group chunk, whole chunks and more
@pytest.mark.parametrize("group", [64, 32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t,n,k", [(65, 51200, 64), (100, 51300, 320), (700, 9000, 576), (1300, 4600, 1024),
                                   (4096, 1700, 1088), (4000, 1800, 2112)])
def test_long_chunk(t, n, k, kind, group):
    m = ref.Matrix(n, k, group, 11)
    dm = device_matrix(m)
    x, s, d = rows(t, k, 11, kind)
    g = torch.Generator().manual_seed(t)
    pick = sorted({0, 1, 31, 32, 63, t - 1, t - 2, t - 33} | set(torch.randint(0, t, (20,), generator=g).tolist()))
    y, err = m.product(d[pick])
    for dtype in (F32, BF16):
        e = err + ref.e4m3_product_error(m, d[pick]) if kind != "bf16" and dtype == BF16 else err
        buf = torch.full((t + 2, n + 3), GUARD, dtype=dtype, device="cuda")
        dm.linear(x, s, out=buf[1:t + 1, :n])
        out = buf[1:t + 1, :n]
        ref.check_rounded(out[pick], y, e, dtype, (t, n, k, kind, group, dtype))
        assert bool((buf[0] == GUARD).all() and (buf[-1] == GUARD).all() and (buf[:, n:] == GUARD).all())
        if dtype == BF16:
            # rounding to bf16: at most half a step each, evenly spread in it; the e4m3 matrix core adds 2^-12 at most
            d2 = out[pick].double().cpu() - y
            assert float(d2.norm() / y.norm()) <= 2.0 ** -8 / 3 ** 0.5 + 2.0 ** -12
        # no row is left out or doubled: the sum over rows is that of the products
        want = torch.stack([d.sum(0)]) @ m.values().t()
        total = out.double().sum(0).cpu()
        bound = t * (e.max() + ref.HALF[dtype] * y.abs().max() * 2)
        assert bool(((total - want[0]).abs() <= bound).all())
    base = torch.randn(t, n, generator=g).to(BF16)
    out = base.cuda()
    dm.linear(x, s, out=out, accumulate=1)
    b = base[pick].double()
    e = err + (ref.e4m3_product_error(m, d[pick]) if kind != "bf16" else 0)
    ref.check_rounded(out[pick], y + b, e + ref.U32 * (y.abs() + b.abs()), BF16, "accumulate")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("width,first", [(25670, 0), (25672, 0), (25672, 1), (25671, 0), (25680, 2)])
def test_long_chunk_output_places(width, first, kind, dtype):
    """Outputs that start at any element, rows any distance apart, whole blocks of 128 rows and part of one."""
    t, n, k = 300, 25670, 128
    m = ref.Matrix(n, k, 64, 5)
    x, s, d = rows(t, k, 9, kind)
    y, err = m.product(d)
    if kind != "bf16" and dtype == BF16:
        err = err + ref.e4m3_product_error(m, d)
    buf = torch.full((t, width), GUARD, dtype=dtype, device="cuda")
    device_matrix(m).linear(x, s, out=buf[:, first:first + n])
    ref.check_rounded(buf[:, first:first + n], y, err, dtype, (width, first, kind, dtype))
    assert bool((buf[:, :first] == GUARD).all() and (buf[:, first + n:] == GUARD).all())


@pytest.mark.parametrize("group", [64, 32])
@pytest.mark.parametrize("kind", ["bf16", "row", "block"])
@pytest.mark.parametrize("t,n,k", [(70, 25600, 128), (1000, 3300, 704), (4096, 896, 1088)])
def test_long_chunk_gated(t, n, k, kind, group):
    g, u = ref.Matrix(n - n % 32, k, group, 1), ref.Matrix(n - n % 32, k, group, 2)
    n = g.n
    dg, du = device_matrix(g), device_matrix(u)
    x, s, d = rows(t, k, 12, kind)
    gen = torch.Generator().manual_seed(t)
    pick = sorted({0, 31, 32, t - 1} | set(torch.randint(0, t, (12,), generator=gen).tolist()))
    (yg, eg), (yu, eu) = g.product(d[pick]), u.product(d[pick])
    y, err = ref.gated((yg, eg), (yu, eu))
    ref.check_rounded(dg.gated(du, x, s, out_dtype=F32)[pick], y, err, F32, (t, n, k, kind, group))
    if kind != "bf16":
        y, err = ref.gated((yg, eg + ref.e4m3_product_error(g, d[pick])), (yu, eu + ref.e4m3_product_error(u, d[pick])))
    ref.check_rounded(dg.gated(du, x, s)[pick], y, err, BF16, (t, n, k, kind, group))
    codes, scale = dg.gated(du, x, s, out_dtype=E4M3)
    ref.check_codes(codes.view(torch.uint8)[pick].view(E4M3), scale[pick], y, err, (t, n, k, kind, group))


def test_long_chunk_bad_rows_and_bits():
    """NaN and infinite rows stay alone; the same call gives the same bits, on another stream too."""
    t, n, k = 4096, 1800, 512
    m = ref.Matrix(n, k, 64)
    dm = device_matrix(m)
    for kind in ("bf16", "block"):
        x, s, _ = rows(t, k, 13, kind)
        for dtype in (F32, BF16):
            want = dm.linear(x, s, out_dtype=dtype)
            bits = torch.int32 if dtype == F32 else torch.int16
            side = torch.cuda.Stream()
            torch.cuda.synchronize()
            again = torch.empty_like(want)
            dm.linear(x, s, out=again, stream=side)
            side.synchronize()
            assert torch.equal(again.view(bits), want.view(bits))
            bad = x.clone()
            if kind == "bf16":
                bad[77, 5], bad[4095, 70] = float("nan"), float("inf")
            else:
                bad.view(torch.uint8)[77, 5] = 0x7F
                bad.view(torch.uint8)[4095, 70] = 0xFF
            got = dm.linear(bad, s, out_dtype=dtype)
            good = torch.ones(t, dtype=torch.bool)
            good[[77, 4095]] = False
            assert torch.equal(got[good.cuda()].view(bits), want[good.cuda()].view(bits))
            assert not bool(torch.isfinite(got[[77, 4095]]).any())


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("t", [3, 40, 300])
def test_gated_8_bit_places_and_bad_rows(t, kind):
    """8-bit outputs that start at any byte have the bits of aligned ones; a bad
    row is NaN codes with the smallest scale, and stays alone."""
    n, k = (12864 if t == 300 else 96), 128
    g, u = device_matrix(ref.Matrix(n, k, 64, 1)), device_matrix(ref.Matrix(n, k, 64, 2))
    x, s, _ = rows(t, k, 21, kind)
    want, scale = g.gated(u, x, s, out_dtype=E4M3)
    for width, first in ((n, 0), (n + 4, 4), (n + 4, 1), (n + 3, 0)):
        buf = torch.full((t, width), 0x55, dtype=torch.uint8, device="cuda").view(E4M3)
        got, gscale = g.gated(u, x, s, out=buf[:, first:first + n])
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)) and torch.equal(gscale, scale)
        rest = torch.cat([buf.view(torch.uint8)[:, :first], buf.view(torch.uint8)[:, first + n:]], 1)
        assert bool((rest == 0x55).all())
    bad = x.clone()
    for r in (1, t - 1):
        if kind == "bf16":
            bad[r] = float("nan")
        else:
            bad.view(torch.uint8)[r] = 0x7F
    got, gscale = g.gated(u, bad, s, out_dtype=E4M3)
    keep = torch.ones(t, dtype=torch.bool, device="cuda")
    keep[[1, t - 1]] = False
    assert torch.equal(got.view(torch.uint8)[keep], want.view(torch.uint8)[keep]) and torch.equal(gscale[keep], scale[keep])
    assert bool(((got.view(torch.uint8)[~keep] & 0x7F) == 0x7F).all()) and bool((gscale[~keep] == 0).all())


def test_same_call_same_bits():
    for t in (1, 20, 200):
        m = ref.Matrix(300, 1024, 64)
        dm = device_matrix(m)
        x, s, _ = rows(t, 1024, 4, "block")
        first = dm.linear(x, s)
        for _ in range(5):
            assert torch.equal(dm.linear(x, s).view(torch.int16), first.view(torch.int16))


# ------------------------------------------------------------------ residual norm

def norm_inputs(t, h, xt, rt, seed=0):
    g = torch.Generator().manual_seed(seed + 3 * t + h)
    x = torch.randn(t, h, generator=g).to(xt)
    r = None if rt is None else (2 * torch.randn(t, h, generator=g)).to(rt)
    gamma = 1 + 0.1 * torch.randn(h, generator=g)
    return x, r, gamma


@pytest.mark.parametrize("scale", ["row", "block"])
@pytest.mark.parametrize("xt,rt", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32), (BF16, None), (F32, None)])
@pytest.mark.parametrize("t,h", [(1, 32), (1, 4096), (3, 96), (5, 512), (6, 544), (9, 1024), (2, 1056), (4, 2048),
                                 (3, 2080), (257, 64), (2, 8192), (1, 8224), (2, 16384)])
def test_residual_norm(t, h, xt, rt, scale):
    import mixture_experts_prefill_amd as mep

    x, r, gamma = norm_inputs(t, h, xt, rt)
    s, y, err = ref.norm(x, r, gamma, 1e-6)
    dx, dr, dg = x.cuda(), None if r is None else r.cuda(), gamma.cuda()
    rout = None if r is None else torch.empty_like(dr)
    out = torch.full((t + 1, h), GUARD, dtype=BF16, device="cuda")
    codes = torch.full((t + 1, h), 0x11, dtype=torch.uint8, device="cuda").view(E4M3)
    sc = torch.full((t,), -1.0, device="cuda") if scale == "row" else torch.full((t, h // 32), 255, dtype=torch.uint8,
                                                                                 device="cuda")
    mep.moe_residual_norm(dx, dg, 1e-6, dr, rout, out[:t], codes[:t], sc)
    if r is not None:
        assert torch.equal(rout.cpu(), s)
    ref.check_rounded(out[:t], y, err, BF16, (t, h, xt, rt))
    ref.check_codes(codes[:t], sc, y, err, (t, h, xt, rt, scale))
    assert bool((out[t] == GUARD).all() and (codes.view(torch.uint8)[t] == 0x11).all())
    # each output alone, and the stream updated in place
    out2, codes2, sc2 = torch.empty_like(out), torch.empty_like(codes), torch.empty_like(sc)
    if r is not None:
        mep.moe_residual_norm(dx, dg, 1e-6, dr, dr, out=out2[:t])
        assert torch.equal(dr, rout)
    else:
        mep.moe_residual_norm(dx, dg, 1e-6, out=out2[:t])
    assert torch.equal(out2[:t].view(torch.int16), out[:t].view(torch.int16))
    r0 = None if r is None else r.cuda()
    mep.moe_residual_norm(dx, dg, 1e-6, r0, None, codes=codes2[:t], scale=sc2)
    assert torch.equal(codes2[:t].view(torch.uint8), codes[:t].view(torch.uint8)) and torch.equal(sc2, sc)


def test_residual_norm_odd_rows():
    """Rows of zeros, of tiny and huge values, with NaN and infinities."""
    import mixture_experts_prefill_amd as mep

    t, h = 7, 1536
    x, r, gamma = norm_inputs(t, h, F32, F32, 5)
    x[0], r[0] = 0, 0
    x[1], r[1] = x[1] * 1e-30, r[1] * 1e-30
    x[2], r[2] = x[2] * 1e15, r[2] * 1e15
    x[3, 7] = float("nan")
    x[4, 9] = float("inf")
    x[5, 64:96], r[5, 64:96] = 0, 0
    gamma[100] = float("inf")
    finite_rows = [0, 1, 2, 5, 6]
    for scale in ("row", "block"):
        sc = torch.empty(t, device="cuda") if scale == "row" else torch.empty((t, h // 32), dtype=torch.uint8, device="cuda")
        codes = torch.empty((t, h), dtype=torch.uint8, device="cuda").view(E4M3)
        out = torch.empty((t, h), dtype=BF16, device="cuda")
        mep.moe_residual_norm(x.cuda(), gamma.cuda(), 1e-6, r.cuda(), None, out, codes, sc)
        _, y, err = ref.norm(x, r, gamma, 1e-6)
        assert bool(torch.isnan(codes.float()[3]).all())
        assert bool(torch.isnan(codes.float()[4, 9]))
        for row in finite_rows:
            keep = torch.isfinite(y[row])
            assert bool(torch.isnan(codes.float()[row].cpu()[~keep]).all())
            yy, ee = y[row:row + 1].clone(), err[row:row + 1].clone()
            yy[:, ~keep], ee[:, ~keep] = 0, 0
            c = codes[row:row + 1].float().cpu()
            c[:, ~keep] = 0
            ref.check_codes(c, sc[row:row + 1], yy, ee + 1e-44, (row, scale))
            o = out[row:row + 1].double().cpu()
            o[:, ~keep] = 0
            ref.check_rounded(o, yy, ee, BF16, row)
        assert bool((codes.float()[0, :64] == 0).all())


def test_residual_norm_strided():
    """x and the residual as column slices, the codes into a wider buffer."""
    import mixture_experts_prefill_amd as mep

    t, h = 33, 256
    x, r, gamma = norm_inputs(t, h, BF16, BF16, 6)
    wide = torch.zeros((t, 3 * h), dtype=BF16, device="cuda")
    wide[:, h:2 * h], wide[:, 2 * h:] = x.cuda(), r.cuda()
    codes = torch.zeros((t, 2 * h), dtype=torch.uint8, device="cuda").view(E4M3)
    sc = torch.empty((t, h // 32), dtype=torch.uint8, device="cuda")
    # out is the buffer's first third: equal strides, no shared byte
    mep.moe_residual_norm(wide[:, h:2 * h], gamma.cuda(), 1e-5, wide[:, 2 * h:], wide[:, 2 * h:], wide[:, :h],
                          codes[:, h:], sc)
    s, y, err = ref.norm(x, r, gamma, 1e-5)
    assert torch.equal(wide[:, 2 * h:].cpu(), s)
    assert torch.equal(wide[:, h:2 * h].cpu(), x)
    ref.check_rounded(wide[:, :h], y, err, BF16, "strided")
    ref.check_codes(codes[:, h:], sc, y, err, "strided")
    assert bool((codes.view(torch.uint8)[:, :h] == 0).all())


# ------------------------------------------------------------------ as a layer runs them

class Layer:
    """Residual norm -> gated pair -> down projection -> residual norm, 8-bit rows in between."""

    def __init__(self, t, h, inter, scale):
        import mixture_experts_prefill_amd as mep

        self.mep, self.t, self.h, self.inter = mep, t, h, inter
        self.hm = [ref.Matrix(inter, h, 64, 1), ref.Matrix(inter, h, 64, 2), ref.Matrix(h, inter, 64, 3)]
        self.gate, self.up, self.down = (device_matrix(m) for m in self.hm)
        g = torch.Generator().manual_seed(t + h)
        self.gamma = 1 + 0.1 * torch.randn(h, generator=g)
        self.dgamma = self.gamma.cuda()
        self.x = torch.randn(t, h, generator=g).to(BF16)
        self.res = torch.randn(t, h, generator=g)
        self.dx, self.dres = self.x.cuda(), self.res.cuda()
        self.s1 = torch.empty_like(self.dres)
        self.s2 = torch.empty_like(self.dres)
        self.codes = torch.empty((t, h), dtype=torch.uint8, device="cuda").view(E4M3)
        self.scale = torch.empty(t, device="cuda") if scale == "row" else torch.empty((t, h // 32), dtype=torch.uint8,
                                                                                      device="cuda")
        self.hg = torch.empty((t, inter), dtype=torch.uint8, device="cuda").view(E4M3)
        self.hg_scale = torch.empty((t, inter // 32), dtype=torch.uint8, device="cuda")
        self.y = torch.empty((t, h), device="cuda")
        self.out = torch.empty((t, h), dtype=BF16, device="cuda")

    def run(self, stream=None):
        m = self.mep
        m.moe_residual_norm(self.dx, self.dgamma, 1e-6, self.dres, self.s1, None, self.codes, self.scale, stream)
        self.gate.gated(self.up, self.codes, self.scale, self.hg, self.hg_scale, stream=stream)
        self.down.linear(self.hg, self.hg_scale, self.y, stream=stream)
        m.moe_residual_norm(self.y, self.dgamma, 1e-6, self.s1, self.s2, self.out, stream=stream)

    def results(self):
        torch.cuda.synchronize()
        return [v.clone() for v in (self.s1, self.codes.view(torch.uint8), self.scale, self.hg.view(torch.uint8),
                                    self.hg_scale, self.y, self.s2, self.out.view(torch.int16))]

    def clear(self):
        for v in (self.s1, self.s2, self.y, self.scale, self.hg_scale):
            v.fill_(1)
        self.codes.view(torch.uint8).fill_(1)
        self.hg.view(torch.uint8).fill_(1)
        self.out.fill_(1)

    def check(self):
        """Every step against 64 bits, each on the step before's own outputs."""
        s, y, err = ref.norm(self.x, self.res, self.gamma, 1e-6)
        assert torch.equal(self.s1.cpu(), s)
        ref.check_codes(self.codes, self.scale, y, err, "norm")
        c = self.codes.cpu().double() * ref.scale_values(self.scale).repeat_interleave(
            self.h // ref.scale_values(self.scale).shape[1], 1)
        y, err = ref.gated(self.hm[0].product(c), self.hm[1].product(c))
        ref.check_codes(self.hg, self.hg_scale, y, err, "gated")
        c = self.hg.cpu().double() * ref.scale_values(self.hg_scale).repeat_interleave(32, 1)
        y, err = self.hm[2].product(c)
        ref.check_rounded(self.y, y, err, F32, "down")
        s, y, err = ref.norm(self.y.cpu(), self.s1.cpu(), self.gamma, 1e-6)
        assert torch.equal(self.s2.cpu(), s)
        ref.check_rounded(self.out, y, err, BF16, "next norm")


@pytest.mark.parametrize("scale", ["row", "block"])
@pytest.mark.parametrize("t,h,inter", [(1, 1024, 384), (13, 512, 768), (200, 768, 512), (600, 512, 640)])
def test_layer(t, h, inter, scale):
    layer = Layer(t, h, inter, scale)
    layer.run()
    torch.cuda.synchronize()
    layer.check()


def test_layer_on_another_stream():
    layer = Layer(40, 512, 384, "block")
    layer.run()
    want = layer.results()
    layer.clear()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    layer.run(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(layer.results(), want))
    layer.clear()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        layer.run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(layer.results(), want))


def test_two_layers_on_two_streams():
    """No shared state between calls that overlap."""
    a, b = Layer(300, 512, 640, "row"), Layer(3, 1024, 512, "block")
    a.run()
    wa = a.results()
    b.run()
    wb = b.results()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for v in (a, b):
        v.clear()
    torch.cuda.synchronize()
    for _ in range(10):
        a.run(sa)
        b.run(sb)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.results(), wa))
    assert all(torch.equal(x, y) for x, y in zip(b.results(), wb))


@pytest.mark.parametrize("t", [1, 50, 300])
def test_layer_graph_replays_match_eager(t):
    layer = Layer(t, 512, 384, "block")
    x0, x1 = layer.dx.clone(), layer.dx * 0.5
    want = []
    for x in (x0, x1):
        layer.dx.copy_(x)
        layer.run()
        want.append(layer.results())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.run()
    torch.cuda.synchronize()
    for rep in range(4):
        layer.dx.copy_((x0, x1)[rep % 2])
        layer.clear()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(layer.results(), want[rep % 2])), rep
        layer.dx.copy_((x1, x0)[rep % 2])
        layer.run()
        torch.cuda.synchronize()
    del g


def test_layer_beside_the_block():
    """The 8-bit rows of the residual norm and the block on its bf16 rows, from one call, as a layer with
    both a dense and a routed part reads them."""
    import mixture_experts_prefill_amd as mep
    import moe_synth as ms
    import numpy as np
    import oracle

    wl = ms.make_workload("tiny", centred=True)
    blk = mep.MoeBlock.from_workload(wl)
    t, h = wl.x.shape
    x, r, gamma = norm_inputs(t, h, BF16, F32, 9)
    codes = torch.empty((t, h), dtype=torch.uint8, device="cuda").view(E4M3)
    sc = torch.empty((t, h // 32), dtype=torch.uint8, device="cuda")
    mep.moe_residual_norm(x.cuda(), gamma.cuda(), 1e-6, r.cuda(), None, blk.x, codes, sc)
    blk.forward()
    m = ref.Matrix(h, h, 64)
    dense = device_matrix(m).linear(codes, sc, out=blk.out.clone(), accumulate=1)
    torch.cuda.synchronize()
    wl.x = blk.x.view(torch.int16).cpu().numpy().view(np.uint16)
    routed = oracle.block(wl)["out"]
    d = blk.out.cpu().numpy().astype(np.float64) - routed
    assert np.linalg.norm(d) <= 5e-3 * np.linalg.norm(routed)   # the block's own tolerance
    y, err = m.product(codes.cpu().double() * ref.scale_values(sc).repeat_interleave(32, 1))
    base = blk.out.cpu().double()
    ref.check_rounded(dense, y + base, err + ref.U32 * (y.abs() + base.abs()), F32, "dense part")
