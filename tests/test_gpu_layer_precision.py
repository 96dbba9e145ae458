"""What the layer operators' sums keep: every row of a long chunk against 64
bits, to the bounds of fp32 sums, and inputs made so that sums held in fewer
bits show.
"""
import pytest
import torch

import layer_ref as ref
from test_gpu_layer_ops import BF16, F32, device_matrix

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
