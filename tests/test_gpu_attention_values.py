"""moe_attention_decode and moe_attention_prefill on values at the ends of
their types: infinities and NaN in values, at any weight; finite values whose
weighted sum passes fp32 before it is divided; scores beyond fp32.

A value that is not finite reaches every row that reads its token, as it is:
two infinities of unequal signs, or a NaN, make a NaN.  All other columns keep
the bounds of `attn_ref`.
"""
import pytest
import torch

import attn_ref as ref
import test_gpu_attention as base
from test_gpu_attention import mep  # noqa: F401  (the fixture)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
MOST = torch.finfo(BF16).max


def set_value(b, s, token, column, v, head=0):
    """One bf16 value of the batch's cache."""
    b.cache.section("v")[b.cache.index("v", [b.slots[s][token]])[0, head, column]] = v


def check(b, s, out, q, positions, scale, weight_half, what):
    """Rows of one sequence: columns that read a value that is not finite are the sum of those, exactly."""
    rows, hq = len(positions), out.shape[1] // b.head
    k, v = b.values(s)
    fin = torch.where(torch.isfinite(v), v, 0.0)
    want, err, var = ref.attention(q.double().view(rows, hq, b.head), k, fin, positions, scale, weight_half)
    wild = torch.where(torch.isfinite(v), 0.0, v).cumsum(0)
    wild = torch.cat([wild.new_zeros(1, b.heads, b.head), wild])[torch.tensor(positions, dtype=torch.int64).clamp_min(-1) + 1]
    wild = wild.repeat_interleave(hq // b.heads, 1)
    got = out.double().cpu().view(rows, hq, b.head)
    at = ~torch.isfinite(wild)
    assert torch.equal(torch.isnan(got[at]), torch.isnan(wild[at])), f"{what}: NaN"
    assert torch.equal(torch.nan_to_num(got[at]), torch.nan_to_num(wild[at])), f"{what}: infinities"
    ref.check_attention(torch.where(at, want, got), want, err, var, what)


def run(mep, b, rows, hq, scale, single, what, q=None):
    """Through moe_attention_decode (one row a sequence) or moe_attention_prefill; every row checked."""
    n = len(b.lengths)
    rows = [1] * n if single else rows
    starts = [sum(rows[:s]) for s in range(n + 1)]
    t = starts[-1]
    q = b.queries(t, hq) if q is None else q
    cache, table, length = b.on_gpu()
    out = torch.full((t, hq * b.head), base.GUARD, dtype=BF16, device="cuda")
    ws = base.workspace(mep, t, n, hq, b.layout)
    if single:
        mep.moe_attention_decode(q.cuda(), b.layout, cache, table, length, scale, out, ws)
    else:
        mep.moe_attention_prefill(q.cuda(), base.ints(starts).cuda(), b.layout, cache, table, length, scale, out, ws)
    torch.cuda.synchronize()
    for s in range(n):
        r0, r1 = starts[s], starts[s + 1]
        positions = [b.lengths[s] - rows[s] + i for i in range(rows[s])]
        check(b, s, out[r0:r1], q[r0:r1], positions, scale, 2.0 ** -16 if single else 2.0 ** -8, f"{what} sequence {s}")
    return out


# ------------------------------------------------------------------ infinities and NaN

def with_infinities(mep, lengths, heads, head, seed=0):
    b = base.Batch(mep, lengths, heads, head, 16, BF16, seed=seed)
    for s, n in enumerate(lengths):
        if n == 0:
            continue
        for h in range(heads):
            set_value(b, s, 0, 3, torch.inf, h)
            set_value(b, s, n - 1, 5 + h, -torch.inf, h)
            set_value(b, s, n // 2, 11, torch.inf, h)
            set_value(b, s, n // 3, 40, torch.nan, h)
            set_value(b, s, 0, 33, torch.inf, h)
            set_value(b, s, n - 1, 33, -torch.inf, h)            # of one token: -inf; else NaN for its reader
            set_value(b, s, n - 1, head - 1, torch.inf, h)
            if n > 2:
                set_value(b, s, n - 2, head - 1, torch.inf, h)
    return b


@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("head", [64, 128, 256])
@pytest.mark.parametrize("heads,g", [(1, 1), (2, 4), (1, 17)])
def test_infinite_values(mep, heads, g, head, single):
    lengths = [1, 2, 17, 0, 33, 64, 65, 300, 1]
    b = with_infinities(mep, lengths, heads, head, seed=g)
    run(mep, b, [1, 2, 5, 0, 33, 3, 65, 70, 0], heads * g, head ** -0.5, single, (heads, g, head, single))


@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("lengths,rows", [([5000], [3]), ([20000, 1, 3000], [1, 1, 200]), ([1700, 900], [700, 40])])
def test_infinite_values_of_sequences_that_are_cut(mep, lengths, rows, single):
    for heads, hq, head in ((1, 1, 64), (2, 16, 128), (1, 2, 256)):
        b = with_infinities(mep, lengths, heads, head)
        run(mep, b, rows, hq, head ** -0.5, single, (lengths, heads, head, single))


@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("n", [65, 700, 5000])
@pytest.mark.parametrize("where", ["first", "last", "middle"])
def test_infinite_values_of_no_weight(mep, where, n, single):
    """A weight that fp32 rounds to 0, at once or when the maximum rises after it, is not 0: 2^-800 of the largest."""
    head, hq = 64, 2
    b = base.Batch(mep, [n], 1, head, 16, BF16)
    k = torch.zeros(n, 1, head)
    at = dict(first=0, last=n - 1, middle=n // 2)[where]
    k[:, 0, 0] = 1.0
    k[at, 0, 0] = -1.0
    b.cache.write("k", b.slots[0], k.to(BF16))
    set_value(b, 0, at, 9, torch.inf)
    set_value(b, 0, at, 50, -torch.inf)
    q = torch.zeros(40, hq * head, dtype=BF16)
    q[:, 0], q[:, head] = 280.0, 290.0
    t = 1 if single else 40
    run(mep, b, [40], hq, 1.0, single, (where, n, single), q=q[:t])


@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("head", [64, 128, 256])
def test_nan_codes(mep, head, single):
    b = base.Batch(mep, [1, 70, 3000], 2, head, 32, E4M3)
    for s, n in enumerate(b.lengths):
        b.cache.section("v").view(torch.uint8)[b.cache.index("v", [b.slots[s][n // 2]])[0, 1, 7]] = 0x7f
    run(mep, b, [1, 70, 20], 6, head ** -0.5, single, (head, single))


# ------------------------------------------------------------------ values that are large, and small ones beside them

def with_large_values(mep, lengths, heads, head, dtype):
    """Columns of the largest values of one sign, of mixed signs, and (bf16) of values of 2^-100 and 2^-120."""
    b = base.Batch(mep, lengths, heads, head, 32, dtype)
    for s, n in enumerate(lengths):
        if n == 0:
            continue
        sign = torch.randint(0, 2, (n, heads, head), generator=b.gen).double() * 2 - 1
        part = torch.rand(n, heads, head, generator=b.gen).double() * 0.5 + 0.5
        x = sign * part
        x[:, :, : head // 4] = 1.0
        x[:, :, head // 4: head // 2] = -part[:, :, head // 4: head // 2]
        if dtype == BF16:
            v = (x * MOST).to(BF16)
            v[:, :, head - 8:head - 4] = (torch.randn(n, heads, 4, generator=b.gen).double() * 2.0 ** -100).to(BF16)
            v[:, :, head - 4:] = (torch.randn(n, heads, 4, generator=b.gen).double() * 2.0 ** -120).to(BF16)
            b.cache.write("v", b.slots[s], v)
        else:
            b.cache.write("v", b.slots[s], (x * 240).to(E4M3), torch.full((n, heads), 247, dtype=torch.uint8))
    return b


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("head", [64, 128, 256])
def test_large_values(mep, head, single, dtype):
    b = with_large_values(mep, [1, 2, 33, 300, 0, 5000], 2, head, dtype)
    run(mep, b, [1, 2, 33, 150, 0, 40], 6, head ** -0.5, single, (head, single, dtype))


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_large_values_joined_by_tiles(mep, dtype):
    b = with_large_values(mep, [900, 1300], 1, 128, dtype)
    run(mep, b, [400, 260], 8, 128 ** -0.5, False, dtype)


# ------------------------------------------------------------------ scores

@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("scale", [2.0 ** 127, 2.0 ** 125])
@pytest.mark.parametrize("n", [1, 50, 700, 5000])
def test_scores_beyond_fp32(mep, n, scale, single):
    """Products q.k of up to 6 that the scale takes out of fp32: the largest one's token is all there is."""
    head, hq, rows = 64, 2, 1 if single else min(n, 30)
    b = base.Batch(mep, [n], 1, head, 16, BF16)
    k = torch.zeros(n, 1, head)
    k[:, 0, 0] = torch.randint(-8, 3, (n,), generator=b.gen).float() * 0.5
    best = (n - rows) // 2
    k[best, 0, 0] = 3.0
    b.cache.write("k", b.slots[0], k.to(BF16))
    q = torch.zeros(rows, hq * head, dtype=BF16)
    q[:, 0], q[:, head] = 1.0, 2.0
    cache, table, length = b.on_gpu()
    out = torch.empty(rows, hq * head, dtype=BF16, device="cuda")
    ws = base.workspace(mep, rows, 1, hq, b.layout)
    if single:
        mep.moe_attention_decode(q.cuda(), b.layout, cache, table, length, scale, out, ws)
    else:
        mep.moe_attention_prefill(q.cuda(), base.ints([0, rows]).cuda(), b.layout, cache, table, length, scale, out, ws)
    want = b.values(0)[1][best].view(1, head).expand(rows * hq, head)
    assert torch.equal(out.double().cpu().view(rows * hq, head), want)


def overflowing(mep, n, head, hq, rows, largest, gen_seed=0):
    """Scores of one head that are twice those of the other, of which token `best` has the largest."""
    b = base.Batch(mep, [n], 1, head, 16, BF16, seed=gen_seed)
    k = torch.zeros(n, 1, head)
    k[:, 0, 0] = largest - torch.randint(1, 9, (n,), generator=b.gen).float() * 0.5
    best = (n - rows) // 2
    k[best, 0, 0] = largest
    b.cache.write("k", b.slots[0], k.to(BF16))
    q = torch.zeros(rows, hq * head, dtype=BF16)
    q[:, 0], q[:, head] = 1.0, 2.0
    return b, q, best


def attend(mep, b, q, hq, scale, single):
    rows = q.shape[0]
    cache, table, length = b.on_gpu()
    out = torch.empty(rows, hq * b.head, dtype=BF16, device="cuda")
    ws = base.workspace(mep, rows, 1, hq, b.layout)
    if single:
        mep.moe_attention_decode(q.cuda(), b.layout, cache, table, length, scale, out, ws)
    else:
        mep.moe_attention_prefill(q.cuda(), base.ints([0, rows]).cuda(), b.layout, cache, table, length, scale, out, ws)
    return out.double().cpu().view(rows * hq, b.head)


@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("n", [1, 50, 700, 5000])
def test_negative_scores_beyond_fp32(mep, n, single):
    """The largest one is below -2^128 too."""
    rows = 1 if single else min(n, 30)
    b, q, best = overflowing(mep, n, 64, 2, rows, -1.5)
    want = b.values(0)[1][best].view(1, 64).expand(rows * 2, 64)
    assert torch.equal(attend(mep, b, q, 2, 2.0 ** 127, single), want)


@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("n", [2, 50, 700, 5000])
def test_infinite_values_beside_scores_beyond_fp32(mep, n, single):
    rows = 1 if single else min(n - 1, 30)
    b, q, best = overflowing(mep, n, 64, 2, rows, 3.0)
    set_value(b, 0, best, 9, torch.inf)
    set_value(b, 0, (best + 1) % n, 50, -torch.inf)               # of no weight
    want = b.values(0)[1][best].view(1, 1, 64).expand(rows, 2, 64).clone()
    reads = torch.tensor([n - rows + i >= (best + 1) % n for i in range(rows)])
    want[reads, :, 50] = -torch.inf
    assert torch.equal(attend(mep, b, q, 2, 2.0 ** 127, single), want.view(rows * 2, 64))


@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("scale", [0.1, 2.0, 2.0 ** 100])
@pytest.mark.parametrize("n,tok,v", [(70, 40, torch.nan), (3000, 2980, torch.nan), (3000, 100, torch.inf)])
def test_scores_that_are_not_finite(mep, n, tok, v, scale, single):
    """A key of NaN, or a score of plus infinity, leaves its readers nothing but NaN, beside an infinite value too."""
    rows, hq, head = 1 if single else 60, 2, 128
    b = base.Batch(mep, [n], 1, head, 16, BF16)
    b.cache.section("k")[b.cache.index("k", [b.slots[0][tok]])[0, 0, 3]] = v
    set_value(b, 0, 5, 17, torch.inf)
    q = b.queries(rows, hq)
    q[:, 3], q[:, head + 3] = 1.0, 0.5
    got = attend(mep, b, q, hq, scale, single).view(rows, hq, head)
    for i in range(rows):
        if n - rows + i >= tok:
            assert bool(torch.isnan(got[i]).all()), i
        else:
            assert bool((got[i, :, 17] == torch.inf).all()) and int((~torch.isfinite(got[i])).sum()) == hq, i


@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("largest", [3.0, -1.5])
@pytest.mark.parametrize("far", [2.0 ** 28, 2.0 ** 36, 2.0 ** 60])
@pytest.mark.parametrize("n", [1, 50, 700, 5000])
def test_far_scores(mep, n, far, largest, single):
    """Scores in fp32 whose rounding alone is many powers of two in weight: the largest one's token is all there is.
    They rise along the sequence, so that the sum is taken relative to one far score after the other."""
    rows = 1 if single else min(n, 30)
    b, q, best = overflowing(mep, n, 64, 2, rows, largest)
    k = b.values(0)[0]
    k[:best, 0, 0] = k[:best, 0, 0].sort().values
    b.cache.write("k", b.slots[0], k.to(BF16))
    q = (q.float() * far).to(BF16)
    want = b.values(0)[1][best].view(1, 64).expand(rows * 2, 64)
    assert torch.equal(attend(mep, b, q, 2, 0.1, single), want)
