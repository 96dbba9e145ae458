"""moe_attention_decode and moe_attention_prefill against 64-bit references:
types, head widths, shared heads, one token to many thousand, pages that end
inside tiles, rows and sequences with nothing to read, bytes of any kind where
no token is, strides, streams, captured graphs; and the whole path together as
a layer runs it.
"""
import random

import pytest
import torch

import attn_ref as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
GUARD = 77.0


@pytest.fixture(scope="module")
def mep():
    import mixture_experts_prefill_amd as mep

    return mep


def ints(v):
    return torch.tensor(v, dtype=torch.int32)


class Batch:
    """Sequences of these lengths in a cache whose other bytes are all ones: NaN in bf16 and e4m3, and the largest
    scale byte.  Tables hold what no page is behind the sequences' own pages."""

    def __init__(self, mep, lengths, heads, head, page, dtype, seed=0, strong=1.0):
        gen = torch.Generator().manual_seed(seed * 7919 + sum(lengths) + head)
        rnd = random.Random(seed)
        self.lengths, self.heads, self.head, self.page, self.dtype = lengths, heads, head, page, dtype
        count = [-(-n // page) for n in lengths]
        pages = sum(count) + 2
        order = rnd.sample(range(pages), pages)
        width = max(count) + 2
        self.cache = ref.Cache(pages, page, heads, head, dtype, fill=0xff)
        self.table, self.slots, at = [], [], 0
        for n, c in zip(lengths, count):
            mine = order[at:at + c]
            at += c
            self.table.append(mine + [rnd.choice([-1, pages, 2 ** 31 - 1, -2 ** 31, 0]) for _ in range(width - c)])
            slots = [mine[i // page] * page + i % page for i in range(n)]
            self.slots.append(slots)
            for which in "kv":
                x = torch.randn(n, heads, head, generator=gen) * (strong if which == "k" else 1.0)
                if dtype == BF16:
                    self.cache.write(which, slots, x.to(BF16))
                elif n:
                    self.cache.write(which, slots, *ref.quantise(x.double() * torch.exp2(torch.randint(
                        -3, 4, (n, heads, 1), generator=gen).double() if which == "v" else torch.zeros(1).double())))
        self.layout = mep.moe_kv_layout_make(pages, page, heads, head, dtype)
        self.gen = gen

    def queries(self, t, hq):
        return (1.5 * torch.randn(t, hq * self.head, generator=self.gen)).to(BF16)

    def values(self, s):
        """float64 keys and values [tokens, heads, head] of a sequence."""
        return tuple(self.cache.read(which, self.slots[s]) for which in "kv")

    def on_gpu(self):
        self.dev = self.cache.bytes.cuda(), ints(self.table).cuda(), ints(self.lengths).cuda()
        return self.dev


def guarded(t, width):
    buf = torch.full((t + 2, width + 24), GUARD, dtype=BF16, device="cuda")
    return buf, buf[1:t + 1, 8:8 + width]


def intact(buf, t, width):
    return bool((buf[0] == GUARD).all() and (buf[-1] == GUARD).all() and (buf[:, :8] == GUARD).all()
                and (buf[:, 8 + width:] == GUARD).all())


def workspace(mep, t, n, hq, L):
    """All ones: NaN wherever a call would use what it has not written."""
    return torch.full((mep.moe_attention_workspace_bytes(t, n, hq, L),), 0xff, dtype=torch.uint8, device="cuda")


def decode(mep, b, hq, what, scale=None, starts=None, q=None):
    n, width = len(b.lengths), hq * b.head
    scale = b.head ** -0.5 if scale is None else scale
    t = n if starts is None else starts[-1] + 2
    q = b.queries(t, hq) if q is None else q
    cache, table, length = b.on_gpu()
    buf, out = guarded(t, width)
    mep.moe_attention_decode(q.cuda(), b.layout, cache, table, length, scale, out, workspace(mep, t, n, hq, b.layout),
                             starts=None if starts is None else ints(starts).cuda())
    torch.cuda.synchronize()
    assert intact(buf, t, width)
    touched = []
    for s in range(n):
        r = s if starts is None else starts[s + 1] - 1
        if starts is not None and starts[s + 1] == starts[s]:
            continue
        touched.append(r)
        k, v = b.values(s)
        o, err, var = ref.attention(q[r:r + 1].double().view(1, hq, b.head), k, v, [b.lengths[s] - 1], scale, 2.0 ** -16)
        ref.check_attention(out[r:r + 1], o, err, var, f"{what} sequence {s} of {b.lengths[s]}")
    for r in set(range(t)) - set(touched):
        assert bool((out[r] == GUARD).all())
    return out


def prefill(mep, b, rows, hq, what, scale=None, q=None, lead=0):
    """rows[s] last tokens of each sequence; `lead` rows before them and two after belong to none."""
    n, width = len(b.lengths), hq * b.head
    scale = b.head ** -0.5 if scale is None else scale
    starts = [lead]
    for m in rows:
        starts.append(starts[-1] + m)
    t = starts[-1] + 2
    q = b.queries(t, hq) if q is None else q
    cache, table, length = b.on_gpu()
    buf, out = guarded(t, width)
    mep.moe_attention_prefill(q.cuda(), ints(starts).cuda(), b.layout, cache, table, length, scale, out,
                              workspace(mep, t, n, hq, b.layout))
    torch.cuda.synchronize()
    assert intact(buf, t, width)
    assert bool((out[:lead] == GUARD).all() and (out[starts[-1]:] == GUARD).all())
    for s in range(n):
        if rows[s] == 0:
            continue
        r0, r1 = starts[s], starts[s + 1]
        k, v = b.values(s)
        positions = [b.lengths[s] - rows[s] + i for i in range(rows[s])]
        o, err, var = ref.attention(q[r0:r1].double().view(r1 - r0, hq, b.head), k, v, positions, scale, 2.0 ** -8)
        ref.check_attention(out[r0:r1], o, err, var, f"{what} sequence {s}: {rows[s]} of {b.lengths[s]}")
    return out


TYPES = [BF16, E4M3]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("head", [64, 128, 256])
@pytest.mark.parametrize("heads,g,page", [(1, 1, 16), (2, 4, 64), (3, 5, 32), (1, 16, 128), (2, 17, 16), (1, 40, 256)])
def test_decode(mep, heads, g, page, head, dtype):
    lengths = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 255, 257, 300, 0, 513, 700]
    decode(mep, Batch(mep, lengths, heads, head, page, dtype, seed=g), heads * g, (heads, g, page, head, dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lengths", [[1], [5000], [20000, 1, 0, 3000], [0], [0, 0, 0]])
def test_decode_cut_along_its_tokens(mep, lengths, dtype):
    for heads, hq, head in ((1, 1, 64), (8, 32, 128)):
        decode(mep, Batch(mep, lengths, heads, head, 64, dtype), hq, (lengths, heads, head, dtype))


@pytest.mark.parametrize("n", [64, 65, 255, 256, 257, 600, 1500])
def test_decode_many_sequences(mep, n):
    rnd = random.Random(n)
    lengths = [rnd.choice([0, 1, rnd.randint(1, 40), rnd.randint(1, 400)]) for _ in range(n)]
    lengths[rnd.randrange(n)] = 6000
    decode(mep, Batch(mep, lengths, 1, 64, 16, BF16, seed=n), 2, n)


@pytest.mark.parametrize("n", [5, 100])
def test_decode_rows_by_starts(mep, n):
    """Sequences without a row, and with several, whose last is computed."""
    rnd = random.Random(n)
    starts = [1]
    for _ in range(n):
        starts.append(starts[-1] + rnd.choice([0, 1, 1, 1, 3]))
    lengths = [rnd.randint(0, 3000 if rnd.random() < 0.05 else 90) for _ in range(n)]
    decode(mep, Batch(mep, lengths, 2, 64, 32, BF16, seed=n), 6, n, starts=starts)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("head", [64, 128, 256])
@pytest.mark.parametrize("heads,g,page", [(1, 1, 16), (2, 4, 64), (1, 7, 32), (1, 16, 128), (2, 3, 256)])
def test_prefill(mep, heads, g, page, head, dtype):
    lengths = [1, 2, 31, 33, 64, 65, 130, 200, 0, 77, 300, 16, 90]
    rows = [1, 2, 31, 20, 64, 1, 130, 7, 0, 0, 150, 3, 90]
    b = Batch(mep, lengths, heads, head, page, dtype, seed=g)
    prefill(mep, b, rows, heads * g, (heads, g, page, head, dtype), lead=3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lengths,rows", [([1], [1]), ([900], [900]), ([9000], [70]), ([6000, 40, 500], [1, 40, 300]),
                                          ([3000, 3000], [0, 33])])
def test_prefill_cut_along_its_tokens(mep, lengths, rows, dtype):
    for heads, hq, head in ((1, 1, 64), (2, 8, 128), (1, 2, 256)):
        prefill(mep, Batch(mep, lengths, heads, head, 64, dtype), rows, hq, (lengths, heads, head, dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,g,head", [(2, 11, 64), (2, 8, 128), (1, 16, 256)])
@pytest.mark.parametrize("lengths,rows", [([1000], [900]), ([1700, 0, 2300], [300, 0, 333]), ([5000, 700, 3], [257, 1, 1])])
def test_prefill_joins_tiles(mep, lengths, rows, heads, g, head, dtype):
    """More rows than are joined one by one: tiles of full, few and no rows, sequences that start between tiles."""
    b = Batch(mep, lengths, heads, head, 32, dtype, seed=sum(rows) + g)
    prefill(mep, b, rows, heads * g, f"prefill {lengths} {rows} {heads}x{g}x{head}")


@pytest.mark.parametrize("tokens", [479, 480, 481, 512])
def test_tables_about_the_length_that_is_cut(mep, tokens):
    """The tables' widths, not the lengths, say whether a joining launch follows: 512 tokens here up to 480."""
    for page, least in ((16, 1), (32, tokens - 1)):
        b = Batch(mep, [tokens, least], 2, 128, page, BF16, seed=tokens)
        decode(mep, b, 8, f"decode {tokens}")
        prefill(mep, b, [tokens // 2, least], 8, f"prefill {tokens}")


@pytest.mark.parametrize("n", [64, 65, 256, 300])
def test_prefill_many_sequences(mep, n):
    rnd = random.Random(n)
    rows = [rnd.choice([0, 1, rnd.randint(1, 20)]) for _ in range(n)]
    lengths = [m + rnd.choice([0, rnd.randint(0, 100)]) for m in rows]
    lengths[rnd.randrange(n)] += 3000
    prefill(mep, Batch(mep, lengths, 1, 64, 16, BF16, seed=n), rows, 3, n)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("head", [64, 128, 256])
def test_rows_before_the_first_token(mep, head, dtype):
    """More rows than tokens: the first rows' positions are negative, and they are 0."""
    b = Batch(mep, [3, 0, 40, 0], 2, head, 16, dtype)
    out = prefill(mep, b, [10, 70, 41, 1], 4, (head, dtype))
    assert bool((out[:7] == 0).all() and (out[10:81] == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("head", [64, 128, 256])
def test_pages_that_are_not_there(mep, head, dtype):
    """Tokens of table entries outside the cache are as if absent, wherever they stand; a row with none is 0."""
    b = Batch(mep, [200, 64, 33, 500], 1, head, 16, dtype)
    for s, i, e in ((0, 0, -1), (0, 5, 10 ** 6), (1, 0, -1), (1, 1, -5), (1, 2, 2 ** 31 - 1), (1, 3, -2 ** 31), (2, 2, -1),
                    (3, 17, -1), (3, 31, b.layout.pages)):
        b.table[s][i] = e
    there = [[0 <= b.table[s][i // 16] < b.layout.pages for i in range(n)] for s, n in enumerate(b.lengths)]
    hq, q = 3, b.queries(130, 3)
    cache, table, length = b.on_gpu()
    rows = [60, 20, 33, 17]
    starts = [0, 60, 80, 113, 130]
    for single in (True, False):
        t = 4 if single else 130
        out = torch.full((t, hq * head), GUARD, dtype=BF16, device="cuda")
        ws = workspace(mep, t, 4, hq, b.layout)
        if single:
            mep.moe_attention_decode(q[:4].cuda(), b.layout, cache, table, length, 0.1, out, ws)
        else:
            mep.moe_attention_prefill(q.cuda(), ints(starts).cuda(), b.layout, cache, table, length, 0.1, out, ws)
        for s, n in enumerate(b.lengths):
            keep = [i for i in range(n) if there[s][i]]
            slots = [b.slots[s][i] if i // 16 < len(b.table[s]) else 0 for i in keep]
            k, v = b.cache.read("k", slots), b.cache.read("v", slots)
            r0, m = (s, 1) if single else (starts[s], rows[s])
            pos = [sum(1 for x in keep if x <= n - m + i) - 1 for i in range(m)]
            o, err, var = ref.attention(q[r0:r0 + m].double().view(m, hq, head), k, v, pos, 0.1, 2.0 ** -16 if single else 2.0 ** -8)
            ref.check_attention(out[r0:r0 + m], o, err, var, (single, s))


@pytest.mark.parametrize("single", [True, False])
def test_lengths_and_starts_out_of_range(mep, single):
    """Lengths past the table or negative count as the nearest possible; starts are held inside the rows.  Rows of
    sequences in order get their result whatever else the integers are."""
    b = Batch(mep, [64, 48, 30, 64], 1, 64, 16, BF16)
    table = [r[:4] for r in b.table]
    b.table = [r if len(r) == 4 else r + [-1] * (4 - len(r)) for r in table]
    hq, q = 2, b.queries(20, 2)
    cache, tab, length = b.on_gpu()
    bad = ints([2 ** 31 - 1, -2 ** 31, 30, 65]).cuda()
    out = torch.full((20, hq * 64), GUARD, dtype=BF16, device="cuda")
    starts = [0, 5, 9, 12, 2 ** 31 - 1]
    ws = workspace(mep, 20, 4, hq, b.layout)
    if single:
        mep.moe_attention_decode(q[:4].cuda(), b.layout, cache, tab, bad, 0.125, out[:4], ws)
    else:
        mep.moe_attention_prefill(q.cuda(), ints(starts).cuda(), b.layout, cache, tab, bad, 0.125, out, ws)
    torch.cuda.synchronize()
    lengths, ends = [64, 0, 30, 64], starts[:4] + [20]
    for s in range(4):
        r0, m = (s, 1) if single else (ends[s], ends[s + 1] - ends[s])
        k, v = (x[:lengths[s]] for x in b.values(s)) if lengths[s] <= b.lengths[s] else b.values(s)
        o, err, var = ref.attention(q[r0:r0 + m].double().view(m, hq, 64), k, v, [lengths[s] - m + i for i in range(m)], 0.125, 2.0 ** -8)
        ref.check_attention(out[r0:r0 + m], o, err, var, s)
    # starts in no order at all: no fault, rows that no sequence has stay
    for starts in ([20, 0, 20, 0, 20], [5, 4, 3, 2, 1], [-7, 2 ** 31 - 1, -2 ** 31, 8, 8], [0, 20, 0, 20, 0]):
        big = ints([64, 64, 64, 64]).cuda()
        (mep.moe_attention_decode(q.cuda(), b.layout, cache, tab, big, 0.125, out, ws, starts=ints(starts).cuda()) if single else
         mep.moe_attention_prefill(q.cuda(), ints(starts).cuda(), b.layout, cache, tab, big, 0.125, out, ws))
        torch.cuda.synchronize()


@pytest.mark.parametrize("g,n", [(1, 18), (5, 6)])
def test_starts_in_no_order_stay_inside_the_workspace(mep, g, n):
    """Every other sequence claims all rows: 576 or 600 partial results, 537 and 557 of which have room."""
    t, length, page = 1000, 24000, 256
    L = mep.moe_kv_layout_make(94, page, 1, 64, BF16)
    cache = torch.zeros(L.bytes, dtype=torch.uint8, device="cuda")
    table = torch.arange(94, dtype=torch.int32, device="cuda").repeat(n, 1)
    size = mep.moe_attention_workspace_bytes(t, n, g, L)
    ws = torch.full((size + (64 << 20),), 0x5a, dtype=torch.uint8, device="cuda")
    q = torch.randn(t, g * 64, device="cuda").to(BF16)
    buf, out = guarded(t, g * 64)
    mep.moe_attention_prefill(q, ints([0, t] * (n // 2) + [0]).cuda(), L, cache, table, ints([length] * n).cuda(),
                              0.125, out, ws[:size])
    torch.cuda.synchronize()
    assert bool((ws[size:] == 0x5a).all()) and intact(buf, t, g * 64)


@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("n", [1, 80])
def test_a_step_without_rows_after_one_that_was_joined(mep, single, n):
    """The same workspace: nothing that the first call left in it is joined again."""
    b = Batch(mep, [3000] + [1] * (n - 1), 1, 64, 64, BF16)
    hq, t = 16, 900
    q = b.queries(t, hq).cuda()
    cache, table, length = b.on_gpu()
    ws = workspace(mep, t, n, hq, b.layout)
    call = mep.moe_attention_decode if single else mep.moe_attention_prefill

    def step(starts):
        out, starts = torch.full((t, hq * 64), GUARD, dtype=BF16, device="cuda"), ints(starts).cuda()
        rest = (b.layout, cache, table, length, 0.125, out, ws)
        call(q, *rest, starts=starts) if single else call(q, starts, *rest)
        torch.cuda.synchronize()
        return out

    first = step([0, 800] + [800] * (n - 1))
    assert bool((first[799] != GUARD).all())
    assert bool((step([0] * (n + 1)) == GUARD).all())
    again = step([0, 5] + [5] * (n - 1))
    assert bool((again[5:] == GUARD).all() and (again[4] != GUARD).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("head", [64, 128, 256])
def test_values_not_finite_reach_their_readers_only(mep, head, dtype):
    """A NaN or infinity in a later token's value or key is not seen by the rows before it; a row's own NaN stays in
    its row."""
    n = 150
    b = Batch(mep, [n], 1, head, 16, dtype)
    bad = torch.tensor([torch.nan, torch.inf, torch.nan])
    for i, tok in enumerate((40, 100, 149)):
        slot = b.slots[0][tok]
        flat = b.cache.section("v")
        at = b.cache.index("v", [slot])[0, 0, 7 + i]
        if dtype == BF16:
            flat[at] = bad[i].to(BF16)
        else:
            flat.view(torch.uint8)[at] = 0x7f
    hq = 2
    q = b.queries(n + 2, hq)
    q[20, 5] = torch.nan                      # head 0 of row 20
    cache, table, length = b.on_gpu()
    out = torch.full((n, hq * head), GUARD, dtype=BF16, device="cuda")
    mep.moe_attention_prefill(q[:n].cuda(), ints([0, n]).cuda(), b.layout, cache, table, length, 0.2, out, workspace(mep, n, 1, hq, b.layout))
    k, v = b.values(0)
    want, err, var = ref.attention(q[:n].double().view(n, hq, head), k, torch.where(torch.isfinite(v), v, 0.0), list(range(n)), 0.2, 2.0 ** -8)
    got = out.double().cpu().view(n, hq, head)
    wild = torch.zeros(n, hq, head, dtype=torch.bool)
    wild[40:, :, 7], wild[100:, :, 8], wild[149:, :, 9], wild[20, 0] = True, True, True, True
    assert not bool(torch.isfinite(got[wild]).any())
    fill = torch.where(wild, want, got)
    ref.check_attention(fill, want, err, var, (head, dtype))
    if dtype == BF16:
        assert bool((got[100:, :, 8] == torch.inf).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("single", [True, False])
def test_sharp_and_flat_scores(mep, single, dtype):
    """Scores that leave one token's weight only, that grow along the sequence (the running maximum rises again and
    again), that fall, and that are all equal."""
    n, head, hq = 400, 64, 2
    for kind in ("grow", "fall", "equal", "huge"):
        b = Batch(mep, [n], 1, head, 16, dtype)
        q = b.queries(42, hq)
        q[:, :] = 0
        q[:, 0], q[:, 64] = 1.0, 2.0
        k = torch.randn(n, 1, head, generator=b.gen).double() * 0.1
        ramp = torch.arange(n).double() * 0.5
        k[:, 0, 0] = dict(grow=ramp, fall=ramp.flip(0), equal=torch.ones(n).double(), huge=ramp * 1000)[kind]
        x = k.float().to(BF16) if dtype == BF16 else None
        b.cache.write("k", b.slots[0], x) if dtype == BF16 else b.cache.write("k", b.slots[0], *ref.quantise(k))
        if single:
            decode(mep, b, hq, kind, scale=1.0, q=q[:1])
        else:
            prefill(mep, b, [40], hq, kind, scale=1.0, q=q)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [2.0 ** -126, 1e-30, 1e-6, 1e3])
def test_scales_of_any_size(mep, scale, dtype):
    """Scales that make all weights equal, or one of them 1."""
    b = Batch(mep, [300, 1, 700], 2, 64, 32, dtype)
    decode(mep, b, 4, scale, scale=scale)
    prefill(mep, b, [20, 1, 150], 4, scale, scale=scale)


def test_scores_of_minus_infinity(mep):
    """They weigh nothing; a row that has no other is 0."""
    b = Batch(mep, [40, 40], 1, 64, 16, BF16)
    x = torch.zeros(40, 1, 64)
    x[:, 0, 0] = -torch.inf
    b.cache.write("k", b.slots[0], x.to(BF16))
    x[5, 0, 0] = 0.0
    b.cache.write("k", b.slots[1], x.to(BF16))
    q = torch.zeros(4, 64).to(BF16)
    q[:, 0] = 1.0
    cache, table, length = b.on_gpu()
    out = torch.full((4, 64), GUARD, dtype=BF16, device="cuda")
    ws = workspace(mep, 4, 2, 1, b.layout)
    v = b.values(1)[1][5].view(-1).to(BF16).cuda()
    mep.moe_attention_decode(q[:2].cuda(), b.layout, cache, table, length, 1.0, out[:2], ws)
    assert bool((out[0] == 0).all()) and torch.equal(out[1], v)
    mep.moe_attention_prefill(q.cuda(), ints([0, 2, 4]).cuda(), b.layout, cache, table, length, 1.0, out, ws)
    assert bool((out[:2] == 0).all()) and torch.equal(out[2], v) and torch.equal(out[3], v)


def test_equal_values_come_back(mep):
    """Weights that sum to 1: where every value is v, so is the output, to half a step."""
    n, head = 333, 128
    b = Batch(mep, [n], 2, head, 16, BF16)
    one = torch.randn(1, 2, head, generator=b.gen).to(BF16)
    b.cache.write("v", b.slots[0], one.expand(n, 2, head))
    out = decode(mep, b, 8, "equal")
    want = one.double().repeat_interleave(4, 1).view(1, -1)
    assert bool(((out.double().cpu() - want).abs() <= 2.0 ** -8 * want.abs()).all())


def test_far_pages(mep):
    """Byte offsets past 32 bits, in both kernels."""
    pages, page, heads, head, hq = 40000, 64, 8, 128, 16
    L = mep.moe_kv_layout_make(pages, page, heads, head)
    assert L.v > 1 << 32
    cache = torch.empty(L.bytes, dtype=torch.uint8, device="cuda")
    n, mine = 200, [pages - 1, 3, pages - 2, pages // 2 + 1]
    gen = torch.Generator().manual_seed(5)
    k, v = (torch.randn(n, heads * head, generator=gen).to(BF16) for _ in range(2))
    q = (1.5 * torch.randn(n, hq * head, generator=gen)).to(BF16)
    slots = ints([mine[i // page] * page + i % page for i in range(n)]).cuda()
    mep.moe_kv_append(k.cuda(), v.cuda(), L, cache, slots)
    table, length = ints([mine]).cuda(), ints([n]).cuda()
    out, last = torch.empty(n, hq * head, dtype=BF16, device="cuda"), torch.empty(1, hq * head, dtype=BF16, device="cuda")
    ws = workspace(mep, n, 1, hq, L)
    mep.moe_attention_prefill(q.cuda(), ints([0, n]).cuda(), L, cache, table, length, 0.1, out, ws)
    mep.moe_attention_decode(q[-1:].cuda(), L, cache, table, length, 0.1, last, ws)
    kd, vd = (x.double().view(n, heads, head) for x in (k, v))
    o, err, var = ref.attention(q.double().view(n, hq, head), kd, vd, list(range(n)), 0.1, 2.0 ** -8)
    ref.check_attention(out, o, err, var, "prefill")
    ref.check_attention(last, o[-1:], err[-1:], var[-1:], "decode")


def test_strides_of_tables_and_rows(mep):
    """q and out as columns of wider buffers, the table as columns of a wider one."""
    b = Batch(mep, [70, 3, 129], 2, 64, 16, BF16)
    hq, n = 4, 3
    cache, table, length = b.on_gpu()
    wide = torch.full((n, table.shape[1] + 7), 2 ** 30, dtype=torch.int32, device="cuda")
    wide[:, 3:3 + table.shape[1]] = table
    q = b.queries(n, hq).cuda()
    qw = torch.full((n, 5 * 64 + 16), torch.nan, dtype=BF16, device="cuda")
    qw[:, 8:8 + 256] = q
    out, ow = torch.empty_like(q), torch.full((n, 400), GUARD, dtype=BF16, device="cuda")
    ws = workspace(mep, n, n, hq, b.layout)
    mep.moe_attention_decode(q, b.layout, cache, table, length, 0.125, out, ws)
    mep.moe_attention_decode(qw[:, 8:264], b.layout, cache, wide[:, 3:3 + table.shape[1]], length, 0.125, ow[:, 16:272], ws)
    assert torch.equal(out, ow[:, 16:272]) and bool((ow[:, :16] == GUARD).all() and (ow[:, 272:] == GUARD).all())


@pytest.mark.parametrize("single", [True, False])
def test_streams_repeats_and_graphs(mep, single):
    """The same bits from another stream, beside another call with a workspace of its own, and from replays of a
    graph captured at other lengths, with the program's own work in between."""
    b = Batch(mep, [5000, 17, 800], 2, 128, 64, BF16)
    hq, n = 8, 3
    t = 3 if single else 90
    q = b.queries(t, hq).cuda()
    cache, table, length = b.on_gpu()
    starts = ints([0, 1, 2, 3] if single else [0, 50, 60, 90]).cuda()
    outs = [torch.empty_like(q) for _ in range(3)]
    spaces = [workspace(mep, t, n, hq, b.layout) for _ in range(3)]

    def call(i, stream=None):
        if single:
            mep.moe_attention_decode(q, b.layout, cache, table, length, 0.09, outs[i], spaces[i], starts=starts, stream=stream)
        else:
            mep.moe_attention_prefill(q, starts, b.layout, cache, table, length, 0.09, outs[i], spaces[i], stream=stream)

    call(0)
    torch.cuda.synchronize()
    first = outs[0].clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        call(1, streams[0])
        call(2, streams[1])
    torch.cuda.synchronize()
    assert torch.equal(outs[1], first) and torch.equal(outs[2], first)
    # captured at the shortest lengths, replayed at others
    other = ints([1, 0, 2]).cuda()
    length, keep = length.clone(), length
    length.copy_(other)
    call(0)
    torch.cuda.synchronize()
    short = outs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(0)
    for i in range(4):
        length.copy_(keep if i % 2 == 0 else other)
        outs[0].fill_(GUARD)
        g.replay()
        (torch.randn(1000, device="cuda") ** 2).sum().item()
        assert torch.equal(outs[0], first if i % 2 == 0 else short), i


def test_decode_is_the_last_row_of_prefill(mep):
    """One row through either kernel gives the same value to the weights' rounding."""
    b = Batch(mep, [700, 60], 1, 128, 32, E4M3)
    q = b.queries(2, 4)
    a = decode(mep, b, 4, "decode", q=q)
    c = prefill(mep, b, [1, 1], 4, "prefill", q=torch.cat([q, q]))
    assert float((a.double() - c[:2].double()).norm() / a.double().norm()) < 2.0 ** -7


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", TYPES)
def test_a_server_runs_a_layer(mep, dtype):
    """Steps of a batch as a server makes them: a 4-bit projection to q, k and v, the plan, the rotated rows into the
    cache, attention (of packed rows, or of single ones), the output projection; prompts in pieces, decodes, a
    sequence that ends and another that takes its place.  Against attention over all tokens in 64 bits."""
    import layer_ref as lref

    n, rows, page, heads, head, hq, hidden, layers = 4, 200, 16, 2, 64, 6, 256, 2
    cache = mep.MoeCache(layers, n, rows, 60, page, heads, head, hq, 24, dtype)
    for c in cache.cache:
        c.fill_(0xff)
    wide = (hq + 2 * heads) * head
    qkv, out_proj = (mep.MoeMatrix.from_codes(m.q.cuda(), m.s.cuda(), m.b.cuda(), 64)
                     for m in (lref.Matrix(wide, hidden, 64, 1), lref.Matrix(hidden, hq * head, 64, 2)))
    half = head // 2
    ang = torch.arange(512, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(half, dtype=torch.float64) / half)
    rope = torch.cat([ang.cos(), ang.sin()], 1).float()
    drope = rope.cuda()
    kept = [[[] for _ in range(n)] for _ in range(layers)]     # per layer and sequence: (k, v) float64 rows
    gen = torch.Generator().manual_seed(3)
    for step, grow in enumerate([[40, 1, 0, 100], [1, 90, 0, 17], [1, 1, 0, 1], [1, 1, 0, 1], [1, -1, 33, 1], [1, 20, 1, 0],
                                 [0, 1, 1, 1], [30, 1, -1, 1], [1, 1, 5, 1]]):
        cache.plan(ints(grow).cuda())
        count = sum(max(x, 0) for x in grow)
        t = count + 3                                            # three padding rows
        single = max(grow) == 1
        for layer in range(layers):
            x = torch.randn(t, hidden, generator=gen).to(BF16).cuda()
            y = qkv.linear(x)
            q, k, v = y.split([hq * head, heads * head, heads * head], dim=1)
            keep = [z.clone() for z in (q, k, v)]
            turned = cache.append(layer, k, v, drope, q)
            o = cache.attend(layer, turned, single=single)
            final = out_proj.linear(o)
            torch.cuda.synchronize()
            assert cache.lacking.item() == 0 and bool((o[count:] == 0).all()) and bool(torch.isfinite(final).all())
            q, k, v = (z.double().cpu() for z in keep)
            at = 0
            for s in range(n):
                if grow[s] < 0:
                    kept[layer][s] = []
                    continue
                m, seq = grow[s], kept[layer][s]
                pos = [len(seq) + i for i in range(m)]
                if m == 0:
                    continue
                a = rope[pos]
                kr = ref.rotate(k[at:at + m].view(m, heads, head), a)
                vr = v[at:at + m].view(m, heads, head)
                qr = turned[at:at + m].double().cpu().view(m, hq, head)
                want = ref.rotate(q[at:at + m].view(m, hq, head), a)
                assert bool(((qr - want).abs() <= 2.0 ** -8 * 1.001 * want.abs() + 1e-30).all())
                # what the cache holds of k and v: their rounding is the append's own test
                table, length = cache.table[s].cpu().tolist(), cache.length[s].item()
                assert length == len(seq) + m
                held = ref.Cache(60, page, heads, head, dtype)
                held.bytes.copy_(cache.cache[layer].cpu())
                slots = [table[p // page] * page + p % page for p in pos]
                kh, vh = held.read("k", slots), held.read("v", slots)
                half_step = ref.HALF[dtype] * 1.001
                for h, w in ((kh, kr), (vh, vr)):
                    floor = 0 if dtype == BF16 else w.abs().amax(-1, keepdim=True) / 224 * 2.0 ** -10
                    assert bool(((h - w).abs() <= half_step * w.abs() + floor + 1e-30).all()), (step, layer, s)
                seq.extend((kh[i], vh[i]) for i in range(m))
                K, V = (torch.stack([e[i] for e in seq]) for i in (0, 1))
                r, err, var = ref.attention(qr, K, V, pos, head ** -0.5, 2.0 ** -16 if single else 2.0 ** -8)
                ref.check_attention(o[at:at + m], r, err, var, (step, layer, s))
                at += m


def test_two_devices_are_refused(mep):
    """Tensors of another GPU than q's, and host tensors, are refused before any launch."""
    b = Batch(mep, [5], 1, 64, 16, BF16)
    cache, table, length = b.on_gpu()
    q = b.queries(1, 1).cuda()
    ws = workspace(mep, 1, 1, 1, b.layout)
    for bad in (dict(cache=cache.cpu()), dict(table=table.cpu()), dict(length=length.cpu()), dict(out=q.cpu()), dict(ws=ws.cpu())):
        a = dict(cache=cache, table=table, length=length, out=torch.empty_like(q), ws=ws)
        a.update(bad)
        with pytest.raises(ValueError, match="GPU"):
            mep.moe_attention_decode(q, b.layout, a["cache"], a["table"], a["length"], 1.0, a["out"], a["ws"])
