"""moe_kv_plan and moe_kv_append against plain implementations: steps of
sequences that grow, end and start, too few pages, integers out of range;
rows of every type and alignment into bf16 and e4m3 pages, rows without a
slot, strides, values that are not finite; captured graphs.
"""
import random

import pytest
import torch

import attn_ref as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
GUARD = -77


@pytest.fixture(scope="module")
def mep():
    import mixture_experts_prefill_amd as mep

    return mep


def ints(v):
    return torch.tensor(v, dtype=torch.int32)


class Guarded:
    """An int32 buffer on the GPU with guard words around it."""

    def __init__(self, n, value=0):
        self.buf = torch.full((n + 16,), GUARD, dtype=torch.int32, device="cuda")
        self.v = self.buf[8:8 + n]
        self.v.fill_(value) if not torch.is_tensor(value) else self.v.copy_(value.view(-1))

    def intact(self):
        return bool((self.buf[:8] == GUARD).all() and (self.buf[-8:] == GUARD).all())


def run_plan(mep, length, grow, page, pages, table, free, free_n, t, ldt=None, in_place=False):
    """The library's plan of a step; returns the same things as ref.plan, and the table and free list after it."""
    n, width = len(length), len(table[0])
    ldt = ldt or width
    L = mep.moe_kv_layout_make(pages, page, 2, 64)
    tab = Guarded(n * ldt, GUARD)
    view = tab.v.view(n, ldt)[:, :width]
    view.copy_(ints(table))
    g = dict(free=Guarded(pages, ints(free)), length=Guarded(n, ints(length)), free_n=Guarded(1, ints([free_n])),
             length_out=Guarded(n), free_n_out=Guarded(1), starts=Guarded(n + 1), positions=Guarded(t), slots=Guarded(t),
             lacking=Guarded(1))
    if in_place:
        g["length_out"], g["free_n_out"] = g["length"], g["free_n"]
    mep.moe_kv_plan(g["length"].v, ints(grow).cuda(), L, view, g["free"].v, g["free_n"].v, g["length_out"].v,
                    g["free_n_out"].v, g["starts"].v, g["positions"].v, g["slots"].v, g["lacking"].v)
    torch.cuda.synchronize()
    assert tab.intact() and all(x.intact() for x in g.values())
    if ldt > width:
        assert bool((tab.v.view(n, ldt)[:, width:] == GUARD).all())
    if not in_place:
        assert g["length"].v.tolist() == length and g["free_n"].v.tolist() == [free_n]
    out = {x: g[x].v.tolist() for x in ("length_out", "free_n_out", "starts", "positions", "slots", "lacking")}
    return out, view.tolist(), g["free"].v.tolist()


def check_plan(mep, length, grow, page, pages, table, free, free_n, t, **kw):
    got, tab, fr = run_plan(mep, length, grow, page, pages, table, free, free_n, t, **kw)
    table, free = [list(r) for r in table], list(free)
    want = ref.plan(length, grow, page, pages, table, free, free_n, t)
    for x in want:
        assert got[x] == want[x], x
    assert tab == table and fr == free
    return got, tab, fr


def a_step(rnd, n, t, page, longest, spare):
    """Lengths, rows and a consistent table and free list."""
    length = [rnd.choice([0, rnd.randint(0, longest), page * rnd.randint(0, longest // page)]) for _ in range(n)]
    grow = [rnd.choice([-1, 0, 1, 1, 1]) for _ in range(n)]
    left = t - sum(max(g, 0) for g in grow)
    for s in rnd.sample(range(n), min(n, 5)):
        if left > 0 and grow[s] > 0:
            more = rnd.randint(0, left)
            grow[s] += more
            left -= more
    up = lambda v: -(-v // page)
    width = max(up(a + max(g, 0)) for a, g in zip(length, grow)) + rnd.randint(1, 3)
    have = sum(up(a) for a in length)
    pages = have + sum(up(a + max(g, 0)) - up(a) for a, g in zip(length, grow)) + spare
    pages = max(pages, have, 1)
    order = list(range(pages))
    rnd.shuffle(order)
    table, at = [], 0
    for a in length:
        table.append([order[at + i] if i < up(a) else rnd.choice([-1, 0, 1 << 30]) for i in range(width)])
        at += up(a)
    free = order[at:]
    return length, grow, page, pages, table, free + [rnd.randint(0, 99) for _ in range(pages - len(free))], len(free), t


@pytest.mark.parametrize("n,t,page,longest", [(1, 1, 16, 100), (1, 4096, 16, 100), (3, 40, 256, 3000), (8, 8, 64, 700),
                                              (64, 512, 32, 500), (65, 513, 16, 300), (255, 512, 64, 900), (256, 300, 16, 40),
                                              (257, 1500, 32, 200), (1023, 4096, 16, 64), (1025, 2000, 16, 90),
                                              (4096, 4096, 16, 33)])
def test_plan(mep, n, t, page, longest):
    rnd = random.Random(n * 31 + t)
    for spare, kw in [(3, {}), (0, dict(in_place=True)), (-2, {}), (5, dict(ldt=40 + longest // page + 4096 // page))]:
        check_plan(mep, *a_step(rnd, n, t, page, longest, spare), **kw)


def test_plan_too_few_pages_and_again(mep):
    """Rows past the last free page have no slot; the step is planned again with fewer rows, as nothing was lost."""
    page, table = 16, [[0, 1, -1, -1], [2, -1, -1, -1], [-1] * 4]
    free = [3, 4, 5, -1, -1, -1]
    got, tab, fr = check_plan(mep, [32, 5, 0], [20, 12, 16], page, 6, table, free, 3, 64)
    assert got["lacking"] == [16] and got["length_out"] == [52, 17, 0] and got["free_n_out"] == [0]
    got, _, _ = check_plan(mep, [32, 5, 0], [20, 12, 0], page, 6, tab, fr, 3, 64)
    assert got["lacking"] == [0]


def test_plan_limits(mep):
    """More rows than t, more tokens than the table has entries for, no free page at all, no rows at all."""
    table, free = [[0, 1], [2, 3], [4, 5]], [6, 7, 8] + [0] * 17
    check_plan(mep, [20, 30, 17], [5, 50, 3], 16, 20, table, free, 3, 10)
    check_plan(mep, [20, 30, 17], [50, 50, 50], 16, 20, table, free, 3, 100)
    check_plan(mep, [20, 30, 17], [5, 5, 5], 16, 20, table, free, 0, 100)
    check_plan(mep, [20, 30, 17], [0, 0, 0], 16, 20, table, free, 3, 7)
    check_plan(mep, [20, 30, 17], [-1, -5, -1], 16, 20, table, free, 3, 7)
    check_plan(mep, [0, 0, 0], [0, -1, 0], 16, 20, table, free, 0, 1)


def test_plan_integers_out_of_range(mep):
    """Whatever the integers are, nothing outside the buffers is read or written, and the result is the stated one."""
    big = 2 ** 31 - 1
    table, free = [[0, 1, big], [-big, 3, 2], [4, -1, 5], [1, 1, 1]], [6, big, -1] + [0] * 17
    check_plan(mep, [-5, 30, big, 17], [5, 3, 1, 20], 16, 20, table, free, 3, 64)
    check_plan(mep, [40, -big - 1, big, 17], [big, big, -big, big], 16, 20, table, free, 20, 64)
    check_plan(mep, [10, 20, 30, 40], [-1, -1, -1, -1], 16, 8, table, free[:8], 7, 64)       # more given back than fits
    check_plan(mep, [10, 20, 30, 40], [3, 30, 8, 1], 16, 20, table, free, big, 64)
    check_plan(mep, [10, 20, 30, 40], [3, 30, 8, 1], 16, 20, table, free, -7, 64)


def test_plan_replayed(mep):
    """A captured plan that writes its lengths and free list in place advances with each replay."""
    page, pages, n, t = 16, 40, 3, 8
    L = mep.moe_kv_layout_make(pages, page, 1, 64)
    table, free = ints([[0] * 10] * n), ints(list(range(pages)))
    dev = dict(length=ints([0, 15, 31]), table=table.clone(), free=free.clone(), free_n=ints([pages]), grow=ints([1, 3, 2]),
               starts=ints([0] * (n + 1)), positions=ints([0] * t), slots=ints([0] * t), lacking=ints([0]))
    dev = {k: v.cuda() for k, v in dev.items()}
    dev["table"][1, 0], dev["table"][2, 0], dev["table"][2, 1] = 39, 38, 37
    dev["free_n"].fill_(37)
    keep = {k: v.clone() for k, v in dev.items()}

    def call():
        mep.moe_kv_plan(dev["length"], dev["grow"], L, dev["table"], dev["free"], dev["free_n"], dev["length"], dev["free_n"],
                        dev["starts"], dev["positions"], dev["slots"], dev["lacking"])

    call()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call()
    for k in dev:
        dev[k].copy_(keep[k])
    tab, fr, length, top = keep["table"].tolist(), keep["free"].tolist(), keep["length"].tolist(), 37
    for step in range(6):
        g.replay()
        torch.cuda.synchronize()
        want = ref.plan(length, [1, 3, 2], page, pages, tab, fr, top, t)
        length, top = want["length_out"], want["free_n_out"][0]
        assert dev["slots"].tolist() == want["slots"] and dev["length"].tolist() == length
        assert dev["table"].tolist() == tab and dev["free_n"].tolist() == [top] and dev["positions"].tolist() == want["positions"]
        (torch.randn(100, device="cuda") * 2).sum().item()      # the program's own work between replays


# ------------------------------------------------------------------ append

def angles(rows, rot, seed=0):
    half = rot // 2
    a = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    return torch.cat([a.cos(), a.sin()], 1).float()


def near(got, want, dtype, what):
    """got (a tensor of dtype) is want rounded once, but for the fp32 rounding of a rotation: two half steps of fp32
    relative to the result, which move a value that lies between two neighbours of dtype by at most a step."""
    g, w = got.double().cpu(), want
    fin = torch.isfinite(w)
    assert torch.equal(torch.isnan(g), torch.isnan(w)), f"{what}: NaN"
    assert torch.equal(g[~fin & ~torch.isnan(w)], w[~fin & ~torch.isnan(w)]), what
    tol = (ref.HALF[dtype] * (1 + 4 * ref.U32) + 4 * ref.U32) * w.abs() + (2.0 ** -10 if dtype == E4M3 else 2.0 ** -134)
    assert bool(((g - w).abs()[fin] <= tol[fin]).all()), f"{what}: {float((g - w).abs()[fin].max())}"


def check_append(mep, t, heads, head, page, ctype, xtype, rot, hq, slots, pages, positions=None, rope_rows=5000, seed=0,
                 in_place=False, change=None, stride=0):
    """Appends rows at these slots (a list) and compares every byte of the cache."""
    gen = torch.Generator().manual_seed(seed * 7919 + t * 31 + head + rot)
    L = mep.moe_kv_layout_make(pages, page, heads, head, ctype)
    cache = ref.Cache(pages, page, heads, head, ctype)
    cache.bytes.copy_(torch.randint(0, 256, cache.bytes.shape, generator=gen, dtype=torch.uint8))
    width = (hq + 2 * heads) * head
    x = torch.randn(t, width + stride, generator=gen) * (1 + 6 * (torch.rand(width + stride, generator=gen) < 0.02).float())
    if change:
        change(x)
    x = x.to(xtype)
    dx = x.cuda()
    off = stride // 2 // 8 * 8
    cut = lambda y: y[:, off:off + width].split([hq * head, heads * head, heads * head], dim=1)
    (q, k, v), (dq, dk, dv) = cut(x), cut(dx)
    table = angles(rope_rows, rot) if rot else None
    pos = ints(positions if positions is not None else [(37 * i) % rope_rows for i in range(t)]) if rot else None
    dev = cache.bytes.cuda()
    buf = torch.full((t + 2, hq * head + 8), 77.0, dtype=BF16, device="cuda") if hq else None
    out = dq if in_place else buf[1:t + 1, :hq * head] if hq else None
    mep.moe_kv_append(dk, dv, L, dev, ints(slots).cuda(), positions=None if pos is None else pos.cuda(),
                      rope=None if table is None else table.cuda(), q=dq if hq else None, q_out=out)
    torch.cuda.synchronize()
    # what it should be
    kd, vd = (y.double().reshape(t, heads, head) for y in (k, v))
    if rot:
        a = torch.full((t, rot), torch.nan)
        ok = (pos >= 0) & (pos < rope_rows)
        a[ok] = table[pos[ok].long()]
        kd = ref.rotate(kd, a)
    kept = [i for i in range(t) if 0 <= slots[i] < pages * page]
    at = [slots[i] for i in kept]
    got = ref.Cache(pages, page, heads, head, ctype)
    got.bytes.copy_(dev.cpu())
    for which, y in (("k", kd), ("v", vd)):
        y = y[kept]
        if not kept:
            continue
        if ctype == BF16:
            g = got.section(which)[got.index(which, at)]
            near(g, y, BF16, which) if which == "k" and rot else None
            if which == "v" or not rot:
                assert torch.equal(torch.isnan(g), torch.isnan(y)) and torch.equal(torch.nan_to_num(g), torch.nan_to_num(y.float().to(BF16))), which
            cache.write(which, at, g)
        else:
            codes, byte = ref.quantise(y)
            g = got.section(which).view(torch.uint8)[got.index(which, at)].view(E4M3)
            gs = got.section(which + "s")[got.index(which + "s", at)]
            if which == "v" or not rot:
                assert torch.equal(gs, byte) and torch.equal(torch.nan_to_num(g.double(), nan=999.0),
                                                             torch.nan_to_num(codes.double(), nan=999.0)), which
            else:
                # the largest magnitude may lie next to 448 * 2^E: a scale twice or half as large is right then
                assert bool(((gs.int() - byte.int()).abs() <= 1).all()) and float((gs != byte).double().mean()) < 0.01
                unit = torch.exp2(gs.double() - 127)[..., None]
                near(g, torch.where(torch.isfinite(y), y, torch.nan) / unit, E4M3, which)
            cache.write(which, at, g, gs)
    assert torch.equal(got.bytes, cache.bytes), "bytes beside the rows' own changed"
    if hq:
        want = ref.rotate(q.double().reshape(t, hq, head), a).reshape(t, -1)
        rows = [i for i in range(t) if slots[i] >= 0]
        left = [i for i in range(t) if slots[i] < 0]
        o = out.cpu()
        near(o[rows], want[rows], BF16, "q")
        if in_place:
            assert torch.equal(torch.nan_to_num(o[left]), torch.nan_to_num(q[left]))
            assert torch.equal(torch.nan_to_num(dx.cpu()[:, off + hq * head:]), torch.nan_to_num(x[:, off + hq * head:]))
        else:
            assert bool((o[left] == 77.0).all())
            assert bool((buf[0] == 77).all() and (buf[-1] == 77).all() and (buf[:, hq * head:] == 77).all())


def scattered(t, pages, page, seed):
    return random.Random(seed).sample(range(pages * page), t)


def run_of(t, first, pages, page, seed):
    """Slots of t consecutive positions from `first` on over pages in any order."""
    order = random.Random(seed).sample(range(pages), pages)
    return [order[p // page] * page + p % page for p in range(first, first + t)]


@pytest.mark.parametrize("xtype", [BF16, F32])
@pytest.mark.parametrize("ctype", [BF16, E4M3])
@pytest.mark.parametrize("head", [64, 128, 256])
@pytest.mark.parametrize("t,heads,g,page,rot", [(1, 1, 1, 16, 1), (3, 2, 3, 32, 2), (33, 3, 1, 16, 4), (70, 1, 7, 64, 1)])
def test_append(mep, t, heads, g, page, rot, head, ctype, xtype):
    rot = max(16, head // rot)
    pages = 300 // page + 4
    for slots in (scattered(t, pages, page, t), run_of(t, 0, pages, page, t), run_of(t, 5, pages, page, t)):
        check_append(mep, t, heads, head, page, ctype, xtype, rot, heads * g, slots, pages)


@pytest.mark.parametrize("ctype", [BF16, E4M3])
@pytest.mark.parametrize("head", [64, 128, 256])
def test_append_without_rotation_or_queries(mep, head, ctype):
    check_append(mep, 45, 2, head, 16, ctype, BF16, 0, 0, run_of(45, 9, 8, 16, 1), 8)
    check_append(mep, 45, 2, head, 16, ctype, F32, 32, 0, run_of(45, 8, 8, 16, 1), 8)


@pytest.mark.parametrize("ctype", [BF16, E4M3])
@pytest.mark.parametrize("head", [64, 128, 256])
def test_append_rows_without_a_slot(mep, head, ctype):
    """Padding rows, slots past the cache, and runs that they break."""
    slots = run_of(40, 0, 8, 16, 2)
    for i, s in ((0, -1), (9, 8 * 16), (17, 2 ** 31 - 1), (23, -2 ** 31), (39, -1)):
        slots[i] = s
    check_append(mep, 40, 2, head, 16, ctype, BF16, head, 4, slots, 8)
    check_append(mep, 7, 2, head, 16, ctype, BF16, head, 4, [-1] * 7, 8)


@pytest.mark.parametrize("ctype", [BF16, E4M3])
def test_append_positions(mep, ctype):
    """Far positions, and positions outside the table, which give NaN keys and queries and ordinary values."""
    pos = [0, 4999, 4998, 1, -1, 5000, 2 ** 31 - 1, -2 ** 31, 17, 2500]
    check_append(mep, 10, 2, 128, 32, ctype, BF16, 128, 6, scattered(10, 4, 32, 3), 4, positions=pos)
    check_append(mep, 10, 2, 128, 32, ctype, F32, 48, 6, scattered(10, 4, 32, 3), 4, positions=pos)


@pytest.mark.parametrize("ctype", [BF16, E4M3])
@pytest.mark.parametrize("head", [64, 256])
def test_append_values_not_finite(mep, head, ctype):
    def change(x):
        x[1, 3], x[2, 70], x[3, -1], x[4, -head] = torch.inf, -torch.inf, torch.nan, torch.inf
        x[5], x[6, 5:] = 0.0, 1e-39
        x[7] *= 1e30
        x[8, -3 * head:] = torch.inf

    check_append(mep, 12, 1, head, 16, ctype, BF16, 0, 0, run_of(12, 0, 2, 16, 1), 2, change=change)
    check_append(mep, 12, 1, head, 16, ctype, F32, 0, 0, run_of(12, 3, 2, 16, 1), 2, change=change)


def test_append_strides_and_in_place(mep):
    for xtype, in_place in ((BF16, True), (BF16, False), (F32, False)):
        check_append(mep, 19, 2, 64, 16, BF16, xtype, 64, 6, run_of(19, 1, 4, 16, 1), 4, stride=48, in_place=in_place)


def test_append_far_slots(mep):
    """Byte offsets past 32 bits."""
    pages, page, heads, head = 40000, 64, 8, 128
    L = mep.moe_kv_layout_make(pages, page, heads, head)
    assert L.v > 1 << 32
    cache = torch.empty(L.bytes, dtype=torch.uint8, device="cuda")
    slots = [pages * page - 1, 0, pages * page // 2 + 3, pages * page - 64]
    k, v = (torch.randn(4, heads * head, generator=torch.Generator().manual_seed(i)).to(BF16) for i in (1, 2))
    mep.moe_kv_append(k.cuda(), v.cuda(), L, cache, ints(slots).cuda())
    c = ref.Cache(1, page, heads, head, BF16)      # indices only, for a page at a time
    for which, x, at in (("k", k, 0), ("v", v, L.v)):
        for i, s in enumerate(slots):
            size = page * heads * head * 2
            part = cache[at + s // page * size:at + (s // page + 1) * size].cpu().view(BF16)
            assert torch.equal(part[c.index(which, [s % page])][0].reshape(-1), x[i])
