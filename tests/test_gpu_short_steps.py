"""Steps of a paged cache that run out of pages or table entries: the rows that
got a slot attend from their own positions, the others are 0, and the step can
be planned again.
"""
import pytest
import torch

import attn_ref as ref
from test_gpu_attention import mep  # noqa: F401  (the fixture)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
HALF = dict(decode=2.0 ** -16, prefill=2.0 ** -8)


def ints(v):
    return torch.tensor(v, dtype=torch.int32)


class Server:
    """A MoeCache of one layer, and what each sequence's tokens were, by position."""

    def __init__(self, mep, n, rows, pages, page, heads, head, hq, max_pages, dtype):
        self.cache = mep.MoeCache(1, n, rows, pages, page, heads, head, hq, max_pages, dtype)
        self.cache.cache[0].fill_(0xff)
        self.n, self.pages, self.page, self.heads, self.head, self.hq, self.dtype = n, pages, page, heads, head, hq, dtype
        self.gen = torch.Generator().manual_seed(7 * n + head)
        self.length = [0] * n

    def step(self, grow, single=False, pad=2, **plan):
        """Plans, appends and attends; every row against the reference.  Returns the lacking rows and the outputs."""
        c, before = self.cache, self.length
        c.plan(ints(grow).cuda(), **plan)
        count = sum(max(g, 0) for g in grow)
        t = count + pad
        k, v = (torch.randn(t, self.heads * self.head, generator=self.gen).to(BF16) for _ in range(2))
        q = (1.5 * torch.randn(t, self.hq * self.head, generator=self.gen)).to(BF16)
        c.append(0, k.cuda(), v.cuda())
        out = c.attend(0, q.cuda(), single=single)
        torch.cuda.synchronize()
        held = ref.Cache(self.pages, self.page, self.heads, self.head, self.dtype)
        held.bytes.copy_(c.cache[0].cpu())
        table, length, slots = c.table.cpu().tolist(), c.length.tolist(), c.slots.tolist()
        row = lacking = 0
        for s, g in enumerate(grow):
            old = 0 if g < 0 else before[s]
            m = max(g, 0)
            placed = sum(slots[row + i] >= 0 for i in range(m))
            lacking += m - placed
            assert length[s] == old + placed
            where = [table[s][p // self.page] * self.page + p % self.page for p in range(length[s])]
            assert slots[row:row + placed] == where[old:]
            if placed:
                K, V = held.read("k", where), held.read("v", where)
                kind = "decode" if single else "prefill"
                o, err, var = ref.attention(q[row:row + placed].double().view(placed, self.hq, self.head), K, V,
                                            [old + i for i in range(placed)], self.head ** -0.5, HALF[kind])
                ref.check_attention(out[row:row + placed], o, err, var, f"{kind} sequence {s}: {placed} of {m} after {old}")
            assert bool((out[row + placed:row + m] == 0).all()), f"rows of sequence {s} without a slot"
            row += m
        assert bool((out[row:] == 0).all()) and c.lacking.item() == lacking
        self.length = length
        return lacking, out


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("heads,g,head", [(2, 3, 64), (1, 8, 128), (1, 2, 256)])
def test_rows_that_have_pages(mep, heads, g, head, dtype):
    """14 rows of one sequence, one of another and all of a third lack pages; a whole sequence beside them."""
    srv = Server(mep, 4, 200, 9, 16, heads, head, heads * g, 8, dtype)
    assert srv.step([20, 5, 0, 31])[0] == 0                       # 2 + 1 + 0 + 2 pages of 9
    assert srv.step([90, 12, 16, 1])[0] == 14 + 1 + 16             # the first gets four pages of five
    assert srv.step([0, -1, 0, 40])[0] == 40 - 16                  # a page comes back


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_rows_of_long_sequences_that_are_cut(mep, dtype):
    """Tiles of several parts and both kinds of joining, with rows past the last page in the middle of a tile."""
    for hq, rows in ((2, 70), (16, 400)):
        srv = Server(mep, 2, 2100, 65, 32, 1, 128, hq, 70, dtype)
        assert srv.step([1990, 20])[0] == 0                        # 63 pages and 1
        assert srv.step([rows, 8])[0] == rows - 26 - 32            # 26 rows in the last page, and one page more


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("head", [64, 128, 256])
def test_single_rows(mep, head, dtype):
    """A row that has no page is 0, and not attention over the tokens before it."""
    srv = Server(mep, 3, 2000, 5, 16, 2, head, 6, 60, dtype)
    assert srv.step([16, 32, 15])[0] == 0
    assert srv.step([1, 1, 1], single=True)[0] == 1
    srv = Server(mep, 2, 2100, 128, 16, 2, head, 6, 100, dtype)    # cut along the tokens
    assert srv.step([1600, 440])[0] == 0
    assert srv.step([1, 1], single=True)[0] == 1                   # the table of the first is full


def test_many_sequences(mep):
    srv = Server(mep, 90, 600, 40, 16, 1, 64, 2, 4, BF16)
    assert srv.step([1 + s % 7 for s in range(90)])[0] > 0
    assert srv.step([s % 3 for s in range(90)])[0] > 0
    assert srv.step([1] * 90, single=True)[0] > 0


@pytest.mark.parametrize("single", [True, False])
def test_before_of_a_whole_step_changes_nothing(mep, single):
    """The same bits with and without the lengths before the step, where every row has a slot."""
    n, hq, head = 5, 4, 64
    L = mep.moe_kv_layout_make(40, 64, 2, head)
    gen = torch.Generator().manual_seed(2)
    cache = torch.randn(L.bytes // 2, generator=gen).to(BF16).view(torch.uint8).cuda()
    table = ints([[7 * s + i for i in range(8)] for s in range(n)]).cuda()
    rows = [1] * n if single else [3, 130, 0, 1, 40]
    length = [500, 300, 17, 1, 40]
    starts = ints([sum(rows[:s]) for s in range(n + 1)]).cuda()
    q = torch.randn(sum(rows), hq * head, generator=gen).to(BF16).cuda()
    ws = torch.empty(mep.moe_attention_workspace_bytes(sum(rows), n, hq, L), dtype=torch.uint8, device="cuda")
    outs = []
    for before in (None, ints([a - b for a, b in zip(length, rows)]).cuda()):
        out = torch.empty_like(q)
        if single:
            mep.moe_attention_decode(q, L, cache, table, ints(length).cuda(), 0.125, out, ws, before=before)
        else:
            mep.moe_attention_prefill(q, starts, L, cache, table, ints(length).cuda(), 0.125, out, ws, before=before)
        outs.append(out)
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("single", [True, False])
def test_lengths_before_out_of_range(mep, single):
    """They count as the nearest of 0 .. max_pages * page; rows that so have no slot are 0, and nothing faults."""
    n, hq, head, rows = 4, 2, 64, 3
    L = mep.moe_kv_layout_make(8, 16, 1, head)
    cache = torch.zeros(L.bytes, dtype=torch.uint8, device="cuda")
    cache.view(BF16)[L.v // 2:] = 1.0
    table = ints([[0, 1]] * n).cuda()
    q = torch.ones(n * rows, hq * head, dtype=BF16, device="cuda")
    starts = ints([rows * s for s in range(n + 1)]).cuda()
    ws = torch.empty(mep.moe_attention_workspace_bytes(n * rows, n, hq, L), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 77.0)
    length, before = ints([20, 32, 1, 10]).cuda(), ints([2 ** 31 - 1, 100, -2 ** 31, 9]).cuda()
    if single:
        mep.moe_attention_decode(q, L, cache, table, length, 0.125, out, ws, starts=starts, before=before)
        there = {8: 0, 2: 0, 5: 0, 11: 0}                          # position 2 of 1 token, 32 and more of 20 and 32, 11 of 10
    else:
        mep.moe_attention_prefill(q, starts, L, cache, table, length, 0.125, out, ws, before=before)
        there = {**{r: 0 for r in range(12)}, 6: 1, 9: 1}          # position 0 of 1 token, 9 of 10
    torch.cuda.synchronize()
    for r in range(n * rows):
        assert bool((out[r] == there.get(r, 77.0)).all()), r


def test_planned_again(mep):
    """The step that lacked pages is planned again with fewer rows, or with a sequence ended, and then holds."""
    for again in ([60, 11, 0, 1], [64, 12, -1, 1], [4, 0, 0, 0], [0, 0, 0, 0]):
        srv = Server(mep, 4, 200, 10, 16, 2, 64, 6, 8, BF16)
        assert srv.step([20, 5, 16, 31])[0] == 0                   # 2 + 1 + 1 + 2 pages
        first, pages = list(srv.length), srv.cache.free_n.item()
        assert srv.step([90, 12, 16, 1])[0] > 0
        srv.length = first
        assert srv.step(again, again=True)[0] == 0
        assert srv.cache.length.tolist() == [0 if g < 0 else a + g for a, g in zip(first, again)]
        up = lambda x: -(-x // 16)
        assert srv.cache.free_n.item() == pages + sum(up(a) for a in first) - sum(up(x) for x in srv.length)
        srv.step([1, 1, 1, 1], single=True)                        # the next step starts where this one ended


def test_first_step_planned_again(mep):
    srv = Server(mep, 2, 100, 3, 16, 1, 64, 2, 4, BF16)
    assert srv.step([40, 20])[0] == 20
    srv.length = [0, 0]
    assert srv.step([30, 16], again=True)[0] == 0
    assert srv.cache.free_n.item() == 0


def test_replayed_steps_advance(mep):
    """A captured plan with its attention: each replay is the next step, also after one that lacked pages."""
    page, pages, n, rows = 16, 6, 2, 24
    c = mep.MoeCache(1, n, rows, pages, page, 1, 64, 1, 8)
    grow = ints([20, 4]).cuda()
    k = torch.randn(rows, 64, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    out = torch.empty(rows, 64, dtype=BF16, device="cuda")

    def call():
        c.plan(grow)
        c.append(0, k, k)
        c.attend(0, k, out=out)

    def again():
        c.length.zero_()
        c.free_n.fill_(pages)
        c.free_pages.copy_(torch.arange(pages - 1, -1, -1, dtype=torch.int32))

    call()
    torch.cuda.synchronize()
    again()
    eager = []
    for _ in range(6):
        call()
        eager.append((out.clone(), c.length.clone(), c.lacking.clone(), c.free_n.clone()))
    assert [x[2].item() for x in eager] == [0, 0, 0, 0, 24, 24]     # 80 tokens and 16 fill the six pages
    again()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call()
    for want in eager:
        g.replay()
        (torch.randn(1000, device="cuda") ** 2).sum().item()
        got = (out, c.length, c.lacking, c.free_n)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
