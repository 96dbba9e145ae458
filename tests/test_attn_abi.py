"""Host-side tests of the paged cache and its attention: layout, workspace and
refusals.  No GPU needed, no kernel is launched: every call here is refused by
its argument checks (the pointers are never dereferenced).
"""
import ctypes
import os

import pytest
import torch

import attn_ref as ref

mep = pytest.importorskip("mixture_experts_prefill_amd")

INVALID, CAPACITY, WORKSPACE = 1, 2, 3
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mep.LIB_PATH):
        from mixture_experts_prefill_amd import build

        build.build()
    return mep.lib()


@pytest.mark.parametrize("pages,page,heads,head,dtype", [(1, 16, 1, 64, BF16), (7, 32, 3, 128, E4M3), (100, 64, 8, 128, BF16),
                                                         (9, 256, 2, 256, E4M3), (1 << 22, 256, 1, 64, BF16),
                                                         (1 << 24, 64, 256, 256, E4M3)])
def test_layout(lib, pages, page, heads, head, dtype):
    L = mep.moe_kv_layout_make(pages, page, heads, head, dtype)
    size = 2 if dtype == BF16 else 1
    values = -(-pages * page * heads * head * size // 256) * 256
    scales = 0 if dtype == BF16 else -(-pages * page * heads // 256) * 256
    assert (L.pages, L.page, L.heads, L.head, L.type, L.k, L.v) == (pages, page, heads, head, 0 if size == 2 else 2, 0, values)
    assert (L.ks, L.vs) == ((0, 0) if size == 2 else (2 * values, 2 * values + scales))
    assert L.bytes == 2 * values + 2 * scales
    if pages <= 100:
        assert ref.Cache(pages, page, heads, head, dtype).bytes.numel() == L.bytes


@pytest.mark.parametrize("a", [(0, 16, 1, 64), (-1, 16, 1, 64), ((1 << 24) + 1, 16, 1, 64), (1 << 23, 256, 1, 64),
                               (4, 8, 1, 64), (4, 48, 1, 64), (4, 512, 1, 64), (4, 0, 1, 64), (4, 16, 0, 64),
                               (4, 16, 257, 64), (4, 16, 1, 32), (4, 16, 1, 96), (4, 16, 1, 512)])
def test_layout_refuses(lib, a):
    with pytest.raises(mep.MoeError) as e:
        mep.moe_kv_layout_make(*a)
    assert e.value.status == INVALID


def test_layout_refuses_other_types(lib):
    for dtype in (torch.float32, torch.float16, torch.uint8):
        with pytest.raises(mep.MoeError):
            mep.moe_kv_layout_make(4, 16, 1, 64, dtype)
    assert lib.moe_kv_layout_make(4, 16, 1, 64, 0, None) == INVALID


def test_workspace_bytes(lib):
    L = mep.moe_kv_layout_make(100, 64, 8, 128)
    size = lambda t, n, hq: mep.moe_attention_workspace_bytes(t, n, hq, L)
    for t, n, hq in [(0, 1, 8), (4097, 1, 8), (1, 0, 8), (1, 4097, 8), (1, 1, 0), (1, 1, 12), (1, 1, 1032)]:
        assert size(t, n, hq) == 0, (t, n, hq)
    bad = mep.moe_kv_layout_make(100, 64, 8, 128)
    bad.v += 256
    assert mep.moe_attention_workspace_bytes(1, 1, 8, bad) == 0
    assert lib.moe_attention_workspace_bytes(1, 1, 8, None) == 0
    for n in (1, 7, 64, 300, 4096):
        last = 0
        for t in (1, 31, 32, 33, 500, 4096):
            assert size(t, n, 32) >= last > -1     # more rows never need less
            last = size(t, n, 32)
    assert size(4096, 4096, 1024) < 1 << 31


# pointers that are never dereferenced: far apart, 256-byte aligned
BASE = 1 << 44
A, B, C, D, E, F, G, H, I, J, K = (BASE + i * (1 << 38) for i in range(11))
N, T, PAGES = 6, 10, 40


def layout(dtype=BF16):
    return mep.moe_kv_layout_make(PAGES, 32, 2, 64, dtype)


def other(L):
    L.bytes += 256
    return L


def call_plan(lib, **over):
    a = dict(length=A, grow=B, n=N, t=T, L=layout(), table=C, max_pages=9, ldt=9, free=D, free_n=E, length_out=F,
             free_n_out=G, starts=H, positions=I, slots=J, lacking=K)
    a.update(over)
    L = a.pop("L")
    v = list(a.values())
    return lib.moe_kv_plan(*v[:4], ctypes.byref(L) if L else None, *v[4:], None)


PLAN_BAD = [(dict(t=0), CAPACITY), (dict(t=4097), CAPACITY), (dict(n=0), CAPACITY), (dict(n=4097), CAPACITY),
            (dict(L=None), INVALID), (dict(L=other(layout())), INVALID), (dict(max_pages=0, ldt=9), INVALID),
            (dict(max_pages=(1 << 25) + 1, ldt=1 << 26), INVALID), (dict(ldt=8), INVALID), (dict(ldt=-9), INVALID),
            (dict(ldt=1 << 33), INVALID)]
PLAN_BAD += [({x: None}, INVALID) for x in ("length", "grow", "table", "free", "free_n", "length_out", "free_n_out",
                                            "starts", "positions", "slots", "lacking")]
PLAN_BAD += [({x: BASE + (1 << 43) + 2}, INVALID) for x in ("length", "grow", "table", "free", "free_n", "length_out",
                                                           "free_n_out", "starts", "positions", "slots", "lacking")]
PLAN_BAD += [(dict(length_out=A + 4), INVALID), (dict(length_out=B), INVALID), (dict(free_n_out=E - 4, length_out=E - 20), INVALID),
             (dict(starts=B + 4 * N - 4), INVALID), (dict(positions=J - 4 * T + 4), INVALID), (dict(slots=A), INVALID),
             (dict(lacking=G), INVALID), (dict(lacking=E), INVALID), (dict(table=D + 4 * PAGES - 4), INVALID),
             (dict(table=J - 4 * (9 * N - 1)), INVALID), (dict(free=C + 4 * (9 * N - 1)), INVALID),
             (dict(free_n_out=A), INVALID), (dict(starts=F - 4 * N), INVALID)]


@pytest.mark.parametrize("i", range(len(PLAN_BAD)))
def test_plan_refuses(lib, i):
    over, status = PLAN_BAD[i]
    assert call_plan(lib, **over) == status, over
    assert lib.moe_last_error()


def call_append(lib, **over):
    a = dict(k=A, ldk=128, v=B, ldv=128, xt=mep.BF16, t=T, L=layout(), cache=C, slots=D, positions=E, rope=F, rope_rows=100,
             rot=64, q=G, ldq=256, hq=4, q_out=H, ldqo=256)
    a.update(over)
    L = a.pop("L")
    v = list(a.values())
    return lib.moe_kv_append(*v[:6], ctypes.byref(L) if L else None, *v[6:], None)


QKV = dict(k=G + 512, ldk=512, v=G + 768, ldv=512, ldq=512)     # one projection's rows: q, k, v beside each other
APPEND_BAD = [(dict(t=0), CAPACITY), (dict(t=4097), CAPACITY), (dict(L=None), INVALID), (dict(L=other(layout())), INVALID),
              (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(cache=None), INVALID), (dict(slots=None), INVALID),
              (dict(xt=mep.E4M3), INVALID), (dict(xt=5), INVALID), (dict(ldk=127), INVALID), (dict(ldk=130), INVALID),
              (dict(ldv=120), INVALID), (dict(ldv=(1 << 22) + 8), INVALID), (dict(k=A + 8), INVALID), (dict(v=B + 2), INVALID),
              (dict(cache=C + 8), INVALID), (dict(slots=D + 1), INVALID), (dict(positions=E + 2), INVALID),
              (dict(rope=F + 8), INVALID), (dict(positions=None), INVALID), (dict(rope=None), INVALID), (dict(rot=0), INVALID),
              (dict(rope=None, positions=None), INVALID), (dict(rope=None, positions=None, rot=0), INVALID),  # q without rope
              (dict(rot=8), INVALID), (dict(rot=24), INVALID), (dict(rot=80), INVALID), (dict(rot=-16), INVALID),
              (dict(rope_rows=0), INVALID), (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(hq=0), INVALID),
              (dict(hq=3), INVALID), (dict(hq=-2), INVALID), (dict(hq=1026, ldq=70000, ldqo=70000), INVALID),
              (dict(ldq=250), INVALID), (dict(ldqo=252), INVALID), (dict(q=G + 8), INVALID), (dict(q_out=H + 4), INVALID),
              (dict(k=C), INVALID), (dict(v=C + 4096), INVALID), (dict(slots=C + 64), INVALID), (dict(rope=C + 64), INVALID),
              (dict(positions=C + 64), INVALID), (dict(q=C + 64), INVALID), (dict(q_out=C + 64), INVALID),
              (dict(q_out=A), INVALID), (dict(q_out=G + 512), INVALID), (dict(q_out=G, ldqo=264), INVALID),
              (dict(q_out=G, xt=mep.F32), INVALID), (dict(q_out=F + 128), INVALID),
              (dict(q_out=G + 512, ldqo=512, **QKV), INVALID)]


@pytest.mark.parametrize("i", range(len(APPEND_BAD)))
def test_append_refuses(lib, i):
    over, status = APPEND_BAD[i]
    assert call_append(lib, **over) == status, over


def call_attention(lib, prefill, **over):
    L = over.pop("L", layout())
    n = over.pop("n", N)
    a = dict(q=A, ldq=256, starts=B, t=T, n=n, hq=4)
    b = dict(cache=C, table=D, max_pages=9, ldt=9, length=E, scale=0.125, out=F, ldo=256, ws=G, ws_bytes=1 << 30)
    for d in (a, b):
        d.update({x: over.pop(x) for x in list(over) if x in d})
    assert not over
    f = lib.moe_attention_prefill if prefill else lib.moe_attention_decode
    return f(*a.values(), ctypes.byref(L) if L else None, *b.values(), None)


ATTENTION_BAD = [(dict(t=0), CAPACITY), (dict(t=4097), CAPACITY), (dict(n=0), CAPACITY), (dict(n=4097), CAPACITY),
                 (dict(L=None), INVALID), (dict(L=other(layout())), INVALID), (dict(q=None), INVALID), (dict(cache=None), INVALID),
                 (dict(table=None), INVALID), (dict(length=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID),
                 (dict(hq=0), INVALID), (dict(hq=5), INVALID), (dict(hq=-4), INVALID), (dict(hq=1026, ldq=70000, ldo=70000), INVALID),
                 (dict(max_pages=0), INVALID), (dict(max_pages=(1 << 25) + 1, ldt=1 << 26), INVALID), (dict(ldt=8), INVALID),
                 (dict(scale=0.0), INVALID), (dict(scale=1e-39), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
                 (dict(scale=float("inf")), INVALID), (dict(ldq=255), INVALID), (dict(ldq=260), INVALID), (dict(ldo=248), INVALID),
                 (dict(ldo=(1 << 22) + 8), INVALID), (dict(q=A + 8), INVALID), (dict(out=F + 4), INVALID),
                 (dict(cache=C + 8), INVALID), (dict(ws=G + 8), INVALID), (dict(table=D + 2), INVALID), (dict(length=E + 1), INVALID),
                 (dict(starts=B + 2), INVALID), (dict(ws_bytes=0), WORKSPACE), (dict(ws_bytes=1000), WORKSPACE),
                 (dict(out=A), INVALID), (dict(out=C + 256), INVALID), (dict(out=G + 256), INVALID), (dict(out=D), INVALID),
                 (dict(out=E), INVALID), (dict(out=B), INVALID), (dict(ws=A), INVALID), (dict(ws=C), INVALID), (dict(ws=D), INVALID),
                 (dict(ws=E), INVALID), (dict(ws=B), INVALID), (dict(out=A - T * 512 + 16), INVALID)]


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("i", range(len(ATTENTION_BAD)))
def test_attention_refuses(lib, prefill, i):
    over, status = ATTENTION_BAD[i]
    assert call_attention(lib, prefill, **over) == status, over
    assert lib.moe_last_error()


def test_attention_needs_starts(lib):
    assert call_attention(lib, True, starts=None) == INVALID
    assert call_attention(lib, False, starts=None) == INVALID       # t rows of n sequences, t != n


def test_workspace_is_what_was_said(lib):
    """One byte less than moe_attention_workspace_bytes is refused by at least one of the two calls it is for."""
    need = mep.moe_attention_workspace_bytes(T, N, 4, layout())
    assert WORKSPACE in [call_attention(lib, p, ws_bytes=need - 1) for p in (False, True)]


def test_python_refuses_before_the_library(lib):
    """Tensors off the GPU, of wrong shapes, types or strides never reach a kernel."""
    L = layout()
    row = torch.zeros(4, 128, dtype=BF16)
    ints = torch.zeros(4, dtype=torch.int32)
    cache = torch.zeros(L.bytes, dtype=torch.uint8)
    with pytest.raises(ValueError, match="one GPU"):
        mep.moe_kv_append(row, row, L, cache, ints)
    with pytest.raises(ValueError, match="one GPU"):
        mep.moe_attention_decode(row, L, cache, torch.zeros(4, 3, dtype=torch.int32), ints, 1.0, row, cache)
    with pytest.raises(ValueError, match="one GPU"):
        mep.moe_kv_plan(ints, ints, L, torch.zeros(4, 3, dtype=torch.int32), torch.zeros(PAGES, dtype=torch.int32), ints[:1],
                        ints, ints[:1], ints, ints, ints, ints[:1])
    with pytest.raises(ValueError, match="heads"):
        mep.moe_attention_decode(row[:, :100], L, cache, torch.zeros(4, 3, dtype=torch.int32), ints, 1.0, row, cache)
    for bad in (torch.zeros(4, 3), torch.zeros(3, 3, dtype=torch.int32), torch.zeros(4, 0, dtype=torch.int32),
                torch.zeros(4, dtype=torch.int32), torch.zeros(4, 6, dtype=torch.int32)[:, ::2],
                torch.zeros(1, 3, dtype=torch.int32).expand(4, 3)):
        with pytest.raises(ValueError):
            mep._table_args(bad, 4, -1)
    with pytest.raises(ValueError, match="int32"):
        mep._ints(ints.long(), 4, -1, "slots")
    with pytest.raises(ValueError, match="contiguous"):
        mep._ints(torch.zeros(8, dtype=torch.int32)[::2], 4, -1, "slots")
    with pytest.raises(ValueError, match="bytes"):
        mep._cache(cache[:-1], L, -1)
    with pytest.raises(ValueError, match="query heads"):
        mep.MoeCache(1, 4, 8, PAGES, 32, 2, 64, 3, 9, device="cpu")


def test_profile_phases(lib):
    assert mep.PHASES[12:14] == ["kv", "attention"]


def test_reference_plan():
    """The reference's own worked example: page size 16, sequence 0 finished, 1 gains a row in a new page, 2 starts."""
    table, free = [[5, 6, 0], [2, 0, 0], [0, 0, 0]], [9, 8, 7, 0, 0, 0, 0, 0, 0, 0]
    got = ref.plan([17, 16, 0], [-1, 1, 18], 16, 10, table, free, 3, 24)
    assert free[:5] == [9, 8, 7, 5, 6]
    assert table == [[5, 6, 0], [2, 6, 0], [5, 7, 0]]
    assert got["slots"] == [96] + list(range(80, 96)) + [112, 113] + [-1] * 5
    assert got["positions"] == [16] + list(range(18)) + [0] * 5
    assert (got["length_out"], got["starts"], got["free_n_out"], got["lacking"]) == ([0, 17, 18], [0, 0, 1, 19], [2], [0])
