"""Refusals of the forms that are told the lengths before a step.  No GPU
needed, no kernel is launched.
"""
import ctypes

import pytest

from test_attn_abi import (A, B, BASE, C, CAPACITY, D, E, F, G, H, I, INVALID, J, K, N, PAGES, T, WORKSPACE, layout,  # noqa: F401
                           lib, other)


def call_plan(lib, **over):  # noqa: F811
    a = dict(length=A, grow=B, n=N, t=T, L=layout(), table=C, max_pages=9, ldt=9, free=D, free_n=E, before=F, again=0,
             starts=H, positions=I, slots=J, lacking=K)
    a.update(over)
    L = a.pop("L")
    v = list(a.values())
    return lib.moe_kv_plan_step(*v[:4], ctypes.byref(L) if L else None, *v[4:], None)


POINTERS = ("length", "grow", "table", "free", "free_n", "before", "starts", "positions", "slots", "lacking")
PLAN_BAD = [(dict(t=0), CAPACITY), (dict(n=4097), CAPACITY), (dict(L=None), INVALID), (dict(L=other(layout())), INVALID),
            (dict(max_pages=0, ldt=9), INVALID), (dict(ldt=8), INVALID)]
PLAN_BAD += [({x: None}, INVALID) for x in POINTERS] + [({x: BASE + (1 << 43) + 2}, INVALID) for x in POINTERS]
PLAN_BAD += [(dict(before=A), INVALID), (dict(before=A - 4 * N), INVALID), (dict(before=E - 4 * N), INVALID),
             (dict(before=B + 4), INVALID), (dict(before=C + 4), INVALID), (dict(before=D), INVALID), (dict(before=H), INVALID),
             (dict(before=I), INVALID), (dict(before=J), INVALID), (dict(before=K - 4 * N), INVALID),
             (dict(length=B), INVALID), (dict(free_n=A), INVALID)]


@pytest.mark.parametrize("again", [0, 1])
@pytest.mark.parametrize("i", range(len(PLAN_BAD)))
def test_plan_refuses(lib, i, again):  # noqa: F811
    over, status = PLAN_BAD[i]
    assert call_plan(lib, again=again, **over) == status, over


def call_attention(lib, prefill, **over):  # noqa: F811
    a = dict(q=A, ldq=256, starts=B, t=T, n=N, hq=4, L=layout(), cache=C, table=D, max_pages=9, ldt=9, length=E, before=H,
             scale=0.125, out=F, ldo=256, ws=G, ws_bytes=1 << 30)
    a.update(over)
    L = a.pop("L")
    v = list(a.values())
    f = lib.moe_attention_prefill_step if prefill else lib.moe_attention_decode_step
    return f(*v[:6], ctypes.byref(L) if L else None, *v[6:], None)


ATTENTION_BAD = [(dict(before=None), INVALID), (dict(before=H + 2), INVALID), (dict(before=F), INVALID),
                 (dict(before=G + 64), INVALID), (dict(length=None), INVALID), (dict(t=0), CAPACITY), (dict(n=0), CAPACITY),
                 (dict(L=other(layout())), INVALID), (dict(scale=0.0), INVALID), (dict(ws_bytes=1000), WORKSPACE),
                 (dict(out=A), INVALID), (dict(ldq=255), INVALID)]


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("i", range(len(ATTENTION_BAD)))
def test_attention_refuses(lib, prefill, i):  # noqa: F811
    over, status = ATTENTION_BAD[i]
    assert call_attention(lib, prefill, **over) == status, over
