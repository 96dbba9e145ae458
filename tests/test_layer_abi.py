"""Host-side tests of the layer operators: layout, packing and refusals.  No
GPU needed, no kernel is launched: every call here is refused by its argument
checks (the pointers are never dereferenced).
"""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import layer_ref as ref
import moe_synth as ms

mep = pytest.importorskip("mixture_experts_prefill_amd")

INVALID, CAPACITY = 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mep.LIB_PATH):
        from mixture_experts_prefill_amd import build

        build.build()
    return mep.lib()


def test_matrix_layout(lib):
    for n, k, group in [(1, 64, 64), (32, 64, 32), (100003, 2048, 64), (1 << 24, 64, 32), (96, 65536, 64)]:
        m = mep.moe_matrix_layout_make(n, k, group)
        rows = -(-n // 32) * 32
        assert (m.n, m.k, m.group, m.w) == (n, k, group, 0)
        assert m.sb % 256 == 0 and m.sb >= rows * k // 2
        assert m.bytes % 256 == 0 and m.bytes >= m.sb + rows * (k // group) * 4 and m.bytes < m.sb + rows * (k // group) * 4 + 256


@pytest.mark.parametrize("n,k,group", [(0, 64, 64), (-5, 64, 64), ((1 << 24) + 1, 64, 64), (32, 0, 64), (32, 96, 32),
                                       (32, 65600, 64), (32, 64, 16), (32, 64, 128)])
def test_matrix_layout_refuses(lib, n, k, group):
    with pytest.raises(mep.MoeError) as e:
        mep.moe_matrix_layout_make(n, k, group)
    assert e.value.status == INVALID


@pytest.mark.parametrize("n,k,group", [(32, 64, 64), (32, 128, 32), (96, 192, 64), (33, 64, 32), (70, 256, 64)])
def test_from_codes_packs_as_the_record_format_says(lib, n, k, group):
    m = ref.Matrix(n, k, group)
    rec = mep.MoeMatrix.from_codes(m.q, m.s, m.b, group)
    pad = -n % 32
    q = np.pad(m.q.numpy(), ((0, pad), (0, 0)))
    s, b = (np.pad(v.numpy(), ((0, pad), (0, 0))) for v in (m.s, m.b))
    L = rec.layout
    codes, sb = ms.pack_codes(q), ms.pack_sb(s, b, group)
    got = rec.record.numpy()
    assert got.size == L.bytes
    assert np.array_equal(got[L.w: L.w + codes.size], codes)
    assert np.array_equal(got[L.sb: L.sb + sb.size], sb)


def test_from_codes_refuses(lib):
    m = ref.Matrix(32, 64, 64)
    with pytest.raises(ValueError):
        mep.MoeMatrix.from_codes(m.q + 16, m.s, m.b, 64)
    with pytest.raises(ValueError):
        mep.MoeMatrix.from_codes(m.q, m.s.float(), m.b, 64)
    with pytest.raises(ValueError):
        mep.MoeMatrix.from_codes(m.q, m.s, m.b[:, :0], 64)
    with pytest.raises(ValueError):
        mep.MoeMatrix(32, 64, 64, torch.zeros(100, dtype=torch.uint8))


# pointers that are never dereferenced: far apart, 256-byte aligned
BASE = 1 << 44
X, XS, REC, REC2, OUT, OS = (BASE + i * (1 << 38) for i in range(6))


def call_linear(lib, **over):
    a = dict(x=X, x_type=mep.BF16, ldx=256, xs=None, xsk=0, t=4, M=mep.moe_matrix_layout_make(96, 256, 64), rec=REC,
             out=OUT, out_type=mep.F32, ldo=96)
    a.update(over)
    M = a["M"]
    return lib.moe_linear(a["x"], a["x_type"], a["ldx"], a["xs"], a["xsk"], a["t"], ctypes.byref(M) if M else None,
                          a["rec"], a["out"], a["out_type"], a["ldo"], 0, None)


def bad_layout():
    m = mep.moe_matrix_layout_make(96, 256, 64)
    m.sb += 256
    return m


LINEAR_BAD = [
    (dict(t=0), CAPACITY), (dict(t=-1), CAPACITY), (dict(t=4097), CAPACITY), (dict(M=None), INVALID),
    (dict(x=None), INVALID), (dict(rec=None), INVALID), (dict(out=None), INVALID),
    (dict(x_type=mep.F32), INVALID), (dict(x_type=7), INVALID), (dict(out_type=mep.E4M3), INVALID),
    (dict(out_type=-1), INVALID), (dict(ldx=255), INVALID), (dict(ldx=260), INVALID), (dict(ldx=-256), INVALID),
    (dict(x=X + 8), INVALID), (dict(rec=REC + 4), INVALID), (dict(ldo=95), INVALID), (dict(out=OUT + 2), INVALID),
    (dict(ldo=1 << 41), INVALID), (dict(ldx=(1 << 22) + 8), INVALID), (dict(xsk=1, xs=XS), INVALID),                     # bf16 rows have no scales
    (dict(x_type=mep.E4M3, xsk=3, xs=XS), INVALID), (dict(x_type=mep.E4M3, xsk=1), INVALID),
    (dict(x_type=mep.E4M3, xsk=1, xs=XS + 2), INVALID), (dict(x_type=mep.E4M3, ldx=264), INVALID),
    (dict(out=X), INVALID), (dict(out=X + 3 * 512 + 508), INVALID), (dict(out=X - 4 * 96 * 4 + 4), INVALID),
    (dict(out=REC + 4096), INVALID), (dict(x_type=mep.E4M3, xsk=2, xs=OUT + 32), INVALID),
]


@pytest.mark.parametrize("i", range(len(LINEAR_BAD)))
def test_linear_refuses(lib, i):
    over, status = LINEAR_BAD[i]
    assert call_linear(lib, **over) == status, over
    assert lib.moe_last_error()


def test_linear_refuses_other_layouts(lib):
    assert call_linear(lib, M=bad_layout()) == INVALID


def call_gated(lib, **over):
    a = dict(x=X, t=4, M=mep.moe_matrix_layout_make(96, 256, 64), gate=REC, up=REC2, out=OUT, out_type=mep.E4M3, ldo=96,
             os=OS)
    a.update(over)
    M = a["M"]
    return lib.moe_linear_gated(a["x"], mep.BF16, 256, None, 0, a["t"], ctypes.byref(M) if M else None, a["gate"],
                                a["up"], a["out"], a["out_type"], a["ldo"], a["os"], None)


GATED_BAD = [
    (dict(t=0), CAPACITY), (dict(M=None), INVALID), (dict(gate=None), INVALID), (dict(up=None), INVALID),
    (dict(up=REC2 + 8), INVALID), (dict(os=None), INVALID), (dict(out_type=mep.BF16), INVALID),
    (dict(out_type=9, os=None), INVALID), (dict(os=OUT + 10), INVALID), (dict(os=X + 100), INVALID),
    (dict(out=REC2 + 64), INVALID), (dict(os=REC + 64), INVALID), (dict(ldo=64), INVALID),
]


@pytest.mark.parametrize("i", range(len(GATED_BAD)))
def test_gated_refuses(lib, i):
    over, status = GATED_BAD[i]
    assert call_gated(lib, **over) == status, over


def test_gated_refuses_a_partial_block_in_8_bits(lib):
    assert call_gated(lib, M=mep.moe_matrix_layout_make(80, 256, 64)) == INVALID


def call_norm(lib, **over):
    a = dict(x=X, x_type=mep.BF16, ldx=256, res=REC, res_out=REC, res_type=mep.F32, ldr=256, gamma=REC2, eps=1e-6, t=4,
             h=256, out=OUT, ldo=256, codes=OS, ldc=256, scale=XS, kind=mep.SCALE_BLOCK)
    a.update(over)
    return lib.moe_residual_norm(a["x"], a["x_type"], a["ldx"], a["res"], a["res_out"], a["res_type"], a["ldr"],
                                 a["gamma"], a["eps"], a["t"], a["h"], a["out"], a["ldo"], a["codes"], a["ldc"],
                                 a["scale"], a["kind"], None)


NORM_BAD = [
    (dict(t=0), CAPACITY), (dict(t=4097), CAPACITY), (dict(h=0), INVALID), (dict(h=240), INVALID),
    (dict(h=16416, ldx=16416, ldr=16416, ldo=16416, ldc=16416), INVALID), (dict(x=None), INVALID),
    (dict(gamma=None), INVALID), (dict(gamma=REC2 + 4), INVALID), (dict(out=None, codes=None), INVALID),
    (dict(x_type=mep.E4M3), INVALID), (dict(res_type=mep.E4M3), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(res=None), INVALID),
    (dict(ldx=248), INVALID), (dict(ldx=257), INVALID), (dict(ldr=254), INVALID), (dict(ldo=250), INVALID),
    (dict(ldc=264), INVALID), (dict(x=X + 8), INVALID), (dict(codes=OS + 8), INVALID), (dict(scale=None), INVALID),
    (dict(kind=0), INVALID), (dict(kind=mep.SCALE_ROW, scale=XS + 2), INVALID), (dict(out=X), INVALID),
    (dict(res_out=REC + 1024), INVALID), (dict(codes=OUT + 1024), INVALID), (dict(scale=OUT + 16), INVALID),
    (dict(out=REC2 + 512), INVALID), (dict(res_out=X), INVALID),
]


@pytest.mark.parametrize("i", range(len(NORM_BAD)))
def test_norm_refuses(lib, i):
    over, status = NORM_BAD[i]
    assert call_norm(lib, **over) == status, over


def test_python_refuses_before_the_library(lib):
    """Tensors off the GPU, of wrong shapes, types or strides never reach a kernel."""
    m = ref.Matrix(32, 64, 64)
    dm = mep.MoeMatrix.from_codes(m.q, m.s, m.b, 64)
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="one GPU"):
        dm.linear(x)
    with pytest.raises(ValueError, match="one GPU"):
        dm.gated(dm, x)
    with pytest.raises(ValueError, match="one GPU"):
        mep.moe_residual_norm(x, torch.ones(64), 1e-6, out=torch.empty_like(x))
    with pytest.raises(ValueError):
        dm.linear(x, accumulate=1)
    with pytest.raises(ValueError, match="same shape"):
        dm.gated(mep.MoeMatrix.from_codes(*[torch.cat([v, v]) for v in (m.q, m.s, m.b)], 64), x)
    for bad, what in [(x[:, :32], "must be"), (x.half(), "bfloat16"), (x.t(), "must be"),
                      (torch.zeros(64, 2).t(), "contiguous"), (torch.zeros(1, 64).expand(2, 64), "overlap")]:
        with pytest.raises(ValueError, match=what):
            mep._row_args(bad, 2, 64, 0, "x")
    for bad in (torch.zeros(3), torch.zeros(2, 2, dtype=torch.float16), torch.zeros(2, 4, dtype=torch.uint8)[:, ::2]):
        with pytest.raises(ValueError):
            mep._scale_args(bad, 2, 64, 0, "scale")


def test_profile_phases_are_the_librarys(lib):
    """moe_profile_end writes as many entries as the binding has names (a shorter
    list would make it write past the binding's arrays), in the header's order."""
    total, launches = np.full(64, -1.0), np.full(64, -1, np.int64)
    assert lib.moe_profile_end(total.ctypes.data, launches.ctypes.data) == 0
    assert int((total == 0).sum()) == int((launches == 0).sum()) == len(mep.PHASES)
    with open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "include", "moe_debug.h")) as f:
        header = dict(re.findall(r"MOE_PHASE_?(\w+) = (\d+)", f.read()))
    assert int(header.pop("S")) == len(mep.PHASES) == len(header)
    assert mep.PHASES[int(header["LINEAR"])] == "linear"
