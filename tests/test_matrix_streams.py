"""MoeMatrix's new outputs belong to the stream that the kernel runs on: memory
of another stream's pool may still be written by what is queued there."""
import contextlib

import pytest
import torch

import layer_ref as ref

mep = pytest.importorskip("mixture_experts_prefill_amd")
matrix = mep.matrix


@pytest.fixture
def recorded(monkeypatch):
    """The handle of the stream that is current at every torch.empty of matrix.py; no launch."""
    current, seen = [None], []

    @contextlib.contextmanager
    def on(stream):
        before, current[0] = current[0], stream
        yield
        current[0] = before

    def empty(shape, **kw):
        seen.append((current[0], kw["dtype"]))
        return real(shape, dtype=kw["dtype"])

    real = torch.empty
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(matrix, "moe_linear", lambda *a: None)
    monkeypatch.setattr(matrix, "moe_linear_gated", lambda *a: None)
    return seen


def test_new_outputs_are_allocated_on_the_launch_stream(recorded):
    m = ref.Matrix(32, 64, 64)
    dm = mep.MoeMatrix.from_codes(m.q, m.s, m.b, 64)
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    recorded.clear()
    dm.linear(x)
    dm.gated(dm, x, out_dtype=torch.float8_e4m3fn)
    assert recorded == [(None, torch.bfloat16), (None, torch.float8_e4m3fn), (None, torch.uint8)]
    recorded.clear()
    side = ("external", 77)
    dm.linear(x, stream=77)
    dm.gated(dm, x, stream=77)
    dm.gated(dm, x, out_dtype=torch.float8_e4m3fn, stream=77)
    dm.gated(dm, x, out=torch.zeros(2, 32).to(torch.float8_e4m3fn), stream=77)
    assert recorded == [(side, torch.bfloat16), (side, torch.bfloat16), (side, torch.float8_e4m3fn), (side, torch.uint8),
                        (side, torch.uint8)]


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")
@pytest.mark.parametrize("raw", [False, True])
def test_new_outputs_are_in_the_launch_streams_pool(raw):
    m = ref.Matrix(96, 256, 64)
    dm = mep.MoeMatrix.from_codes(m.q.cuda(), m.s.cuda(), m.b.cuda(), 64)
    x = torch.randn(5, 256, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    want = [dm.linear(x), *dm.gated(dm, x, out_dtype=torch.float8_e4m3fn)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    stream = side.cuda_stream if raw else side
    got = [dm.linear(x, stream=stream), *dm.gated(dm, x, out_dtype=torch.float8_e4m3fn, stream=stream)]
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        owner = [s["stream"] for s in torch.cuda.memory_snapshot()
                 if s["address"] <= a.data_ptr() < s["address"] + s["total_size"]]
        assert owner == [side.cuda_stream]
    assert torch.cuda.current_stream() != side
    assert torch.equal(dm.linear(x, stream=0).view(torch.uint8), want[0].view(torch.uint8))   # the default stream's handle
