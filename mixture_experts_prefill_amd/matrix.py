"""One 4-bit matrix on the device, and the projections that read it.

Owns the record (the tiled bytes that ``moe_linear`` and ``moe_linear_gated``
read, laid out once when weights are loaded) and its layout.  Only the byte
layout and output allocation live here; the arithmetic is in libmoe.
"""
from __future__ import annotations

import contextlib
from typing import Optional

import torch

from . import moe_linear, moe_linear_gated, moe_matrix_layout_make


def _allocating_on(stream, device: torch.device):
    """A context whose allocations belong to the stream that the kernel runs on
    (memory of the current stream's pool may still be written by what is queued there)."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


class MoeMatrix:
    def __init__(self, n: int, k: int, group: int, record: torch.Tensor):
        """A matrix whose record exists already (at least layout.bytes bytes)."""
        self.layout = moe_matrix_layout_make(n, k, group)
        self.n, self.k, self.group = n, k, group
        if record.dtype != torch.uint8 or not record.is_contiguous() or record.numel() < self.layout.bytes:
            raise ValueError(f"record must be {self.layout.bytes} contiguous uint8 values")
        self.record = record

    @classmethod
    def from_codes(cls, codes: torch.Tensor, scale: torch.Tensor, bias: torch.Tensor, group: int) -> "MoeMatrix":
        """codes uint8 [n, k] (0..15), scale and bias fp16 [n, k/group]:
        W[j, i] = scale[j, i/group] * codes[j, i] + bias[j, i/group]."""
        n, k = codes.shape
        layout = moe_matrix_layout_make(n, k, group)
        if codes.dtype != torch.uint8 or (codes.numel() and int(codes.max()) > 15):
            raise ValueError("codes must be uint8 values 0..15")
        for v in (scale, bias):
            if v.dtype != torch.float16 or tuple(v.shape) != (n, k // group):
                raise ValueError(f"scale and bias must be float16 [{n}, {k // group}]")
        pad = -n % 32
        q = torch.nn.functional.pad(codes, (0, 0, 0, pad))
        sb = torch.nn.functional.pad(torch.stack([scale, bias], -1), (0, 0, 0, 0, 0, pad))
        rows = n + pad
        v = q.view(rows // 32, 32, k // 64, 2, 4, 8)
        word = v[..., 0].int()
        for j in range(1, 8):
            word |= v[..., j].int() << (4 * (j // 2) + 16 * (j % 2))
        record = torch.zeros(layout.bytes, dtype=torch.uint8, device=codes.device)
        w = word.permute(0, 2, 3, 1, 4).contiguous().view(torch.uint8).view(-1)
        record[layout.w: layout.w + w.numel()] = w
        e = sb.view(rows // 32, 32, k // 64, 64 // group, 2).permute(0, 2, 3, 1, 4).contiguous().view(torch.uint8)
        record[layout.sb: layout.sb + e.numel()] = e.view(-1)
        return cls(n, k, group, record)

    def linear(self, x: torch.Tensor, x_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               out_dtype: torch.dtype = torch.bfloat16, accumulate: int = 0, stream=None) -> torch.Tensor:
        """x times this matrix (moe_linear), into `out` or a new tensor, which is
        `stream`'s like any tensor allocated on it."""
        if out is None:
            if accumulate:
                raise ValueError("accumulate adds into a given out")
            with _allocating_on(stream, x.device):
                out = torch.empty((x.shape[0], self.n), dtype=out_dtype, device=x.device)
        moe_linear(x, self.layout, self.record, out, x_scale, accumulate, stream)
        return out

    def gated(self, up: "MoeMatrix", x: torch.Tensor, x_scale: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, out_scale: Optional[torch.Tensor] = None,
              out_dtype: torch.dtype = torch.bfloat16, stream=None):
        """silu(x times this matrix) * (x times `up`) (moe_linear_gated); with
        8-bit output returns (codes, scale).  New tensors are `stream`'s."""
        if (up.n, up.k, up.group) != (self.n, self.k, self.group):
            raise ValueError("gate and up must have the same shape and group")
        if out is None or (out.dtype == torch.float8_e4m3fn and out_scale is None):
            with _allocating_on(stream, x.device):
                if out is None:
                    out = torch.empty((x.shape[0], self.n), dtype=out_dtype, device=x.device)
                if out.dtype == torch.float8_e4m3fn and out_scale is None:
                    out_scale = torch.empty((x.shape[0], self.n // 32), dtype=torch.uint8, device=x.device)
        moe_linear_gated(x, self.layout, self.record, up.record, out, x_scale, out_scale, stream)
        return out if out_scale is None else (out, out_scale)
