"""A linear layer in 8-bit integers (W8A8) over the C ABI: an nn.Linear whose
weight is held as int8 codes with one scale per output channel, and whose
activations are quantized per token on the way in.

Beside Linear4bit: the 4-bit weights halve what decode has to read once more,
the 8-bit integer product runs prompts and large batches on the tensor cores'
8-bit rate without a dequantization step.  All compute is on the GPU; there is
no CPU path.
"""
from __future__ import annotations

import torch

from . import q4


class Linear8bit(torch.nn.Module):
    """y = x . W^T + b with W as (int8 codes [N, K], float32 scales [N])."""

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor, bias: torch.Tensor | None = None,
                 compute_dtype: torch.dtype = torch.float16):
        super().__init__()
        if compute_dtype not in (torch.float16, torch.bfloat16):
            raise q4.Q4Error("compute_dtype must be torch.float16 or torch.bfloat16")
        q4._check_codes("W", codes, scale)
        self.out_features, self.in_features = codes.shape
        why = unsupported_reason(self.in_features)
        if why:
            raise q4.Q4Error(f"Linear8bit cannot run this layer: {why}")
        self.compute_dtype = compute_dtype
        # the whole padded rows are the buffer: module copies and moves keep them
        rows, ld = codes.shape[0], (codes.shape[1] + 15) // 16 * 16
        if codes.stride(0) == ld and codes.storage_offset() + rows * ld <= codes.untyped_storage().nbytes():
            codes = codes.as_strided((rows, ld), (ld, 1))
        else:  # part of a wider buffer
            padded = codes.new_zeros(rows, ld)
            padded[:, :self.in_features] = codes
            codes = padded
        self.register_buffer("codes", codes)
        self.register_buffer("scale", scale)
        self.bias = None if bias is None else torch.nn.Parameter(bias.detach().to(compute_dtype), requires_grad=False)

    @classmethod
    def from_linear(cls, lin: torch.nn.Linear, compute_dtype: torch.dtype = torch.float16) -> "Linear8bit":
        """Quantize an nn.Linear's weight (on its CUDA device) once, at load time."""
        why = unsupported_reason(lin.in_features)
        if why:
            raise q4.Q4Error(f"Linear8bit cannot run this layer: {why}")
        w = lin.weight.detach()
        if w.dtype not in (torch.float16, torch.bfloat16):
            w = w.float()
        codes, scale = q4.int8_quantize_rows(w)
        return cls(codes, scale, lin.bias, compute_dtype)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.in_features:
            raise q4.Q4Error(f"expected last dimension {self.in_features}, got {x.shape[-1]}")
        a = x.reshape(-1, self.in_features).to(self.compute_dtype)
        bias = self.bias
        if bias is not None and bias.dtype == torch.float64:  # model.double()
            bias = bias.float()
        y = q4.int8_linear(a, self.codes[:, :self.in_features], self.scale, bias)
        return y.reshape(*x.shape[:-1], self.out_features)

    def _apply(self, fn, recurse=True):
        # moves apply to the codes and scales, casts (model.half()) to neither
        scale = self.scale
        super()._apply(fn, recurse)
        if self.scale.dtype != torch.float32:
            self.scale = scale.to(self.codes.device)
        return self

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, int8, "
                f"compute_dtype={self.compute_dtype}")


def unsupported_reason(in_features: int) -> str | None:
    """Why the 8-bit product cannot run a layer, or None when it can."""
    if not 1 <= in_features <= q4.INT8_MAX_K:
        return f"in_features {in_features} is not in 1 .. {q4.INT8_MAX_K}"
    return None
