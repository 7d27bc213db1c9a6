"""The serving operators without a GPU: refusals at the borders of their ranges."""
import pytest
import torch

from bit_blockwise_weight_absmax_b200 import q4
from test_int8_cpu import ALIGN, ARG, NO_DEVICE, SHAPE, A, lib  # noqa: F401  (lib: the fixture)


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers: only where nothing can be launched")
def test_float32_rows_are_refused_like_16_bit_ones(lib):
    def quant(X=A, rows=4, cols=64, ldx=64, codes=A, ldc=64, scale=A):
        return lib.q4_int8_quantize_rows_f32(X, rows, cols, ldx, codes, ldc, scale, None)

    assert quant() == NO_DEVICE
    for kw, rc in [(dict(X=None), ARG), (dict(codes=None), ARG), (dict(scale=None), ARG), (dict(rows=0), SHAPE),
                   (dict(cols=0), SHAPE), (dict(cols=131072, ldx=131072, ldc=131072), SHAPE), (dict(ldx=63), SHAPE),
                   (dict(ldc=48), SHAPE), (dict(ldc=72), SHAPE), (dict(codes=A + 8), ALIGN), (dict(X=A + 2), ALIGN)]:
        assert quant(**kw) == rc, kw


def test_other_types_are_refused():
    for dtype in (torch.float64, torch.int8):
        with pytest.raises(q4.Q4Error, match="float32"):
            q4.int8_quantize_rows(torch.zeros(2, 64, dtype=dtype))
