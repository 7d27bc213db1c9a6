"""The serving operators without a GPU: refusals at the borders of their ranges."""
import ctypes

import pytest
import torch

from bit_blockwise_weight_absmax_b200 import linear8bit, q4
from test_int8_cpu import ALIGN, ARG, NO_DEVICE, SHAPE, A, lib  # noqa: F401  (lib: the fixture)
from test_kv_cpu import cache


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


def test_sizes_whose_row_numbers_would_leave_32_bits_are_refused(lib):
    """A product's last row plus the rows that a grid takes at once; a query row in front of every key less a window."""
    n = ctypes.c_size_t(0)
    most = 2 ** 31 - 2 ** 16
    for M, N, rc in ((1, most, 0), (1, most + 1, SHAPE), (1, 2 ** 31 - 1, SHAPE), (most, 1, 0), (most + 1, 1, SHAPE)):
        assert lib.q4_int8_gemm_workspace_size(M, N, 16, ctypes.byref(n)) == rc
        assert lib.q4_int8_linear_scratch_size(M, 16, ctypes.byref(n)) == (SHAPE if M > most else 0)
    for total, rc in ((2 ** 30, 0), (2 ** 30 + 1, SHAPE), (2 ** 31 - 1, SHAPE)):
        assert lib.q4_kv_attention_workspace_size(cache(), 4, total, 8, ctypes.byref(n)) == rc


def test_linear8bit_takes_codes_that_are_part_of_a_wider_buffer():
    wide = torch.randint(-127, 128, (5, 96), dtype=torch.int8)
    for codes in (wide[:, 16:80], wide[:, :64], wide[:, 32:86], wide[1:2, 16:80], wide[::2, 80:], wide[:, 16:]):
        m = linear8bit.Linear8bit(codes, torch.ones(codes.shape[0]))
        assert torch.equal(m.codes[:, :m.in_features], codes) and m.codes.shape[1] == (codes.shape[1] + 15) // 16 * 16
