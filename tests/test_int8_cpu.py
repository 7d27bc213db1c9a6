"""The 8-bit integer linear layer without a GPU: what the C ABI and the binding
refuse before anything is launched, and the workspace sizes."""
import ctypes

import pytest
import torch

from bit_blockwise_weight_absmax_b200 import linear8bit, q4

ARG, SHAPE, ALIGN, NO_DEVICE, WORKSPACE = -1, -2, -3, -4, -7
A = 1 << 20  # a 16-byte aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    from bit_blockwise_weight_absmax_b200 import build
    build.build()
    return q4.library()


def quant(lib, X=A, dt=0, rows=4, cols=64, ldx=64, codes=A, ldc=64, scale=A):
    return lib.q4_int8_quantize_rows(X, dt, rows, cols, ldx, codes, ldc, scale, None)


def gemm(lib, Ap=A, lda=64, sa=A, M=4, W=A, ldw=64, sw=A, N=8, K=64, bias=None, bdt=0, Y=A, ldy=8, ydt=0, ws=A,
         wsb=1 << 40):
    return lib.q4_int8_gemm(Ap, lda, sa, M, W, ldw, sw, N, K, bias, bdt, Y, ldy, ydt, ws, wsb, None)


def linear(lib, X=A, dt=0, ldx=64, M=4, W=A, ldw=64, sw=A, N=8, K=64, bias=None, bdt=0, Y=A, ldy=8, ydt=0, scr=A,
           scb=1 << 40, ws=A, wsb=1 << 40):
    return lib.q4_int8_linear(X, dt, ldx, M, W, ldw, sw, N, K, bias, bdt, Y, ldy, ydt, scr, scb, ws, wsb, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers: only where nothing can be launched")
def test_refusals(lib):
    assert quant(lib) == gemm(lib) == linear(lib) == NO_DEVICE
    for kw, rc in [(dict(X=None), ARG), (dict(codes=None), ARG), (dict(scale=None), ARG), (dict(dt=2), ARG),
                   (dict(rows=0), SHAPE), (dict(cols=0), SHAPE), (dict(cols=131072, ldx=131072, ldc=131072), SHAPE),
                   (dict(ldx=63), SHAPE), (dict(ldc=48), SHAPE), (dict(ldc=72), SHAPE), (dict(codes=A + 8), ALIGN)]:
        assert quant(lib, **kw) == rc, kw
    assert quant(lib, X=A + 2, ldx=65) == NO_DEVICE  # any 2-byte alignment of the input is taken
    for kw, rc in [(dict(Ap=None), ARG), (dict(sa=None), ARG), (dict(W=None), ARG), (dict(sw=None), ARG),
                   (dict(Y=None), ARG), (dict(ydt=3), ARG), (dict(bias=A, bdt=7), ARG), (dict(M=0), SHAPE),
                   (dict(N=0), SHAPE), (dict(K=0), SHAPE), (dict(K=131072, lda=131072, ldw=131072), SHAPE),
                   (dict(lda=48), SHAPE), (dict(lda=72), SHAPE), (dict(ldw=72), SHAPE), (dict(ldy=7), SHAPE),
                   (dict(Ap=A + 8), ALIGN), (dict(W=A + 8), ALIGN)]:
        assert gemm(lib, **kw) == rc, kw
    for kw, rc in [(dict(X=None), ARG), (dict(dt=2), ARG), (dict(ldx=63), SHAPE), (dict(ldw=72), SHAPE),
                   (dict(ldy=7), SHAPE), (dict(W=A + 8), ALIGN), (dict(M=9, scr=None), WORKSPACE),
                   (dict(M=9, scb=16), WORKSPACE), (dict(ws=A + 8), ALIGN), (dict(scr=A + 8), ALIGN),
                   (dict(M=9, K=4096, ldx=4096, ldw=4096, ws=None), WORKSPACE),
                   (dict(M=9, K=4096, ldx=4096, ldw=4096, wsb=16), WORKSPACE)]:
        assert linear(lib, **kw) == rc, kw


def test_workspace_sizes(lib):
    n = ctypes.c_size_t(0)
    for M, N, K in [(1, 1, 1), (1, 4096, 4096), (33, 4096, 4095), (300, 300, 300), (4096, 28672, 8192)]:
        assert lib.q4_int8_gemm_workspace_size(M, N, K, ctypes.byref(n)) == 0
        assert n.value <= q4.WORKSPACE_HEAD + 148 * 2 * 256 * 128 * 4  # two unfinished tiles of 128 x 256 a CTA
        assert lib.q4_int8_linear_scratch_size(M, K, ctypes.byref(n)) == 0
        assert n.value >= 4 * M + M * ((K + 15) // 16 * 16) or (M <= 4 and n.value == 0)  # few tokens need none
    assert lib.q4_int8_gemm_workspace_size(0, 1, 1, ctypes.byref(n)) == SHAPE
    assert lib.q4_int8_linear_scratch_size(1, 131072, ctypes.byref(n)) == SHAPE
    assert lib.q4_int8_gemm_workspace_size(1, 1, 1, None) == ARG


def _codes(n=4, k=64):
    return torch.zeros(n, k, dtype=torch.int8), torch.ones(n)


def test_binding_refuses_before_the_library():
    c, s = _codes()
    x = torch.zeros(2, 64, dtype=torch.float16)
    for bad in (lambda: q4.int8_linear(x.float(), c, s), lambda: q4.int8_linear(x[:, :60], c, s),
                lambda: q4.int8_linear(x, c, s.double()), lambda: q4.int8_linear(x, c[:, :60][:, ::2], s),
                lambda: q4.int8_linear(x, c, s[:3]), lambda: q4.int8_linear(x, c.to(torch.uint8), s),
                lambda: q4.int8_gemm(c, s, *_codes(4, 48)), lambda: q4.int8_gemm(c, s, c, s, out_dtype=torch.float64),
                lambda: q4.int8_quantize_rows(x.float()), lambda: q4.int8_quantize_rows(x[0]),
                lambda: q4.int8_linear(x, torch.zeros(4, 70, dtype=torch.int8)[:, :64], s)):
        with pytest.raises(q4.Q4Error):
            bad()


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_no_cpu_fallback():
    c, s = _codes()
    x = torch.zeros(2, 64, dtype=torch.float16)
    for call in (lambda: q4.int8_linear(x, c, s), lambda: q4.int8_gemm(c, s, c, s), lambda: q4.int8_quantize_rows(x),
                 lambda: linear8bit.Linear8bit(c, s)(x)):
        with pytest.raises(q4.Q4Error, match="no CUDA device"):
            call()


def test_linear8bit_module_holds_codes_and_float32_scales():
    c, s = _codes(4, 50 + 14)
    m = linear8bit.Linear8bit(c[:, :50], s, torch.ones(4))
    assert (m.in_features, m.out_features) == (50, 4) and m.codes.shape == (4, 64)
    m.half()
    assert m.scale.dtype == torch.float32 and m.codes.dtype == torch.int8
    with pytest.raises(q4.Q4Error, match="last dimension"):
        m(torch.zeros(1, 64))
    with pytest.raises(q4.Q4Error):
        linear8bit.Linear8bit(c, s, compute_dtype=torch.float32)
