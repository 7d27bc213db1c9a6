"""The 8-bit integer linear layer on a B200 at the borders of its kernels' ranges."""
import numpy as np
import pytest
import torch

from test_int8_gpu import q4, random_codes, rows_reference  # noqa: F401  (q4: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,most", [(1, 49152), (2, 24576), (3, 12288), (4, 12288)])
@pytest.mark.parametrize("past", [-32, -31, -1, 0, 1])
def test_linear_at_the_longest_rows_of_the_one_launch_kernel(q4, M, most, past):
    """The tokens' codes fill a CTA's 48 KB of shared memory at K = most; one more takes the other kernel."""
    K, N = most + past, 40
    g = torch.Generator().manual_seed(M + K)
    x = torch.randn(M, K, generator=g).half().cuda()
    W, sw = q4.int8_quantize_rows((torch.randn(N, K, generator=g) * 0.02).half().cuda())
    qa, sa = q4.int8_quantize_rows(x)
    want = (qa.double() @ W.double().t()).float() * (sa[:, None] * sw[None])
    for out in (torch.float32, torch.bfloat16):
        y = q4.int8_linear(x, W, sw, out_dtype=out)
        assert torch.equal(y, q4.int8_gemm(qa, sa, W, sw, out_dtype=out))
        assert torch.equal(y, want.to(out))
    assert q4.last_device_status() == 0


@pytest.mark.parametrize("K", [1, 64, 1001, 4104, 28672])
def test_float32_rows_are_quantized_with_all_their_bits(q4, K):
    """A checkpoint's float32 weights: the definition's codes and scales, not those of the weights in 16 bits."""
    g = torch.Generator().manual_seed(K)
    w = torch.randn(37, K, generator=g) * torch.exp(3 * torch.randn(37, 1, generator=g))
    w[3] = 0
    w[5] *= 1e-36
    w[7] = 2.0 ** -140
    codes, scale = q4.int8_quantize_rows(w.cuda())
    want, s = rows_reference(w)
    assert s[7] == 4 * 2.0 ** -149  # 2^-140 / 127, rounded to a subnormal: the quotient is 128
    want[7] = 127
    assert np.array_equal(scale.cpu().numpy(), s) and np.array_equal(codes.cpu().numpy(), want)
    codes, scale = q4.int8_quantize_rows(w.cuda().t().contiguous().t())  # columns first: copied
    assert np.array_equal(codes.cpu().numpy(), want)
    if K > 9:
        view = w[::2, 3:K - 2]
        codes, scale = q4.int8_quantize_rows(w.cuda()[::2, 3:K - 2])
        want, s = rows_reference(view)
        assert np.array_equal(scale.cpu().numpy(), s) and np.array_equal(codes.cpu().numpy(), want)
    assert q4.last_device_status() == 0


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_float32_row_that_is_not_finite_spoils_itself_alone(q4, bad):
    w = torch.ones(3, 700, device="cuda")
    w[1, 699] = bad
    codes, scale = q4.int8_quantize_rows(w)
    assert torch.isnan(scale).tolist() == [False, True, False] and not codes[1].any() and (codes[::2] == 127).all()
    assert q4.last_device_status() == 1
    q4.clear_device_status()


def test_linear8bit_quantizes_float32_weights_themselves(q4):
    from bit_blockwise_weight_absmax_b200 import linear8bit
    torch.manual_seed(1)
    lin = torch.nn.Linear(777, 130).cuda()
    m = linear8bit.Linear8bit.from_linear(lin)
    want, s = rows_reference(lin.weight)
    assert np.array_equal(m.scale.cpu().numpy(), s) and np.array_equal(m.codes[:, :777].cpu().numpy(), want)
    # half a step of a code for each weight, and no more
    back = m.codes[:, :777].double() * m.scale.double()[:, None]
    assert ((back - lin.weight.double()).abs() <= m.scale.double()[:, None] * (0.5 + 127 * 2.0 ** -23)).all()


@pytest.mark.parametrize("M,N,K", [(9, 600, 4096), (100, 4096, 4096), (1024, 1024, 8192), (3000, 4096, 2048)])
def test_waits_that_run_out_while_copies_are_on_their_way(q4, M, N, K):
    """Limits around a copy's own time, single CTAs and pairs: any wait may run out (a probe of a barrier blocks for a
    while itself, so none has to).  Every call returns, with the right result or with its status, and the next is right."""
    g = torch.Generator().manual_seed(M)
    A, sa = random_codes(g, M, K)
    W, sw = random_codes(g, N, K)
    want = q4.int8_gemm(A, sa, W, sw, None, torch.float32)
    try:
        for limit in (1, 300, 1000, 2000, 5000) * 4:
            q4.set_wait_limit_ns(limit)
            y = q4.int8_gemm(A, sa, W, sw, None, torch.float32)
            torch.cuda.synchronize()
            status = q4.last_device_status()
            assert status in (0, 2)
            assert status or torch.equal(y, want)
            q4.reset_workspaces()
            q4.clear_device_status()
    finally:
        q4.set_wait_limit_ns(0)
        q4.reset_workspaces()
        q4.clear_device_status()
    assert torch.equal(q4.int8_gemm(A, sa, W, sw, None, torch.float32), want)


def test_linear8bit_after_casts_of_the_model(q4):
    """The codes and scales stay as they are; a bias of any type is added in binary32."""
    from bit_blockwise_weight_absmax_b200 import linear8bit
    torch.manual_seed(2)
    m = linear8bit.Linear8bit.from_linear(torch.nn.Linear(300, 70).cuda(), torch.float16)
    x = torch.randn(6, 300, device="cuda").half()
    want = m(x)
    for cast in ("half", "double", "float"):
        getattr(m, cast)()
        assert torch.equal(m(x), want)
