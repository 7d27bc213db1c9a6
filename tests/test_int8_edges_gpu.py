"""The 8-bit integer linear layer on a B200 at the borders of its kernels' ranges."""
import pytest
import torch

from test_int8_gpu import q4  # noqa: F401  (the fixture)

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

