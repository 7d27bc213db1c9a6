"""The 8-bit integer linear layer on a B200 against 64-bit arithmetic."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24  # half a step of binary32
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: U}  # half a step, relative


@pytest.fixture(scope="module")
def q4():
    from bit_blockwise_weight_absmax_b200 import build
    build.build()
    from bit_blockwise_weight_absmax_b200 import q4
    q4.clear_device_status()
    yield q4
    q4.clear_device_status()


def rows_reference(x):
    """Codes and scales of the definition; a binary32 quotient is the binary64 one rounded (53 >= 2 * 24 + 2 bits)."""
    v = x.detach().float().cpu().numpy()
    top = np.abs(v).max(1)
    s = (top.astype(np.float64) / 127).astype(np.float32)
    safe = np.where(s > 0, s, 1).astype(np.float64)
    q = np.rint((v.astype(np.float64) / safe[:, None]).astype(np.float32))
    return np.where(s[:, None] > 0, q, 0).astype(np.int8), s


@pytest.mark.parametrize("rows,K", [(1, 1), (3, 7), (5, 64), (2, 1001), (300, 576), (7, 4096), (3, 4104), (2, 16390),
                                    (2, 28672), (1, 131071)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_quantize_rows_is_the_definition_bit_for_bit(q4, rows, K, dtype):
    g = torch.Generator().manual_seed(rows * 7 + K)
    x = torch.randn(rows, K, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))
    x[0] *= 1e-6
    x = x.to(dtype)
    x.view(-1)[:: 37] = x.view(-1)[0] / 2  # halves of one value: quotients near ties
    codes, scale = q4.int8_quantize_rows(x.cuda())
    want, s = rows_reference(x)
    assert codes.shape == (rows, K) and codes.stride(0) % 16 == 0
    assert np.array_equal(scale.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), want)


def test_quantize_rows_strides_zero_rows_and_tiny_values(q4):
    g = torch.Generator().manual_seed(3)
    big = torch.randn(9, 133, generator=g).bfloat16()
    big[2] = 0
    big[4] = big[4] * 1e-38 * 0.5  # scales below 2^-90
    big[6] = -0.0
    for view in (big[:, 1:130], big[::2, 3:100], big.t(), big[:, :128]):
        codes, scale = q4.int8_quantize_rows(big.cuda()[:, 1:130] if view is big else view.cuda())
        want, s = rows_reference(view)
        assert np.array_equal(scale.cpu().numpy(), s) and np.array_equal(codes.cpu().numpy(), want)
    dev = big.cuda()
    codes, scale = q4.int8_quantize_rows(dev[:, 1:130])  # rows at odd 2-byte addresses
    want, s = rows_reference(big[:, 1:130])
    assert np.array_equal(codes.cpu().numpy(), want)
    codes, scale = q4.int8_quantize_rows(dev[:, :1].expand(9, 1))
    assert codes.shape == (9, 1)
    assert q4.last_device_status() == 0
    assert q4.int8_quantize_rows(dev[:0])[0].shape == (0, 133)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_row_that_is_not_finite_spoils_itself_alone(q4, bad):
    x = torch.ones(4, 100, dtype=torch.float16, device="cuda")
    x[2, 99] = bad
    w, sw = q4.int8_quantize_rows(torch.ones(24, 100, dtype=torch.float16, device="cuda"))
    codes, scale = q4.int8_quantize_rows(x)
    assert torch.isnan(scale).tolist() == [False, False, True, False] and not codes[2].any()
    assert q4.last_device_status() == 1
    q4.clear_device_status()
    y = q4.int8_linear(x, w, sw)
    assert torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 3]]).all()
    q4.clear_device_status()


def random_codes(g, rows, K, dev="cuda"):
    buf = torch.randint(-128, 128, (rows, (K + 15) // 16 * 16), generator=g, dtype=torch.int8).to(dev)  # garbage past K
    return buf[:, :K], (torch.rand(rows, generator=g) + 0.5).to(dev)


def product_reference(A, sa, W, sw, bias):
    """(value, bound of the binary32 roundings) in binary64: the integer sum to binary32, the product of the scales,
    their product, and the bias: a relative half step each."""
    acc = A.double() @ W.double().t()
    y = acc * sa.double()[:, None] * sw.double()[None]
    err = 3.1 * U * y.abs()
    if bias is not None:
        y = y + bias.double()[None]
        err = err + U * y.abs() * 1.01
    return y, err


MNK = [(1, 1, 1), (1, 8, 16), (1, 128, 4096), (2, 129, 31), (3, 577, 1000), (16, 256, 129), (17, 100, 128), (31, 1536, 576),
       (33, 127, 127), (64, 640, 255), (65, 130, 2048), (127, 300, 64), (129, 257, 513), (256, 128, 1024), (257, 513, 385),
       (512, 384, 4096), (700, 1111, 333), (2, 4096, 8192),
       (4, 50, 20000), (3, 2000, 12272), (5, 4096, 4096), (24, 11008, 1000), (513, 11008, 640), (1024, 2304, 4224),
       (130, 20000, 2064)]


@pytest.mark.parametrize("M,N,K", MNK)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_product(q4, M, N, K, dtype):
    g = torch.Generator().manual_seed(M + 3 * N + 7 * K)
    A, sa = random_codes(g, M, K)
    W, sw = random_codes(g, N, K)
    if dtype == torch.float16:
        sa = sa * 2.0 ** -13  # |sums| reach K 2^14
    bias = torch.randn(N, generator=g).to(dtype).cuda() if (M + N) % 2 else None
    y = q4.int8_gemm(A, sa, W, sw, bias, dtype)
    ref, err = product_reference(A, sa, W, sw, bias)
    tol = err + HALF[dtype] * (ref.abs() + err) + (2.0 ** -25 if dtype == torch.float16 else 0)
    assert ((y.double() - ref).abs() <= tol).all()
    assert torch.equal(y, q4.int8_gemm(A, sa, W, sw, bias, dtype))
    assert q4.last_device_status() == 0


@pytest.mark.parametrize("value", [-128, 127])
@pytest.mark.parametrize("M", [1, 40])
def test_the_largest_sums_are_exact(q4, value, M):
    K = 131071  # 131071 * 128^2 < 2^31
    A = torch.full((M, K + 1), value, dtype=torch.int8, device="cuda")[:, :K]
    W = torch.full((3, K + 1), value, dtype=torch.int8, device="cuda")[:, :K]
    W[1] = -127
    one = torch.ones(M, device="cuda"), torch.ones(3, device="cuda")
    y = q4.int8_gemm(A, one[0], W, one[1], None, torch.float32)
    want = torch.tensor([value * value * K, -127 * value * K, value * value * K], dtype=torch.float64).float()
    assert torch.equal(y.cpu(), want.expand(M, 3))


def test_linear_is_quantize_then_product_and_takes_strides(q4):
    g = torch.Generator().manual_seed(5)
    for M, N, K, dt in [(1, 100, 576, torch.float16), (40, 300, 577, torch.bfloat16), (300, 64, 4096, torch.float16)]:
        x = torch.randn(M, K + 5, generator=g).to(dt).cuda()[:, 2:K + 2]
        W, sw = q4.int8_quantize_rows((torch.randn(N, K, generator=g) * 0.02).to(dt).cuda())
        for bdt in (None, torch.float32, torch.float16, torch.bfloat16):
            bias = None if bdt is None else torch.randn(N, generator=g).to(bdt).cuda()
            wide = torch.full((M, N + 9), 7.0, dtype=torch.float32, device="cuda")
            y = q4.int8_linear(x, W, sw, bias, torch.float32, out=wide[:, :N])
            qa, sa = q4.int8_quantize_rows(x)
            assert torch.equal(y, q4.int8_gemm(qa, sa, W, sw, bias, torch.float32))
            assert (wide[:, N:] == 7).all()
            ref, err = product_reference(qa, sa, W, sw, bias)
            assert ((y.double() - ref).abs() <= err).all()
    assert q4.int8_linear(x[:0], W, sw).shape == (0, 64)


def test_other_streams_and_graphs_that_run_at_once(q4):
    g = torch.Generator().manual_seed(6)
    W, sw = q4.int8_quantize_rows((torch.randn(512, 2048, generator=g) * 0.02).half().cuda())
    xs = [torch.randn(m, 2048, generator=g).half().cuda() for m in (1, 24, 3)]
    want = [q4.int8_linear(x, W, sw) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [q4.int8_linear(x, W, sw, stream=s) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs, ins = [], [], [torch.zeros_like(x) for x in xs]
    for x in ins:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(q4.int8_linear(x, W, sw))
        graphs.append(graph)
    for x, y in zip(ins, xs):
        x.copy_(y)
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("M,N,K", [(9, 600, 4096), (100, 4096, 4096), (1024, 1024, 8192)])
def test_wait_limit_times_out_and_recovers(q4, M, N, K):
    """With the copy-stall hook on no stage is ever filled: the waits run out, the call reports it, and after the
    workspaces are zeroed again the next call is right (single CTAs, and CTA pairs for many tokens)."""
    g = torch.Generator().manual_seed(8)
    A, sa = random_codes(g, M, K)
    W, sw = random_codes(g, N, K)
    try:
        q4.set_wait_limit_ns(200_000)
        q4.set_copy_stall(True)
        q4.int8_gemm(A, sa, W, sw, None, torch.float32)
        torch.cuda.synchronize()
        assert q4.last_device_status() & 2  # Q4_STATUS_TIMEOUT
    finally:
        q4.set_copy_stall(False)
        q4.set_wait_limit_ns(0)
        q4.reset_workspaces()
        q4.clear_device_status()
    y = q4.int8_gemm(A, sa, W, sw, None, torch.float32)
    ref, err = product_reference(A, sa, W, sw, None)
    assert ((y.double() - ref).abs() <= err).all()
    assert q4.last_device_status() == 0


def test_linear8bit_and_replace_linear(q4):
    from bit_blockwise_weight_absmax_b200 import linear4bit, linear8bit
    torch.manual_seed(0)
    model = torch.nn.Sequential(torch.nn.Linear(250, 512), torch.nn.GELU(), torch.nn.Linear(512, 256))
    model.lm_head = torch.nn.Linear(256, 64)
    model = model.bfloat16().cuda()
    before = linear4bit.memory_footprint(model)
    x = torch.randn(3, 5, 250, device="cuda").bfloat16()
    with torch.no_grad():
        plain = [model[0](x), None]
        linear4bit.replace_linear(model, linear=linear8bit.Linear8bit, compute_dtype=torch.bfloat16)
        assert isinstance(model[0], linear8bit.Linear8bit) and type(model.lm_head) is torch.nn.Linear
        assert linear4bit.memory_footprint(model) < 0.6 * before
        y = model[0](x)
        h = model[2](model[1](y))
    assert y.shape == (3, 5, 512) and h.shape == (3, 5, 256) and y.dtype == torch.bfloat16
    m = model[0]
    ref, err = product_reference(*q4.int8_quantize_rows(x.view(15, 250)), m.codes[:, :250], m.scale, m.bias)
    assert ((y.view(15, 512).double() - ref).abs() <= err + HALF[torch.bfloat16] * (ref.abs() + err)).all()
    # 8-bit codes: a step is top / 127, so an error of at most half a step of each factor
    assert ((y - plain[0]).float().norm() / plain[0].float().norm()).item() < 0.03
    assert q4.last_device_status() == 0
