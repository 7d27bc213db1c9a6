"""The 4-bit key/value cache and its attention on a B200 where they are easily wrong."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import bits, is_bf16
from test_kv_gpu import HALF, INDEX, check, fill_cache, q4, reference, values  # noqa: F401  (q4: the fixture)

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("rows,length", [(2, 500), (14, 500), (150, 500), (130, 30000)])
def test_rows_that_are_nan_have_a_nan_log_sum_exp(q4, rows, length):
    """A NaN in a query: every score of its row is one (both kernels, and parts that are joined)."""
    g = torch.Generator().manual_seed(rows)
    c, table = fill_cache(q4, g, [length], 2, 128, 64, 64)
    q = torch.randn(rows, 4, 128, generator=g).half().cuda()
    bad = torch.zeros(rows, 4, dtype=torch.bool)
    for row, head in ((0, 1), (rows // 2, 3), (rows - 1, 0)):
        q[row, head, 5] = math.nan
        bad[row, head] = True
    out, lse = q4.kv_attention(q, c, table.cuda(), ints([length]), ints([0, rows]), return_lse=True)
    assert torch.equal(torch.isnan(lse).cpu(), bad) and torch.equal(torch.isnan(out).all(-1).cpu(), bad)
    assert torch.isfinite(lse).cpu()[~bad].all() and torch.isfinite(out).cpu()[~bad].all()


@pytest.mark.parametrize("name", ["k_state", "v_state"])
@pytest.mark.parametrize("rows,length", [(300, 300), (1000, 1000)])
def test_a_first_key_that_could_not_be_held_makes_every_log_sum_exp_nan(q4, rows, length, name):
    """Row 0 of a whole prompt attends to that key alone."""
    g = torch.Generator().manual_seed(rows)
    c, table = fill_cache(q4, g, [length], 2, 128, 64, 64)
    getattr(c, name)[int(table[0, 0]), 1, 0, 1, 0] = math.nan
    q = torch.randn(rows, 4, 128, generator=g).half().cuda()
    out, lse = q4.kv_attention(q, c, table.cuda(), ints([length]), ints([0, rows]), return_lse=True)
    assert torch.isnan(lse[:, 2:]).all() and torch.isnan(out[:, 2:]).all()
    assert torch.isfinite(lse[:, :2]).all() and torch.isfinite(out[:, :2]).all()



@pytest.mark.parametrize("rows,length", [(1, 300), (3, 40000), (12, 3000), (300, 700), (130, 30000)])
def test_waits_that_run_out_while_copies_are_on_their_way(q4, rows, length):
    """Limits around a copy's own time: any of the warps' waits may run out (a probe of a barrier blocks for a while
    itself, so none has to).  Every call returns, with the right result or with its status, and the next one is right."""
    g = torch.Generator().manual_seed(rows)
    c, table = fill_cache(q4, g, [length], 2, 64, 64, 64)
    q = torch.randn(rows, 4, 64, generator=g).half()
    args = (q.cuda(), c, table.cuda(), ints([length]), ints([0, rows]))
    want = q4.kv_attention(*args)
    try:
        for limit in (1, 300, 1000, 2000, 5000) * 4:
            q4.set_wait_limit_ns(limit)
            out = q4.kv_attention(*args)
            torch.cuda.synchronize()
            status = q4.last_device_status()
            assert status in (0, 2)
            assert status or torch.equal(out, want)
            q4.reset_workspaces()
            q4.clear_device_status()
    finally:
        q4.set_wait_limit_ns(0)
        q4.reset_workspaces()
        q4.clear_device_status()
    check(q4, c, table, [length], [rows], q, implicit=False)


def one_large_weight(q4, D, length, gap, first):
    """A cache whose first key's score lies 2^gap above all the others', which are zero, and whose first value is `first`
    in elements 1, 4, 7, .. and the others' 15 in elements 0, 3, 6, ..: every number is an integer that the cache and binary16 hold exactly.
    Returns the cache, its table, the query vector and the scale."""
    page = 256
    pages = (length + page - 1) // page
    c = q4.kv_cache(pages, 1, D, page, 64)
    k, v = torch.zeros(2, length, 1, D, dtype=torch.float16, device="cuda")
    k[0, :, ::64] = 15
    v[0, :, 1::3] = first
    v[1:, :, ::3] = 15
    q4.kv_append(c, k, v, torch.arange(length, device="cuda"))
    query = torch.zeros(D, dtype=torch.float16, device="cuda")
    query[0] = 1
    return c, torch.arange(pages, dtype=torch.int32, device="cuda")[None], query, float(np.float32(gap * math.log(2) / 15))


@pytest.mark.parametrize("first", [0, 15])
@pytest.mark.parametrize("gap", [20.356, 25.1])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("batch,rows,group", [(300, 1, 1), (300, 1, 12), (1, 1024, 37), (1, 130, 1)])
def test_many_small_weights_beside_a_large_one(q4, D, batch, rows, group, gap, first):
    """131072 keys whose weights are 2^-gap of the first key's: none of them may be lost.  A weight's binary16 rounding
    is half a step, 2^-11, or below the normal range 2^-25, where the largest weight is at least 2^8 (so 2^(gap - 33) of
    it); binary32 sums of at most 8192 MMAs of 16 keys and 300 joined parts, terms of one sign, a step (2^-23, an MMA may
    truncate) each; exponentials 2^-20."""
    length = 131073
    c, table, query, scale = one_large_weight(q4, D, length, gap, first)
    q = query.expand(batch * rows, group, D).contiguous()
    cu = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * rows
    out, lse = q4.kv_attention(q, c, table.expand(batch, -1).contiguous(), ints([length] * batch), cu, max_q=rows,
                               scale=scale, return_lse=True)
    tail = (length - rows + torch.arange(rows, dtype=torch.float64)) * 2.0 ** (-scale * 15 / math.log(2))  # of each row
    share = (tail / (1 + tail))[None, :, None, None].cuda()
    got = out.double().view(batch, rows, group, D)
    sums = 8492 * 2.0 ** -23
    rel = max(2.0 ** -11, 2.0 ** (gap - 33)) + 2 * sums + HALF[torch.float16] + 2.0 ** -19
    for at, want in ((0, 15 * share), (1, first * (1 - share)), (2, 0 * share)):
        assert ((got[..., at::3] - want).abs() <= rel * want + 2.0 ** -25).all()
    wl = scale * 15 + torch.log1p(tail)[None, :, None].cuda()
    # eight roundings of numbers up to 2^5 (the score, its factor and the reference in base 2), and the sum's
    assert ((lse.double().view(batch, rows, group) - wl).abs() <= 8 * 2.0 ** -19 + sums).all()
    assert q4.last_device_status() == 0


@pytest.mark.parametrize("rows", [1, 5, 14, 140])
def test_a_vector_whose_blocks_differ_in_size(q4, rows):
    """The values of a vector's two blocks, 2^20 apart, are both right to their own size."""
    g = torch.Generator().manual_seed(rows + 3)
    n, D = 700, 128
    c = q4.kv_cache(11, 2, D, 64, 64)
    k, v = torch.randn(2, n, 2, D, generator=g)
    v[:, :, :64] *= 2000
    v[:, :, 64:] *= 2e-3
    v[:, 1] = v[:, 1].roll(64, 1)
    q4.kv_append(c, k.half().cuda(), v.half().cuda(), torch.arange(n).cuda())
    check(q4, c, torch.arange(11, dtype=torch.int32)[None], [n], [rows], torch.randn(rows, 6, D, generator=g).bfloat16(),
          implicit=False)


@pytest.mark.parametrize("D,B", [(64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("rows", [1, 5, 14, 150])
@pytest.mark.parametrize("name", ["k_state", "v_state"])
def test_a_block_that_could_not_be_held_spoils_whole_rows_in_either_kernel(q4, D, B, rows, name):
    """Whichever block of the key or the value it is, and whichever kernel the hint chooses: the rows that attend to it
    are NaN in every element and in the log sum exp, the others are not."""
    g = torch.Generator().manual_seed(rows)
    lens, qs = [260, 260], [rows, rows]
    c, table = fill_cache(q4, g, lens, 2, D, B, 64)
    getattr(c, name)[int(table[0, 1]), 1, 3, D // B - 1, 0] = math.nan  # key 67 of the first sequence, head 1
    q = torch.randn(2 * rows, 4, D, generator=g).half().cuda()
    for max_q in (1, rows, 1000):
        out, lse = q4.kv_attention(q, c, table.cuda(), ints(lens), ints([0, rows, 2 * rows]), max_q=max_q, return_lse=True)
        for t in (out[:rows, 2:], lse[:rows, 2:]):
            assert torch.isnan(t).all()
        for t in (out[:rows, :2], out[rows:], lse[:rows, :2], lse[rows:]):
            assert torch.isfinite(t).all()


def test_the_hint_left_out_takes_the_kernel_for_few_rows_where_the_rows_are_as_many_as_the_sequences(q4):
    """A decode step given by its row ranges: the same kernel, and so the same bits, as with the hint 1."""
    g = torch.Generator().manual_seed(3)
    lens = [(37 * b) % 900 + 1 for b in range(64)]
    c, table = fill_cache(q4, g, lens, 2, 128, 64, 64)
    q = torch.randn(64, 8, 128, generator=g).half().cuda()
    args = (q, c, table.cuda(), ints(lens), torch.arange(65, dtype=torch.int32, device="cuda"))
    want = q4.kv_attention(*args, max_q=1)
    assert not torch.equal(q4.kv_attention(*args, max_q=64), want)  # the other kernel rounds otherwise
    assert torch.equal(q4.kv_attention(*args), want)


@pytest.mark.parametrize("D,B,qh,kh", [(64, 64, 9, 3), (128, 64, 8, 2), (128, 128, 4, 4)])
@pytest.mark.parametrize("max_q", [1, 3, 10 ** 6])
def test_a_hint_that_is_off_changes_no_result(q4, D, B, qh, kh, max_q):
    """Either kernel takes any rows: many row tiles of a sequence in the one for few, single rows in the one for many."""
    g = torch.Generator().manual_seed(D + B)
    for lens, qs in (([64, 900, 2, 333], [64, 450, 1, 333]), ([200, 1, 90], [1, 1, 1])):
        c, table = fill_cache(q4, g, lens, kh, D, B, 32)
        q = torch.randn(sum(qs), qh, D, generator=g).half()
        cu = ints([0] + list(np.cumsum(qs)))
        out, lse = q4.kv_attention(q.cuda(), c, table.cuda(), ints(lens), cu, max_q=max_q, return_lse=True)
        ref, rl, tol, ltol = reference(c, table, lens, qs, q, D ** -0.5, True, 0)
        assert ((out.double().cpu() - ref).abs() <= tol + HALF[q.dtype] * (ref.abs() + tol) + 2.0 ** -25).all()
        assert ((lse.double().cpu() - rl).abs() <= ltol).all()
    assert q4.last_device_status() == 0


@pytest.mark.parametrize("D,B", [(64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_calls_of_many_tokens_write_and_read_the_same_bits(q4, oracle, D, B, dtype):
    """Threads take several tokens each; slots outside the cache near the end, where a thread's tokens run out."""
    T, H, page = 8191, 32, 64
    g = torch.Generator().manual_seed(D + B)
    k, v = (torch.randn(T, H, D, generator=g).to(dtype) for _ in range(2))
    pages = T // page + 3
    c = q4.kv_cache(pages, H, D, page, B)
    for t in (c.k_codes, c.v_codes):
        t.fill_(0xAB)
    slots = torch.randperm(pages * page, generator=g)[:T]
    for at, slot in ((0, -1), (63, -5), (T - 130, -1), (T - 65, pages * page), (T - 2, -1), (T - 1, pages * page + 7)):
        slots[at] = slot
    q4.kv_append(c, k.cuda(), v.cuda(), slots.cuda())
    assert q4.last_device_status() == INDEX
    q4.clear_device_status()
    some = (slots >= 0) & (slots < pages * page)
    for x, codes, state in ((k, c.k_codes, c.k_state), (v, c.v_codes, c.v_state)):
        ost = oracle.quantize(bits(x), is_bf16(x), B, oracle.QT_INT4_ASYM, False, True)
        nb = D // B
        z = np.empty(2 * ost.zero.size, dtype=np.uint8)
        z[0::2], z[1::2] = ost.zero & 15, ost.zero >> 4
        s = ost.scale_f16_bits().view(np.float16).reshape(T, H, nb)[some]
        got = state.cpu().numpy().transpose(0, 2, 1, 3, 4).reshape(-1, H, nb, 2)
        at = slots[some].numpy()
        assert np.array_equal(got[at][..., 0], s)
        assert np.array_equal(got[at][..., 1], z[:T * H * nb].reshape(T, H, nb)[some])
        want = ost.codes().reshape(T, H, nb, B // 8, 8).swapaxes(2, 3).reshape(T, H, D // 2, 2)[some]
        got = codes.cpu().numpy().transpose(0, 2, 1, 3).reshape(-1, H, D // 2)
        assert np.array_equal(got[at], want[..., 0] | (want[..., 1] << 4))
        rest = np.ones(pages * page, dtype=bool)
        rest[at] = False
        assert (got[rest] == 0xAB).all()
    for out in (torch.float16, torch.bfloat16):
        for x, codes, state in zip(q4.kv_dequantize(c, slots.cuda(), out), (c.k_codes, c.v_codes), (c.k_state, c.v_state)):
            flat_c, flat_s = (t.cpu().transpose(1, 2).flatten(0, 1) for t in (codes, state))
            assert torch.equal(x.cpu()[some], values(flat_c[slots[some]], flat_s[slots[some]]).to(out))
            assert not x.cpu()[~some].any()
    assert q4.last_device_status() == INDEX
    q4.clear_device_status()


@pytest.mark.parametrize("D,B", [(64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("window", [1, 0])
@pytest.mark.parametrize("few", [False, True])
def test_the_log_sum_exp_has_all_bits_of_the_keys(q4, D, B, window, few):
    """Queries along what rounding their own keys to binary16 leaves over, where the rounding costs most.  The bound has
    binary32 terms alone.  An MMA adds 16 products to its sum, each cut at the last bit of the largest (17 terms, a step
    of 2^-23 of at most sum |q k| each); many rows take D / 16 MMAs for the rounded keys and as many for what is left.
    Few rows sum code - 8 and take (z - 8) sum(q) off, each up to 8 s |q| (a window's units lie at the ends of its
    keys; whole units sum the codes, and z, up to 15).  Then a dozen roundings of the score in base 2, exponentials
    and logarithm (2^-21), and the sum over n keys, n / 64 + 20 additions in a row."""
    n, H = 300, 2
    g = torch.Generator().manual_seed(D + B + window)
    c, table = fill_cache(q4, g, [n], H, D, B, 64)
    at = table[0, torch.arange(n) // 64].long(), torch.arange(n) % 64
    k = values(c.k_codes, c.k_state)[at[0], :, at[1]]  # [n, H, D]
    s = c.k_state.cpu().double()[at[0], :, at[1]][..., 0].repeat_interleave(B, -1)
    rest = k - k.half().double()
    q = torch.where(rest != 0, rest.sign(), torch.randn(n, H, D, generator=g).sign().double())
    q = (q * (1 + torch.randint(0, 8, q.shape, generator=g) / 8)).half()
    lse = q4.kv_attention(q.cuda(), c, table.cuda(), ints([n]), ints([0, n]), max_q=1 if few else n, window=window,
                          return_lse=True)[1].double().cpu()
    scale = D ** -0.5
    seen = torch.ones(n, n).tril().bool() & (torch.ones(n, n).triu().bool() if window else True)
    step = 2.0 ** -23
    for h in range(H):
        qh = q[:, h].double()
        want = torch.logsumexp((qh @ k[:, h].t() * scale).masked_fill(~seen, -math.inf), 1)
        if few:
            most = 8 if window else 15
            off = most * (D / 16 * 17 * step + (D + 4) * step / 2) * (qh.abs() @ s[:, h].t())
        else:
            off = D / 8 * 17 * step * (qh.abs() @ k[:, h].abs().t())
        x = qh @ k[:, h].t() * scale
        tol = scale * torch.where(seen, off, 0.0).amax(1) + 12 * step / 2 * (1.45 * torch.where(seen, x.abs(), 0.0).amax(1) + 16)
        tol += 2.0 ** -21 + (0 if window else (n / 64 + 20) * step / 2)
        assert ((lse[:, h] - want).abs() <= tol).all(), ((lse[:, h] - want).abs() / tol).max()
        if window and not few:  # keys rounded to binary16 would not pass
            lost = scale * (qh * rest[:, h]).sum(1).abs()
            assert (lost > tol).double().mean() > 0.5
    assert q4.last_device_status() == 0


@pytest.mark.parametrize("D,B,qh,kh", [(64, 64, 9, 3), (128, 64, 8, 2), (128, 128, 4, 4)])
@pytest.mark.parametrize("lens,qs", [([129, 600], [129, 300]), ([9000], [260]), ([700] * 20, [3] * 20)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 100)])
def test_the_call_without_the_log_sum_exp(q4, D, B, qh, kh, lens, qs, causal, window):
    """The default: prompts run another loop, with the keys rounded to binary16 (inside the reference's bound)."""
    g = torch.Generator().manual_seed(sum(lens) + D)
    dtype = torch.float16 if B == 64 else torch.bfloat16
    c, table = fill_cache(q4, g, lens, kh, D, B, 64, dtype)
    q = torch.randn(sum(qs), qh, D, generator=g).to(dtype)
    out = q4.kv_attention(q.cuda(), c, table.cuda(), ints(lens), ints([0] + list(np.cumsum(qs))), max_q=max(qs),
                          causal=causal, window=window)
    ref, _, tol, _ = reference(c, table, lens, qs, q, D ** -0.5, causal, window)
    assert ((out.double().cpu() - ref).abs() <= tol + HALF[dtype] * (ref.abs() + tol) + 2.0 ** -25).all()
    assert q4.last_device_status() == 0
