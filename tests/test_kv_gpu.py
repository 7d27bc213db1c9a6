"""The paged 4-bit key/value cache and the attention over it on a B200, against
the 4-bit oracle and 64-bit arithmetic."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import bits, is_bf16

pytestmark = pytest.mark.gpu
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a step, relative
NONFINITE, INDEX = 1, 8


@pytest.fixture(scope="module")
def q4():
    from bit_blockwise_weight_absmax_b200 import build
    build.build()
    from bit_blockwise_weight_absmax_b200 import q4
    q4.clear_device_status()
    yield q4
    q4.clear_device_status()


def values(codes, state):
    """The binary64 values of cached vectors [..., D], from the documented layout (on the CPU)."""
    codes, state = codes.cpu(), state.cpu().double()
    nb, d = state.shape[-2], 2 * codes.shape[-1]
    e = torch.arange(d)
    j, i = e // (d // nb), e % (d // nb)
    byte = ((i // 8) * nb + j) * 4 + (i % 8) // 2
    q = (codes[..., byte].to(torch.int64) >> (4 * (i % 2))) % 16
    return state[..., j, 0] * (q - state[..., j, 1])


# -------------------------------------------------------------- append, dequantize ----

@pytest.mark.parametrize("D,B", [(64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,heads,page", [(1, 1, 16), (5, 3, 32), (33, 8, 64), (130, 2, 256), (17, 5, 128)])
def test_append_is_the_asymmetric_rule_bit_for_bit(q4, oracle, D, B, dtype, tokens, heads, page):
    g = torch.Generator().manual_seed(tokens + D + B + heads)
    k, v = (torch.randn(tokens, heads, D, generator=g) * torch.exp(2 * torch.randn(tokens, heads, 1, generator=g))
            for _ in range(2))
    k[0] = 0
    k[-1, 0] = k[-1, 0].abs() + 1  # a block without negative values
    v[-1, -1] *= 1e-6              # a subnormal binary16 scale
    k, v = k.to(dtype), v.to(dtype)
    pages = (tokens + page - 1) // page + 2
    c = q4.kv_cache(pages, heads, D, page, B)
    slots = torch.randperm(pages * page, generator=g)[:tokens]
    for t in (c.k_codes, c.v_codes):
        t.fill_(0xAB)
    for t in (c.k_state, c.v_state):
        t.fill_(float("nan"))
    q4.kv_append(c, k.cuda(), v.cuda(), slots.cuda())
    for x, codes, state in ((k, c.k_codes, c.k_state), (v, c.v_codes, c.v_state)):
        ost = oracle.quantize(bits(x), is_bf16(x), B, oracle.QT_INT4_ASYM, False, True)
        nb = D // B
        z = np.empty(2 * ost.zero.size, dtype=np.uint8)
        z[0::2], z[1::2] = ost.zero & 15, ost.zero >> 4
        s = ost.scale_f16_bits().view(np.float16).reshape(tokens, heads, nb)
        got = state.cpu().numpy().transpose(0, 2, 1, 3, 4).reshape(-1, heads, nb, 2)[slots.numpy()]
        assert np.array_equal(got[..., 0], s) and np.array_equal(got[..., 1], z[:tokens * heads * nb].reshape(s.shape))
        want = ost.codes().reshape(tokens, heads, nb, B // 8, 8).swapaxes(2, 3).reshape(tokens, heads, D // 2, 2)
        got = codes.cpu().numpy().transpose(0, 2, 1, 3).reshape(-1, heads, D // 2)
        assert np.array_equal(got[slots.numpy()], want[..., 0] | (want[..., 1] << 4))
        rest = np.ones(pages * page, dtype=bool)
        rest[slots.numpy()] = False
        assert (got[rest] == 0xAB).all()  # no other place is written
    for out in (torch.float16, torch.bfloat16):
        for x, codes, state in zip(q4.kv_dequantize(c, slots.cuda(), out), (c.k_codes, c.v_codes), (c.k_state, c.v_state)):
            ref = values(codes, state).transpose(1, 2).reshape(-1, heads, D)[slots]
            assert torch.equal(x.cpu(), ref.to(out))
    assert q4.last_device_status() == 0


def test_append_passes_over_slots_and_takes_strides(q4):
    g = torch.Generator().manual_seed(1)
    T, H, D = 9, 2, 128
    qkv = torch.randn(T, 3 * H, D, generator=g).half().cuda()  # a fused projection's keys and values
    k, v = qkv[:, H:2 * H], qkv[:, 2 * H:]
    a, b = (q4.kv_cache(3, H, D, 16, 64) for _ in range(2))
    for c in (a, b):
        for t in (c.k_codes, c.v_codes, c.k_state, c.v_state):
            t.zero_()
    slots = torch.tensor([0, -1, 47, 5, -7, 16, 31, 32, 6], device="cuda")
    q4.kv_append(a, k, v, slots)
    keep = slots >= 0
    q4.kv_append(b, k[keep].contiguous(), v[keep].contiguous(), slots[keep])
    assert torch.equal(a.k_codes, b.k_codes) and torch.equal(a.v_state, b.v_state)
    assert q4.last_device_status() == 0
    kd, vd = q4.kv_dequantize(a, slots)
    assert not kd[~keep].any() and not vd[~keep].any() and kd[keep].any(-1).all()
    odd = torch.randn(T, H, D + 1, generator=g).half().cuda()[:, :, 1:]  # vectors at odd addresses: copied
    q4.kv_append(b, odd, odd, slots)
    q4.kv_append(a, odd.contiguous(), odd.contiguous(), slots)
    assert torch.equal(a.k_codes, b.k_codes)
    q4.kv_append(a, k[:0], v[:0], slots[:0])
    assert q4.kv_dequantize(a, slots[:0])[0].shape == (0, H, D)


def test_slots_past_the_cache_are_passed_over_and_reported(q4):
    c = q4.kv_cache(2, 1, 64, 16, 64)
    for t in (c.k_codes, c.v_codes, c.k_state, c.v_state):
        t.zero_()
    x = torch.ones(3, 1, 64, dtype=torch.float16, device="cuda")
    slots = torch.tensor([32, 1 << 40, 31], device="cuda")
    q4.kv_append(c, x, x, slots)
    assert q4.last_device_status() == INDEX
    q4.clear_device_status()
    assert int((c.k_codes != 0).any(-1).sum()) == 1
    k, _ = q4.kv_dequantize(c, slots)
    assert q4.last_device_status() == INDEX
    q4.clear_device_status()
    assert not k[:2].any() and (k[2] != 0).all()


@pytest.mark.parametrize("bad", [float("inf"), float("nan"), 65000.0])
def test_blocks_that_cannot_be_held_become_nan(q4, bad):
    c = q4.kv_cache(1, 2, 128, 16, 64)
    x = torch.ones(2, 2, 128, dtype=torch.float16, device="cuda")
    x[1, 0, 70] = bad
    q4.kv_append(c, x, x, torch.tensor([3, 4], device="cuda"))
    assert q4.last_device_status() == NONFINITE
    q4.clear_device_status()
    k, v = q4.kv_dequantize(c, torch.tensor([3, 4], device="cuda"))
    for t in (k, v):
        nan = torch.isnan(t)
        assert nan[1, 0, 64:].all() and int(nan.sum()) == 64


# -------------------------------------------------------------------------- attention ----

def fill_cache(q4, g, lens, heads, D, B, page, dtype=torch.float16, spare=3, size=1.0):
    """A cache with a shuffled table, its places past the lengths holding NaN; the tables' rest points nowhere."""
    need = [(n + page - 1) // page for n in lens]
    pages = sum(need) + spare
    c = q4.kv_cache(pages, heads, D, page, B)
    for t in (c.k_codes, c.v_codes):
        t.fill_(0xF7)
    for t in (c.k_state, c.v_state):
        t.fill_(float("nan"))
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    slots, at = [], 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        j = torch.arange(n)
        slots.append(table[b, j // page].long() * page + j % page)
    slots = torch.cat(slots)
    k = torch.randn(len(slots), heads, D, generator=g) * torch.exp(0.5 * torch.randn(D, generator=g)) * size
    v = torch.randn(len(slots), heads, D, generator=g) + torch.randn(D, generator=g)
    if len(slots):
        q4.kv_append(c, k.to(dtype).cuda(), v.to(dtype).cuda(), slots.cuda())
    return c, table


def reference(c, table, lens, qs, q, scale, causal, window):
    """(out, lse, bound of out, bound of lse) in binary64.  The bounds: keys, values and weights may each be rounded to
    binary16 on the way (half a step, 2^-11, each), so a score is off by at most 2^-11 sum |q k| scale, plus a
    binary32 sum's 2^-24 per term and addition (D + 2 of them, on codes of up to 15 before the zero-point of up to 15
    is taken off: 30 |q| s each)."""
    D, heads = c.head_dim, c.kv_heads
    k_all, v_all = values(c.k_codes, c.k_state), values(c.v_codes, c.v_state)
    ks, vs = c.k_state[..., 0].cpu().double(), c.v_state[..., 0].cpu().double()
    group = q.shape[1] // heads
    q = q.cpu().double()
    out = torch.zeros(q.shape, dtype=torch.float64)
    tol = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    ltol = torch.zeros(q.shape[:2], dtype=torch.float64)
    row = 0
    for b, (n, length) in enumerate(zip(qs, lens)):
        if n == 0 or length == 0:
            row += n
            continue
        pg = table[b, :(length + c.page_size - 1) // c.page_size].long()
        pos = torch.arange(length - n, length)[:, None]
        j = torch.arange(length)[None]
        seen = (j <= pos) if causal else torch.ones(n, length, dtype=torch.bool)
        if window:
            seen = seen & (j > pos - window)
        for h in range(q.shape[1]):
            hk = h // group
            k = k_all[pg, hk].reshape(-1, D)[:length]
            v = v_all[pg, hk].reshape(-1, D)[:length]
            s, sv = (x[pg, hk].reshape(-1, x.shape[-1])[:length].repeat_interleave(D // x.shape[-1], 1) for x in (ks, vs))
            qh = q[row:row + n, h]
            x = (qh @ k.t() * scale).masked_fill(~seen, -math.inf)
            dx = abs(scale) * (2.0 ** -11 * (qh.abs() @ k.abs().t()) + (D + 2) * 2.0 ** -24 * (qh.abs() @ (30 * s).t()))
            dx = torch.where(seen, dx, 0.0).amax(1) + 2.0 ** -20  # 2^-20: the exponential
            some = seen.any(1)
            m = torch.logsumexp(x, 1)
            p = torch.where(some[:, None], torch.exp(x - torch.where(some, m, 0.0)[:, None]), 0.0)
            out[row:row + n, h] = p @ v
            lse[row:row + n, h] = torch.where(some, m, -math.inf)
            # e^dx - 1 on every weight and on their sum, 2^-11 on weights and values each; weights below binary16's
            # smallest normal lose up to 2^-24 of the largest weight's value each
            rel = 2 * torch.expm1(dx) + 2.0 ** -10 + 2.0 ** -20
            tiny = 2.0 ** -23 * length
            tol[row:row + n, h] = rel[:, None] * (p @ v.abs()) + tiny * p.amax(1, keepdim=True) * v.abs().amax(0)
            # sum w code - sum w z, each up to 15 sum w s, where both are summed in binary32: a step of 2^-23 for each
            # of length / 16 accumulations of 16 keys and of the joins of up to 32 partial sums
            tol[row:row + n, h] += (length / 16 + 32) * 2.0 ** -23 * 15 * (p @ sv)
            ltol[row:row + n, h] = dx + 2.0 ** -22 * (m.abs().nan_to_num(posinf=0) + 1)
        row += n
    return out, lse, tol, ltol


def check(q4, c, table, lens, qs, q, scale=None, causal=True, window=0, implicit=True, **kw):
    dev = q.cuda() if not q.is_cuda else q
    cu = torch.tensor([0] + list(np.cumsum(qs)), dtype=torch.int32, device="cuda")
    args = (dev, c, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
            None if implicit and all(n == 1 for n in qs) else cu)
    out, lse = q4.kv_attention(*args, scale=scale, causal=causal, window=window, return_lse=True, max_q=max(qs + [1]), **kw)
    ref, rl, tol, ltol = reference(c, table, lens, qs, q, 1 / math.sqrt(c.head_dim) if scale is None else scale, causal, window)
    off = (out.double().cpu() - ref).abs()
    tol = tol + HALF[q.dtype] * (ref.abs() + tol) + 2.0 ** -25
    assert torch.isfinite(out).all()
    assert (off <= tol).all(), (off / tol).max()
    empty = rl == -math.inf
    assert torch.equal(lse.cpu() == -math.inf, empty) and not out[empty.cuda()].any()
    assert ((lse.double().cpu() - rl).abs()[~empty] <= ltol[~empty]).all()
    again = q4.kv_attention(*args, scale=scale, causal=causal, window=window, return_lse=True, max_q=max(qs + [1]), **kw)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert q4.last_device_status() == 0
    return out, lse


FORMATS = [(64, 64, 9, 3), (128, 64, 8, 2), (128, 128, 4, 4)]


@pytest.mark.parametrize("D,B,qh,kh", FORMATS + [(128, 64, 24, 2), (64, 64, 20, 1), (128, 128, 16, 1)])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_single_tokens_over_ragged_lengths(q4, D, B, qh, kh, page, dtype):
    g = torch.Generator().manual_seed(D + B + page + qh)
    lens = [1, 15, 16, 17, 31, 33, 64, 0, 100, 255, 257, 700]
    c, table = fill_cache(q4, g, lens, kh, D, B, page, dtype)
    check(q4, c, table, lens, [1] * len(lens), torch.randn(len(lens), qh, D, generator=g).to(dtype))


@pytest.mark.parametrize("D,B,qh,kh", FORMATS)
@pytest.mark.parametrize("length", [1, 2, 63, 65, 1000, 5003])
def test_one_sequence(q4, D, B, qh, kh, length):
    g = torch.Generator().manual_seed(length + D)
    c, table = fill_cache(q4, g, [length], kh, D, B, 32)
    check(q4, c, table, [length], [1], torch.randn(1, qh, D, generator=g).half())


@pytest.mark.parametrize("D,B,qh,kh", FORMATS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 20, 130])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_several_rows_a_sequence(q4, D, B, qh, kh, causal, window, dtype):
    g = torch.Generator().manual_seed(D + window)
    lens, qs = [40, 5, 200, 3, 0, 130, 70], [4, 5, 7, 0, 0, 2, 33]
    c, table = fill_cache(q4, g, lens, kh, D, B, 16, dtype)
    check(q4, c, table, lens, qs, torch.randn(sum(qs), qh, D, generator=g).to(dtype), causal=causal, window=window)


@pytest.mark.parametrize("D,B,qh,kh", FORMATS)
@pytest.mark.parametrize("lens,qs", [([127], [127]), ([128, 129], [128, 129]), ([500, 300, 40], [200, 300, 7]),
                                     ([1025], [600]), ([64, 900, 2, 333], [64, 450, 1, 333])])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 100), (False, 64)])
def test_prompts(q4, D, B, qh, kh, lens, qs, causal, window):
    g = torch.Generator().manual_seed(sum(lens) + D)
    dtype = torch.bfloat16 if B == 64 else torch.float16
    c, table = fill_cache(q4, g, lens, kh, D, B, 64, dtype)
    check(q4, c, table, lens, qs, torch.randn(sum(qs), qh, D, generator=g).to(dtype), causal=causal, window=window)


@pytest.mark.parametrize("rows", [3, 40, 300])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_in_front_of_every_key_are_empty(q4, rows, causal):
    """More query rows than keys: the first rows stand before position 0."""
    g = torch.Generator().manual_seed(rows)
    lens, qs = [rows - 2, rows // 2], [rows, rows]
    c, table = fill_cache(q4, g, lens, 2, 128, 64, 16)
    check(q4, c, table, lens, qs, torch.randn(2 * rows, 4, 128, generator=g).half(), causal=causal, window=0 if causal else 1)


@pytest.mark.parametrize("rows", [1, 6, 200])
def test_large_scores_and_scales(q4, rows):
    """Scores of several hundred (one key takes nearly all), a negative scale, values of very different sizes."""
    g = torch.Generator().manual_seed(rows)
    c, table = fill_cache(q4, g, [900], 2, 128, 64, 32, size=8.0)
    q = (torch.randn(rows, 8, 128, generator=g) * 4).half()
    qs = [rows]
    for scale in (0.02, -0.02):
        check(q4, c, table, [900], qs, q, scale=scale, implicit=False)


@pytest.mark.parametrize("rows", [1, 5, 150])
def test_queries_of_any_size(q4, rows):
    """bf16 queries far outside binary16's range, and tiny ones."""
    g = torch.Generator().manual_seed(rows + 1)
    c, table = fill_cache(q4, g, [300], 1, 128, 128, 16, torch.bfloat16)
    q = torch.randn(rows, 3, 128, generator=g)
    check(q4, c, table, [300], [rows], (q * 1e30).bfloat16(), scale=1e-31, implicit=False)
    check(q4, c, table, [300], [rows], (q * 1e-30).bfloat16(), scale=1e29, implicit=False)
    check(q4, c, table, [300], [rows], (q * 0).bfloat16(), implicit=False)


@pytest.mark.parametrize("rows", [1, 4, 140])
def test_values_of_any_size(q4, rows):
    """Values of one head very small, another's large, constant ones, zeros."""
    g = torch.Generator().manual_seed(rows + 2)
    n, D = 333, 64
    c = q4.kv_cache(8, 4, D, 64, 64)
    k, v = torch.randn(2, n, 4, D, generator=g)
    v[:, 0] *= 2e-4
    v[:, 1] *= 3000
    v[:, 2] = 0
    v[:, 3] = 1
    v[::3, 1] *= 1e-6
    slots = torch.arange(n)
    q4.kv_append(c, k.half().cuda(), v.half().cuda(), slots.cuda())
    table = torch.arange(8, dtype=torch.int32)[None]
    check(q4, c, table, [n], [rows], torch.randn(rows, 8, D, generator=g).half(), implicit=False)


def test_long_cache_whose_offsets_pass_32_bits(q4):
    """More than 2^32 bytes of codes: the last pages are read at their places."""
    D, heads, page = 128, 32, 256
    pages = (1 << 32) // (heads * page * 64) + 40
    c = q4.kv_cache(pages, heads, D, page, 128)
    g = torch.Generator().manual_seed(9)
    n = 300
    table = torch.tensor([[pages - 1, pages - 39]], dtype=torch.int32)
    j = torch.arange(n)
    slots = table[0, j // page].long() * page + j % page
    k, v = torch.randn(2, n, heads, D, generator=g).half().cuda()
    q4.kv_append(c, k, v, slots.cuda())
    kd, vd = q4.kv_dequantize(c, slots.cuda())
    assert ((kd - k).float().norm() / k.float().norm()).item() < 0.15
    small = q4.kv_cache(2, heads, D, page, 128)
    t2 = torch.tensor([[1, 0]], dtype=torch.int32)
    q4.kv_append(small, k, v, (t2[0, j // page].long() * page + j % page).cuda())
    for rows in (1, 3, 200):
        q = torch.randn(rows, heads, D, generator=g).half().cuda()
        lens, cu = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        a = q4.kv_attention(q, c, table.cuda(), lens, cu)
        b = q4.kv_attention(q, small, t2.cuda(), lens, cu)
        assert torch.equal(a, b) and torch.isfinite(a).all()
    assert q4.last_device_status() == 0


@pytest.mark.parametrize("rows", [1, 7, 160])
def test_strides_rows_outside_and_padded_batches(q4, rows):
    g = torch.Generator().manual_seed(rows + 4)
    H, D, lens = 4, 128, [rows + 30, rows]
    c, table = fill_cache(q4, g, lens, 2, D, 64, 16)
    qkv = torch.randn(2 * rows + 3, H + 4, D, generator=g).bfloat16().cuda()
    q = qkv[:, :H]  # heads of a fused projection
    wide = torch.full((2, table.shape[1] + 5), 9999, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    tb = wide.cuda()[:, :table.shape[1]]
    cu = torch.tensor([1, rows + 1, 2 * rows + 1], dtype=torch.int32, device="cuda")
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full((2 * rows + 3, H, D), 5.0, dtype=torch.bfloat16, device="cuda")
    q4.kv_attention(q, c, tb, ln, cu, out=out)
    want = q4.kv_attention(q[1:2 * rows + 1].contiguous(), c, table.cuda(), ln, cu - 1)
    assert torch.equal(out[1:2 * rows + 1], want)
    assert (out[0] == 5).all() and (out[2 * rows + 1:] == 5).all()
    # padded sequences: no rows, no keys
    cu2 = torch.cat([cu, cu[-1:], cu[-1:]])
    ln2 = torch.cat([ln, ln[:1] * 0, ln[:1]])
    tb2 = torch.cat([table, torch.full_like(table, -1)]).cuda()
    tb2[3, 0] = int(table[0, 0])
    assert torch.equal(q4.kv_attention(q, c, tb2, ln2, cu2, out=out.clone()), out)
    assert q4.last_device_status() == 0


@pytest.mark.parametrize("rows", [1, 5, 140])
def test_bad_pages_lengths_and_ranges_are_cut_off_and_reported(q4, rows):
    g = torch.Generator().manual_seed(rows)
    c, table = fill_cache(q4, g, [200], 1, 64, 64, 16)
    q = torch.randn(rows, 2, 64, generator=g).half().cuda()
    lens = torch.tensor([200], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    good = q4.kv_attention(q, c, table.cuda(), lens, cu)
    assert q4.last_device_status() == 0
    for bad in (-1, c.pages, 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = bad
        out = q4.kv_attention(q, c, t.cuda(), lens, cu)
        assert q4.last_device_status() == INDEX and torch.isfinite(out).all()
        q4.clear_device_status()
    for n in (10 ** 9, -4):
        out = q4.kv_attention(q, c, table.cuda(), lens * 0 + n, cu)
        assert q4.last_device_status() == INDEX
        q4.clear_device_status()
    assert not out.any()  # a negative length: no keys
    out = torch.zeros_like(q)
    q4.kv_attention(q, c, table.cuda(), lens, torch.tensor([0, rows + 9], dtype=torch.int32, device="cuda"), out=out)
    assert q4.last_device_status() == INDEX
    q4.clear_device_status()
    q4.kv_attention(q, c, table.cuda(), lens, torch.tensor([rows, 0], dtype=torch.int32, device="cuda"), out=out)
    assert q4.last_device_status() == INDEX
    q4.clear_device_status()
    assert torch.equal(q4.kv_attention(q, c, table.cuda(), lens, cu, max_q=1), q4.kv_attention(q, c, table.cuda(), lens, cu, max_q=1))
    assert good.any()


@pytest.mark.parametrize("rows", [1, 130])
def test_nan_states_reach_the_rows_that_attend_to_them(q4, rows):
    g = torch.Generator().manual_seed(rows)
    for name in ("k_state", "v_state"):
        c, table = fill_cache(q4, g, [260, 260], 2, 128, 64, 64)
        getattr(c, name)[int(table[0, 1]), 1, 3, 1, 0] = float("nan")  # key 67 of the first sequence, head 1
        q = torch.randn(2 * rows, 2, 128, generator=g).half().cuda()
        out = q4.kv_attention(q, c, table.cuda(), torch.tensor([260, 260], dtype=torch.int32, device="cuda"),
                              torch.tensor([0, rows, 2 * rows], dtype=torch.int32, device="cuda"))
        assert torch.isfinite(out[:, 0]).all() and torch.isfinite(out[rows:]).all()
        assert torch.isnan(out[:rows, 1]).any(-1).all()


@pytest.mark.parametrize("rows,length,at", [(5, 40, 37), (300, 300, 150), (200, 700, 600)])
@pytest.mark.parametrize("name", ["k_state", "v_state"])
def test_nan_states_spare_the_rows_in_front_of_them(q4, rows, length, at, name):
    """A bad block meets zero weights in the rows that do not attend to its key: they keep their values."""
    g = torch.Generator().manual_seed(rows)
    c, table = fill_cache(q4, g, [length], 2, 128, 64, 64)
    q = torch.randn(rows, 4, 128, generator=g).half().cuda()
    args = (q, c, table.cuda(), torch.tensor([length], dtype=torch.int32, device="cuda"),
            torch.tensor([0, rows], dtype=torch.int32, device="cuda"))
    want = q4.kv_attention(*args)
    getattr(c, name)[int(table[0, at // 64]), 1, at % 64, 0, 0] = float("nan")
    out = q4.kv_attention(*args)
    before = at - (length - rows)  # rows in front of the key
    assert torch.equal(out[:, :2], want[:, :2]) and torch.equal(out[:before], want[:before])
    assert torch.isnan(out[before:, 2:]).any(-1).all()


def test_an_attention_block_in_a_graph_and_on_streams(q4):
    """Projections in 8-bit integers, the cache, attention and a 4-bit output projection as they are used together:
    eagerly, captured once and replayed for later tokens, and two batches at once on two streams."""
    from bit_blockwise_weight_absmax_b200 import linear4bit, linear8bit
    torch.manual_seed(0)
    hid, H, KH, D, page = 512, 8, 2, 64, 16
    qkv = linear8bit.Linear8bit.from_linear(torch.nn.Linear(hid, (H + 2 * KH) * D).bfloat16().cuda(), torch.bfloat16)
    o = linear4bit.Linear4bit.from_linear(torch.nn.Linear(H * D, hid, bias=False).bfloat16().cuda(), compute_dtype=torch.bfloat16)

    def block(x, c, table, slots, lens, cu=None, max_q=None):
        y = qkv(x).view(-1, H + 2 * KH, D)
        q4.kv_append(c, y[:, H:H + KH], y[:, H + KH:], slots)
        a = q4.kv_attention(y[:, :H], c, table, lens, cu, max_q=max_q)
        return o(a.view(-1, H * D)), a, y

    def start(seed):
        g = torch.Generator().manual_seed(seed)
        c = q4.kv_cache(40, KH, D, page, 64)
        table = torch.randperm(40, generator=g)[:24].view(2, 12).to(torch.int32)
        return g, c, table

    def slot(table, b, j):
        return table[b, j // page].long() * page + j % page

    def prompt(g, c, table, lens):
        x = torch.randn(sum(lens), hid, generator=g).bfloat16().cuda()
        slots = torch.cat([slot(table, b, torch.arange(n)) for b, n in enumerate(lens)]).cuda()
        cu = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda")
        return block(x, c, table.cuda(), slots, torch.tensor(lens, dtype=torch.int32, device="cuda"), cu, max(lens))

    g, c, table = start(1)
    lens = [70, 33]
    _, a, y = prompt(g, c, table, lens)
    ref, _, tol, _ = reference(c, table, lens, lens, y[:, :H], 1 / 8, True, 0)
    assert ((a.double().cpu() - ref).abs() <= tol + HALF[a.dtype] * (ref.abs() + tol) + 2.0 ** -25).all()
    # decode: captured once, replayed with new inputs
    xs = torch.zeros(2, hid, dtype=torch.bfloat16, device="cuda")
    slots, ln, tb = torch.zeros(2, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"), table.cuda()

    def step_inputs(i):
        xs.copy_(torch.randn(2, hid, generator=torch.Generator().manual_seed(100 + i)))
        slots.copy_(torch.stack([slot(table, b, torch.tensor(lens[b] + i)) for b in range(2)]))
        ln.copy_(torch.tensor([n + i + 1 for n in lens]))

    step_inputs(0)
    block(xs, c, tb, slots, ln)  # also warms up
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = block(xs, c, tb, slots, ln)
    for i in range(1, 40):
        step_inputs(i)
        graph.replay()
        if i % 13 == 0:
            got = [t.clone() for t in res]
            now = [n + i + 1 for n in lens]
            ref, _, tol, _ = reference(c, table, now, [1, 1], got[2][:, :H], 1 / 8, True, 0)
            assert ((got[1].double().cpu() - ref).abs() <= tol + HALF[a.dtype] * (ref.abs() + tol) + 2.0 ** -25).all()
            eager = block(xs, c, tb, slots, ln)
            assert all(torch.equal(u, v) for u, v in zip(got, eager))
    # two batches at once on two streams
    both = [start(s) for s in (2, 3)]
    want = [prompt(*b, lens)[0] for b in both]
    both = [start(s) for s in (2, 3)]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    got = []
    for b, s in zip(both, streams):
        with torch.cuda.stream(s):
            got.append(prompt(*b, lens)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    assert q4.last_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows", [2, 14, 150])
def test_queries_that_are_not_finite_spoil_their_own_rows(q4, rows, dtype):
    g = torch.Generator().manual_seed(rows)
    c, table = fill_cache(q4, g, [500], 2, 128, 64, 64)
    q = torch.randn(rows, 4, 128, generator=g).to(dtype).cuda()
    args = (c, table.cuda(), torch.tensor([500], dtype=torch.int32, device="cuda"),
            torch.tensor([0, rows], dtype=torch.int32, device="cuda"))
    _, _, tol, _ = reference(c, table, [500], [rows], q, 128 ** -0.5, True, 0)
    want = q4.kv_attention(q, *args)
    bad = torch.zeros(rows, 4, dtype=torch.bool)
    for row, head, value in ((0, 1, math.nan), (rows // 2, 3, math.inf), (rows - 1, 0, -math.inf)):
        q[row, head, 5] = value
        bad[row, head] = True
    out = q4.kv_attention(q, *args).cpu()
    assert torch.isnan(out[bad]).all()
    # the others: both within the bound (the reference of a softmax may move at another unit of keys)
    off, tol = (out.double() - want.cpu().double()).abs(), 2 * (tol + HALF[dtype] * (want.cpu().double().abs() + tol) + 2.0 ** -25)
    assert (off <= tol)[~bad].all()


def test_row_ranges_that_overlap_leave_the_workspace_usable(q4):
    """The second range begins before the first ends: more row tiles than rows.  No result is promised, but the next
    call's is right."""
    g = torch.Generator().manual_seed(5)
    rows, length = 2432, 20000  # 38 tiles of 256 rows for each of the four ranges: past the SMs by a few
    c, table = fill_cache(q4, g, [length], 1, 64, 64, 64)
    q = torch.randn(rows, 4, 64, generator=g).half().cuda()
    args = (q, c, table.cuda().expand(8, -1), torch.full((8,), length, dtype=torch.int32, device="cuda"))
    fine = torch.arange(9, dtype=torch.int32, device="cuda") * (rows // 8)
    over = torch.tensor([0, rows] * 4 + [0], dtype=torch.int32, device="cuda")
    for max_q in (8, rows):
        want = q4.kv_attention(*args, fine, max_q)
        q4.kv_attention(*args, over, max_q)
        q4.clear_device_status()
        assert torch.equal(q4.kv_attention(*args, fine, max_q), want)
        assert q4.last_device_status() == 0


@pytest.mark.parametrize("rows,length", [(1, 100), (3, 40000), (300, 700), (130, 30000)])
def test_wait_limit_times_out_and_recovers(q4, rows, length):
    """With the copy-stall hook on no keys arrive: the waits run out, the call reports it, and after the workspaces are
    zeroed again the next call is right (whole segments and parts that are joined, both kernels)."""
    g = torch.Generator().manual_seed(rows)
    c, table = fill_cache(q4, g, [length], 1, 64, 64, 64)
    q = torch.randn(rows, 2, 64, generator=g).half()
    args = (q.cuda(), c, table.cuda(), torch.tensor([length], dtype=torch.int32, device="cuda"),
            torch.tensor([0, rows], dtype=torch.int32, device="cuda"))
    try:
        q4.set_wait_limit_ns(200_000)
        q4.set_copy_stall(True)
        q4.kv_attention(*args)
        torch.cuda.synchronize()
        assert q4.last_device_status() & 2  # Q4_STATUS_TIMEOUT
    finally:
        q4.set_copy_stall(False)
        q4.set_wait_limit_ns(0)
        q4.reset_workspaces()
        q4.clear_device_status()
    check(q4, c, table, [length], [rows], q, implicit=False)


@pytest.mark.parametrize("rows", [1, 9, 200])
def test_windows_longer_than_every_sequence_are_none(q4, rows):
    """The first rows stand in front of position 0, where a far window's begin would leave 32 bits."""
    g = torch.Generator().manual_seed(rows)
    lens, qs = [rows, max(rows - 5, 1)], [rows, rows]
    c, table = fill_cache(q4, g, lens, 2, 64, 64, 16)
    q = torch.randn(2 * rows, 4, 64, generator=g).half()
    want = check(q4, c, table, lens, qs, q, implicit=False)
    for window in (rows, 10 ** 6, 2 ** 31 - 1, 2 ** 40):
        got = check(q4, c, table, lens, qs, q, window=window, implicit=False)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) or window == rows  # cut at other keys, it may round otherwise
