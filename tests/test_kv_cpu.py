"""The 4-bit key/value cache and its attention without a GPU: what the C ABI and
the binding refuse before anything is launched."""
import ctypes

import pytest
import torch

from bit_blockwise_weight_absmax_b200 import q4

ARG, SHAPE, ALIGN, NO_DEVICE, WORKSPACE = -1, -2, -3, -4, -7
A = 1 << 20  # a 16-byte aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    from bit_blockwise_weight_absmax_b200 import build
    build.build()
    return q4.library()


def cache(**kw):
    c = q4._CKVCache()
    base = dict(head_dim=128, blocksize=64, kv_heads=8, page_size=64, pages=10, k_codes=A, k_state=A, v_codes=A, v_state=A)
    for name, v in {**base, **kw}.items():
        setattr(c, name, v)
    return ctypes.byref(c)


def append(lib, c=None, K=A, V=A, dt=0, tokens=4, kt=1024, kh=128, vt=1024, vh=128, slots=A):
    return lib.q4_kv_append(c or cache(), K, V, dt, tokens, kt, kh, vt, vh, slots, None)


def deq(lib, c=None, slots=A, n=4, K=A, V=A, dt=0):
    return lib.q4_kv_dequantize(c or cache(), slots, n, K, V, dt, None)


def attend(lib, c=None, Q=A, dt=0, total=4, heads=64, qt=8192, qh=128, cu=None, lens=A, table=A, stride=5, pages=5, batch=4,
           max_q=1, scale=0.1, causal=1, window=0, out=A, lse=None, ws=A, wsb=1 << 40):
    return lib.q4_kv_attention(c or cache(), Q, dt, total, heads, qt, qh, cu, lens, table, stride, pages, batch, max_q,
                               scale, causal, window, out, lse, ws, wsb, None)


BAD_CACHES = [(dict(head_dim=96), ARG), (dict(head_dim=256), ARG), (dict(blocksize=32), ARG),
              (dict(head_dim=64, blocksize=128), ARG), (dict(page_size=8), ARG), (dict(page_size=48), ARG),
              (dict(page_size=512), ARG), (dict(k_codes=None), ARG), (dict(k_state=None), ARG), (dict(v_codes=None), ARG),
              (dict(v_state=None), ARG), (dict(kv_heads=0), SHAPE), (dict(pages=0), SHAPE), (dict(pages=1 << 31), SHAPE),
              (dict(k_codes=A + 8), ALIGN), (dict(k_state=A + 4), ALIGN), (dict(v_codes=A + 1), ALIGN),
              (dict(v_state=A + 2), ALIGN)]


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers: only where nothing can be launched")
def test_refusals(lib):
    assert append(lib) == deq(lib) == attend(lib) == NO_DEVICE
    for kw, rc in BAD_CACHES:
        assert append(lib, cache(**kw)) == deq(lib, cache(**kw)) == attend(lib, cache(**kw)) == rc, kw
    for kw, rc in [(dict(K=None), ARG), (dict(V=None), ARG), (dict(slots=None), ARG), (dict(dt=2), ARG),
                   (dict(tokens=0), SHAPE), (dict(kt=-8), SHAPE), (dict(K=A + 8), ALIGN), (dict(vt=1020), ALIGN),
                   (dict(kh=132), ALIGN)]:
        assert append(lib, **kw) == rc, kw
    for kw, rc in [(dict(K=None), ARG), (dict(slots=None), ARG), (dict(dt=2), ARG), (dict(n=0), SHAPE), (dict(V=A + 8), ALIGN)]:
        assert deq(lib, **kw) == rc, kw
    for kw, rc in [(dict(Q=None), ARG), (dict(lens=None), ARG), (dict(table=None), ARG), (dict(out=None), ARG),
                   (dict(dt=2), ARG), (dict(causal=2), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
                   (dict(total=5), SHAPE), (dict(heads=12), SHAPE), (dict(heads=0), SHAPE), (dict(batch=0, total=0), SHAPE),
                   (dict(window=-1), SHAPE), (dict(pages=0), SHAPE), (dict(stride=4), SHAPE), (dict(max_q=0), SHAPE),
                   (dict(pages=1 << 26, stride=1 << 26), SHAPE), (dict(batch=65536, total=65536), SHAPE),
                   (dict(Q=A + 8), ALIGN), (dict(out=A + 2), ALIGN), (dict(qt=8190), ALIGN), (dict(ws=A + 8), ALIGN)]:
        assert attend(lib, **kw) == rc, kw
    n = ctypes.c_size_t(0)
    assert lib.q4_kv_attention_workspace_size(cache(), 4, 4, 64, ctypes.byref(n)) == 0
    if n.value:
        assert attend(lib, ws=None) == attend(lib, wsb=n.value - 1) == WORKSPACE
    assert lib.q4_kv_attention_workspace_size(cache(), 4, 4, 64, None) == ARG


def test_kv_cache_refuses_formats_before_allocating():
    for kw in (dict(head_dim=96), dict(head_dim=64, blocksize=128), dict(head_dim=128, blocksize=32),
               dict(head_dim=128, page_size=48), dict(head_dim=128, pages=0), dict(head_dim=128, kv_heads=0)):
        with pytest.raises(q4.Q4Error):
            q4.kv_cache(**{**dict(pages=2, kv_heads=1, device="cpu"), **kw})


def test_binding_refuses_before_the_library():
    c = q4.kv_cache(4, 2, 64, 16, 64, device="cpu")
    assert (c.pages, c.kv_heads, c.head_dim, c.page_size, c.blocksize) == (4, 2, 64, 16, 64)
    assert c.held_bytes() == 2 * 4 * 2 * 16 * (32 + 4)
    with pytest.raises(q4.Q4Error, match="fixed"):
        c.k_codes = c.v_codes
    with pytest.raises(q4.Q4Error):
        q4.KVCache(c.k_codes, c.k_state.float(), c.v_codes, c.v_state)
    with pytest.raises(q4.Q4Error):
        q4.KVCache(c.k_codes, c.k_state[:, :, :8], c.v_codes, c.v_state)
    with pytest.raises(q4.Q4Error):
        q4.KVCache(c.k_codes, c.k_state, c.v_codes[:2], c.v_state)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_no_cpu_fallback():
    c = q4.kv_cache(4, 2, 64, 16, 64, device="cpu")
    x = torch.zeros(3, 2, 64, dtype=torch.float16)
    slots = torch.zeros(3, dtype=torch.int64)
    table, lens = torch.zeros(3, 1, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: q4.kv_append(c, x, x, slots), lambda: q4.kv_dequantize(c, slots),
                 lambda: q4.kv_attention(x, c, table, lens)):
        with pytest.raises(q4.Q4Error, match="no CUDA device"):
            call()
