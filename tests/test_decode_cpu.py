"""Refusals of the decoding step's calls: through the C ABI (argument errors are returned before any device
work, so they need no GPU) and through the binding's checks on CPU tensors."""
import ctypes

import pytest
import torch

import bit_integer_gemm_b200 as imq
from bit_integer_gemm_b200 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return imq.lib()


def _cache(**over):
    f = dict(k=4096, v=8192, steps=12288, n_pages=4, k_page_stride=2 * 16 * 64, v_page_stride=2 * 16 * 64,
             steps_page_stride=2 * 16 * 2, page_size=16, n_heads=2, head_dim=64, bits=8)
    f.update(over)
    return imq.imq_kv_cache(*[f[n] for n, _ in imq.imq_kv_cache._fields_])


P = 1 << 20  # a 16-byte aligned address that no refused call reads

W4 = dict(codes=P, ldc=64, steps=P, lds=1, K=128, N=16, group=128)
BAD_WEIGHT = [
    (dict(group=0), imq.IMQ_ERR_ARG), (dict(group=48), imq.IMQ_ERR_ARG), (dict(group=256), imq.IMQ_ERR_ARG),
    (dict(K=-1), imq.IMQ_ERR_ARG), (dict(N=-1), imq.IMQ_ERR_ARG), (dict(ldc=48), imq.IMQ_ERR_ARG),
    (dict(ldc=72), imq.IMQ_ERR_ARG), (dict(K=129), imq.IMQ_ERR_ARG), (dict(lds=0), imq.IMQ_ERR_ARG),
    (dict(codes=None), imq.IMQ_ERR_ARG), (dict(codes=P + 4), imq.IMQ_ERR_ARG), (dict(steps=None), imq.IMQ_ERR_ARG),
    (dict(steps=P + 2), imq.IMQ_ERR_ARG), (dict(K=1 << 31, ldc=1 << 40, lds=1 << 40), imq.IMQ_ERR_UNSUPPORTED),
    (dict(N=1 << 31), imq.IMQ_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("over,want", BAD_WEIGHT)
def test_bad_weights_are_refused(lib, over, want):
    w = {**W4, **over}
    big = 1 << 40
    assert lib.imq_w4_quantize(P, imq.IMQ_BF16, w["K"], w["N"], big, 0, w["group"], w["codes"], w["ldc"], w["steps"], w["lds"], None) == want
    h = tuple(w[k] for k in ("codes", "ldc", "steps", "lds", "K", "N", "group"))
    assert lib.imq_w4_dequantize(*h, P, imq.IMQ_BF16, big, 0, None) == want
    assert lib.imq_w4_matvec(*h, P, imq.IMQ_BF16, 1, big, P, imq.IMQ_BF16, big, None) == want


@pytest.mark.parametrize("over,want", [
    (dict(xt=imq.IMQ_I16), imq.IMQ_ERR_ARG), (dict(yt=imq.IMQ_I32), imq.IMQ_ERR_ARG), (dict(M=-1), imq.IMQ_ERR_ARG),
    (dict(ldx=127), imq.IMQ_ERR_ARG), (dict(ldy=15), imq.IMQ_ERR_ARG), (dict(X=None), imq.IMQ_ERR_ARG),
    (dict(Y=None), imq.IMQ_ERR_ARG), (dict(X=P + 1), imq.IMQ_ERR_ARG), (dict(Y=P + 2, yt=imq.IMQ_F32), imq.IMQ_ERR_ARG),
    (dict(M=1 << 40), imq.IMQ_ERR_UNSUPPORTED), (dict(M=0, X=None, Y=None), imq.IMQ_OK)])
def test_bad_products_are_refused(lib, over, want):
    a = {**dict(X=P, xt=imq.IMQ_BF16, M=1, ldx=128, Y=P, yt=imq.IMQ_BF16, ldy=16), **over}
    h = tuple(W4[k] for k in ("codes", "ldc", "steps", "lds", "K", "N", "group"))
    assert lib.imq_w4_matvec(*h, a["X"], a["xt"], a["M"], a["ldx"], a["Y"], a["yt"], a["ldy"], None) == want


@pytest.mark.parametrize("W,wt,ldw,trans", [(None, 1, 16, 0), (P, 2, 16, 0), (P, 1, 15, 0), (P, 1, 127, 1), (P, 1, 128, 2), (P + 1, 1, 128, 1)])
def test_bad_quantisations_are_refused(lib, W, wt, ldw, trans):
    assert lib.imq_w4_quantize(W, wt, 128, 16, ldw, trans, 128, P, 64, P, 1, None) == imq.IMQ_ERR_ARG
    assert lib.imq_w4_dequantize(P, 64, P, 1, 128, 16, 128, W, wt, ldw, trans, None) == imq.IMQ_ERR_ARG


BAD_CACHE = [
    (dict(bits=5), imq.IMQ_ERR_ARG), (dict(n_pages=-1), imq.IMQ_ERR_ARG), (dict(n_heads=0), imq.IMQ_ERR_ARG),
    (dict(page_size=0), imq.IMQ_ERR_ARG), (dict(head_dim=0), imq.IMQ_ERR_ARG), (dict(k=None), imq.IMQ_ERR_ARG),
    (dict(v=None), imq.IMQ_ERR_ARG), (dict(steps=None), imq.IMQ_ERR_ARG), (dict(k=4104), imq.IMQ_ERR_ARG),
    (dict(v=4104), imq.IMQ_ERR_ARG), (dict(steps=12292), imq.IMQ_ERR_ARG), (dict(k_page_stride=2032), imq.IMQ_ERR_ARG),
    (dict(v_page_stride=2056), imq.IMQ_ERR_ARG), (dict(steps_page_stride=62), imq.IMQ_ERR_ARG),
    (dict(steps_page_stride=66), imq.IMQ_ERR_ARG), (dict(head_dim=32), imq.IMQ_ERR_UNSUPPORTED),
    (dict(head_dim=96), imq.IMQ_ERR_UNSUPPORTED), (dict(head_dim=320), imq.IMQ_ERR_UNSUPPORTED),
    (dict(page_size=8), imq.IMQ_ERR_UNSUPPORTED), (dict(page_size=40), imq.IMQ_ERR_UNSUPPORTED),
    (dict(page_size=1 << 17), imq.IMQ_ERR_UNSUPPORTED), (dict(n_heads=65536), imq.IMQ_ERR_UNSUPPORTED),
    (dict(n_pages=1 << 31), imq.IMQ_ERR_UNSUPPORTED),
]


def _attend(lib, c, **over):
    a = dict(Q=P, qt=imq.IMQ_BF16, qb=128, qh=64, batch=1, heads=2, table=P, stride=4, width=4, lens=P, max_len=64, scale=1.0,
             out=P, ot=imq.IMQ_BF16, ob=128, oh=64, lse=P, lb=2, ws=P, wn=1 << 30)
    a.update(over)
    return lib.imq_paged_attention(None if c is None else ctypes.addressof(c), *a.values(), None)


@pytest.mark.parametrize("over,want", BAD_CACHE)
def test_bad_caches_are_refused(lib, over, want):
    c = _cache(**over)
    r = ctypes.addressof(c)
    n = ctypes.c_size_t(7)
    assert lib.imq_kv_write(r, P, 0, 0, P, 0, 0, imq.IMQ_BF16, 1, P, None) == want
    assert lib.imq_kv_read(r, P, 1, P, 0, 0, P, 0, 0, imq.IMQ_BF16, None) == want
    assert lib.imq_paged_attention_workspace(r, 1, 2, 64, ctypes.addressof(n)) == want and n.value == 7
    assert _attend(lib, c) == want


def test_missing_caches_are_refused(lib):
    assert lib.imq_kv_write(None, P, 0, 0, P, 0, 0, imq.IMQ_BF16, 1, P, None) == imq.IMQ_ERR_ARG
    assert lib.imq_kv_read(None, P, 1, P, 0, 0, P, 0, 0, imq.IMQ_BF16, None) == imq.IMQ_ERR_ARG
    assert _attend(lib, None) == imq.IMQ_ERR_ARG


@pytest.mark.parametrize("a", [(None, 0, 0, P, 0, 0, 1, 1, P), (P, 0, 0, None, 0, 0, 1, 1, P), (P, -1, 0, P, 0, 0, 1, 1, P),
                               (P, 0, 0, P, 0, -1, 1, 1, P), (P, 0, 0, P, 0, 0, 2, 1, P), (P, 0, 0, P, 0, 0, 1, -1, P),
                               (P, 0, 0, P, 0, 0, 1, 1, None), (P, 0, 0, P, 0, 0, 1, 1, P + 4), (P + 1, 0, 0, P, 0, 0, 1, 1, P)])
def test_bad_writes_are_refused(lib, a):
    c = _cache()
    assert lib.imq_kv_write(ctypes.addressof(c), *a, None) == imq.IMQ_ERR_ARG


@pytest.mark.parametrize("a", [(None, 1, P, 0, 0, P, 0, 0, 1), (P, 1, None, 0, 0, None, 0, 0, 1), (P, -1, P, 0, 0, P, 0, 0, 1),
                               (P, 1, P, -1, 0, P, 0, 0, 1), (P, 1, P, 0, 0, P, 0, 0, 4), (P, 1, P, 0, 0, P + 2, 0, 0, 0)])
def test_bad_reads_are_refused(lib, a):
    c = _cache()
    assert lib.imq_kv_read(ctypes.addressof(c), *a, None) == imq.IMQ_ERR_ARG


@pytest.mark.parametrize("over,want", [
    (dict(Q=None), imq.IMQ_ERR_ARG), (dict(out=None), imq.IMQ_ERR_ARG), (dict(lens=None), imq.IMQ_ERR_ARG),
    (dict(table=None), imq.IMQ_ERR_ARG), (dict(qt=imq.IMQ_I16), imq.IMQ_ERR_ARG), (dict(ot=imq.IMQ_I64), imq.IMQ_ERR_ARG),
    (dict(qb=-1), imq.IMQ_ERR_ARG), (dict(oh=-1), imq.IMQ_ERR_ARG), (dict(lb=-1), imq.IMQ_ERR_ARG), (dict(stride=-1), imq.IMQ_ERR_ARG),
    (dict(heads=3), imq.IMQ_ERR_ARG), (dict(heads=0), imq.IMQ_ERR_ARG), (dict(batch=-1), imq.IMQ_ERR_ARG),
    (dict(max_len=65), imq.IMQ_ERR_ARG), (dict(max_len=-1), imq.IMQ_ERR_ARG), (dict(width=-1, max_len=0), imq.IMQ_ERR_ARG),
    (dict(ws=P + 8), imq.IMQ_ERR_ARG), (dict(lse=P + 2), imq.IMQ_ERR_ARG), (dict(Q=P + 1), imq.IMQ_ERR_ARG),
    (dict(batch=65536), imq.IMQ_ERR_UNSUPPORTED), (dict(heads=65536), imq.IMQ_ERR_UNSUPPORTED),
    (dict(max_len=1 << 31, width=1 << 30), imq.IMQ_ERR_UNSUPPORTED), (dict(batch=0, Q=None, out=None), imq.IMQ_OK)])
def test_bad_attention_is_refused(lib, over, want):
    assert _attend(lib, _cache(), **over) == want


def test_the_binding_refuses_what_does_not_fit():
    c = imq.KVCache.zeros(3, 16, 2, 64, 8, device="cpu")
    f = torch.zeros
    for bad in (dict(head_dim=128, bits=8), dict(head_dim=64, bits=3), dict(head_dim=64, bits=4)):
        with pytest.raises(ValueError):
            imq.KVCache(c.k, c.v, c.steps, **bad)
    with pytest.raises(ValueError):
        imq.KVCache(c.k, c.v[:2], c.steps, 64, 8)
    with pytest.raises(ValueError):
        imq.KVCache(c.k.transpose(1, 2), c.v.transpose(1, 2), f(3, 16, 2, 2), 64, 8)
    with pytest.raises(ValueError):
        imq.KVCache(c.k, c.v, c.steps.double(), 64, 8)
    slots = torch.zeros(4, dtype=torch.int64)
    for K, V, s in ((f(4, 2, 64), f(4, 2, 64).bfloat16(), slots), (f(4, 2, 64).half(), f(4, 2, 64).half(), slots),
                    (f(3, 2, 64), f(3, 2, 64), slots), (f(4, 2, 64), f(4, 2, 64), slots.int()), (f(4, 2, 32), f(4, 2, 32), slots),
                    (f(4, 2, 64), f(4, 2, 64), slots)):  # the last: not on the GPU
        with pytest.raises(ValueError):
            imq.imq_kv_write(c, K, V, s)
    table, lens = torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    q = f(4, 4, 64)
    for args, kw in (((q.half(), table, lens), {}), ((f(4, 3, 64), table, lens), {}), ((f(4, 4, 32), table, lens), {}),
                     ((q, table.long(), lens), {}), ((q, table[:3], lens), {}), ((q, table, lens.long()), {}),
                     ((q, table, lens), dict(out=f(4, 4, 128))), ((q, table, lens), dict(out=f(4, 4, 64), out_dtype=torch.bfloat16)),
                     ((q, table, lens), dict(lse=f(4, 3))), ((q, table, lens), dict(out_dtype=torch.float16))):
        with pytest.raises(ValueError):
            imq.imq_paged_attention(c, *args, **kw)
    codes, steps = torch.zeros(5, 64, dtype=torch.uint8), f(5, 1)
    for K, N, group in ((129, 5, 128), (128, 6, 128), (128, 5, 64), (128, 5, 100)):
        with pytest.raises(ValueError):
            imq.W4Weight(codes, steps, K, N, group)
    w = imq.W4Weight(codes, steps, 128, 5, 128)
    for X, kw in ((f(2, 127), {}), (f(128), {}), (f(2, 128).half(), {}), (f(2, 128), dict(out=f(2, 6))),
                  (f(2, 128), dict(out=f(2, 5), out_dtype=torch.bfloat16)), (f(2, 128), {})):
        with pytest.raises(ValueError):
            imq.imq_w4_matvec(w, X, **kw)
    with pytest.raises(ValueError):
        imq.imq_w4_quantize(f(128, 5), 128)
    with pytest.raises(ValueError):
        imq.imq_w4_dequantize(w, torch.float32, out=f(5, 128))


def test_struct_layout_matches_header():
    assert ctypes.sizeof(imq.imq_kv_cache) == 3 * 8 + 4 * 8 + 4 * 4
