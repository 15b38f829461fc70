"""The decoding step's operators on the GPU against plain 64-bit implementations of their formulas.

Codes, steps and dequantised values are compared exactly: every fp32 operation of the quantisation rule is a
correctly rounded quotient or product, which numpy's float32 gives too.  Sums are compared within bounds that count the
roundings of the kernels: u = 2^-23 a sum (the tensor cores may cut off where IEEE rounds), and half a step
of the output type.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def imq():
    import bit_integer_gemm_b200 as m
    assert torch.cuda.is_available(), "a GPU is required"
    m.lib()
    m.imq_device_status(clear=True)
    return m


def leaves(status):
    """The status that a test leaves in the device's status word (every other one leaves it at IMQ_OK)."""
    def mark(f):
        f.leaves = status
        return f
    return mark


@pytest.fixture(autouse=True)
def _status(imq, request):
    yield
    torch.cuda.synchronize()
    assert imq.imq_device_status(clear=True) == getattr(request.function, "leaves", 0)


def _randn(seed, *shape, dtype=torch.float32, heavy=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda")
    if heavy:
        x = torch.where(torch.rand(*shape, generator=g, device="cuda") < 0.02, x * heavy, x)
    return x.to(dtype)


# ---------------------------------------------------------------------------------------------------------------
# plain implementations
# ---------------------------------------------------------------------------------------------------------------
def plain_quantise(x: np.ndarray, bits: int):
    """Codes and steps of fp32 groups along the last axis."""
    beta = np.float32(2 ** (bits - 1) - 1)
    q = np.abs(x).max(-1)
    bad = ~np.isfinite(q)
    with np.errstate(all="ignore"):
        s, step = beta / q, q / beta
    unit = (q == 0) | ~np.isfinite(s) & ~bad
    s, step = np.where(unit, np.float32(1), s), np.where(unit, np.float32(1), step)
    with np.errstate(all="ignore"):
        codes = np.rint(x * s[..., None])
    return np.where(bad[..., None], 0, codes).astype(np.int64), np.where(bad, np.float32(np.nan), step).astype(np.float32)


def plain_nibbles(b: np.ndarray):
    """(..., 4 n) bytes as (..., 8 n) codes."""
    w = np.ascontiguousarray(b).view("<u4").astype(np.int64)
    return np.stack([(w >> (4 * (e // 2 + 4 * (e % 2)))) & 15 for e in range(8)], -1).reshape(*b.shape[:-1], -1) - 8


def plain_weight_codes(codes: torch.Tensor, K: int):
    c = plain_nibbles(codes.cpu().numpy())
    r = np.arange(c.shape[1])
    place = r // 128 * 128 + ((r % 32) // 8 * 4 + r % 128 // 32) * 8 + r % 8
    full = c[:, place]
    assert (full[:, K:] == 0).all()
    return full[:, :K]


def plain_vectors(b: torch.Tensor, bits: int):
    return plain_nibbles(b.cpu().numpy()) if bits == 4 else b.cpu().numpy().astype(np.int64) - 128


def f64(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------------------------------------------------------
# 4-bit weights
# ---------------------------------------------------------------------------------------------------------------
WEIGHTS = [(1, 1, 32), (7, 3, 64), (32, 16, 32), (33, 17, 32), (64, 31, 64), (127, 33, 128), (128, 16, 128), (129, 48, 128),
           (200, 65, 64), (256, 40, 32), (1000, 100, 128), (4096, 70, 128), (4099, 37, 64)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K,N,group", WEIGHTS)
def test_weight_codes_steps_and_values(imq, K, N, group, dtype, trans):
    W = _randn(K * 7 + N, N, K, dtype=dtype, heavy=30.0)
    W[0, : K // 2] = 0  # groups of zeros
    stored = W if trans else W.t().contiguous()
    w = imq.imq_w4_quantize(stored, group, transW=trans)
    x = W.float().cpu().numpy()
    pad = np.zeros((N, -(-K // group) * group), np.float32)
    pad[:, :K] = x
    codes, steps = plain_quantise(pad.reshape(N, -1, group), 4)
    codes = codes.reshape(N, -1)[:, :K]
    assert np.array_equal(w.steps.cpu().numpy(), steps)
    assert np.array_equal(plain_weight_codes(w.codes, K), codes)
    values = (codes.astype(np.float32) * np.repeat(steps, group, 1)[:, :K]).astype(np.float32)
    for out in (torch.float32, torch.bfloat16):
        for t in (False, True):
            want = torch.from_numpy(values).to(out)
            assert torch.equal(imq.imq_w4_dequantize(w, out, transW=t).cpu(), want if t else want.t())


def test_weight_groups_are_the_quantisers(imq):
    """A group is a row of imq_rtn_quantize with p = 1."""
    W = _randn(3, 64, 1024, dtype=torch.bfloat16, heavy=30.0)
    w = imq.imq_w4_quantize(W, 128, transW=True)
    q = imq.imq_rtn_quantize(W.view(-1, 128), imq.IMQ_PER_ROW, 1.0, 7)
    assert torch.equal(w.steps.view(-1), q.delta)
    assert np.array_equal(plain_weight_codes(w.codes, 1024), q.xint.view(64, 1024).cpu().numpy())


def test_weight_strides(imq):
    """Parts of larger matrices in and out, rows that are not 16-byte aligned, padded rows of codes and steps."""
    big = _randn(5, 300, 410, dtype=torch.bfloat16)
    for W, trans in ((big[3:60, 5:333], True), (big[7:200, 9:40], False)):
        K, N = (W.shape[1], W.shape[0]) if trans else W.shape
        codes = torch.full((N, 64 * -(-K // 128) + 48), 7, dtype=torch.uint8, device="cuda")
        steps = torch.full((N, -(-K // 32) + 3), 7.0, device="cuda")
        w = imq.imq_w4_quantize(W, 32, transW=trans, codes=codes, steps=steps)
        dense = imq.imq_w4_quantize(W.contiguous(), 32, transW=trans)
        n, m = dense.codes.size(1), dense.steps.size(1)
        assert torch.equal(codes[:, :n], dense.codes) and torch.equal(steps[:, :m], dense.steps)
        assert (codes[:, n:] == 7).all() and (steps[:, m:] == 7).all()
        out = torch.full((W.shape[0] + 2, W.shape[1] + 7), 5.0, device="cuda")
        imq.imq_w4_dequantize(w, transW=trans, out=out[1:-1, 3:-4])
        assert torch.equal(out[1:-1, 3:-4], imq.imq_w4_dequantize(dense, transW=trans))
        out[1:-1, 3:-4] = 5.0
        assert (out == 5.0).all()
        X = _randn(6, 3, K + 5)
        y = torch.full((3, N + 4), 9.0, device="cuda")
        imq.imq_w4_matvec(w, X[:, 3:-2], out=y[:, 1:-3])
        assert torch.equal(y[:, 1:-3], imq.imq_w4_matvec(dense, X[:, 3:-2].contiguous()))
        assert (y[:, 0] == 9).all() and (y[:, -3:] == 9).all()


def matvec_bound(codes, steps, group, x, M, f32):
    """fp64 product and how far an fp32 sum of exact products may be from it: a product passes the sums of its
    group's inner steps of 16 (and, for fp32 entries, of their three parts), of its warp's blocks and of the
    warps."""
    K = codes.shape[1]
    W = codes * np.repeat(steps.astype(np.float64), group, 1)[:, :K]
    y, mass = x @ W.T, np.abs(x) @ np.abs(W).T
    sums = 16 + group // 16 + 128 // group * (-(-K // 128) // 8 + 1) + (24 if f32 else 8)
    return y, (sums + 2) * U * mass


@pytest.mark.parametrize("xt,yt", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                   (torch.float32, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("M", [1, 2, 3, 5, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("K,N,group", [(1, 1, 32), (96, 17, 32), (129, 15, 128), (1024, 33, 64), (2056, 130, 128), (4099, 64, 32)])
def test_matvec(imq, K, N, group, M, xt, yt):
    W = _randn(K + N, N, K, heavy=30.0)
    X = _randn(M, M, K, dtype=xt, heavy=60.0)
    w = imq.imq_w4_quantize(W, group, transW=True)
    y = imq.imq_w4_matvec(w, X, out_dtype=yt)
    want, tol = matvec_bound(plain_weight_codes(w.codes, K), w.steps.cpu().numpy(), group, f64(X), M, xt == torch.float32)
    assert y.dtype == yt and y.shape == (M, N)
    tol = tol + HALF_STEP[yt] * (np.abs(want) + tol)
    assert (np.abs(f64(y) - want) <= tol).all()
    assert torch.equal(y, imq.imq_w4_matvec(w, X, out_dtype=yt))  # the same bits again


@pytest.mark.parametrize("xt,yt", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)])
@pytest.mark.parametrize("M", [1, 2, 3, 8, 9, 16, 17])
@pytest.mark.parametrize("K,N,group", [(514, 2369, 32), (130, 10007, 64), (2049, 4737, 128)])
def test_matvec_of_many_channels(imq, K, N, group, M, xt, yt):
    """More channels than the SMs hold at once; rows of X on 4-byte and, in bf16, on 2-byte boundaries."""
    W = _randn(K + N + 1, N, K, heavy=30.0)
    X = _randn(M + 1, M, K, dtype=xt, heavy=60.0)
    w = imq.imq_w4_quantize(W, group, transW=True)
    y = imq.imq_w4_matvec(w, X, out_dtype=yt)
    want, tol = matvec_bound(plain_weight_codes(w.codes, K), w.steps.cpu().numpy(), group, f64(X), M, xt == torch.float32)
    tol = tol + HALF_STEP[yt] * (np.abs(want) + tol)
    assert (np.abs(f64(y) - want) <= tol).all()
    assert torch.equal(y, imq.imq_w4_matvec(w, X, out_dtype=yt))


@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("M", [2, 3, 9, 12])
@pytest.mark.parametrize("N,group", [(15, 32), (15, 64), (15, 128), (2400, 128)])
def test_matvec_rows_on_any_boundary(imq, N, group, M, pad, xt):
    """Rows of X that begin on multiples of 16, 8, 4 and 2 bytes, in every stage of the rings."""
    K = 2056
    W = _randn(9, N, K)
    X = _randn(10, M, K + pad, dtype=xt)[:, pad:]
    w = imq.imq_w4_quantize(W, group, transW=True)
    y = imq.imq_w4_matvec(w, X, out_dtype=torch.float32)
    want, tol = matvec_bound(plain_weight_codes(w.codes, K), w.steps.cpu().numpy(), group, f64(X), M, xt == torch.float32)
    assert (np.abs(f64(y) - want) <= tol + HALF_STEP[torch.float32] * (np.abs(want) + tol)).all()


@leaves(2)
@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M", [1, 3, 9])
@pytest.mark.parametrize("K,N,group", [(130, 300, 64), (514, 5000, 32), (33, 40, 32)])
def test_matvec_after_values_that_are_not_finite(imq, K, N, group, M, xt):
    """A last block with fewer groups than others, where steps and tokens that are NaN were multiplied before."""
    bad = imq.imq_w4_quantize(torch.full((N, 1024), float("nan"), device="cuda"), group, transW=True)
    w = imq.imq_w4_quantize(_randn(3, N, K), group, transW=True)
    X = _randn(4, M, K, dtype=xt)
    for _ in range(3):
        assert torch.isnan(imq.imq_w4_matvec(bad, torch.full((16, 1024), float("nan"), device="cuda", dtype=xt)[:M])).all()
        y = imq.imq_w4_matvec(w, X, out_dtype=torch.float32)
        want, tol = matvec_bound(plain_weight_codes(w.codes, K), w.steps.cpu().numpy(), group, f64(X), M, xt == torch.float32)
        assert (np.abs(f64(y) - want) <= tol + HALF_STEP[torch.float32] * (np.abs(want) + tol)).all()


def test_matvec_of_nothing(imq):
    w = imq.imq_w4_quantize(_randn(1, 0, 24), 32)
    assert (w.K, w.N) == (0, 24)
    assert torch.equal(imq.imq_w4_matvec(w, torch.zeros(3, 0, device="cuda")), torch.zeros(3, 24, device="cuda"))
    w = imq.imq_w4_quantize(_randn(1, 64, 0), 32)
    assert imq.imq_w4_matvec(w, _randn(2, 3, 64)).shape == (3, 0)
    w = imq.imq_w4_quantize(_randn(1, 64, 24), 32)
    assert imq.imq_w4_matvec(w, _randn(2, 0, 64)).shape == (0, 24)
    assert imq.imq_w4_dequantize(imq.imq_w4_quantize(_randn(1, 0, 24), 32)).shape == (0, 24)


@leaves(2)
def test_weights_that_are_not_finite(imq):
    W = _randn(1, 20, 256)
    W[3, 40], W[5, 200], W[7, 0] = math.nan, math.inf, -math.inf
    W[9] = 1e-40  # so small that 7 / q leaves fp32: stored as zeros
    w = imq.imq_w4_quantize(W, 128, transW=True)
    codes, steps = plain_quantise(W.cpu().numpy().reshape(20, 2, 128), 4)
    assert np.array_equal(plain_weight_codes(w.codes, 256), codes.reshape(20, 256))
    assert np.array_equal(w.steps.cpu().numpy(), steps, equal_nan=True)
    y = imq.imq_w4_matvec(w, _randn(2, 2, 256))
    bad = torch.zeros(20, dtype=torch.bool)
    bad[[3, 5, 7]] = True
    assert torch.equal(y.isnan().cpu(), bad.expand(2, 20))
    assert (y[:, 9] == 0).all()


@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16])
def test_tokens_that_are_not_finite_stay_alone(imq, xt):
    w = imq.imq_w4_quantize(_randn(1, 40, 256), 64, transW=True)
    X = _randn(2, 11, 256, dtype=xt)
    want = imq.imq_w4_matvec(w, X)
    X[2, 7], X[9, 200] = math.nan, math.inf
    y = imq.imq_w4_matvec(w, X)
    rows = [r for r in range(11) if r not in (2, 9)]
    assert torch.equal(y[rows], want[rows]) and y[2].isnan().all() and not y[9].isfinite().any()


def test_weight_rows_behind_32_bit_offsets(imq):
    N, K, ld = 40, 256, 128 << 20
    dense = imq.imq_w4_quantize(_randn(1, N, K), 128, transW=True)
    codes = torch.empty(N * ld, dtype=torch.uint8, device="cuda").view(N, ld)[:, :128]
    codes.copy_(dense.codes)
    w = imq.W4Weight(codes, dense.steps, K, N, 128)
    X = _randn(2, 2, K)
    assert torch.equal(imq.imq_w4_matvec(w, X), imq.imq_w4_matvec(dense, X))
    assert torch.equal(imq.imq_w4_dequantize(w), imq.imq_w4_dequantize(dense))


# ---------------------------------------------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------------------------------------------
def cache_values(cache):
    """fp64 values of every slot's key and value, (slots, heads, head_dim)."""
    steps = cache.steps.cpu().numpy().astype(np.float32)
    out = []
    for t, i in ((cache.k, 0), (cache.v, 1)):
        v = plain_vectors(t, cache.bits).astype(np.float32) * steps[..., i, None]
        out.append(v.transpose(0, 2, 1, 3).reshape(-1, cache.n_heads, cache.head_dim))
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("n,H,page", [(1, 1, 16), (5, 3, 16), (77, 2, 48), (300, 8, 64), (5003, 9, 48), (5003, 8, 64)])
def test_cache_write_and_read(imq, n, H, page, D, bits, dtype):
    pages = -(-n // page) + 3
    cache = imq.KVCache.zeros(pages, page, H, D, bits)
    K, V = _randn(1, n, H, D, dtype=dtype, heavy=20.0), _randn(2, n, H, D, dtype=dtype, heavy=20.0)
    K[0, 0] = 0
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(n))[:n].cuda()
    skip = torch.zeros(n, dtype=torch.bool)
    skip[2::5] = True
    slots[skip.cuda()] = -1
    imq.imq_kv_write(cache, K, V, slots)
    at = slots.cpu().numpy()[~skip.numpy()]
    kc, ks = plain_quantise(K.float().cpu().numpy(), bits)
    vc, vs = plain_quantise(V.float().cpu().numpy(), bits)
    page_at, pos = at // page, at % page
    keep = ~skip.numpy()
    assert np.array_equal(plain_vectors(cache.k, bits)[page_at, :, pos], kc[keep])
    assert np.array_equal(plain_vectors(cache.v, bits)[page_at, :, pos], vc[keep])
    assert np.array_equal(cache.steps.cpu().numpy()[page_at, :, pos], np.stack((ks, vs), -1)[keep])
    untouched = np.ones((pages, page), bool)
    untouched[page_at, pos] = False
    assert not cache.k.cpu().numpy().transpose(0, 2, 1, 3)[untouched].any()
    assert not cache.steps.cpu().numpy().transpose(0, 2, 1, 3)[untouched].any()
    for out in (torch.float32, torch.bfloat16):
        k, v = (torch.full((n, H, D), 3.0, dtype=out, device="cuda") for _ in range(2))
        imq.imq_kv_read(cache, slots, K=k, V=v)
        for got, c, s in ((k, kc, ks), (v, vc, vs)):
            want = torch.from_numpy(c.astype(np.float32) * s[..., None]).to(out)
            want[skip] = 3.0
            assert torch.equal(got.cpu(), want)


def test_cache_vectors_are_the_quantisers(imq):
    K, V = _randn(1, 40, 4, 128, dtype=torch.bfloat16, heavy=20.0), _randn(2, 40, 4, 128, dtype=torch.bfloat16)
    cache = imq.KVCache.zeros(3, 16, 4, 128, 8)
    imq.imq_kv_write(cache, K, V, torch.arange(40, device="cuda"))
    q = imq.imq_rtn_quantize(K.view(-1, 128), imq.IMQ_PER_ROW, 1.0, 127)
    codes = plain_vectors(cache.k, 8).transpose(0, 2, 1, 3).reshape(48, 4, 128)[:40]
    assert np.array_equal(codes.reshape(-1, 128), q.xint.cpu().numpy())
    assert torch.equal(cache.steps[..., 0].transpose(1, 2).reshape(48, 4)[:40].reshape(-1), q.delta)


def test_cache_strides(imq):
    """Keys and values inside one projection's output (unaligned too), pages of keys and values in one buffer."""
    n, H, D, page = 21, 2, 64, 16
    row = H * D * page // 2
    buf = torch.full((5, 3 * row + 32), 9, dtype=torch.uint8, device="cuda")
    k, v = (buf[:, i * row:(i + 1) * row].unflatten(1, (H, page, D // 2)) for i in (0, 2))
    cache = imq.KVCache(k, v, torch.zeros(5, H, page, 8, device="cuda").flatten(1)[:, : H * page * 2].unflatten(1, (H, page, 2)), D, 4)
    plain = imq.KVCache.zeros(5, page, H, D, 4)
    slots = torch.randperm(80, device="cuda")[:n]
    for off in (0, 3):
        qkv = _randn(off, n, 6 * H * D + 9, dtype=torch.bfloat16)
        K = qkv[:, off:off + H * D].unflatten(1, (H, D))
        V = qkv[:, off + 2 * H * D:off + 4 * H * D].unflatten(1, (H, 2 * D))[..., :D]
        imq.imq_kv_write(cache, K, V, slots)
        imq.imq_kv_write(plain, K.contiguous(), V.contiguous(), slots)
        k1, v1 = imq.imq_kv_read(cache, slots)
        k2, v2 = imq.imq_kv_read(plain, slots)
        assert torch.equal(k1, k2) and torch.equal(v1, v2)
        out = torch.full((n, 2 * H * D + 7), 5.0, dtype=torch.bfloat16, device="cuda")
        imq.imq_kv_read(cache, slots, K=out[:, off:off + H * D].unflatten(1, (H, D)),
                        V=out[:, off + H * D:off + 2 * H * D].unflatten(1, (H, D)))
        assert torch.equal(out[:, off:off + H * D], k2.bfloat16().flatten(1))
        assert torch.equal(out[:, off + H * D:off + 2 * H * D], v2.bfloat16().flatten(1))
        assert (out[:, :off] == 5).all() and (out[:, off + 2 * H * D:] == 5).all()
    assert (buf[:, row:2 * row] == 9).all() and (buf[:, 3 * row:] == 9).all()
    # one key head's vector for every head
    one = _randn(9, n, 1, D)
    imq.imq_kv_write(plain, one.expand(n, H, D), one.expand(n, H, D), slots)
    k2, _ = imq.imq_kv_read(plain, slots)
    assert torch.equal(k2[:, 0], k2[:, 1])


@leaves(9)
def test_slots_outside_the_cache(imq):
    cache = imq.KVCache.zeros(2, 16, 2, 64, 8)
    K = _randn(1, 5, 2, 64)
    slots = torch.tensor([3, 32, 1 << 40, -7, 31], device="cuda")
    imq.imq_kv_write(cache, K, K, slots)
    torch.cuda.synchronize()
    assert imq.imq_device_status(clear=True) == imq.IMQ_ERR_BOUNDS
    out = torch.full((5, 2, 64), 4.0, device="cuda")
    imq.imq_kv_read(cache, slots, K=out, V=out.clone())
    assert (out[1:4] == 4).all()
    assert ((out[[0, 4]] - K[[0, 4]]).abs() <= K[[0, 4]].abs().amax(-1, keepdim=True) / 127).all()
    assert int((cache.steps != 0).sum()) == 2 * 2 * 2


@leaves(2)
@pytest.mark.parametrize("bits", [4, 8])
def test_cached_vectors_that_are_not_finite(imq, bits):
    cache = imq.KVCache.zeros(1, 16, 2, 64, bits)
    K, V = _randn(1, 3, 2, 64), _randn(2, 3, 2, 64)
    K[0, 1, 5], V[1, 0, 9] = math.inf, math.nan
    imq.imq_kv_write(cache, K, V, torch.arange(3, device="cuda"))
    k, v = imq.imq_kv_read(cache, torch.arange(3, device="cuda"))
    assert k[0, 1].isnan().all() and v[1, 0].isnan().all()
    assert int(k.isnan().sum()) == 64 and int(v.isnan().sum()) == 64


# ---------------------------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------------------------
def make_cache(imq, lens, page, H, D, bits, seed=0, width=None, poison=True):
    """A cache holding sequences of these lengths on shuffled pages.  Slots that no token uses are poisoned: codes
    of all ones and NaN steps; table entries behind a sequence's pages point outside the cache."""
    need = [-(-max(n, 0) // page) for n in lens]
    n_pages = sum(need) + 2
    width = max(max(need, default=0), 1) if width is None else width
    cache = imq.KVCache.zeros(n_pages, page, H, D, bits)
    if poison:
        cache.k.fill_(255)
        cache.v.fill_(255)
        cache.steps.fill_(math.nan)
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(lens), width), 1 << 30, dtype=torch.int32)
    slots, at = [], 0
    for b, n in enumerate(lens):
        pages = order[at:at + need[b]]
        at += need[b]
        table[b, : need[b]] = torch.tensor(pages, dtype=torch.int32)
        slots += [pages[t // page] * page + t % page for t in range(n)]
    total = len(slots)
    K, V = _randn(seed + 1, total, H, D, heavy=8.0), _randn(seed + 2, total, H, D, heavy=8.0)
    if total:
        imq.imq_kv_write(cache, K, V, torch.tensor(slots, device="cuda"))
    return cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def plain_attention(cache, Q, table, lens, scale):
    """fp64 outputs and log sums, and their error bounds.
    A score is sum of D products, exact but for the query's 22 bits (2^-22 of its largest entry, each entry) and the
    roundings of D / 16 + 16 sums, then three more roundings: dx in all.  A weight exp(x - max) is off by two such
    errors and 2^-21 (the exponential, its argument's rounding), the value's part by 2^-21; the sums over the tokens
    pass at most len / 64 + 60 roundings.  A weight times its step, in units of the largest step and of 2^-11, goes into
    two fp16 parts; the second is rounded to fp16's smallest spacing, 2^-24, where it is below 2^-14, so off by up to
    2^-25 of those units whatever the weight: 2^-36 of the largest step, times a code of up to beta, per token.  (That
    counts where a token that takes all the weight has a code of 0 and far smaller weights make the output.)"""
    k, v = cache_values(cache)
    B, Hq, D = Q.shape
    G, page = Hq // cache.n_heads, cache.page_size
    out, tol = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    lse, ltol = np.full((B, Hq), -np.inf), np.zeros((B, Hq))
    q = f64(Q)
    steps = f64(cache.steps[..., 1]).transpose(0, 2, 1).reshape(-1, cache.n_heads)
    for b, n in enumerate(lens.tolist()):
        if n <= 0:
            continue
        t = np.arange(n)
        slot = table[b].cpu().numpy().astype(np.int64)[t // page] * page + t % page
        for h in range(Hq):
            kk, vv = k[slot, h // G].astype(np.float64), v[slot, h // G].astype(np.float64)
            x = scale * (kk @ q[b, h])
            dx = abs(scale) * (np.abs(kk) @ (np.abs(q[b, h]) * (D // 16 + 16) * U + 2.0 ** -22 * np.abs(q[b, h]).max())) + 4 * U * np.abs(x)
            top = x.max()
            p = np.exp(x - top)
            # errors of the scores, weighted: terms far below the maximum do not count
            e = p * (dx + dx[x.argmax()] + 2.0 ** -20 + U * np.abs(x - top))
            s = p.sum()
            out[b, h], lse[b, h] = p @ vv / s, top + np.log(s)
            rel = (n / 64 + 60) * U
            floor = n * 2.0 ** -36 * (2 ** (cache.bits - 1) - 1) * steps[slot, h // G].max()
            tol[b, h] = (floor + e @ np.abs(vv) + rel * (p @ np.abs(vv))) / s + (e.sum() / s + rel) * np.abs(out[b, h])
            ltol[b, h] = dx[x.argmax()] + e.sum() / s + rel + 4 * U * (1 + abs(lse[b, h]) + abs(top))
    return out, tol, lse, ltol


def check_attention(imq, cache, Q, table, lens, scale=None, **kw):
    out, lse = imq.imq_paged_attention(cache, Q, table, lens, scale=scale, **kw)
    want, tol, wl, ltol = plain_attention(cache, Q, table, lens, Q.shape[2] ** -0.5 if scale is None else scale)
    tol = tol + HALF_STEP[out.dtype] * (np.abs(want) + tol)
    err = np.abs(f64(out) - want)
    assert (err <= tol).all(), (float((err / np.maximum(tol, 1e-300)).max()), np.unravel_index((err - tol).argmax(), err.shape))
    got = f64(lse)
    assert np.array_equal(np.isneginf(got), np.isneginf(wl))
    live = ~np.isneginf(wl)
    assert (np.abs(got[live] - wl[live]) <= ltol[live]).all()
    return out, lse


LENS = {"short": [1, 2, 15, 16, 17, 0, 31, 33], "mixed": [63, 64, 65, 0, 127, 129, 200, 1, 500], "long": [1537, 3, 4000]}


@pytest.mark.parametrize("lens", LENS, ids=list(LENS))
@pytest.mark.parametrize("G", [1, 3, 8, 9, 16, 21])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
def test_attention(imq, D, bits, G, lens):
    lens = LENS[lens]
    page = (16, 32, 48, 64)[(D // 64 + G) % 4]
    H = 2 if G < 9 else 1
    cache, table, n = make_cache(imq, lens, page, H, D, bits, seed=G)
    dt = torch.float32 if (G + bits) % 2 else torch.bfloat16
    check_attention(imq, cache, _randn(G, len(lens), H * G, D, dtype=dt), table, n)
    other = torch.bfloat16 if dt == torch.float32 else torch.float32
    check_attention(imq, cache, _randn(G + 1, len(lens), H * G, D, dtype=dt), table, n, out_dtype=other)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_attention_scales(imq, scale):
    """Equal weights, a negative scale, and scores so far apart that one token takes all."""
    cache, table, n = make_cache(imq, [70, 5, 300], 16, 2, 64, 8)
    check_attention(imq, cache, _randn(1, 3, 4, 64), table, n, scale=scale)


@pytest.mark.parametrize("size", [1e-30, 1e-38, 1e-44, 1e30])
def test_attention_of_very_small_and_large_values(imq, size):
    """Queries (and values) near the ends of fp32's range: scaled by powers of two, they lose nothing."""
    cache, table, n = make_cache(imq, [70, 5], 16, 1, 64, 8)
    q = _randn(1, 2, 2, 64) * size
    scale = 0.1 if size > 1 else 0.1 / max(size, 1e-30)
    if size > 1:
        scale = 0.1 / size
    check_attention(imq, cache, q, table, n, scale=scale)


def test_attention_of_queries_at_the_end_of_fp32(imq):
    """Rows whose largest entries are 3.3e38, 2^126 and just beside it."""
    cache, table, n = make_cache(imq, [70, 5, 33], 16, 1, 64, 4)
    q = _randn(1, 3, 3, 64).clamp(-3, 3) / 3
    q = q / q.abs().amax(-1, keepdim=True) * torch.tensor([3.3e38, 2.0 ** 126, 8.4e37], device="cuda")[None, :, None]
    check_attention(imq, cache, q, table, n, scale=1e-37)


def test_attention_of_steps_of_very_different_sizes(imq):
    """Values that grow a millionfold from token to token: the sums' unit grows with them."""
    H, D, page, n = 1, 64, 16, 200
    cache = imq.KVCache.zeros(14, page, H, D, 8)
    K, V = _randn(1, n, H, D), _randn(2, n, H, D)
    V *= 10.0 ** (torch.arange(n, device="cuda") % 13 - 6.0)[:, None, None]
    imq.imq_kv_write(cache, K, V, torch.arange(n, device="cuda"))
    table = torch.arange(14, dtype=torch.int32, device="cuda")[None]
    check_attention(imq, cache, _randn(3, 1, 4, D), table, torch.tensor([n], dtype=torch.int32, device="cuda"))


def test_attention_strides_and_rows_behind_the_batch(imq):
    cache, table, n = make_cache(imq, [40, 0, 90], 16, 2, 64, 8)
    wide = torch.full((3, 5 + table.size(1)), -5, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + table.size(1)] = table
    qkv = _randn(1, 3, 4 * 64 * 3 + 7, dtype=torch.bfloat16)
    Q = qkv[:, 3:3 + 4 * 64 * 2].unflatten(1, (4, 128))[..., 64:]
    out = torch.full((5, 4, 80), 6.0, device="cuda")
    lse = torch.full((5, 9), 6.0, device="cuda")
    part = wide[:, 2:2 + table.size(1)]
    o, l = check_attention(imq, cache, Q, part, n, out=out[1:4, :, 8:72], lse=lse[1:4, 2:6])
    assert o.data_ptr() == out[1:4, :, 8:72].data_ptr()
    assert (out[[0, 4]] == 6).all() and (out[:, :, :8] == 6).all() and (out[:, :, 72:] == 6).all()
    assert (lse[[0, 4]] == 6).all() and (lse[:, :2] == 6).all() and (lse[:, 6:] == 6).all()
    o2, none = imq.imq_paged_attention(cache, Q, part, n, out_dtype=torch.float32, want_lse=False)
    assert none is None and torch.equal(o, o2)
    # a query for all heads
    one = _randn(2, 3, 1, 64)
    o3, _ = check_attention(imq, cache, one.expand(3, 4, 64), table, n)
    assert torch.equal(o3[:, 0], o3[:, 1])


def test_attention_of_sequences_that_share_pages(imq):
    """One prefix on the same pages, read by several sequences of several lengths."""
    cache, table, n = make_cache(imq, [500], 32, 2, 128, 4)
    check_attention(imq, cache, _randn(1, 4, 4, 128), table.expand(4, -1), torch.tensor([500, 100, 31, 499], dtype=torch.int32, device="cuda"))


def test_attention_of_many_short_sequences(imq):
    """More sequences than the device holds CTAs, a quarter of them empty."""
    lens = [(7 * i) % 41 if i % 4 else 0 for i in range(1100)]
    cache, table, n = make_cache(imq, lens, 16, 1, 64, 4)
    check_attention(imq, cache, _randn(1, len(lens), 2, 64), table, n)


@pytest.mark.parametrize("H,L,bits", [(32, 40000, 4), (30, 36001, 8)])
def test_attention_of_long_parts(imq, H, L, bits):
    """So many tokens and heads that a warp takes more than 32 runs of one row; page numbers are read in batches."""
    cache, table, n = make_cache(imq, [L], 48, H, 64, bits, poison=False)
    check_attention(imq, cache, _randn(1, 1, H, 64), table, n)


def test_two_graphs_replayed_at_once(imq):
    """Each with a workspace of its own."""
    cache, table, n = make_cache(imq, [3000, 0, 5000], 64, 2, 128, 8)
    Qs = [_randn(i, 3, 8, 128) for i in range(2)]
    want = [imq.imq_paged_attention(cache, q, table, n) for q in Qs]
    graphs, got, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for q in Qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(imq.imq_paged_attention(cache, q, table, n))
        graphs.append(g)
    for _ in range(10):
        for (o, l), g, s in zip(got, graphs, streams):
            with torch.cuda.stream(s):
                o.zero_(), l.zero_()
                g.replay()
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


def test_attention_does_not_depend_on_the_bound_or_the_workspace(imq):
    """max_len only sizes the launch (other splits, other roundings); a workspace's old contents do not matter."""
    cache, table, n = make_cache(imq, [3000, 17, 0], 16, 2, 128, 8)
    Q = _randn(1, 3, 8, 128)
    for max_len in (3000, 3008, table.size(1) * 16):
        need = imq.imq_paged_attention_workspace(cache, 3, 8, max_len)
        assert need > 0
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        a, _ = check_attention(imq, cache, Q, table, n, max_len=max_len, workspace=ws)
        b, _ = imq.imq_paged_attention(cache, Q, table, n, max_len=max_len)
        assert torch.equal(a, b)
        with pytest.raises(imq.ImqError) as e:
            imq.imq_paged_attention(cache, Q, table, n, max_len=max_len, workspace=ws[:-16])
        assert e.value.status == imq.IMQ_ERR_BUFFER


def test_attention_of_an_empty_batch_and_of_empty_sequences(imq):
    cache, table, n = make_cache(imq, [0, -3, 0], 16, 1, 64, 8)
    out, lse = imq.imq_paged_attention(cache, _randn(1, 3, 2, 64), table, n)
    assert (out == 0).all() and torch.isneginf(lse).all()
    out, lse = imq.imq_paged_attention(cache, _randn(1, 3, 2, 64), table, n, max_len=0)
    assert (out == 0).all() and torch.isneginf(lse).all()
    out, lse = imq.imq_paged_attention(cache, _randn(1, 0, 2, 64), table[:0], n[:0])
    assert out.shape == (0, 2, 64)
    # a table without entries, a cache without pages
    none = imq.KVCache.zeros(0, 16, 1, 64, 8)
    out, _ = imq.imq_paged_attention(none, _randn(1, 3, 2, 64), table[:, :0], n)
    assert (out == 0).all()


@leaves(9)
@pytest.mark.parametrize("long", [False, True])
def test_bad_pages_and_lengths(imq, long):
    """A page outside the cache, or a sequence longer than max_len, makes that sequence NaN and no other."""
    top = 3000 if long else 60
    cache, table, n = make_cache(imq, [40, top, 20, 50], 16, 2, 64, 8)
    Q = _randn(1, 4, 4, 64)
    good, glse = imq.imq_paged_attention(cache, Q, table, n)
    assert imq.imq_device_status() == imq.IMQ_OK and good.isfinite().all()
    t = table.clone()
    t[0, 2], t[3, 0] = cache.n_pages, -1
    out, lse = imq.imq_paged_attention(cache, Q, t, n)
    assert out[[0, 3]].isnan().all() and lse[[0, 3]].isnan().all()
    assert torch.equal(out[1:3], good[1:3]) and torch.equal(lse[1:3], glse[1:3])
    assert imq.imq_device_status(clear=True) == imq.IMQ_ERR_BOUNDS
    n2 = n.clone()
    n2[2] = table.size(1) * 16 + 1
    out, lse = imq.imq_paged_attention(cache, Q, table, n2)
    assert out[2].isnan().all() and lse[2].isnan().all()
    assert torch.equal(out[[0, 1, 3]], good[[0, 1, 3]]) and torch.equal(lse[[0, 1, 3]], glse[[0, 1, 3]])
    assert imq.imq_device_status() == imq.IMQ_ERR_BOUNDS


def test_queries_that_are_not_finite_stay_alone(imq):
    cache, table, n = make_cache(imq, [40, 70], 16, 2, 64, 8)
    Q = _randn(1, 2, 8, 64)
    good, _ = imq.imq_paged_attention(cache, Q, table, n)
    Q[0, 1, 3], Q[1, 6, 0] = math.nan, math.inf
    out, lse = imq.imq_paged_attention(cache, Q, table, n)
    bad = torch.zeros(2, 8, dtype=torch.bool)
    bad[0, 1] = bad[1, 6] = True
    assert torch.equal(out.isnan().all(-1).cpu(), bad) and torch.equal(lse.isnan().cpu(), bad)
    assert torch.equal(out[~bad.cuda()], good[~bad.cuda()])


@leaves(2)
def test_cached_tokens_that_are_not_finite(imq):
    """They reach the sequences that read them and no others."""
    cache, table, n = make_cache(imq, [40, 70, 30], 16, 1, 64, 8)
    Q = _randn(1, 3, 2, 64)
    good, _ = imq.imq_paged_attention(cache, Q, table, n)
    K, V = _randn(2, 1, 1, 64), _randn(3, 1, 1, 64)
    at = lambda b, t: (table[b, t // 16].long() * 16 + t % 16).reshape(1)  # noqa: E731
    imq.imq_kv_write(cache, K * math.inf, V, at(0, 39))
    imq.imq_kv_write(cache, K, V * math.nan, at(1, 3))
    out, lse = imq.imq_paged_attention(cache, Q, table, n)
    assert out[:2].isnan().all() and torch.equal(out[2], good[2]) and lse[0].isnan().all() and lse[1].isfinite().all()
    n[0] = 39  # the sequence before that token
    out, _ = imq.imq_paged_attention(cache, Q, table, n)
    assert out[0].isfinite().all()


def test_pages_behind_32_bit_offsets(imq):
    """Pages 1.2 GB apart: the last ones lie behind 2^32 bytes of codes (and 2^32 bytes of steps)."""
    H, D, page, gap = 1, 64, 16, 1200 << 20
    k = torch.empty(4 * gap + 4096, dtype=torch.uint8, device="cuda")
    dense = imq.KVCache.zeros(5, page, H, D, 8)
    strided = k.as_strided((5, H, page, D), (gap, page * D, D, 1))
    steps = torch.empty(gap + 64, device="cuda").as_strided((5, H, page, 2), (gap // 4, page * 2, 2, 1))
    cache = imq.KVCache(strided, strided.as_strided((5, H, page, D), (gap, page * D, D, 1), 2048), steps, D, 8)
    K, V = _randn(1, 80, H, D), _randn(2, 80, H, D)
    slots = torch.arange(80, device="cuda")
    for c in (cache, dense):
        imq.imq_kv_write(c, K, V, slots)
    assert torch.equal(imq.imq_kv_read(cache, slots)[1], imq.imq_kv_read(dense, slots)[1])
    table, n = torch.arange(5, dtype=torch.int32, device="cuda")[None], torch.tensor([77], dtype=torch.int32, device="cuda")
    Q = _randn(3, 1, 4, D)
    assert torch.equal(imq.imq_paged_attention(cache, Q, table, n)[0], imq.imq_paged_attention(dense, Q, table, n)[0])


def test_two_streams_at_once(imq):
    cache, table, n = make_cache(imq, [6000, 100, 3000], 64, 4, 128, 4)
    Qs = [_randn(i, 3, 16, 128) for i in range(2)]
    want = [imq.imq_paged_attention(cache, q, table, n)[0] for q in Qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(imq.imq_paged_attention(cache, Qs[i], table, n, stream=s)[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


# ---------------------------------------------------------------------------------------------------------------
# the run of them together
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("bits", [4, 8])
def test_decoding_steps_eager_and_in_a_graph(imq, bits):
    """Several steps of one attention layer: project, write the new key and value, attend, project back.  The steps run
    eagerly and then from one captured graph whose lengths and slots change in place, and give the same bits; each
    step's attention is within its bounds of the formula on the cache that the step left."""
    B, Hq, H, D, page, width = 3, 8, 2, 64, 16, 6
    E = Hq * D
    wq = imq.imq_w4_quantize(_randn(1, E, (Hq + 2 * H) * D, dtype=torch.bfloat16) * 0.05, 128)
    wo = imq.imq_w4_quantize(_randn(2, E, E, dtype=torch.bfloat16) * 0.05, 64)
    table = torch.randperm(B * width, device="cuda").int().view(B, width)
    starts = [0, 15, 63]

    def step(cache, x, lens, slots):
        qkv = imq.imq_w4_matvec(wq, x)
        q = qkv[:, :E].unflatten(1, (Hq, D))
        k, v = qkv[:, E:].unflatten(1, (2, H, D)).unbind(1)
        imq.imq_kv_write(cache, k, v, slots)
        a, _ = imq.imq_paged_attention(cache, q, table, lens)
        return q, a, imq.imq_w4_matvec(wo, a.flatten(1))

    def slots_of(lens):
        t = lens.long() - 1
        return table.gather(1, (t // page)[:, None])[:, 0].long() * page + t % page

    def fresh():
        cache = imq.KVCache.zeros(B * width, page, H, D, bits)
        for b, n in enumerate(starts):
            if n:
                t = torch.arange(n, device="cuda")
                imq.imq_kv_write(cache, _randn(10 + b, n, H, D), _randn(20 + b, n, H, D), table[b].long()[t // page] * page + t % page)
        return cache

    xs = [_randn(30 + i, B, E, dtype=torch.bfloat16) for i in range(5)]
    cache = fresh()
    eager, x = [], xs[0]
    for i in range(5):
        lens = torch.tensor([n + i + 1 for n in starts], dtype=torch.int32, device="cuda")
        q, a, y = step(cache, xs[i], lens, slots_of(lens))
        want, tol, _, _ = plain_attention(cache, q, table, lens, D ** -0.5)
        assert (np.abs(f64(a) - want) <= tol + HALF_STEP[a.dtype] * (np.abs(want) + tol)).all()
        eager.append(y.clone())

    cache = fresh()
    x = xs[0].clone()
    lens = torch.tensor([n + 1 for n in starts], dtype=torch.int32, device="cuda")
    slots = slots_of(lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cache, x, lens, slots)  # first calls outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, _, y = step(cache, x, lens, slots)
    for i in range(5):
        x.copy_(xs[i])
        lens.copy_(torch.tensor([n + i + 1 for n in starts], dtype=torch.int32))
        slots.copy_(slots_of(lens))
        graph.replay()
        assert torch.equal(y, eager[i])
