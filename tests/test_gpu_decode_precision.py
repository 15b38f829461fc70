"""Precision of attention over the cache where operands of very different sizes meet: bounds from fp32 arithmetic and from
the weights and queries that make the output, not from the largest entry of anything."""
import numpy as np
import pytest
import torch

from test_gpu_decode import _randn, _status, cache_values, f64, imq  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def filled(imq, K, V, bits, page=32):  # noqa: F811
    """A cache that holds one sequence, its table and its length."""
    n, H, D = K.shape
    pages = -(-n // page)
    cache = imq.KVCache.zeros(pages, page, H, D, bits)
    imq.imq_kv_write(cache, K, V, torch.arange(n, device="cuda"))
    return cache, torch.arange(pages, dtype=torch.int32, device="cuda")[None], torch.tensor([n], dtype=torch.int32, device="cuda")


def bounds(cache, Q, n, scale, grid):
    """fp64 outputs of one sequence and how far they may be off.
    A score: D products whose sums and scalings pass D / 16 + 16 roundings, and query entries off by `grid` of their row's
    largest, times the keys they meet.  A weight exp(x - max): two such errors and 2^-20.  Its product with the value's step is
    cut to 22 bits, or to 2^-36 of the head's largest such product over the vectors that are not zero; the sums over
    the tokens pass n / 64 + 60 roundings."""
    k, v = (x[:n] for x in cache_values(cache))
    steps = f64(cache.steps[..., 1]).transpose(0, 2, 1).reshape(-1, cache.n_heads)[:n]
    q, G = f64(Q)[0], Q.shape[1] // cache.n_heads
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(len(q)):
        kk, vv = k[:, h // G].astype(np.float64), v[:, h // G].astype(np.float64)
        x = scale * (kk @ q[h])
        dx = abs(scale) * (np.abs(kk) @ ((cache.head_dim // 16 + 16) * U * np.abs(q[h]) + grid * np.abs(q[h]).max())) + 4 * U * np.abs(x)
        p = np.exp(x - x.max())
        e = p * (dx + dx[x.argmax()] + 2.0 ** -20 + U * np.abs(x - x.max()))
        s, rel = p.sum(), (n / 64 + 60) * U
        out[h] = p @ vv / s
        live = np.abs(vv).max(-1) > 0
        floor = n * 2.0 ** -36 * (2 ** (cache.bits - 1) - 1) * (p * steps[:, h // G])[live].max(initial=0.0)
        tol[h] = (floor + e @ np.abs(vv) + rel * (p @ np.abs(vv))) / s + (e.sum() / s + rel + 2.0 ** -24) * np.abs(out[h])
    return out, tol


def check(imq, cache, Q, table, lens, scale=None, grid=2.0 ** -22):  # noqa: F811
    scale = Q.shape[2] ** -0.5 if scale is None else scale
    out, _ = imq.imq_paged_attention(cache, Q, table, lens, scale=scale, out_dtype=torch.float32)
    want, tol = bounds(cache, Q, int(lens[0]), scale, grid)
    err = np.abs(f64(out)[0] - want)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())
    return out


SHAPES = [(D, bits, G) for D in (64, 128, 192, 256) for bits in (4, 8) for G in (1, 8, 9, 16)]


@pytest.mark.parametrize("D,bits,G", SHAPES)
def test_zero_vectors_among_small_values(imq, D, bits, G):  # noqa: F811
    """A vector of zeros, or of entries that are stored as zeros, has the step 1; it adds nothing and costs the others
    nothing, wherever it stands.  With equal weights every operation behind the quantiser is a product or a sum
    of the steps, so values that are 2^-k times as large give exactly 2^-k times the output."""
    H, n = 2, 700
    K, V, Q = _randn(1, n, H, D), _randn(2, n, H, D), _randn(3, 1, H * G, D)
    zeros = torch.rand(n, H, generator=torch.Generator().manual_seed(4)) < 0.1
    zeros[0] = zeros[640:] = True  # the first of the sequence, and whole runs
    V[zeros.cuda()] = 0
    tiny = V.clone()
    tiny[5] = 1e-41  # 127 / q leaves fp32
    outs = []
    for k in (0, 10, 20, 40, 60):
        cache, table, lens = filled(imq, K, V * 2.0 ** -k, bits)
        check(imq, cache, Q, table, lens)
        outs.append(check(imq, cache, Q, table, lens, scale=0.0) * 2.0 ** k)
        cache, table, lens = filled(imq, K, torch.where(tiny == 1e-41, tiny, tiny * 2.0 ** -k), bits)
        check(imq, cache, Q, table, lens)
    assert all(torch.equal(o, outs[0]) for o in outs[1:])


def test_zero_vectors_alone(imq):  # noqa: F811
    cache, table, lens = filled(imq, _randn(1, 50, 1, 64), torch.zeros(50, 1, 64, device="cuda"), 8)
    out, lse = imq.imq_paged_attention(cache, _randn(2, 1, 4, 64), table, lens)
    assert (out == 0).all() and lse.isfinite().all()


@pytest.mark.parametrize("D,bits,G", SHAPES)
@pytest.mark.parametrize("size", [0.0, 1e-9, 1e-3])
def test_sinks(imq, size, D, bits, G):  # noqa: F811
    """A token that takes nearly all the weight and has a small or no value: the others, 2^-34 of its weight, make
    the output."""
    H, n = 2, 300
    K, V, Q = _randn(1, n, H, D), _randn(2, n, H, D), _randn(3, 1, H * G, D)
    for at in (0, 170):
        k, v = K.clone(), V.clone()
        k[..., 3] = 0
        k[at], v[at] = 0, V[at] * size
        k[at, :, 3], Q[..., 3] = 40.0, 0.6 * D ** 0.5
        cache, table, lens = filled(imq, k, v, bits)
        check(imq, cache, Q, table, lens)


@pytest.mark.parametrize("D,bits,G", SHAPES)
def test_large_values_of_no_weight(imq, D, bits, G):  # noqa: F811
    """A token with values a millionfold, and a weight of 2^-86: it adds 2^-66 of what the others do."""
    H, n = 2, 300
    K, V, Q = _randn(1, n, H, D), _randn(2, n, H, D), _randn(3, 1, H * G, D)
    for at in (0, 170):
        k, v = K.clone(), V.clone()
        k[..., 3] = 0
        k[at], v[at] = 0, V[at] * 1e6
        k[at, :, 3], Q[..., 3] = -40.0, 1.5 * D ** 0.5
        cache, table, lens = filled(imq, k, v, bits)
        check(imq, cache, Q, table, lens)


@pytest.mark.parametrize("heavy", [30.0, 1e3, 1e5, 2.0 ** 20])
@pytest.mark.parametrize("D,bits,G", SHAPES)
def test_heavy_query_dimensions(imq, D, bits, G, heavy):  # noqa: F811
    """A query entry far above its row's others, on keys that are zero there.  The scores of the others are off by what fp32
    sums cost and by 2^-30 of the largest entry; entries of few bits, down to 2^-22 of the largest, lose nothing.  One
    token a sequence: its log sum is the score."""
    H, n, page, at = 2, 40, 16, D - 5
    K, V = _randn(1, n, H, D), _randn(2, n, H, D)
    K[..., at] = 0
    cache = imq.KVCache.zeros(n, page, H, D, bits)
    imq.imq_kv_write(cache, K, V, torch.arange(n, device="cuda") * page)
    table, lens = torch.arange(n, dtype=torch.int32, device="cuda")[:, None], torch.ones(n, dtype=torch.int32, device="cuda")
    k = cache_values(cache)[0][::page].astype(np.float64)  # (n, H, D)
    v = cache_values(cache)[1][::page]
    whole = torch.randint(-8, 9, (n, H * G, D), generator=torch.Generator().manual_seed(3)).cuda()
    for Q, grid in ((_randn(4, n, H * G, D), 2.0 ** -30), (_randn(5, n, H * G, D, dtype=torch.bfloat16), 2.0 ** -30),
                    (whole.float(), 0.0), (whole.bfloat16(), 0.0)):
        Q[..., at] = heavy
        out, lse = imq.imq_paged_attention(cache, Q, table, lens, out_dtype=torch.float32)
        q = f64(Q).reshape(n, H, G, D)
        scale = D ** -0.5
        x = scale * np.einsum("nhgd,nhd->nhg", q, k)
        mass = np.einsum("nhgd,nhd->nhg", np.abs(q), np.abs(k))
        tol = scale * ((D // 16 + 16) * U * mass + grid * np.abs(q).max(-1) * np.abs(k).sum(-1)[..., None]) + 8 * U * np.abs(x)
        assert (np.abs(f64(lse).reshape(x.shape) - x) <= tol).all()
        want = np.broadcast_to(v[:, :, None], q.shape)
        assert (np.abs(f64(out).reshape(q.shape) - want) <= 2.0 ** -20 * np.abs(want)).all()


@pytest.mark.parametrize("top", [1.0, 1.984375, 1.9999999, 1.9921875, 1.5])
@pytest.mark.parametrize("exponent", [-99, -3, 0, 40, 127])
def test_largest_query_entries(imq, top, exponent):  # noqa: F811
    """Rows whose largest entries stand at the ends of what the first digit holds, both signs, over fp32's exponents."""
    D, n = 128, 1
    K = torch.full((n, 1, D), 127.0, device="cuda")  # codes of 127 and -127, a step of 1
    K[..., ::2] = -127.0
    cache, table, lens = filled(imq, K, K, 8, page=16)
    Q = torch.zeros(1, 4, D, device="cuda")
    big = float(np.float32(top) * np.float32(2.0) ** exponent)
    Q[0, 0, 0], Q[0, 1, 1], Q[0, 2, ::2], Q[0, 3, 1::2] = big, -big, big, big
    Q[0, 2, 6] = -big
    scale = 2.0 ** -exponent / 128
    _, lse = imq.imq_paged_attention(cache, Q, table, lens, scale=scale)
    x = scale * f64(Q)[0] @ f64(K)[0, 0]
    assert (np.abs(f64(lse)[0] - x) <= 8 * U * np.abs(x)).all()


@pytest.mark.parametrize("D,bits,G", SHAPES)
def test_values_that_grow_from_nothing(imq, D, bits, G):  # noqa: F811
    """Whole runs of zeros and of 1e-30, then values of 1, 1e4 and 1e30, with equal and with unequal weights."""
    H, n = 2, 320
    K, V, Q = _randn(1, n, H, D), _randn(2, n, H, D), _randn(3, 1, H * G, D)
    size = torch.zeros(n, device="cuda")
    size[64:128], size[128:192], size[192:256], size[256:] = 1e-30, 1.0, 1e4, 1e30
    for at in (64, 128, 192, 256, 320):
        cache, table, lens = filled(imq, K, V * size[:, None, None], bits)
        lens[0] = at
        check(imq, cache, Q, table, lens)
        check(imq, cache, Q, table, lens, scale=0.0)
