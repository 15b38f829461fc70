"""Refusals of the decoding step's calls that need no GPU: through the C ABI, where argument errors are returned before any
device work, and through the binding's checks on CPU tensors."""
import ctypes

import pytest
import torch

import bit_integer_gemm_b200 as imq
from bit_integer_gemm_b200 import build


def _attention():
    c = imq.KVCache.zeros(3, 16, 2, 64, 8, device="cpu")
    return c, torch.zeros(4, 4, 64), torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)


@pytest.mark.parametrize("workspace", [torch.zeros(1, dtype=torch.uint8).expand(1 << 24), torch.zeros(1 << 12, dtype=torch.uint8)[::2],
                                       torch.zeros(64, 64).t()])
def test_workspaces_with_gaps_or_repeats_are_refused(workspace):
    """Their element count says nothing of the bytes behind their address."""
    with pytest.raises(ValueError, match="contiguous"):
        imq.imq_paged_attention(*_attention(), workspace=workspace)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return imq.lib()


P = 1 << 20  # a 16-byte aligned address that no refused call reads
# (n, step, heads, head step, dim) of vectors that share entries
OVERLAPS = [(2, 0, 2, 64, 64), (2, 128, 2, 0, 64), (2, 63, 1, 0, 64), (1, 0, 2, 63, 64), (2, 64, 2, 64, 64), (3, 128, 2, 256, 64),
            (2, 64, 3, 96, 64), (4, 100, 3, 230, 64), (2, 300, 4, 120, 64)]
APART = [(2, 128, 2, 64, 64), (2, 64, 2, 128, 64), (1, 0, 2, 64, 64), (2, 64, 1, 0, 64), (2, 128, 2, 192, 64), (3, 1 << 40, 2, 1 << 50, 64),
         (2, 192, 4, 64 * 6, 64)]


def _apart(n, step, heads, head_step, dim):
    at = sorted(i * step + h * head_step for i in range(n) for h in range(heads))
    return all(b - a >= dim for a, b in zip(at, at[1:]))


def test_what_overlaps():
    assert not any(_apart(*a) for a in OVERLAPS) and all(_apart(*a) for a in APART)


def _cache(heads, dim):
    return imq.imq_kv_cache(4096, 8192, 12288, 4, heads * 16 * dim, heads * 16 * dim, heads * 32, 16, heads, dim, 8)


@pytest.mark.parametrize("n,step,heads,head_step,dim", OVERLAPS)
def test_outputs_that_overlap_are_refused(lib, n, step, heads, head_step, dim):
    """Two results for one place: which of them stays would be left to chance."""
    c = _cache(heads, dim)
    r, good = ctypes.addressof(c), (heads * dim, dim)
    assert lib.imq_kv_read(r, P, n, P, step, head_step, None, 0, 0, imq.IMQ_F32, None) == imq.IMQ_ERR_ARG
    assert lib.imq_kv_read(r, P, n, P, *good, P, step, head_step, imq.IMQ_BF16, None) == imq.IMQ_ERR_ARG
    for lse, rows in ((None, 0), (P, heads)):
        assert lib.imq_paged_attention(r, P, imq.IMQ_BF16, 0, 0, n, heads, P, 4, 4, P, 64, 1.0, P, imq.IMQ_BF16, step, head_step,
                                       lse, rows, P, 1 << 30, None) == imq.IMQ_ERR_ARG


def test_log_sums_that_overlap_are_refused(lib):
    c = _cache(2, 64)
    for rows in (0, 1):
        assert lib.imq_paged_attention(ctypes.addressof(c), P, imq.IMQ_BF16, 0, 0, 2, 2, P, 4, 4, P, 64, 1.0, P, imq.IMQ_BF16, 128, 64, P,
                                       rows, P, 1 << 30, None) == imq.IMQ_ERR_ARG


def test_workspace_sizes_are_the_current_devices():
    """They count the device's SMs, and the binding keeps them with the cache: asked of another device, they would be
    another's."""
    c = imq.KVCache.zeros(3, 16, 2, 64, 8, device="cpu")
    with pytest.raises(ValueError, match="current CUDA device"):
        imq.imq_paged_attention_workspace(c, 1, 2, 48)
    assert not c._workspace
