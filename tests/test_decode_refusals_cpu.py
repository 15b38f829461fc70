"""Refusals of the decoding step's calls that need no GPU: through the C ABI, where argument errors are returned before any
device work, and through the binding's checks on CPU tensors."""
import pytest
import torch

import bit_integer_gemm_b200 as imq


def _attention():
    c = imq.KVCache.zeros(3, 16, 2, 64, 8, device="cpu")
    return c, torch.zeros(4, 4, 64), torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)


@pytest.mark.parametrize("workspace", [torch.zeros(1, dtype=torch.uint8).expand(1 << 24), torch.zeros(1 << 12, dtype=torch.uint8)[::2],
                                       torch.zeros(64, 64).t()])
def test_workspaces_with_gaps_or_repeats_are_refused(workspace):
    """Their element count says nothing of the bytes behind their address."""
    with pytest.raises(ValueError, match="contiguous"):
        imq.imq_paged_attention(*_attention(), workspace=workspace)
