"""Calls of the decoding step that its other tests do not make: layouts of outputs, first calls, ends of ranges."""
import pytest
import torch

from test_gpu_decode import _randn, _status, imq, make_cache  # noqa: F401

pytestmark = pytest.mark.gpu


def test_outputs_laid_out_by_heads(imq):  # noqa: F811
    """Outputs whose heads are the outer axis, and vectors between another tensor's."""
    lens, H, G, D = [70, 0, 33, 16], 2, 3, 64
    cache, table, n = make_cache(imq, lens, 16, H, D, 8)
    Q = _randn(1, len(lens), H * G, D)
    want, wl = imq.imq_paged_attention(cache, Q, table, n)
    out = torch.full((H * G, len(lens), 2, D), 7.0, device="cuda")
    got, lse = imq.imq_paged_attention(cache, Q, table, n, out=out[:, :, 1].transpose(0, 1))
    assert torch.equal(got, want) and torch.equal(lse, wl) and (out[:, :, 0] == 7).all()
    slots = table[0, :4].long() * 16
    k, v = imq.imq_kv_read(cache, slots)
    both = torch.full((H, 4, 2, D), 7.0, device="cuda")
    imq.imq_kv_read(cache, slots, K=both[:, :, 0].transpose(0, 1), V=both[:, :, 1].transpose(0, 1))
    assert torch.equal(both[:, :, 0].transpose(0, 1), k) and torch.equal(both[:, :, 1].transpose(0, 1), v)
    with pytest.raises(imq.ImqError) as e:
        imq.imq_paged_attention(cache, Q, table, n, out=torch.zeros(len(lens), 1, D, device="cuda").expand(-1, H * G, -1))
    assert e.value.status == imq.IMQ_ERR_ARG
