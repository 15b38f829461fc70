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


@pytest.mark.parametrize("exponent", [-109, -100, 0, 100, 117])
def test_ends_of_a_products_range(imq, exponent):  # noqa: F811
    """fp32 entries from 2^-109 to 2^118 keep all their bits: their last part lies above bf16's smallest spacing, and a
    group's sum, up to 128 entries times codes of 7, within fp32.  One weight of step 1 and code 7 and its product, then
    groups whose sum has one sign.  (An exact product passes the sums of three parts; one of 128 of them, its inner steps, too.)"""
    x = (1 + torch.rand(9, 1, generator=torch.Generator().manual_seed(exponent), dtype=torch.float64)).float().cuda() * 2.0 ** exponent
    one = imq.imq_w4_quantize(torch.full((1, 5), 7.0, device="cuda"), 32)
    y = imq.imq_w4_matvec(one, x).double()
    assert ((y - 7 * x.double()).abs() <= 3 * 2.0 ** -23 * y).all()
    many = imq.imq_w4_quantize(torch.full((128, 5), 7.0, device="cuda"), 128)
    y = imq.imq_w4_matvec(many, x.expand(9, 128).contiguous()).double()
    assert ((y - 896 * x.double()).abs() <= 40 * 2.0 ** -23 * y).all()
