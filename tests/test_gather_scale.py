"""mla_kv_gather's kv_scale: asked of the formats that use it, ignored by the others."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def mla():
    from mla_attention_paged_gb300 import build
    build.build()
    from mla_attention_paged_gb300 import mla as m
    return m


@pytest.mark.parametrize("kind", [1, 2, 4])
@pytest.mark.parametrize("scale", [0.0, -1.0, math.nan])
def test_a_scale_that_is_used_is_positive(mla, kind, scale):
    at = [ctypes.c_void_p(1 << n) for n in (20, 8, 10, 28)]
    assert mla.lib.mla_kv_gather(at[0], 10, 64, kind, scale, None, at[1], 4, at[2], 2, 100, at[3], 576, None) == mla.MLA_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -1.0, math.nan])
def test_a_scale_that_is_not_used_is_ignored(mla, scale):
    g = torch.Generator().manual_seed(1)
    table = torch.tensor([[2, 0], [3, 3]], dtype=torch.int32)
    rows = torch.cat([torch.arange(32, 48), torch.arange(0, 4), torch.arange(48, 57)])
    cu = torch.tensor([0, 20, 29], dtype=torch.int32, device="cuda")
    x = torch.randn(4, 16, 576, generator=g)
    codes = (x * 25).round().clamp(-127, 127).to(torch.int8)
    scales = torch.rand(4, generator=g) * 0.05
    for pool, kind, ps, value in ((x.bfloat16(), mla.MLA_KV_BF16, None, x.bfloat16()),
                                  (codes, mla.MLA_KV_INT8_PAGE, scales.cuda(), (codes.float() * scales[:, None, None]).bfloat16())):
        out = torch.zeros(29, 576, device="cuda").bfloat16()
        mla.kv_gather(pool.cuda(), table.cuda(), cu, out, kv_dtype=kind, kv_scale=scale, page_scales=ps)
        assert mla.get_status() == mla.MLA_OK
        assert torch.equal(out.cpu(), value.view(-1, 576)[rows])
