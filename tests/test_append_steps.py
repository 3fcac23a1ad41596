"""mla_kv_append of 64-column queries: how many heads a warp takes changes no bit of what is written."""
import pytest
import torch


@pytest.fixture(scope="module")
def mla():
    from mla_attention_paged_gb300 import build
    build.build()
    from mla_attention_paged_gb300 import mla as m
    return m


# tokens x heads around the border (4256 warps of two steps, key warps among them), heads that fill four steps or not
SIZES = [(2000, 9), (2300, 9), (2100, 12), (2200, 12), (2120, 16), (2140, 16), (1690, 16), (1720, 16), (1400, 17), (1500, 17),
         (1300, 24), (3000, 24), (1060, 25), (1070, 32), (500, 40), (860, 33), (270, 128), (40, 1000)]


@pytest.mark.gpu
@pytest.mark.parametrize("n,heads", SIZES)
@pytest.mark.parametrize("keys", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_many_rows_as_few_at_a_time(mla, n, heads, keys, interleaved):
    """One call against calls of at most 12288 rows, which take one step (keys without a norm, whose sum has an order)."""
    g = torch.Generator().manual_seed(n + heads)
    d = "cuda"
    q = torch.randn(n, heads, 64, generator=g).bfloat16().to(d)
    kv = torch.randn(n, 576, generator=g).bfloat16().to(d) if keys else None
    angles = torch.rand(n, 32, generator=g) * 6
    cos_sin = torch.cat([angles.cos(), angles.sin()], 1).to(d)
    pos = torch.randperm(n, generator=g).int().to(d)
    pages = -(-n // 64)
    slots = torch.randperm(pages * 64, generator=g)[:n].to(d) if keys else None

    def run(step):
        pool = torch.full((pages, 64, 576), 7.0, device=d).bfloat16() if keys else None
        out = torch.empty_like(q)
        for a in range(0, n, step):
            s = slice(a, min(n, a + step))
            mla.kv_append(q[s], kv[s] if keys else None, pos[s], slots[s] if keys else None, cos_sin, pool, interleaved=interleaved,
                          q_out=out[s])
        assert mla.get_status() == mla.MLA_OK
        return out, pool
    out, pool = run(n)
    few, few_pool = run(max(1, 12288 // heads))
    assert torch.equal(out, few)
    assert not keys or torch.equal(pool, few_pool)
