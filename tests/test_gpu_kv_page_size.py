"""The binding's page size: what a page's bytes come to at the call's head_dim, or as the caller
says, which must agree."""
import pytest
import torch

from linear_attention_recurrence_gb300 import gdn

pytestmark = pytest.mark.gpu


def call(cache, D, **kw):
    dev = "cuda"
    x = torch.ones(3, 2, D, device=dev).bfloat16()
    table, lens = torch.zeros(1, 1, device=dev, dtype=torch.int32), torch.tensor([3], device=dev, dtype=torch.int32)
    gdn.gdn_kv_append(x, x, cache, table, lens, **kw)
    return gdn.gdn_kv_attention(x, cache, table, lens, **kw)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_a_page_size_that_agrees(D, page):
    cache = gdn.gdn_kv_cache(2, 2, page, D)
    assert torch.equal(call(cache, D, page_size=page), call(cache.clone(), D))


def test_a_cache_of_another_head_width_is_refused():
    """Pages of 32 tokens of 64 are as long as pages of 16 tokens of 128."""
    for made, used in (((32, 64), 128), ((16, 128), 64)):
        cache = gdn.gdn_kv_cache(2, 2, *made)
        with pytest.raises(ValueError, match="made for head_dim"):
            call(cache, used)
        with pytest.raises(ValueError, match="page_size"):  # a view does not know
            call(cache[:], used, page_size=made[0])
        with pytest.raises(ValueError, match="page_size"):
            gdn.gdn_kv_attention(torch.ones(3, 2, used, device="cuda").bfloat16(), cache[:],
                                 torch.zeros(1, 1, device="cuda", dtype=torch.int32),
                                 torch.tensor([3], device="cuda", dtype=torch.int32), page_size=made[0])
        assert not bool(cache.any())
