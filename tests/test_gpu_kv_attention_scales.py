"""gdn_kv_attention under heads' scales of any size: a scale that is a power of two moves its
results by that power, to the bit."""
import pytest
import torch

from linear_attention_recurrence_gb300 import gdn
from test_gpu_kv_attention import make

pytestmark = pytest.mark.gpu
SHAPES = [([1] * 3, [9000, 30, 700]), ([1], [200]), ([4, 1], [5000, 64]), ([150], [200]), ([70], [9000])]


@pytest.mark.parametrize("new,lens", SHAPES)
@pytest.mark.parametrize("power", [-120, -100, 100])
def test_values(new, lens, power):
    q, cache, table, kv, cu, _, _ = make(new, lens, 6, 2, 128, 32, "bf16", torch.Generator().manual_seed(1))
    by = torch.tensor([2.0 ** power, 1.0], device="cuda")
    got = gdn.gdn_kv_attention(q, cache, table, kv, cu_seqlens=cu, v_scale=by)
    want = gdn.gdn_kv_attention(q, cache, table, kv, cu_seqlens=cu)
    for head in range(6):
        a, b = got[:, head].double(), want[:, head].double()
        sure = b.abs() >= 2.0 ** -5  # (BF16's normal range ends at 2^-126)
        assert bool(sure.any()) and torch.equal(a[sure], b[sure] * float(by[head % 2]))


@pytest.mark.parametrize("new,lens", SHAPES)
@pytest.mark.parametrize("power,up", [(-140, 120), (-120, 120), (-126, 110), (100, -90), (120, -100)])
def test_keys(new, lens, power, up):
    """Queries sized against the scale: the scores are ordinary ones."""
    q, cache, table, kv, cu, _, _ = make(new, lens, 6, 2, 128, 32, "bf16", torch.Generator().manual_seed(2))
    q = torch.where(q.abs() < 2.0 ** -10, 0, q)  # (those times 2^-100 are normal numbers)
    lse, same = (torch.empty(q.shape[:2], device="cuda") for _ in range(2))
    got = gdn.gdn_kv_attention(q * 2.0 ** up, cache, table, kv, cu_seqlens=cu, lse=lse,
                               k_scale=torch.full((2,), 2.0 ** power, device="cuda"))
    want = gdn.gdn_kv_attention(q * 2.0 ** (up + power), cache, table, kv, cu_seqlens=cu, lse=same)
    assert torch.equal(got, want) and torch.equal(lse, same)
