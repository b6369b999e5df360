"""gdn_launch_count counts the paged cache's kernels: of the few-row form one, and one more that
joins pieces; of the prompt form one, and one more where units are split."""
import pytest
import torch

from linear_attention_recurrence_gb300 import gdn
from test_gpu_kv_attention import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,lens,with_bounds,launches", [
    ([1] * 3, [60, 200, 9], False, 1),        # short caches: units stay whole
    ([1] * 3, [60, 5000, 9], False, 2),       # pieces, joined
    ([70], [200], False, 1),                  # a prompt over few blocks
    ([70], [5000], False, 2),                 # split between CTAs
    ([70, 1], [200, 60], True, 2),            # both forms
    ([70, 1], [5000, 60], True, 4),
])
def test_attention(new, lens, with_bounds, launches):
    q, cache, table, kv, cu, _, _ = make(new, lens, 4, 2, 128, 64, "bf16", torch.Generator().manual_seed(1))
    before = gdn.gdn_launch_count()
    gdn.gdn_kv_attention(q, cache, table, kv, cu_seqlens=cu if with_bounds else None)
    assert gdn.gdn_launch_count() - before == launches


def test_append():
    k = torch.ones(5, 2, 64, device="cuda").half()
    before = gdn.gdn_launch_count()
    gdn.gdn_kv_append(k, k, gdn.gdn_kv_cache(1, 2, 16, 64), torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                      torch.tensor([5], dtype=torch.int32, device="cuda"), q=k)
    assert gdn.gdn_launch_count() - before == 1
