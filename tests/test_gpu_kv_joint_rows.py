"""Outputs of gdn_kv_append and gdn_kv_attention among the columns of a joint q, k, v row."""
import pytest
import torch

from linear_attention_recurrence_gb300 import gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 2, 33, 500])
@pytest.mark.parametrize("dtype,H,G,D,pad", [(torch.bfloat16, 6, 2, 128, 0), (torch.float16, 8, 1, 64, 24), (torch.float32, 4, 2, 64, 3)])
def test_queries_in_place_in_a_joint_row(T, dtype, H, G, D, pad):
    gen = torch.Generator().manual_seed(T)
    row = torch.randn(T, (H + 2 * G) * D + pad, generator=gen).to(dtype).cuda()
    cut = lambda x: [x[:, a * D:(a + n) * D].unflatten(1, (n, D)) for a, n in ((0, H), (H, G), (H + G, G))]
    table = torch.randperm(T // 16 + 1, generator=gen).int().cuda()[None]
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    freq = torch.rand(D // 2, generator=gen).cuda()
    caches = [gdn.gdn_kv_cache(T // 16 + 1, G, 16, D) for _ in range(2)]
    q, k, v = cut(row)
    want = gdn.gdn_kv_append(k.contiguous(), v.contiguous(), caches[0], table, lens, q=q.contiguous(), inv_freq=freq)
    joint = row.clone()
    q, k, v = cut(joint)
    assert gdn.gdn_kv_append(k, v, caches[1], table, lens, q=q, inv_freq=freq, q_out=q) is q
    assert torch.equal(q, want) and torch.equal(caches[0], caches[1])
    assert torch.equal(joint[:, H * D:], row[:, H * D:])  # the keys and values are as they were


@pytest.mark.parametrize("T", [2, 200])
def test_attention_into_columns_of_its_queries_rows(T):
    H, G, D = 4, 2, 128
    gen = torch.Generator().manual_seed(T)
    row = torch.randn(T, 2 * H * D, generator=gen).bfloat16().cuda()
    q, out = row[:, H * D:].unflatten(1, (H, D)), row[:, :H * D].unflatten(1, (H, D))
    k = torch.randn(T, G, D, generator=gen).bfloat16().cuda()
    cache = gdn.gdn_kv_cache(T // 16 + 1, G, 16, D)
    table = torch.arange(T // 16 + 1, device="cuda", dtype=torch.int32)[None]
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    gdn.gdn_kv_append(k, k, cache, table, lens)
    want = gdn.gdn_kv_attention(q.contiguous(), cache, table, lens)
    before = q.clone()
    gdn.gdn_kv_attention(q, cache, table, lens, out=out)
    assert torch.equal(out, want) and torch.equal(q, before)
