"""Heads' scales of any size: codes and scales have one right answer for each positive FP32
number, the smallest and the largest among them."""
import math

import pytest
import torch

import kv_reference as ref
from linear_attention_recurrence_gb300 import gdn
from test_gpu_kv_append import held

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rotary", [0, 64])
@pytest.mark.parametrize("scale", [2.0 ** -149, 3 * 2.0 ** -149, 1e-40, 2.0 ** -126, 1.2e-38, 1e-36, 2.0 ** -101, 2.0 ** -99, 1e-20,
                                   1e20, 2.0 ** 99, 2.0 ** 101, 1e35, 1e37, 2.0 ** 127, 3.4e38])
def test_heads_scales(dtype, rotary, scale):
    gen = torch.Generator().manual_seed(2)
    T, G, D = 6, 2, 64
    hs = torch.tensor([scale, 1.0], dtype=torch.float32)
    most = min(1.0, 3e38 / (float(hs[0]) * 8))  # (finite elements)
    x = (torch.randn(T, G, D, generator=gen, dtype=torch.float64) * most).clamp(-4 * most, 4 * most) * hs.double()[:, None]
    x[1, :, :16] *= 40
    x[2, :, :7] = 0
    x[2, :, 16:32] = 0
    x[3, :, 5] = -0.0
    x = x.clamp(-3.3e38, 3.3e38).to(dtype)
    assert bool(x.isfinite().all())
    freq = 1e4 ** (-torch.arange(0, rotary, 2).float() / max(rotary, 1))
    cache = gdn.gdn_kv_cache(1, G, 16, D)
    gdn.gdn_kv_append(x.cuda(), x.cuda(), cache, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                      torch.tensor([T], dtype=torch.int32, device="cuda"), inv_freq=freq.cuda() if rotary else None,
                      k_scale=hs.cuda(), v_scale=hs.cuda())
    cache = cache.cpu()
    n = 16 * D // 2
    for which, y in ((0, ref.rotate(x, torch.arange(T), freq, False)), (1, x.double())):
        codes, scales, _ = held(y, hs, dtype)
        got = cache[0, :, which, :n].view(G, 16, D // 2)[:, :T].transpose(0, 1).int()
        assert torch.equal(cache[0, :, which, n:].view(G, 16, D // 16)[:, :T].transpose(0, 1).int(), scales)
        assert torch.equal(torch.stack([got & 15, got >> 4], -1).flatten(-2), codes)
