"""gdn_kv_attention through the C entry, with a workspace of the test's own: what it held before
does not reach the results, and nothing is written behind it."""
import pytest
import torch

from linear_attention_recurrence_gb300 import gdn
from test_gpu_kv_attention import make

pytestmark = pytest.mark.gpu

CASES = [([1] * 5, [3000, 9, 700, 64, 1], True), ([1] * 5, [3000, 9, 700, 64, 1], False), ([4] * 3, [900, 50, 2000], False),
         ([70], [5000], False), ([200, 1, 90, 4], [4200, 900, 90, 33], True), ([20, 0, 40], [20, 5, 3000], True)]


def arguments(new, lens, with_bounds, D, H=6, G=2, page=32):
    q, cache, table, kv, cu, ks, vs = make(new, lens, H, G, D, page, "bf16", torch.Generator().manual_seed(5), True)
    T, n = q.shape[0], len(new)
    need = gdn.load_library().gdn_kv_attention_workspace_bytes(T, n, 0 if with_bounds else 1, page, table.shape[1], H, G, D)
    out, lse = torch.empty_like(q), torch.empty(T, H, device="cuda")

    def call(workspace, size=need):
        out.fill_(7), lse.fill_(7)
        rc = gdn.load_library().gdn_kv_attention(
            q.data_ptr(), H * D, cache.data_ptr(), cache.shape[0], page, table.data_ptr(), table.shape[1], table.shape[1],
            kv.data_ptr(), cu.data_ptr() if with_bounds else None, n, ks.data_ptr(), vs.data_ptr(), D ** -0.5, 1, 0,
            out.data_ptr(), H * D, lse.data_ptr(), T, H, G, D, gdn.GDN_BF16, None if workspace is None else workspace.data_ptr(),
            size, torch.cuda.current_stream().cuda_stream)
        return rc, out.clone(), lse.clone()
    keep = (q, cache, table, kv, cu, ks, vs)
    return call, need, keep


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,lens,with_bounds", CASES)
def test_what_the_workspace_held(new, lens, with_bounds, D):
    call, need, keep = arguments(new, lens, with_bounds, D)
    assert need > 0
    results = []
    for byte in (0x00, 0xFF, 0x7F, 0x01):  # (0xff: NaN and -1, 0x7f: 3.4e38 and large numbers)
        ws = torch.full((need + 4096,), byte, dtype=torch.uint8, device="cuda")
        rc, out, lse = call(ws)
        assert rc == gdn.GDN_OK
        assert bool((ws[need:] == byte).all())
        results.append((out, lse))
    for out, lse in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(lse, results[0][1])
    q, cache, table, kv, cu, ks, vs = keep
    want = gdn.gdn_kv_attention(q, cache, table, kv, k_scale=ks, v_scale=vs, cu_seqlens=cu if with_bounds else None)
    assert torch.equal(want, results[0][0])
    assert gdn.gdn_device_status() == 0


def test_a_workspace_that_is_missing_or_too_small():
    call, need, _ = arguments([1] * 5, [3000, 9, 700, 64, 1], True, 128)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for got in (call(None), call(ws, need - 1)):
        assert got[0] == gdn.GDN_ERR_INVALID_ARG and bool((got[1] == 7).all())
    assert call(ws)[0] == gdn.GDN_OK
