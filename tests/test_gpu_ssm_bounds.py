"""Sequence bounds and slots that are not sound: what a call may still touch.

Bounds live on the device, so a call cannot refuse them; whatever they hold, the kernels
read and write within the arrays that they were given."""
import pytest
import torch

from linear_attention_recurrence_gb300 import gdn

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_recurrence_gb300 import build

    build.build()


@pytest.mark.parametrize("ch", [64, 37])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("bounds", [(0, 2, 1, 40), (1, 1, 1, 0, 40), (5, 0, 1, 0, 40), (0, 17, 16, 40)])
def test_conv_reads_no_row_before_its_array(bounds, width, ch):
    """A sequence that begins below the end of an earlier one is taken up behind its own first
    row.  The window is then not its own, but it is made of the array's rows: the 8 rows of
    NaN before the array (and behind it) reach no output."""
    gen = torch.Generator().manual_seed(41)
    T = 40
    wide = torch.full((T + 16, ch), float("nan"))
    wide[8:8 + T] = torch.randn(T, ch, generator=gen)
    x = wide.cuda()[8:8 + T]
    w = torch.rand(ch, width, generator=gen).cuda() + 0.1
    cu = torch.tensor(bounds, dtype=torch.int32).cuda()
    out = torch.zeros(T, ch).cuda()
    gdn.gdn_ssm_conv(x, w, cu_seqlens=cu, out=out)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out).all())


def layer(gen, T, H, G, P, N, dtype, lead):
    """A scan's inputs as rows `lead` .. of arrays with NaN in the `lead` rows around them."""

    def rows(*shape):
        v = torch.full((T + 2 * lead, *shape), float("nan"))
        v[lead:lead + T] = torch.randn(T, *shape, generator=gen)
        return v.to(dtype).cuda()[lead:lead + T]

    A_log = torch.log(torch.rand(H, generator=gen) * 15 + 1).cuda()
    dt_bias = (torch.randn(H, generator=gen) - 3).cuda()
    return rows(H, P), rows(H), rows(G, N), rows(G, N), A_log, dt_bias


# dtype, P, N, T, heads: the token form, the tensor form with whole sequences, and with segments
FORMS = [(F32, 64, 64, 400, 2), (F16, 32, 64, 400, 2), (BF16, 64, 128, 400, 40), (F16, 128, 64, 400, 40),
         (BF16, 128, 128, 1900, 2), (F16, 64, 64, 1900, 2)]


@pytest.mark.parametrize("dtype,P,N,T,H", FORMS)
def test_scan_with_bounds_out_of_range(dtype, P, N, T, H):
    """Bounds below 0 and above the rows make their own sequence empty: the others, their slots and
    everything else are as if that sequence had no rows.  Slots out of range keep nothing."""
    gen = torch.Generator().manual_seed(42)
    x, a, B, C, A_log, dt_bias = layer(gen, T, H, 1, P, N, dtype, 130)
    mid = T // 3
    cu = torch.tensor([-5, 3, mid, mid, T - 9, T + 7, T + 9], dtype=torch.int32).cuda()
    as_if = torch.tensor([3, 3, mid, mid, T - 9, T - 9, T - 9], dtype=torch.int32).cuda()
    slots = torch.tensor([6, 7, 1, 2, 3, 4], dtype=torch.int32).cuda()  # [3, mid) has slot 7 of 7: none
    pool = torch.randn(7, H, N, P, generator=gen).cuda()
    got, want = pool.clone(), pool.clone()
    out = torch.full((T, H, P), 3.0, dtype=dtype).cuda()
    ref = out.clone()
    gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, got, cu_seqlens=cu, slots=slots, out=out)
    gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, want, cu_seqlens=as_if, slots=slots, out=ref)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(got, want)
    assert bool((out[:3] == 3.0).all()) and bool((out[T - 9:] == 3.0).all())
    kept = [0, 1, 3, 4, 5, 6]  # slot 2 alone has a sequence with rows
    assert torch.equal(got[kept], pool[kept]) and not torch.equal(got[2], pool[2])
    assert gdn.gdn_device_status() == gdn.GDN_OK


DECREASING = [(0, 10, 5, 390, 60), (20, 40, 0, 10, 400), (0, 400, 0, 400, 0, 400), (400, 300, 200, 100, 0),
              (0, 400, 399, 0, 399, 1, 400), (-7, 400, 0, 500, 130)]


@pytest.mark.parametrize("bounds", DECREASING)
@pytest.mark.parametrize("dtype,P,N,T,H", FORMS)
def test_decreasing_bounds_stay_inside_the_arrays(dtype, P, N, T, H, bounds):
    """What such a call gives is undefined; what lies around its arrays stays as it was, its waits end,
    and the same call with sound bounds is right behind it."""
    gen = torch.Generator().manual_seed(43)
    x, a, B, C, A_log, dt_bias = layer(gen, T, H, 1, P, N, dtype, 130)
    k = T // 400
    cu = torch.tensor([b * k for b in bounds], dtype=torch.int32).cuda()
    n = len(bounds) - 1
    slots = torch.arange(1, n + 1, dtype=torch.int32).cuda()
    pool = torch.randn(n + 2, H, N, P, generator=gen).cuda()
    wide = torch.full((T + 16, H, P), 3.0, dtype=dtype).cuda()
    args = (x, a, B, C, A_log, dt_bias)
    want = gdn.gdn_ssm_scan(*args)
    states = pool.clone()
    gdn.gdn_ssm_scan(*args, states, cu_seqlens=cu, slots=slots, out=wide[8:8 + T])
    torch.cuda.synchronize()
    assert bool((wide[:8] == 3.0).all()) and bool((wide[8 + T:] == 3.0).all())
    assert torch.equal(states[[0, -1]], pool[[0, -1]])
    assert gdn.gdn_device_status() == gdn.GDN_OK
    assert torch.equal(gdn.gdn_ssm_scan(*args), want)


@pytest.mark.parametrize("dtype,ch", [(F32, 64), (BF16, 256), (F16, 37)])
def test_conv_with_bounds_out_of_range(dtype, ch):
    gen = torch.Generator().manual_seed(44)
    T = 90
    x = torch.randn(T, ch, generator=gen).to(dtype).cuda()
    w = torch.rand(ch, 4, generator=gen).cuda()
    cu = torch.tensor([-5, 3, 31, 31, 81, 97, 99], dtype=torch.int32).cuda()
    as_if = torch.tensor([3, 3, 31, 31, 81, 81, 81], dtype=torch.int32).cuda()
    slots = torch.tensor([6, 7, 1, 2, 3, 4], dtype=torch.int32).cuda()
    pool = torch.randn(7, 3, ch, generator=gen).to(dtype).cuda()
    got, want = pool.clone(), pool.clone()
    out = torch.full((T, ch), 3.0, dtype=dtype).cuda()
    ref = out.clone()
    gdn.gdn_ssm_conv(x, w, hist=got, cu_seqlens=cu, slots=slots, out=out)
    gdn.gdn_ssm_conv(x, w, hist=want, cu_seqlens=as_if, slots=slots, out=ref)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(got, want)
    kept = [0, 1, 3, 4, 5, 6]
    assert torch.equal(got[kept], pool[kept]) and torch.equal(got[2], x[78:81])


@pytest.mark.parametrize("bounds", DECREASING)
@pytest.mark.parametrize("dtype,ch", [(F32, 64), (BF16, 256), (F16, 37)])
def test_conv_with_decreasing_bounds_stays_inside_the_arrays(dtype, ch, bounds):
    gen = torch.Generator().manual_seed(45)
    T, n = 400, len(bounds) - 1
    x = torch.randn(T, ch, generator=gen).to(dtype).cuda()
    w = torch.rand(ch, 4, generator=gen).cuda()
    cu = torch.tensor(bounds, dtype=torch.int32).cuda()
    slots = torch.arange(1, n + 1, dtype=torch.int32).cuda()
    pool = torch.randn(n + 2, 3, ch, generator=gen).to(dtype).cuda()
    hist, wide = pool.clone(), torch.full((T + 16, ch), 3.0, dtype=dtype).cuda()
    gdn.gdn_ssm_conv(x, w, hist=hist, cu_seqlens=cu, slots=slots, out=wide[8:8 + T])
    torch.cuda.synchronize()
    assert bool((wide[:8] == 3.0).all()) and bool((wide[8 + T:] == 3.0).all())
    assert torch.equal(hist[[0, -1]], pool[[0, -1]])
