"""The tensor form of the scan in FP16, whose range is short: steps of any size, against the
definition in 64 bits.

Tolerances: as in test_gpu_ssm.py, (4 tokens + 2 state_dim + 32) 2^-24 + 2^-21 of the states'
magnitudes, and the parts' smallest step (fp16_steps there): 2^-24 of a chunk's largest w
times |B|, never more than the product itself."""
import pytest
import torch

import ssm_reference as ref
from linear_attention_recurrence_gb300 import gdn
from test_gpu_ssm import F16, F32, check, fp16_steps, packed, rnd, scan_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_recurrence_gb300 import build

    build.build()


def inputs(gen, T, H, P, N):
    x, B, C = rnd(gen, T, H, P, dtype=F16), rnd(gen, T, 1, N, dtype=F16), rnd(gen, T, 1, N, dtype=F16)
    return x, rnd(gen, T, H, dtype=F16), B, C


@pytest.mark.parametrize("carried", [False, True])
@pytest.mark.parametrize("lens", [(300,), (127, 128, 129, 40), (1500,)])
@pytest.mark.parametrize("base", [-7.0, -14.0, -18.0, -25.0, -38.0])
def test_small_steps(base, lens, carried):
    """Steps of 2^-10 down to 2^-57 in every chunk: the states keep their precision."""
    gen = torch.Generator().manual_seed(51)
    cu, T = packed(lens)
    n, H, P, N = len(lens), 4, 128, 64
    x, a, B, C = inputs(gen, T, H, P, N)
    A_log, dt_bias = rnd(gen, H), torch.full((H,), base).cuda()
    states = rnd(gen, n, H, N, P, scale=0.3)
    has = torch.full((n,), carried)
    out = torch.zeros(T, H, P, dtype=F16).cuda()
    _, st, _, smag = ref.scan(x, a, B, C, A_log, dt_bias, states, None, None, cu, None, has, out)
    gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, states, cu_seqlens=cu, has_state=has.cuda(), out=out)
    torch.cuda.synchronize()
    more = fp16_steps(x, a, B, A_log, dt_bias, states, cu, torch.arange(n))
    check(states, st, smag, scan_bound(F32, P, N, max(lens)), "states", more)
    assert bool(torch.isfinite(out).all()) and gdn.gdn_device_status() == gdn.GDN_OK


@pytest.mark.parametrize("T", [200, 900])
def test_steps_of_every_size(T):
    """Chunks of large steps, of small ones and of none (dt = 0) in turn, and extreme decays."""
    gen = torch.Generator().manual_seed(52)
    H, P, N = 4, 128, 128
    x, a, B, C = inputs(gen, T, H, P, N)
    A_log = torch.tensor([-100.0, -3.0, 6.0, 88.0]).cuda()
    dt_bias = torch.tensor([0.0, 1.0, 2.0, 3.0]).cuda()
    a -= (torch.arange(T) // 128 % 3 * 14).to(F16).cuda()[:, None]
    a[::3] = -float("inf")
    a[128:256] = -float("inf")
    states = rnd(gen, 1, H, N, P, scale=0.3)
    cu = torch.tensor([0, T], dtype=torch.int32).cuda()
    out = torch.zeros(T, H, P, dtype=F16).cuda()
    y, st, mag, smag = ref.scan(x, a, B, C, A_log, dt_bias, states, None, None, None, None, None, out)
    gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, states, out=out)
    torch.cuda.synchronize()
    check(states, st, smag, scan_bound(F32, P, N, T), "states",
          fp16_steps(x, a, B, A_log, dt_bias, states, cu, torch.arange(1)))
    assert bool(torch.isfinite(out).all()) and gdn.gdn_device_status() == gdn.GDN_OK
