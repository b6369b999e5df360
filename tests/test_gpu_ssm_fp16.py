"""The tensor form of the scan in FP16, whose range is short: steps, scores and states of any
size, against the definition in 64 bits.

Tolerances: as in test_gpu_ssm.py, (4 tokens + 2 state_dim + 32) 2^-24 + 2^-21 of the states'
magnitudes, and the parts' smallest step (fp16_steps there): 2^-24 of a chunk's largest w
times |B|, never more than the product itself.  Outputs: the same and eps / 2 of the
magnitude, and what smallest steps cost them (floors below)."""
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


def floors(x, a, B, C, A_log, dt_bias, hmax):
    """What FP16's smallest step, off by 2^-25, costs an output (one head group).  A score C.B dt is rounded times
    2^s / ds, ds <= 2 max dt of the chunk; s is 0, or 16 2^-s < the largest of 32 rows' |C.B| / 2^16
    where that is above the range: 2^-24 max dt max(1, 2^-12 max |C.B|) off, times |x|, over a
    chunk's tokens.  The state is rounded times a power of two that brings the largest of 32
    columns to 2^14 at least: 2^-39 of it off, times |C|.  (Maxima over the whole call.)  And the
    state itself is off by what its parts lose in the chunks before (fp16_steps), times |C|."""
    T, H, P = x.shape
    N = B.shape[2]
    state = torch.zeros(T, H, P, dtype=torch.float64)
    for b in range(128, T, 128):
        off = fp16_steps(x, a, B, A_log, dt_bias, torch.zeros(1, H, N, P), [0, b], torch.arange(1))[0]
        c = C[b:b + 128, 0].cpu().double().abs().nan_to_num(0, posinf=0)
        state[b:b + 128] = torch.einsum("tn,hnp->thp", c, off.nan_to_num(0))
    x, a, B, C, dt_bias = (t.cpu().double() for t in (x, a, B, C, dt_bias))
    dt = torch.logaddexp(a + dt_bias, torch.zeros((), dtype=torch.float64)).amax(0)
    s = float((C[:, 0] @ B[:, 0].T).abs().nan_to_num(0, posinf=0).max())
    sums = x.abs().cumsum(0)
    sums = sums - torch.cat([torch.zeros_like(sums[:128]), sums[:-128]])[:len(sums)] if len(sums) > 128 else sums
    scores = 2.0 ** -24 * max(1.0, 2.0 ** -12 * s) * dt[:, None] * sums
    return state + scores + 2.0 ** -39 * hmax * C[:, 0].abs().nan_to_num(0, posinf=0).sum(-1)[:, None, None]


def run(x, a, B, C, A_log, dt_bias, states, D=None, z=None):
    """(got, want, magnitudes of y; the states' after, wanted, magnitudes and bound)."""
    T = len(x)
    cu = torch.tensor([0, T], dtype=torch.int32)
    out = torch.zeros_like(x)
    y, st, mag, smag = ref.scan(x, a, B, C, A_log, dt_bias, states, D, z, None, None, None, out)
    more = fp16_steps(x, a, B, A_log, dt_bias, states, cu, torch.arange(1))
    gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, states, D=D, z=z, out=out)
    torch.cuda.synchronize()
    assert gdn.gdn_device_status() == gdn.GDN_OK
    return out, y, mag, st, smag, more


@pytest.mark.parametrize("T", [128, 300, 900])
@pytest.mark.parametrize("big", [(0, 128, 0, 128), (70, 100, 0, 128), (0, 40, 96, 128), (100, 101, 110, 113), (3, 4, 3, 4)])
@pytest.mark.parametrize("size", [60.0, 4000.0])
def test_scores_above_the_range(size, big, T):
    """C . B up to 2^37 where B's and C's tokens (of every chunk) are large: in the first half of a
    chunk's columns, in the second, in both, for all rows or a few."""
    gen = torch.Generator().manual_seed(53)
    H, P, N = 4, 128, 128
    x, a, B, C = inputs(gen, T, H, P, N)
    at = torch.arange(T) % 128
    B[(at >= big[0]) & (at < big[1])] *= size
    C[(at >= big[2]) & (at < big[3])] *= size
    x *= 2.0 ** -12 if size > 1000 else 2.0 ** -4
    A_log, dt_bias = torch.log(torch.rand(H, generator=gen) * 15 + 1).cuda(), torch.full((H,), -6.0).cuda()
    states = torch.zeros(1, H, N, P).cuda()
    got, y, mag, st, smag, more = run(x, a, B, C, A_log, dt_bias, states, D=rnd(gen, H))
    assert float(y.abs().max()) < 60000
    check(got, y, mag, scan_bound(F16, P, N, T), "y", floors(x, a, B, C, A_log, dt_bias, float(smag.max())))
    check(states, st, smag, scan_bound(F32, P, N, T), "states", more)


@pytest.mark.parametrize("size,c_size", [(3e5, 2.0 ** -10), (1e9, 2.0 ** -22), (1e-9, 3000.0), (1e-20, 3000.0)])
@pytest.mark.parametrize("P,N,T", [(128, 128, 200), (64, 64, 900), (64, 128, 300), (128, 64, 40)])
def test_states_of_every_size(size, c_size, P, N, T):
    """Carried states far above FP16's range, seen through a small C, and far below it, through a large one."""
    gen = torch.Generator().manual_seed(54)
    H = 4
    x, a, B, C = inputs(gen, T, H, P, N)
    C = (C.float() * c_size).to(F16)
    A_log, dt_bias = rnd(gen, H) - 4, torch.full((H,), -7.0 if size > 1 else -25.0).cuda()
    states = rnd(gen, 1, H, N, P, scale=size)
    states[:, :, :, P // 2:] *= 2.0 ** -6
    got, y, mag, st, smag, more = run(x, a, B, C, A_log, dt_bias, states, z=rnd(gen, T, H, P, dtype=F16))
    assert float(y.abs().max()) < 60000
    check(got, y, mag, scan_bound(F16, P, N, T), "y", floors(x, a, B, C, A_log, dt_bias, float(smag.max())) * 8)  # (|silu(z)| < 8)
    check(states, st, smag, scan_bound(F32, P, N, T), "states", more)


@pytest.mark.parametrize("size", [1.0, 60.0])
def test_infinities_stay_with_their_row(size):
    """An infinite C of one token and an infinite element of a state: that token's outputs and that
    column's are not finite, all others are as precise as without them, also above the range."""
    gen = torch.Generator().manual_seed(55)
    T, H, P, N, at, col = 300, 4, 128, 128, 170, 37
    x, a, B, C = inputs(gen, T, H, P, N)
    B *= size
    C *= size
    x *= 2.0 ** -4
    A_log, dt_bias = rnd(gen, H) - 2, torch.full((H,), -6.0).cuda()
    states = rnd(gen, 1, H, N, P, scale=0.3)
    states[0, 1, 5, col] = float("inf")
    C[at, 0, 9] = float("inf")
    got, y, mag, _, smag, _ = run(x, a, B, C, A_log, dt_bias, states)
    rest = torch.ones(T, H, P, dtype=torch.bool)
    rest[at] = False
    rest[:, 1, col] = False
    assert not torch.isfinite(got.cpu()[~rest]).any()
    tol = floors(x, a, B, C, A_log, dt_bias, float(smag[smag.isfinite()].max()))
    for u in (y, mag, tol):
        u[~rest] = 0
    check(torch.where(rest.cuda(), got, 0), y, mag, scan_bound(F16, P, N, T), "y", tol)
