"""The scan's token form with 16-bit rows, held to its own bound.

Which form runs goes by sizes: the tensor form takes BF16 and FP16 with head_dim and state_dim
64 or 128, T >= 32 n_seq, and rows of 16-byte pieces.  The calls here are
outside of that, so nothing but y is rounded to the type: the bound is the token form's,
(4 tokens + 2 state_dim + 32) 2^-24 + 2^-21 of the magnitude, for y and the states."""
import pytest
import torch

import ssm_reference as ref
from linear_attention_recurrence_gb300 import gdn
from test_gpu_ssm import BF16, F16, F32, check, layer, packed, rnd, scan_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_recurrence_gb300 import build

    build.build()


CASES = [
    # lens, H, G, P, N, wide (columns before x), strong
    ((70, 70), 2, 2, 96, 32, 0, False),      # sizes
    ((200,), 2, 1, 256, 64, 3, True),
    ((150,), 3, 1, 32, 16, 0, False),
    ((90, 1, 60), 4, 2, 128, 32, 5, True),
    ((1,), 3, 1, 128, 128, 0, False),        # tokens per sequence
    ((28,), 4, 2, 64, 64, 0, True),
    ((40, 1, 3, 50), 2, 1, 128, 128, 0, False),
    ((300,), 2, 1, 128, 128, 4, False),      # rows off 16-byte boundaries
    ((127, 129), 4, 2, 64, 128, 1, True),
    ((640,), 3, 3, 64, 64, 2, False),
]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens,H,G,P,N,wide,strong", CASES)
def test_token_form_keeps_its_bound(lens, H, G, P, N, wide, strong, dtype):
    gen = torch.Generator().manual_seed(sum(lens) + P + N + 1)
    n = len(lens)
    cu, end = packed(lens, lead=1)
    T = end + 2
    assert P not in (64, 128) or N not in (64, 128) or T < 32 * n or wide % 8
    x, a, B, C, A_log, dt_bias = layer(gen, T, H, G, P, N, dtype, wide, strong)
    z, D = rnd(gen, T, H, P, dtype=dtype), rnd(gen, H)
    states, out = rnd(gen, n + 2, H, N, P, scale=0.3), rnd(gen, T, H, P, dtype=dtype)
    slots = torch.randperm(n + 2, generator=gen)[:n].to(torch.int32)
    has = torch.tensor([i % 3 != 1 for i in range(n)])
    y, st, mag, smag = ref.scan(x, a, B, C, A_log, dt_bias, states, D, z, cu, slots, has, out)
    gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, states, D=D, z=z, cu_seqlens=cu, slots=slots.cuda(),
                     has_state=has.cuda(), out=out)
    torch.cuda.synchronize()
    check(out, y, mag, scan_bound(F32, P, N, max(lens)), "y")
    check(states, st, smag, scan_bound(F32, P, N, max(lens)), "states")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,H", [(300, 40), (900, 4)])
def test_nan_in_x_stays_in_its_column_and_32_tokens(dtype, T, H):
    """The tensor form: a NaN in x reaches its column's later outputs and those of the same 32 tokens
    of its chunk, the column's state, and nothing else."""
    gen = torch.Generator().manual_seed(61)
    P, N, at, h, col = 128, 64, 170, 1, 9
    x, a, B, C, A_log, dt_bias = layer(gen, T, H, 2, P, N, dtype)
    states = rnd(gen, 1, H, N, P)
    want_st = states.clone()
    want = gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, want_st)
    x[at, h, col] = float("nan")
    y = gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, states)
    torch.cuda.synchronize()
    first = at // 32 * 32
    assert torch.equal(y[:first], want[:first])
    assert bool(y[at:, h, col].isnan().all()) and bool(states[0, h, :, col].isnan().all())
    keep = torch.ones(H, P, dtype=torch.bool).cuda()
    keep[h, col] = False
    assert torch.equal(y[:, keep], want[:, keep])
    assert torch.equal(states[0].transpose(1, 2)[keep], want_st[0].transpose(1, 2)[keep])


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_token_form_on_request(dtype):
    """The option takes every call to the token form: its bound where the tensor form would run, the
    same bits for a sequence alone, split over calls and beside others, and no workspace."""
    gen = torch.Generator().manual_seed(62)
    T, H, P, N = 420, 4, 128, 128
    x, a, B, C, A_log, dt_bias = layer(gen, T, H, 2, P, N, dtype)
    start = rnd(gen, 1, H, N, P, scale=0.3)
    y, st, mag, smag = ref.scan(x, a, B, C, A_log, dt_bias, start, None, None, None, None, None, torch.zeros(T, H, P))
    tensor = gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, start.clone())
    with gdn.options(ssm_scan_form=1):
        assert gdn.load_library().gdn_ssm_scan_workspace_bytes(T, 1, H, P, N, gdn.GDN_BF16) == 0
        s1, s2 = start.clone(), start.clone()
        whole = gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, s1)
        parts, at = [], 0
        for n in (100, 3, 200, 117):
            r = slice(at, at + n)
            parts.append(gdn.gdn_ssm_scan(x[r], a[r], B[r], C[r], A_log, dt_bias, s2))
            at += n
        cu, _ = packed((T, 1))
        more = [torch.cat([v, v[:1]]) for v in (x, a, B, C)]
        s3 = torch.cat([start, start])
        beside = gdn.gdn_ssm_scan(*more, A_log, dt_bias, s3, cu_seqlens=cu)
    torch.cuda.synchronize()
    check(whole, y, mag, scan_bound(F32, P, N, T), "y")
    check(s1, st, smag, scan_bound(F32, P, N, T), "states")
    assert at == T and torch.equal(whole, torch.cat(parts)) and torch.equal(s1, s2)
    assert torch.equal(whole, beside[:T]) and torch.equal(s1[0], s3[0])
    assert not torch.equal(whole, tensor)  # (the default is the other form here)
    assert torch.equal(gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, start.clone()), tensor)


@pytest.mark.parametrize("dtype,T", [(F32, 40), (BF16, 200)])
def test_heads_of_a_layer_whose_neighbours_share_a_group(dtype, T):
    """Heads reordered as gdn.h says give that layer's results: its head i reads group i / r."""
    gen = torch.Generator().manual_seed(63)
    H, G, P, N = 6, 2, 64, 64
    r = H // G
    x, a, B, C, A_log, dt_bias = layer(gen, T, H, G, P, N, dtype)
    D, z, states = rnd(gen, H), rnd(gen, T, H, P, dtype=dtype), rnd(gen, 1, H, N, P, scale=0.3)
    order = torch.tensor([(h % G) * r + h // G for h in range(H)]).cuda()
    st = states[:, order].contiguous()
    got = gdn.gdn_ssm_scan(x[:, order], a[:, order], B, C, A_log[order], dt_bias[order], st, D=D[order], z=z[:, order])
    torch.cuda.synchronize()
    for i in range(H):  # the layer's own order: a head and its group, alone
        g, h = i // r, int((order == i).nonzero())
        one = [v[:, i:i + 1] for v in (x, a)] + [v[:, g:g + 1] for v in (B, C)] + [A_log[i:i + 1], dt_bias[i:i + 1]]
        y, s, mag, smag = ref.scan(*one, states[:, i:i + 1], D[i:i + 1], z[:, i:i + 1], None, None, None,
                                   torch.zeros(T, 1, P))
        check(got[:, h:h + 1], y, mag, scan_bound(dtype, P, N, T), f"y {i}")
        check(st[:, h:h + 1], s, smag, scan_bound(F32, P, N, T), f"states {i}")
