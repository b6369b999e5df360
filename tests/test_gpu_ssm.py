"""The selective state space operators (convolution, scan, step) against their
definitions in 64 bits.

Tolerances.  A value rounded to type t is off by eps_t / 2 of itself.  Sums in FP32 of
terms with magnitudes m_i are off by at most (roundings per term) * 2^-24 * sum m_i:
the reference returns sum m_i beside each result.  Per term and token the scan rounds
the decay, the product, the update and the output product, and its gates carry a few
ulp of exp and log1p (2^-21 covers them, and the fast exponential of silu): the token
form's bound is (4 tokens + 2 state_dim + 32) 2^-24 of the magnitude.  The tensor form
of 16-bit types also rounds the decayed score and the state once each to that type
(disjoint terms: one eps_t / 2 of the magnitude).
"""
import pytest
import torch

import ssm_reference as ref
from linear_attention_recurrence_gb300 import gdn

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U32 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_recurrence_gb300 import build

    build.build()


def rnd(gen, *shape, scale=1.0, dtype=F32):
    return (scale * torch.randn(shape, generator=gen)).to(dtype).cuda()


def uni(gen, lo, hi, *shape):
    return (torch.rand(shape, generator=gen) * (hi - lo) + lo).cuda()


def check(got, want, mag, c, what="", more=0.0):
    """|got - want| <= eps/2 |want| + c mag + the type's smallest step (+ more)."""
    fi = torch.finfo(got.dtype)
    g = got.detach().cpu().double()
    assert torch.isfinite(g).all(), what
    tol = fi.eps / 2 * (1 + 1e-3) * want.abs() + c * mag + fi.smallest_normal * fi.eps + more
    over = (g - want).abs() - tol
    assert bool((over <= 0).all()), (what, float(over.max()), float((g - want).abs().max()), float(mag.max()))


def packed(lens, lead=0):
    cu = [lead]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32).cuda(), cu[-1]


# ---------------------------------------------------------------- convolution

CONV = [
    # lens, channels, width, dtype, bias, column offset, row padding
    ((1,), 8, 4, BF16, True, 0, 0),
    ((0, 3, 0, 1, 2, 0), 37, 4, F32, False, 0, 0),
    ((16, 17, 15, 1, 33), 72, 3, BF16, True, 8, 16),
    ((5, 200, 31), 513, 4, F16, True, 1, 3),
    ((2, 1, 13, 1, 1, 14, 2, 2, 60), 256, 4, F32, True, 0, 4),
    ((64, 1, 1), 128, 2, F16, False, 0, 0),
    (tuple(1 + i % 5 for i in range(70)), 40, 4, BF16, True, 0, 0),
    ((1100,), 2056, 4, BF16, True, 0, 0),
]


@pytest.mark.parametrize("lens,ch,width,dtype,bias,off,padc", CONV)
def test_conv(lens, ch, width, dtype, bias, off, padc):
    gen = torch.Generator().manual_seed(len(lens) * 100 + ch)
    n = len(lens)
    cu, end = packed(lens, lead=2)
    T = end + 3
    wide = rnd(gen, T, ch + off + padc, dtype=dtype)
    wide[:2] = float("nan")  # rows of no sequence
    wide[end:] = float("nan")
    x = wide[:, off:off + ch]
    w, b = uni(gen, -0.5, 0.5, ch, width), rnd(gen, ch, scale=0.1) if bias else None
    hist = rnd(gen, n + 2, width - 1, ch, dtype=dtype)
    slots = torch.randperm(n + 2, generator=gen)[:n].to(torch.int32)
    if n > 2:
        slots[n // 2] = -1
    has = torch.tensor([i % 3 != 1 for i in range(n)])
    out = rnd(gen, T, ch, dtype=dtype)
    y, h, mag = ref.conv(x, w, b, hist, cu, slots, has, out)
    got = gdn.gdn_ssm_conv(x, w, bias=b, hist=hist, cu_seqlens=cu, slots=slots.cuda(), has_state=has.cuda(), out=out)
    torch.cuda.synchronize()
    assert got is out
    # width + 1 sums, then silu (its slope is at most 1.1) with a few ulp
    check(out, y, mag, (width + 1) * 1.1 * U32 + 2.0 ** -21)
    assert torch.equal(hist.cpu().double(), h)


def test_conv_one_sequence_without_history_or_activation():
    gen = torch.Generator().manual_seed(5)
    x, w = rnd(gen, 50, 64), uni(gen, -1, 1, 64, 4)
    y, _, mag = ref.conv(x, w, None, None, None, None, None, torch.zeros(50, 64), activation=0)
    check(gdn.gdn_ssm_conv(x, w, activation=0), y, mag, 5 * U32)
    assert gdn.gdn_ssm_conv(x[:0], w).shape == (0, 64)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_conv_split_calls_give_the_same_bits(dtype):
    gen = torch.Generator().manual_seed(6)
    T, ch = 77, 96
    x, w = rnd(gen, T, ch, dtype=dtype), uni(gen, -0.5, 0.5, ch, 4)
    h1 = rnd(gen, 1, 3, ch, dtype=dtype)
    h2 = h1.clone()
    whole = gdn.gdn_ssm_conv(x, w, hist=h1)
    parts, at = [], 0
    for n in (1, 1, 30, 2, 43):
        parts.append(gdn.gdn_ssm_conv(x[at:at + n], w, hist=h2))
        at += n
    assert at == T and torch.equal(whole, torch.cat(parts)) and torch.equal(h1, h2)


# ---------------------------------------------------------------- scan


def layer(gen, T, H, G, P, N, dtype, wide=0, strong=False):
    """The inputs of a scan, x, B and C as columns of one row (`wide` extra columns before them)."""
    row = rnd(gen, T, wide + H * P + 2 * G * N, dtype=dtype)
    x = row[:, wide:wide + H * P].unflatten(1, (H, P))
    B = row[:, wide + H * P:wide + H * P + G * N].unflatten(1, (G, N))
    C = row[:, wide + H * P + G * N:].unflatten(1, (G, N))
    A_log = torch.log(uni(gen, 1.0, 16.0, H))
    dt_bias = torch.log(torch.expm1(torch.exp(uni(gen, -6.9, 2.0 if strong else -2.3, H))))
    return x, rnd(gen, T, H, dtype=dtype), B, C, A_log, dt_bias


def tensor_form(dtype, P, N):
    return dtype != F32


def scan_bound(dtype, P, N, tokens):
    c = (4 * tokens + 2 * N + 32) * U32 + 2.0 ** -21
    return c + (torch.finfo(dtype).eps / 2 if tensor_form(dtype, P, N) else 0)


def fp16_steps(x, a, B, A_log, dt_bias, states, cu, slots):
    """What FP16's smallest step, 2^-24, costs the states (the tensor form).  A chunk of 128
    tokens brings sum_t (w_t x_t) B_t^T, w_t the token's step times the decay behind it; the
    products enter divided by a power of two 2^k <= 2 max w, in two parts, the second of
    which rounds to that step: at most 2^-25 2^k <= 2^-24 max w off (and never more than
    w_t |x_t|), times |B_t|; later chunks decay it."""
    x, a, B, A_log, dt_bias = (t.cpu().double() for t in (x, a, B, A_log, dt_bias))
    H = x.shape[1]
    of = torch.arange(H) % B.shape[1]
    out = torch.zeros(states.shape, dtype=torch.float64)
    cu = [int(v) for v in cu]
    for i, slot in enumerate(slots.tolist()):
        if slot < 0:
            continue
        for b in range(cu[i], cu[i + 1], 128):
            r = slice(b, min(b + 128, cu[i + 1]))
            dt = torch.logaddexp(a[r] + dt_bias, torch.zeros((), dtype=torch.float64))
            g = -torch.exp(A_log) * dt
            w = dt * torch.exp(g.flip(0).cumsum(0).flip(0) - g)
            off = torch.minimum(2.0 ** -24 * w.amax(0)[None, :, None].expand_as(x[r]), w[..., None] * x[r].abs())
            out[slot] = torch.exp(g.sum(0))[:, None, None] * out[slot] + torch.einsum("thp,thn->hnp", off, B[r][:, of].abs())
    return out


SCAN = [
    # lens, H, G, P, N, dtype, z, D, column offset, strong decay
    ((1,), 3, 1, 128, 128, BF16, True, True, 0, False),
    ((0, 5, 0, 16, 17, 1, 0), 6, 2, 64, 128, F32, True, True, 0, False),
    ((33, 2), 4, 4, 32, 16, F32, False, False, 1, True),
    ((127, 128, 129), 6, 2, 128, 128, BF16, True, True, 0, False),
    ((127, 128, 129), 6, 2, 128, 128, F16, True, True, 8, True),
    ((300, 1, 40), 2, 1, 64, 128, BF16, False, True, 0, False),
    ((300, 1, 40), 4, 2, 128, 64, F16, True, False, 0, False),
    ((257, 64, 65, 31), 3, 3, 64, 64, BF16, True, True, 0, True),
    ((70, 70), 2, 2, 96, 32, BF16, True, True, 0, False),
    ((200,), 2, 1, 256, 64, F16, True, True, 3, False),
    ((640,), 3, 1, 128, 128, BF16, True, True, 0, False),
    ((1500,), 3, 1, 128, 128, F16, False, True, 0, False),
    # one sequence over segments of one, two and more chunks
    ((170,), 4, 2, 128, 128, BF16, True, True, 0, False),
    ((300,), 5, 1, 64, 64, F16, True, True, 0, True),
    ((1000,), 8, 8, 64, 128, BF16, True, True, 0, False),
    ((2300,), 2, 1, 128, 64, F16, True, False, 0, False),
    ((900,), 40, 2, 64, 64, BF16, False, True, 0, True),
]


@pytest.mark.parametrize("lens,H,G,P,N,dtype,gate,skip,wide,strong", SCAN)
def test_scan(lens, H, G, P, N, dtype, gate, skip, wide, strong):
    gen = torch.Generator().manual_seed(sum(lens) + P + N)
    n = len(lens)
    cu, end = packed(lens, lead=1)
    T = end + 130  # rows behind the last sequence, as many as a tile
    x, a, B, C, A_log, dt_bias = layer(gen, T, H, G, P, N, dtype, wide, strong)
    z = rnd(gen, T, H, P, dtype=dtype) if gate else None
    D = rnd(gen, H) if skip else None
    for v in (x, a, B, C):  # what no sequence holds must not matter
        v[:1] = float("nan")
        v[end:] = float("nan")
    states = rnd(gen, n + 2, H, N, P, scale=0.3)
    slots = torch.randperm(n + 2, generator=gen)[:n].to(torch.int32)
    if n > 2:
        slots[n // 2] = -1
    has = torch.tensor([i % 3 != 1 for i in range(n)])
    out = rnd(gen, T, H, P, dtype=dtype)
    y, st, mag, smag = ref.scan(x, a, B, C, A_log, dt_bias, states, D, z, cu, slots, has, out)
    gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, states, D=D, z=z, cu_seqlens=cu, slots=slots.cuda(),
                     has_state=has.cuda(), out=out)
    torch.cuda.synchronize()
    check(out, y, mag, scan_bound(dtype, P, N, max(lens)), "y")
    more = fp16_steps(x, a, B, A_log, dt_bias, states, cu, slots) if dtype == F16 else 0.0
    check(states, st, smag, scan_bound(F32, P, N, max(lens)), "states", more)
    assert gdn.gdn_device_status() == gdn.GDN_OK


@pytest.mark.parametrize("dtype,T", [(F32, 40), (BF16, 40), (BF16, 300)])
def test_scan_without_states(dtype, T):
    gen = torch.Generator().manual_seed(9)
    x, a, B, C, A_log, dt_bias = layer(gen, T, 4, 2, 128, 128, dtype)
    y, _, mag, _ = ref.scan(x, a, B, C, A_log, dt_bias, None, None, None, None, None, None, torch.zeros(T, 4, 128))
    check(gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias), y, mag, scan_bound(dtype, 128, 128, T))
    assert gdn.gdn_ssm_scan(x[:0], a[:0], B[:0], C[:0], A_log, dt_bias).shape == (0, 4, 128)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_extreme_gates(dtype):
    """No step (dt = 0), no decay, and decays that leave nothing (2^-256 and below) or overflow exp(A_log) dt."""
    gen = torch.Generator().manual_seed(10)
    T, H, P, N = 200, 4, 128, 128
    x, a, B, C, A_log, dt_bias = layer(gen, T, H, 2, P, N, dtype)
    A_log = torch.tensor([-100.0, 3.0, 6.0, 88.0]).cuda()
    dt_bias = torch.tensor([0.0, 1.0, 2.0, 3.0]).cuda()
    a[::3] = -float("inf")
    states = rnd(gen, 1, H, N, P, scale=0.3)
    out = torch.zeros(T, H, P, dtype=dtype).cuda()
    y, st, mag, smag = ref.scan(x, a, B, C, A_log, dt_bias, states, None, None, None, None, None, out)
    gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, states, out=out)
    check(out, y, mag, scan_bound(dtype, P, N, T), "y")
    check(states, st, smag, scan_bound(F32, P, N, T), "states")


def test_scan_token_form_split_calls_give_the_same_bits():
    gen = torch.Generator().manual_seed(11)
    T, H, P, N = 75, 3, 64, 64
    x, a, B, C, A_log, dt_bias = layer(gen, T, H, 1, P, N, F32)
    s1 = rnd(gen, 1, H, N, P)
    s2 = s1.clone()
    whole = gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, s1)
    parts, at = [], 0
    for n in (1, 16, 3, 40, 15):
        r = slice(at, at + n)
        parts.append(gdn.gdn_ssm_scan(x[r], a[r], B[r], C[r], A_log, dt_bias, s2))
        at += n
    assert at == T and torch.equal(whole, torch.cat(parts)) and torch.equal(s1, s2)


@pytest.mark.parametrize("dtype,lens", [(F32, (40, 9)), (BF16, (400, 130, 7))])
def test_scan_repeats_its_bits(dtype, lens):
    gen = torch.Generator().manual_seed(12)
    cu, T = packed(lens)
    x, a, B, C, A_log, dt_bias = layer(gen, T, 6, 2, 128, 128, dtype)
    s0 = rnd(gen, len(lens), 6, 128, 128)
    got = []
    for _ in range(5):
        s = s0.clone()
        got.append((gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, s, cu_seqlens=cu), s))
    for y, s in got[1:]:
        assert torch.equal(y, got[0][0]) and torch.equal(s, got[0][1])


def test_bad_bounds_and_slots_touch_nothing():
    """cu_seqlens out of order or out of range, slots out of range: those sequences are empty or keep nothing."""
    gen = torch.Generator().manual_seed(13)
    T, H, P, N = 60, 2, 64, 64
    x, a, B, C, A_log, dt_bias = layer(gen, T, H, 1, P, N, F32)
    cu = torch.tensor([0, 10, 5, 70, 60, 60], dtype=torch.int32).cuda()  # only [0, 10) is sound
    slots = torch.tensor([7, 0, 1, 2, 3], dtype=torch.int32).cuda()  # and its slot is none of the 5
    states, out = rnd(gen, 5, H, N, P), torch.full((T, H, P), 3.0).cuda()
    before = states.clone()
    gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, states, cu_seqlens=cu, slots=slots, out=out)
    torch.cuda.synchronize()
    y, _, mag, _ = ref.scan(x[:10], a[:10], B[:10], C[:10], A_log, dt_bias, None, None, None, None, None, None,
                            torch.zeros(10, H, P))
    check(out[:10], y, mag, scan_bound(F32, P, N, 10))
    assert torch.equal(states, before) and bool((out[10:] == 3.0).all())


# ---------------------------------------------------------------- step

STEP = [
    # batch, H, G, P, N, width, dtype, z, D, conv bias
    (1, 48, 16, 128, 128, 4, BF16, True, True, True),
    (5, 6, 2, 64, 64, 3, F32, True, True, False),
    (70, 4, 4, 32, 16, 2, F16, False, False, True),
    (9, 20, 1, 128, 128, 4, BF16, True, True, True),
    (130, 6, 2, 128, 128, 4, F32, True, False, True),
    (3, 2, 1, 256, 32, 4, F16, True, True, True),
    # a group of 32 and of 64 tiles; many requests with groups of 1 to 4 tiles
    (3, 16, 1, 64, 128, 4, BF16, True, True, True),
    (2, 32, 1, 64, 64, 4, F32, True, True, False),
    (460, 4, 4, 32, 32, 4, BF16, True, True, True),
    (250, 8, 8, 64, 64, 2, F16, True, True, True),
    (110, 18, 6, 32, 128, 4, F32, False, True, True),
    (130, 16, 8, 64, 16, 3, BF16, True, False, True),
]


@pytest.mark.parametrize("n,H,G,P,N,width,dtype,gate,skip,bias", STEP)
def test_step(n, H, G, P, N, width, dtype, gate, skip, bias):
    gen = torch.Generator().manual_seed(n + H)
    cw = H * P + 2 * G * N
    A_log = torch.log(uni(gen, 1.0, 16.0, H))
    dt_bias = rnd(gen, H)
    w, cb = uni(gen, -0.5, 0.5, cw, width), rnd(gen, cw, scale=0.1) if bias else None
    D = rnd(gen, H) if skip else None
    hist, states = rnd(gen, n + 2, width - 1, cw, dtype=dtype), rnd(gen, n + 2, H, N, P, scale=0.3)
    slots = torch.randperm(n + 2, generator=gen)[:n].to(torch.int32)
    if n > 2:
        slots[1] = -1
        slots[2] = n + 2
    for _ in range(2):
        xbc, a = rnd(gen, n, cw + 5, dtype=dtype)[:, 5:], rnd(gen, n, H, dtype=dtype)
        z = rnd(gen, n, H, P, dtype=dtype) if gate else None
        out = rnd(gen, n, H, P, dtype=dtype)
        y, h, st, mag, smag = ref.step(xbc, a, w, cb, A_log, dt_bias, hist, states, D, z, slots, out)
        gdn.gdn_ssm_step(xbc, a, w, A_log, dt_bias, hist, states, conv_bias=cb, D=D, z=z, slots=slots.cuda(), out=out)
        torch.cuda.synchronize()
        # A convolved value u = silu(s) is off by 1.1 (width + 1) 2^-24 of the sum's magnitude
        # m >= |u| and a few ulp of itself, however small it is next to m.  So a product
        # like B x is off by at most (e_B m_x + m_B e_x) = 2 (6 + 2^5) 2^-24 m_B m_x: the
        # magnitudes of y and the states are formed from those of x, B and C.
        c = (2 * N + 64 + 128) * U32 + 2.0 ** -19
        check(out, y, mag, c, "y")
        check(states, st, smag, c, "states")
        assert torch.equal(hist.cpu().double(), h)


def test_step_of_an_empty_batch():
    gen = torch.Generator().manual_seed(3)
    H, P, N, cw = 2, 64, 64, 2 * 64 + 2 * 64
    y = gdn.gdn_ssm_step(rnd(gen, 0, cw), rnd(gen, 0, H), rnd(gen, cw, 4), rnd(gen, H), rnd(gen, H), rnd(gen, 1, 3, cw),
                         rnd(gen, 1, H, N, P))
    assert y.shape == (0, H, P)


# ---------------------------------------------------------------- together


def run_layer(rows, a, z, prm, hist, states, cu=None, slots=None, has=None):
    H, G, P, N = prm["dims"]
    u = gdn.gdn_ssm_conv(rows, prm["w"], bias=prm["cb"], hist=hist, cu_seqlens=cu, slots=slots, has_state=has)
    x = u[:, :H * P].unflatten(1, (H, P))
    B = u[:, H * P:H * P + G * N].unflatten(1, (G, N))
    C = u[:, H * P + G * N:].unflatten(1, (G, N))
    return gdn.gdn_ssm_scan(x, a, B, C, prm["A_log"], prm["dt_bias"], states, D=prm["D"], z=z, cu_seqlens=cu,
                            slots=slots, has_state=has)


def params(gen, H, G, P, N):
    cw = H * P + 2 * G * N
    return {"dims": (H, G, P, N), "w": uni(gen, -0.5, 0.5, cw, 4), "cb": rnd(gen, cw, scale=0.1),
            "A_log": torch.log(uni(gen, 1.0, 16.0, H)), "dt_bias": rnd(gen, H) - 3, "D": rnd(gen, H)}


@pytest.mark.parametrize("dtype,tol", [(F32, 2.0 ** -12), (BF16, 2.0 ** -5)])
def test_layer_prompts_then_steps(dtype, tol):
    """Norms around the layer, packed prompts, then single tokens: as one longer prompt.
    FP32: the library's product of another row count may add its 768 terms in another
    order, each sum off by up to 768 * 2^-24 of its terms' magnitudes, which are
    768^0.5 / 5 = 5.5 times the largest value: 2^-12.  BF16: the prompt's convolution is
    rounded to the type, the step's is not, and the scan's forms round differently: a few
    eps of the largest value."""
    gen = torch.Generator().manual_seed(21)
    H, G, P, N = 6, 2, 128, 128
    cw, dim, lens, more = H * P + 2 * G * N, H * P, (150, 37), 3
    prm = params(gen, H, G, P, N)
    w_in = rnd(gen, dim, cw + H + H * P, scale=dim ** -0.5)
    w_pre, w_post = 1 + rnd(gen, dim, scale=0.1), 1 + rnd(gen, dim, scale=0.1)

    def block(stream, body):
        """One block: norm, projections, the layer, the norm behind it with the residual."""
        zero = torch.zeros_like(stream, dtype=dtype)
        _, u = gdn.gdn_block_norm(zero, stream, w_pre, residual_out=torch.empty_like(stream))
        p = (u.float() @ w_in).to(dtype)
        y = body(p[:, :cw], p[:, cw:cw + H], p[:, cw + H:].unflatten(1, (H, P)))
        return gdn.gdn_block_norm(y.flatten(1), stream, w_pre, w_post=w_post, scale=0.5,
                                  residual_out=torch.empty_like(stream))

    whole_lens = tuple(n + more for n in lens)
    streams = [rnd(gen, n, dim) for n in whole_lens]

    def pools():
        return torch.zeros(3, 3, cw, dtype=dtype).cuda(), torch.zeros(3, H, N, P).cuda()

    slots = torch.tensor([2, 0], dtype=torch.int32).cuda()
    hist, states = pools()
    cu, _ = packed(whole_lens)
    r_all, y_all = block(torch.cat(streams), lambda q, a, z: run_layer(q, a, z, prm, hist, states, cu, slots))
    hist2, states2 = pools()
    cu2, _ = packed(lens)
    r_p, y_p = block(torch.cat([s[:n] for s, n in zip(streams, lens)]),
                     lambda q, a, z: run_layer(q, a, z, prm, hist2, states2, cu2, slots))
    at = [0, whole_lens[0]]
    scale_y, scale_r = float(y_all.abs().max()), float(r_all.abs().max())
    off = 0
    for i, n in enumerate(lens):
        assert float((y_p[off:off + n].float() - y_all[at[i]:at[i] + n].float()).abs().max()) <= tol * scale_y
        off += n
    for t in range(more):
        r_s, y_s = block(torch.stack([s[n + t] for s, n in zip(streams, lens)]),
                         lambda q, a, z: gdn.gdn_ssm_step(q, a, prm["w"], prm["A_log"], prm["dt_bias"], hist2, states2,
                                                          conv_bias=prm["cb"], D=prm["D"], z=z, slots=slots))
        for i, n in enumerate(lens):
            row = at[i] + n + t
            assert float((y_s[i].float() - y_all[row].float()).abs().max()) <= tol * scale_y, (t, i)
            assert float((r_s[i] - r_all[row]).abs().max()) <= tol * scale_r, (t, i)
    assert float((hist - hist2).abs().max()) <= tol * float(hist.abs().max())
    assert float((states - states2).abs().max()) <= tol * float(states.abs().max())


def test_captured_and_replayed():
    """The layer captured into two graphs that share their pools, replayed on new inputs, in turn and beside eager calls."""
    gen = torch.Generator().manual_seed(22)
    H, G, P, N, T = 4, 2, 128, 128, 300
    cw = H * P + 2 * G * N
    prm = params(gen, H, G, P, N)
    rows, a, z = rnd(gen, T, cw, dtype=BF16), rnd(gen, T, H, dtype=BF16), rnd(gen, T, H, P, dtype=BF16)
    one, a1, z1 = rnd(gen, 1, cw, dtype=BF16), rnd(gen, 1, H, dtype=BF16), rnd(gen, 1, H, P, dtype=BF16)
    hist, states = torch.zeros(1, 3, cw, dtype=BF16).cuda(), torch.zeros(1, H, N, P).cuda()

    def prompt():
        return run_layer(rows, a, z, prm, hist, states)

    def token():
        return gdn.gdn_ssm_step(one, a1, prm["w"], prm["A_log"], prm["dt_bias"], hist, states, conv_bias=prm["cb"],
                                D=prm["D"], z=z1)

    prompt(), token()  # everything is loaded before the capture
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        y1 = prompt()
    with torch.cuda.graph(g2):
        y2 = token()
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        rows.copy_(rnd(g, T, cw, dtype=BF16))
        one.copy_(rnd(g, 1, cw, dtype=BF16))
        hist.zero_(), states.zero_()
        want = prompt().clone(), token().clone(), states.clone()
        hist.zero_(), states.zero_()
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(y1, want[0]) and torch.equal(y2, want[1]) and torch.equal(states, want[2])


def test_another_stream():
    """Two calls at once on two streams, each with its own slots' pool; and a stream given by argument."""
    gen = torch.Generator().manual_seed(23)
    H, G, P, N, T = 4, 2, 128, 128, 500
    sets = []
    for _ in range(2):
        x, a, B, C, A_log, dt_bias = layer(gen, T, H, G, P, N, BF16)
        sets.append((x, a, B, C, A_log, dt_bias, rnd(gen, 1, H, N, P)))
    want = []
    for s in sets:
        st = s[6].clone()
        want.append((gdn.gdn_ssm_scan(*s[:6], st), st))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        got = []
        for s, q in zip(sets, streams):
            q.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(q):
                st = s[6].clone()
            got.append((gdn.gdn_ssm_scan(*s[:6], st, stream=q), st))
        torch.cuda.synchronize()
        for (y, st), (wy, ws) in zip(got, want):
            assert torch.equal(y, wy) and torch.equal(st, ws)


@pytest.mark.parametrize("dtype,T", [(BF16, 1000), (F16, 1300)])
def test_segmented_scans_in_a_row(dtype, T):
    """Scans over segments one right behind the other, each reusing the workspace of the one before and
    going on from its state, eager and as replays of one graph: always the bits of calls far apart."""
    gen = torch.Generator().manual_seed(T)
    H, G, P, N = 8, 2, 128, 128
    sets = [layer(gen, T, H, G, P, N, dtype) for _ in range(3)]
    start = rnd(gen, 1, H, N, P)
    apart, st = [], start.clone()
    for s in sets:
        apart.append(gdn.gdn_ssm_scan(*s, st).clone())
        torch.cuda.synchronize()
    end = st.clone()

    def run(st):
        return [gdn.gdn_ssm_scan(*s, st) for s in sets]

    for _ in range(5):
        st = start.clone()
        got = run(st)
        torch.cuda.synchronize()
        assert torch.equal(st, end) and all(torch.equal(u, v) for u, v in zip(got, apart))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run(st)
    for _ in range(5):
        st.copy_(start)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(st, end) and all(torch.equal(u, v) for u, v in zip(got, apart))
    assert gdn.gdn_device_status() == gdn.GDN_OK


def test_more_sequences_than_threads():
    gen = torch.Generator().manual_seed(31)
    lens = [(20, 50, 31)[i % 3] for i in range(800)]
    cu, T = packed(lens)
    H, G, P, N = 2, 1, 64, 64
    x, a, B, C, A_log, dt_bias = layer(gen, T, H, G, P, N, BF16)
    states = rnd(gen, len(lens), H, N, P, scale=0.3)
    out = torch.empty_like(x, memory_format=torch.contiguous_format)
    y, st, mag, smag = ref.scan(x, a, B, C, A_log, dt_bias, states, None, None, cu, None, None, out)
    gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, states, cu_seqlens=cu, out=out)
    torch.cuda.synchronize()
    check(out, y, mag, scan_bound(BF16, P, N, 50), "y")
    check(states, st, smag, scan_bound(F32, P, N, 50), "states")


@pytest.mark.parametrize("dtype,T", [(F32, 60), (BF16, 700)])
def test_nan_in_a_gate_reaches_its_head_from_there_on(dtype, T):
    gen = torch.Generator().manual_seed(32)
    H, G, P, N, at = 4, 2, 128, 128, T // 2
    x, a, B, C, A_log, dt_bias = layer(gen, T, H, G, P, N, dtype)
    states = rnd(gen, 1, H, N, P)
    want_st = states.clone()
    want = gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, want_st)
    a[at, 1] = float("nan")
    y = gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, states)
    torch.cuda.synchronize()
    other = [0, 2, 3]
    assert torch.equal(y[:, other], want[:, other]) and torch.equal(states[:, other], want_st[:, other])
    assert torch.equal(y[:at, 1], want[:at, 1]) and bool(y[at:, 1].isnan().all()) and bool(states[:, 1].isnan().all())


def test_one_row_for_every_token():
    """Inputs expanded along the tokens (stride 0) give what their copies give in the same form."""
    gen = torch.Generator().manual_seed(33)
    H, G, P, N, T = 2, 1, 64, 64, 150
    x, a, B, C, A_log, dt_bias = layer(gen, T, H, G, P, N, F32)
    B1, a1 = B[:1].expand(T, G, N), a[:1].expand(T, H)
    got = gdn.gdn_ssm_scan(x, a1, B1, C, A_log, dt_bias, z=x[:1].expand(T, H, P))
    want = gdn.gdn_ssm_scan(x, a1.contiguous(), B1.contiguous(), C, A_log, dt_bias, z=x[:1].expand(T, H, P).contiguous())
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    rows = rnd(gen, 1, 40).expand(T, 40)
    w = rnd(gen, 40, 4)
    assert torch.equal(gdn.gdn_ssm_conv(rows, w), gdn.gdn_ssm_conv(rows.contiguous(), w))
