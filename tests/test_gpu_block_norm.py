"""gdn_block_norm against its definition in 64 bits.

Tolerances: a value rounded to type t is off by eps_t / 2 of itself.  The residual's sum
has two FP32 terms (one rounding each of the product, the sum, the norm's factor, its
sum of squares (dim / 256 serial additions, then 13) and the gate's fast exponential):
(dim / 256 + 32) 2^-24 of the terms' magnitudes.  y is that sum (whose error counts
relative to itself, so by magnitude / |sum|) times a factor with the same count."""
import pytest
import torch

import ssm_reference as ref
from linear_attention_recurrence_gb300 import gdn

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_recurrence_gb300 import build

    build.build()


CASES = [
    # T, dim, dtype, stream, post, gate, sigmoid, column offset, in place
    (1, 6144, BF16, BF16, True, "row", True, 0, True),
    (5, 1, F32, F32, True, "token", False, 0, False),
    (3, 37, F16, F32, True, "token", True, 1, True),
    (7, 130, BF16, F32, False, "none", False, 0, False),
    (4, 2052, F16, F16, True, "row", False, 4, True),
    (300, 1024, BF16, F32, True, "token", True, 0, True),
    (2, 16384, F32, F32, True, "token", True, 0, False),
    (2, 16383, BF16, F32, True, "row", True, 0, False),
    (3, 9999, F32, F32, False, "token", True, 0, True),
    (3, 8190, F16, F16, True, "none", False, 0, True),
    # rows through shared memory: one row, and several in turn of every CTA
    (1, 1024, F32, F32, True, "token", True, 0, False),
    (700, 2056, BF16, F32, True, "token", True, 8, True),
    (950, 1536, F32, F32, True, "row", False, 0, False),
    (640, 6144, F16, F16, False, "token", True, 0, True),
    (7, 6136, BF16, BF16, False, "none", False, 0, False),
    (200, 8192, BF16, F32, True, "token", True, 0, True),
]


def check(got, want, mag, c):
    fi = torch.finfo(got.dtype)
    g = got.cpu().double()
    tol = fi.eps / 2 * (1 + 1e-3) * want.abs() + c * mag + fi.smallest_normal * fi.eps
    over = (g - want).abs() - tol
    assert bool((over <= 0).all()), float(over.max())


@pytest.mark.parametrize("T,dim,dtype,stream,post,gate,sig,off,inplace", CASES)
def test_block_norm(T, dim, dtype, stream, post, gate, sig, off, inplace):
    gen = torch.Generator().manual_seed(T + dim)

    def rnd(*shape, dtype=F32):
        return torch.randn(shape, generator=gen).to(dtype).cuda()

    b = rnd(T, dim + off, dtype=dtype)[:, off:]
    r = (2 * rnd(T, dim + off)).to(stream)[:, off:]
    w_pre, w_post = 1 + 0.1 * rnd(dim), 1 + 0.1 * rnd(dim) if post else None
    g = {"none": None, "row": rnd(1, dim, dtype=dtype), "token": rnd(T, dim, dtype=dtype)}[gate]
    want_r, want_y, mag = ref.block_norm(b, r, w_pre, w_post, g, sig, 0.7, 1e-6)
    keep = r.clone()
    out_r, y = gdn.gdn_block_norm(b, r, w_pre, w_post=w_post, gate=g, gate_sigmoid=sig, scale=0.7, eps=1e-6,
                                  residual_out=None if inplace else torch.empty_like(r))
    torch.cuda.synchronize()
    assert out_r is r if inplace else torch.equal(r, keep)
    c = (dim / 256 + 32) * 2.0 ** -24
    check(out_r, want_r, mag, c)
    factor = w_pre.cpu().double().abs() / torch.sqrt(want_r.square().mean(-1, keepdim=True) + 1e-6)
    check(y, want_y, mag * factor, 2 * c)


def test_zero_rows_and_empty_calls():
    w = torch.ones(64).cuda()
    r, y = gdn.gdn_block_norm(torch.zeros(3, 64).cuda(), torch.zeros(3, 64).cuda(), w, w_post=w)
    assert not r.any() and not y.any()
    r, y = gdn.gdn_block_norm(torch.zeros(0, 64).cuda(), torch.zeros(0, 64).cuda(), w)
    assert y.shape == (0, 64)


def test_agrees_with_out_norm_convention():
    """With no gate and a zero stream, out is the RMSNorm of the block twice over: of weight 1, its own fixed point."""
    gen = torch.Generator().manual_seed(1)
    b, w = torch.randn(9, 512, generator=gen).cuda(), torch.ones(512).cuda()
    r, y = gdn.gdn_block_norm(b, torch.zeros_like(b), w, w_post=w, eps=0.0)
    assert float((r - y).abs().max()) <= 64 * 2.0 ** -24 * float(r.abs().max())
