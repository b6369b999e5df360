"""The scan where strong and weak decays meet inside a chunk, against the definition in 64 bits.

Every head has one token of x that is not 0, there a power of two, and C . B = 1: an output of
the tensor form is one score times a power of two, so y's own rounding leaves it as it is, and
its error is the score's rounding, eps / 2, and the decay's own.  (For FP16 the score's smallest
step besides, 2^-25 of a power of two below 2 max dt.)  The exponent is a sum of at most 36
terms (31 groups of 4 tokens, those inside a group, the difference), each rounding 2^-24 of a sum
up to the exponent or, inside a group, to 3 * 256: (36 * 126 * 2^-24 + 2^-15) ln 2 < 2^-12 as
long as the decay is above FP32's smallest normal 2^-126.  The token form's bound is that of
test_gpu_ssm.py."""
import math

import pytest
import torch

import ssm_reference as ref
from linear_attention_recurrence_gb300 import gdn
from test_gpu_ssm import BF16, F16, F32, U32, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_recurrence_gb300 import build

    build.build()


def strong_tokens(pattern, T):
    t = torch.arange(T)
    if pattern == "first half":
        return t % 128 < 64
    if pattern == "first quarter":
        return t % 128 < 32
    if pattern == "all but two of 8":
        return t % 8 < 6
    if pattern == "second of 4":
        return t % 4 == 1
    return torch.rand(T, generator=torch.Generator().manual_seed(7)) < 0.5


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("strong", [5.0, 10.0, 30.0])
@pytest.mark.parametrize("pattern", ["first half", "first quarter", "all but two of 8", "second of 4", "half of them"])
def test_weak_decays_between_strong_ones(pattern, strong, dtype):
    T, H, P, N = 128, 12, 64, 64
    of = strong_tokens(pattern, T)
    a = torch.where(of, strong, -4.0)[:, None].expand(T, H).to(dtype).cuda()
    x = torch.zeros(T, H, P)
    for h in range(H):
        x[5 + 11 * h if h < 11 else 66, h] = 2.0 ** (torch.arange(P) % 4)
    x = x.to(dtype).cuda()
    B, C = torch.ones(T, 1, N, dtype=dtype).cuda(), torch.full((T, 1, N), 1 / N, dtype=dtype).cuda()
    A_log, dt_bias = torch.full((H,), math.log(16.0)).cuda(), torch.zeros(H).cuda()
    out = torch.zeros(T, H, P, dtype=dtype).cuda()
    y, _, mag, _ = ref.scan(x, a, B, C, A_log, dt_bias, None, None, None, None, None, None, out)
    gdn.gdn_ssm_scan(x, a, B, C, A_log, dt_bias, out=out)
    torch.cuda.synchronize()
    # (check allows eps / 2 of the output: y's rounding here, or the score's)
    c = (4 * T + 2 * N + 32) * U32 + 2.0 ** -21 if dtype == F32 else 2.0 ** -12 + (2 * N + 32) * U32
    more = 2.0 ** -24 * strong * float(x.max()) if dtype == F16 else 2.0 ** -126 * 64
    check(out, y, mag, c, "y", more)
