"""Refusals of the selective state space operators and the block norm: every call
below fails its host-side checks, so no pointer in it is used."""
import ctypes

import pytest
import torch

from linear_attention_recurrence_gb300 import gdn

P = ctypes.c_void_p
NIL = None


@pytest.fixture(scope="module")
def lib():
    from linear_attention_recurrence_gb300 import build

    build.build()
    return gdn.load_library()


def ptr(i):
    return P((1 << 30) + (i << 24))  # 16 MB apart


CONV = dict(x=ptr(0), xs=64, w=ptr(1), bias=NIL, hist=ptr(2), cu=ptr(3), slots=NIL, has=NIL, n=2, n_slots=2, y=ptr(4),
            ys=64, T=10, ch=64, width=4, act=1, dt=gdn.GDN_BF16, stream=NIL)
SCAN = dict(x=ptr(0), xs=256, a=ptr(1), as_=2, B=ptr(2), bs=64, C=ptr(3), cs=64, z=ptr(4), zs=256, A_log=ptr(5),
            dtb=ptr(6), D=NIL, states=ptr(7), cu=NIL, slots=NIL, has=NIL, n=1, n_slots=1, y=ptr(8), ys=256, T=5, H=2, G=1,
            P=128, N=64, dt=gdn.GDN_F32, ws=NIL, wsb=0, stream=NIL)
STEP = dict(xbc=ptr(0), xs=384, a=ptr(1), as_=2, z=NIL, zs=0, w=ptr(2), cb=NIL, A_log=ptr(3), dtb=ptr(4), D=NIL,
            hist=ptr(5), states=ptr(6), slots=NIL, n_slots=4, y=ptr(7), ys=256, batch=4, H=2, G=1, P=128, N=64, width=4,
            act=1, dt=gdn.GDN_F32, stream=NIL)
NORM = dict(b=ptr(0), bs=64, r=ptr(1), rs=64, gate=NIL, gs=0, sig=0, w_post=NIL, w_pre=ptr(2), scale=1.0, eps=1e-6,
            ro=ptr(3), ros=64, y=ptr(4), ys=64, T=4, dim=64, dt=gdn.GDN_F32, rdt=gdn.GDN_F32, stream=NIL)

INV, UNS = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INV), (dict(n=-1), INV), (dict(cu=NIL), INV), (dict(n_slots=0), INV), (dict(ch=0), INV),
    (dict(width=1), UNS), (dict(width=5), UNS), (dict(act=2), INV), (dict(dt=3), INV), (dict(x=NIL), INV),
    (dict(w=NIL), INV), (dict(y=NIL), INV), (dict(ys=63), INV), (dict(xs=-64), INV), (dict(x=P((1 << 30) + 1)), INV),
    (dict(y=ptr(0)), INV), (dict(hist=ptr(4)), INV), (dict(y=P((1 << 30) + 256)), INV), (dict(T=1 << 31), UNS),
])
def test_conv_refusals(lib, change, status):
    assert lib.gdn_ssm_conv(*{**CONV, **change}.values()) == status
    assert lib.gdn_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INV), (dict(n=2), INV), (dict(n_slots=0), INV), (dict(H=0), INV), (dict(H=3, G=2), INV),
    (dict(P=48), UNS), (dict(P=288), UNS), (dict(N=48), UNS), (dict(N=256), UNS), (dict(dt=-1), INV), (dict(a=NIL), INV),
    (dict(y=NIL), INV), (dict(A_log=NIL), INV), (dict(ys=255), INV), (dict(bs=-1), INV), (dict(y=ptr(4)), INV),
    (dict(states=ptr(8)), INV), (dict(states=P((1 << 30) + (7 << 24) + 4)), INV), (dict(cu=P(2)), INV),
    (dict(T=1 << 31), UNS), (dict(H=70000, ys=70000 * 128), UNS),
])
def test_scan_refusals(lib, change, status):
    assert lib.gdn_ssm_scan(*{**SCAN, **change}.values()) == status
    assert lib.gdn_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), INV), (dict(batch=65536, n_slots=70000), UNS), (dict(n_slots=0), INV), (dict(n_slots=3), INV),
    (dict(H=3, G=2), INV), (dict(width=5), UNS), (dict(act=-1), INV), (dict(dt=9), INV), (dict(hist=NIL), INV),
    (dict(states=NIL), INV), (dict(xbc=NIL), INV), (dict(y=ptr(0)), INV), (dict(ys=100), INV),
    (dict(hist=ptr(6)), INV), (dict(N=24), UNS),
])
def test_step_refusals(lib, change, status):
    assert lib.gdn_ssm_step(*{**STEP, **change}.values()) == status
    assert lib.gdn_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INV), (dict(dim=0), INV), (dict(dim=16385, ros=16385, ys=16385), UNS), (dict(dt=4), INV),
    (dict(dt=gdn.GDN_F32, rdt=gdn.GDN_BF16), UNS), (dict(dt=gdn.GDN_F16, rdt=gdn.GDN_BF16), UNS), (dict(sig=2), INV),
    (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(b=NIL), INV),
    (dict(w_pre=NIL), INV), (dict(y=ptr(3)), INV), (dict(y=ptr(1)), INV), (dict(ro=ptr(0)), INV), (dict(ys=63), INV),
    (dict(ro=ptr(1), ros=128), INV),
])
def test_block_norm_refusals(lib, change, status):
    assert lib.gdn_block_norm(*{**NORM, **change}.values()) == status
    assert lib.gdn_last_error()


def test_nothing_to_do(lib):
    assert lib.gdn_ssm_conv(*{**CONV, "T": 0}.values()) == gdn.GDN_OK
    assert lib.gdn_ssm_conv(*{**CONV, "n": 0}.values()) == gdn.GDN_OK
    assert lib.gdn_ssm_scan(*{**SCAN, "T": 0}.values()) == gdn.GDN_OK
    assert lib.gdn_ssm_scan(*{**SCAN, "n": 0}.values()) == gdn.GDN_OK
    assert lib.gdn_ssm_step(*{**STEP, "batch": 0}.values()) == gdn.GDN_OK
    assert lib.gdn_block_norm(*{**NORM, "T": 0}.values()) == gdn.GDN_OK
    assert lib.gdn_ssm_scan_workspace_bytes(0, 0, 48, 128, 128, gdn.GDN_BF16) == 0


def test_binding_refuses_what_is_not_on_the_gpu():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_ssm_conv(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_block_norm(x, x, torch.zeros(8))
    with pytest.raises(TypeError):
        gdn.gdn_ssm_scan(None, x, x, x, x, x)
