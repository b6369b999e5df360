"""Refusals of the paged cache's operators: every call below fails its host-side checks, so no
pointer in it is used."""
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


APPEND = dict(q=ptr(0), qs=512, k=ptr(1), ks=128, v=ptr(2), vs=128, freq=ptr(3), rotary=64, inter=0, pos=NIL, k_scale=NIL,
              v_scale=NIL, cache=ptr(4), n_pages=8, page=16, table=ptr(5), ts=4, width=4, lens=ptr(6), cu=ptr(7), n=2,
              qo=ptr(8), qos=512, ko=NIL, kos=0, vo=NIL, vos=0, T=6, H=4, G=1, D=128, dt=gdn.GDN_BF16, stream=NIL)
ATTEND = dict(q=ptr(0), qs=512, cache=ptr(1), n_pages=8, page=16, table=ptr(2), ts=4, width=4, lens=ptr(3), cu=ptr(4), n=2,
              k_scale=NIL, v_scale=NIL, scale=0.1, causal=1, window=0, out=ptr(5), os=512, lse=NIL, T=6, H=4, G=1, D=128,
              dt=gdn.GDN_BF16, ws=ptr(6), wsb=1 << 23, stream=NIL)

INV, UNS = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED
BOTH = [
    (dict(T=-1), INV), (dict(n=-1), INV), (dict(cu=NIL, T=7), INV), (dict(H=0), INV), (dict(G=0), INV),
    (dict(H=5, G=2), INV), (dict(D=96), UNS), (dict(D=256), UNS), (dict(page=8), UNS), (dict(page=48), UNS),
    (dict(page=512), UNS), (dict(page=0), UNS), (dict(page=-16), UNS), (dict(n_pages=-1), INV), (dict(width=-1), INV),
    (dict(ts=3), INV), (dict(lens=NIL), INV), (dict(table=NIL), INV), (dict(cache=NIL), INV), (dict(dt=7), INV),
    (dict(T=1 << 31), UNS), (dict(H=70000, qs=70000 * 128), UNS), (dict(q=P((1 << 30) + 1)), INV), (dict(qs=-1), INV),
    (dict(cache=P((1 << 30) + (9 << 24) + 8)), INV), (dict(table=P((1 << 30) + (9 << 24) + 2)), INV),
]


@pytest.mark.parametrize("change,status", BOTH + [
    (dict(rotary=-32), INV), (dict(rotary=160), INV), (dict(rotary=16), UNS), (dict(inter=2), INV), (dict(freq=NIL), INV),
    (dict(q=NIL), INV), (dict(qo=NIL), INV), (dict(k=NIL), INV), (dict(v=NIL), INV), (dict(qos=511), INV),
    (dict(ko=ptr(9), kos=127), INV), (dict(qo=ptr(1)), INV), (dict(ko=ptr(2), kos=128), INV), (dict(cache=ptr(8)), INV),
    (dict(vo=ptr(4), vos=128), INV), (dict(qo=ptr(0), qos=1024), INV),
])
def test_append_refusals(lib, change, status):
    assert lib.gdn_kv_append(*{**APPEND, **change}.values()) == status
    assert lib.gdn_last_error()


@pytest.mark.parametrize("change,status", BOTH + [
    (dict(dt=gdn.GDN_F32), UNS), (dict(causal=2), INV), (dict(window=-1), INV), (dict(causal=0, window=5), INV),
    (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(q=NIL), INV), (dict(out=NIL), INV),
    (dict(os=511), INV), (dict(out=ptr(0)), INV), (dict(out=ptr(1)), INV), (dict(lse=ptr(5)), INV),
    (dict(lse=P((1 << 30) + (9 << 24) + 2)), INV), (dict(ws=P((1 << 30) + (9 << 24) + 8)), INV),
])
def test_attention_refusals(lib, change, status):
    assert lib.gdn_kv_attention(*{**ATTEND, **change}.values()) == status
    assert lib.gdn_last_error()


@pytest.mark.parametrize("change", [dict(T=0), dict(n=0, T=0, cu=NIL)])
def test_nothing_to_do(lib, change):
    assert lib.gdn_kv_append(*{**APPEND, **change}.values()) == gdn.GDN_OK
    assert lib.gdn_kv_attention(*{**ATTEND, **change}.values()) == gdn.GDN_OK


def test_the_binding_names_what_is_wrong():
    k = torch.zeros(2, 1, 64)
    with pytest.raises(ValueError, match="k must be a CUDA tensor"):
        gdn.gdn_kv_append(k, k, None, None, None)
    with pytest.raises(TypeError, match="q must be a torch.Tensor"):
        gdn.gdn_kv_attention(None, None, None, None)
    assert gdn.gdn_kv_cache(3, 2, 16, 64, "cpu").shape == (3, 2, 2, 16 * 36)
