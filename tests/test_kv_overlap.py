"""Which arguments of the paged cache's operators overlap: columns of joint rows.  Calls that are
refused use no pointer; those that pass the checks are made only where there is no device to
launch on."""
import ctypes

import pytest
import torch

from linear_attention_recurrence_gb300 import gdn
from test_kv_abi import APPEND, ATTEND, NIL, lib, ptr  # noqa: F401

no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="would run on pointers that are none")
ROW = (4 + 1 + 1) * 128  # q of 4 heads, k and v of one


def col(i, elements):
    return ctypes.c_void_p(ptr(i).value + 2 * elements)


JOINT = dict(q=ptr(0), qs=ROW, k=col(0, 512), ks=ROW, v=col(0, 640), vs=ROW, qo=ptr(0), qos=ROW)


def append(lib, **change):  # noqa: F811
    return lib.gdn_kv_append(*{**APPEND, **JOINT, **change}.values())


def attend(lib, **change):  # noqa: F811
    return lib.gdn_kv_attention(*{**ATTEND, "qs": 1024, "os": 1024, "out": col(0, 512), **change}.values())


@no_device
@pytest.mark.parametrize("change", [
    dict(), dict(T=2), dict(T=1, n=1, cu=NIL), dict(qs=ROW + 7, ks=ROW + 7, vs=ROW + 7, qos=ROW + 7),
    dict(q=ptr(9), qs=512),                                                  # out of place into the joint row
    dict(q=col(0, 256), qo=col(0, 256), k=ptr(0), v=col(0, 128)),            # the keys and values first
    dict(ko=col(0, 768), kos=896, qs=896, ks=896, vs=896, qos=896),          # the kept keys behind
    dict(k=col(0, 512 + 3 * ROW), v=col(0, 640 + 3 * ROW)),                  # of later rows
])
def test_append_takes_other_columns(lib, change):  # noqa: F811
    assert append(lib, **change) == gdn.GDN_ERR_CUDA, lib.gdn_last_error()


@pytest.mark.parametrize("change", [
    dict(k=col(0, 511)), dict(k=col(0, 511 + ROW)), dict(v=col(0, 641)), dict(v=col(0, 641 + ROW)),  # (the next row's q)
    dict(k=col(0, 511), q=ptr(9), qs=512), dict(ks=ROW + 1), dict(vs=ROW - 1), dict(ko=col(0, 768), kos=ROW),
    dict(q=col(0, 1)), dict(q=col(0, ROW)),  # (in place, but not its own row)
    dict(ko=col(0, 512), kos=ROW), dict(freq=col(0, 512)), dict(cache=col(0, 512)), dict(lens=col(0, 640)),
    dict(qs=0, q=col(0, 8)), dict(ks=0, k=col(0, 8)),
])
def test_append_refuses_shared_columns(lib, change):  # noqa: F811
    assert append(lib, **change) == gdn.GDN_ERR_INVALID_ARG
    assert b"overlap" in lib.gdn_last_error() or b"in place" in lib.gdn_last_error()


@no_device
def test_attention_takes_other_columns(lib):  # noqa: F811
    assert attend(lib) == gdn.GDN_ERR_CUDA, lib.gdn_last_error()
    assert attend(lib, q=col(0, 512), out=ptr(0)) == gdn.GDN_ERR_CUDA, lib.gdn_last_error()


@pytest.mark.parametrize("change", [dict(out=col(0, 511)), dict(out=col(0, 513)), dict(os=1025), dict(out=ptr(0)),
                                    dict(lse=col(0, 600))])
def test_attention_refuses_shared_columns(lib, change):  # noqa: F811
    assert attend(lib, **change) == gdn.GDN_ERR_INVALID_ARG
    assert b"overlap" in lib.gdn_last_error()
