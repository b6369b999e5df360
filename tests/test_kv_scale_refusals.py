"""Scales whose product with log2 e, which the kernels' exponentials are in, leaves FP32."""
import pytest
import torch

from linear_attention_recurrence_gb300 import gdn
from test_kv_abi import ATTEND, lib  # noqa: F401


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38, -3e38, float("inf"), float("nan")])
def test_refused(lib, scale):  # noqa: F811
    assert lib.gdn_kv_attention(*{**ATTEND, "scale": scale}.values()) == gdn.GDN_ERR_INVALID_ARG
    assert b"scale" in lib.gdn_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="would run on pointers that are none")
@pytest.mark.parametrize("scale", [2.3e38, -2.3e38, 0.0, 1e-45])
def test_taken(lib, scale):  # noqa: F811
    assert lib.gdn_kv_attention(*{**ATTEND, "scale": scale}.values()) == gdn.GDN_ERR_CUDA
