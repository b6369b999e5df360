"""What the binding of the selective state space operators and the block norm refuses, by the
argument's name, before anything is launched."""
import pytest
import torch

from linear_attention_recurrence_gb300 import gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_recurrence_gb300 import build

    build.build()


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).cuda()


CONV = dict(x=(4, 8), w=(8, 4), hist=(1, 3, 8))
SCAN = dict(x=(4, 2, 32), a=(4, 2), B=(4, 1, 16), C=(4, 1, 16), A_log=(2,), dt_bias=(2,), states=(1, 2, 16, 32))
STEP = dict(xbc=(3, 96), a=(3, 2), conv_w=(96, 4), A_log=(2,), dt_bias=(2,), hist=(3, 3, 96), states=(3, 2, 16, 32))
NORM = dict(b=(4, 8), residual=(4, 8), w_pre=(8,))
CALLS = {"conv": (gdn.gdn_ssm_conv, CONV), "scan": (gdn.gdn_ssm_scan, SCAN), "step": (gdn.gdn_ssm_step, STEP),
         "norm": (gdn.gdn_block_norm, NORM)}


@pytest.mark.parametrize("call,name,value,error", [
    ("conv", "x", None, TypeError), ("conv", "w", None, TypeError), ("conv", "w", (8,), ValueError),
    ("conv", "hist", (3, 8), ValueError), ("conv", "hist", "list", TypeError), ("conv", "cu_seqlens", "list", TypeError),
    ("conv", "cu_seqlens", (), ValueError), ("conv", "has_state", "list", TypeError), ("conv", "slots", "list", TypeError),
    ("conv", "out", (4, 9), ValueError),
    ("scan", "B", None, TypeError), ("scan", "B", (4, 16), ValueError), ("scan", "C", None, TypeError),
    ("scan", "states", (2, 16, 32), ValueError), ("scan", "states", "list", TypeError), ("scan", "z", (4, 2, 31), ValueError),
    ("scan", "has_state", (), ValueError), ("scan", "cu_seqlens", "list", TypeError), ("scan", "a", (4, 3), ValueError),
    ("step", "states", None, TypeError), ("step", "hist", None, TypeError), ("step", "conv_w", None, TypeError),
    ("step", "hist", (3, 96), ValueError), ("step", "xbc", (3, 97), ValueError), ("step", "slots", "list", TypeError),
    ("norm", "residual", None, TypeError), ("norm", "w_pre", None, TypeError), ("norm", "gate", "list", TypeError),
    ("norm", "gate", (8,), ValueError), ("norm", "gate", (2, 8), ValueError), ("norm", "residual_out", (4, 7), ValueError),
])
def test_refused_by_name(call, name, value, error):
    fn, shapes = CALLS[call]
    args = {k: t(*v) for k, v in shapes.items()}
    fn(**args)  # (as it is, the call goes through)
    args[name] = value if value is None else [0, 4] if value == "list" else t(*value)
    before = gdn.gdn_launch_count()
    with pytest.raises(error, match=name):
        fn(**args)
    assert gdn.gdn_launch_count() == before
    torch.cuda.synchronize()
