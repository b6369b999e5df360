"""Sequence bounds and slots that are not sound: what a call may still touch.

Bounds live on the device, so a call cannot refuse them; whatever they hold, the kernels
read and write within the arrays that they were given."""
import pytest
import torch

from linear_attention_recurrence_gb300 import gdn

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from linear_attention_recurrence_gb300 import build

    build.build()


@pytest.mark.parametrize("ch", [64, 37])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("bounds", [(0, 2, 1, 40), (1, 1, 1, 0, 40), (5, 0, 1, 0, 40), (0, 17, 16, 40)])
def test_conv_reads_no_row_before_its_array(bounds, width, ch):
    """A sequence that begins below the end of an earlier one is taken up behind its own first
    row.  The window is then not its own, but it is made of the array's rows: the 8 rows of
    NaN before the array (and behind it) reach no output."""
    gen = torch.Generator().manual_seed(41)
    T = 40
    wide = torch.full((T + 16, ch), float("nan"))
    wide[8:8 + T] = torch.randn(T, ch, generator=gen)
    x = wide.cuda()[8:8 + T]
    w = torch.rand(ch, width, generator=gen).cuda() + 0.1
    cu = torch.tensor(bounds, dtype=torch.int32).cuda()
    out = torch.zeros(T, ch).cuda()
    gdn.gdn_ssm_conv(x, w, cu_seqlens=cu, out=out)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out).all())
