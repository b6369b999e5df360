"""Refusals of the paged cache's operators that need tensors on a GPU."""
import pytest
import torch

from linear_attention_recurrence_gb300 import gdn

pytestmark = pytest.mark.gpu


def good():
    dev = "cuda"
    return dict(q=torch.zeros(2, 4, 64, device=dev).half(), k=torch.zeros(2, 2, 64, device=dev).half(),
                cache=gdn.gdn_kv_cache(2, 2, 16, 64), table=torch.zeros(1, 2, device=dev, dtype=torch.int32),
                lens=torch.full((1,), 2, device=dev, dtype=torch.int32))


@pytest.mark.parametrize("change,match", [
    (lambda a: a.update(q=a["q"].float()), "16-bit"), (lambda a: a.update(q=a["q"][..., :32].contiguous()), "head_dim"),
    (lambda a: a.update(cache=a["cache"][..., :-1]), "hold tokens"), (lambda a: a.update(cache=a["cache"].int()), "cache must be"),
    (lambda a: a.update(table=a["table"].long()), "block_table must be"), (lambda a: a.update(table=a["table"][0]), "2 dimensions"),
    (lambda a: a.update(lens=a["lens"].cpu()), "kv_lens must be on"), (lambda a: a.update(lens=a["lens"].expand(3)), "shape|contiguous|need"),
    (lambda a: a.update(q=a["q"].transpose(0, 1)), "contiguous"), (lambda a: a.update(q=a["q"][:, :3].contiguous()), "multiple"),
])
def test_attention(change, match):
    a = good()
    change(a)
    with pytest.raises((ValueError, TypeError, gdn.GDNError), match=match):
        gdn.gdn_kv_attention(a["q"], a["cache"], a["table"], a["lens"])


@pytest.mark.parametrize("kw,match", [
    (dict(inv_freq=torch.ones(8)), "inv_freq must be on"), (dict(positions=torch.zeros(2)), "positions"),
    (dict(k_scale=torch.ones(3)), "k_scale"), (dict(q_out=torch.zeros(2, 4, 64)), "q_out without q"),
])
def test_append(kw, match):
    a = good()
    with pytest.raises((ValueError, TypeError, gdn.GDNError), match=match):
        gdn.gdn_kv_append(a["k"], a["k"], a["cache"], a["table"], a["lens"], **kw)
    with pytest.raises(gdn.GDNError, match="multiple of 32"):
        gdn.gdn_kv_append(a["k"], a["k"], a["cache"], a["table"], a["lens"], inv_freq=torch.ones(8, device="cuda"))
    with pytest.raises(gdn.GDNError, match="overlaps"):
        gdn.gdn_kv_append(a["k"], a["k"], a["cache"], a["table"], a["lens"], k_out=a["k"])
