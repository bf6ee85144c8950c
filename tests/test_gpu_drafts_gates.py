"""The conv over drafted tokens of a layer whose gates are drawn elsewhere: q, k and v alone."""
import pytest
import torch

from gpu_util import DEV, Guarded, f32_dev, sync
from test_gpu_drafts import SHAPES, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_the_conv_without_gates(shape):
    """As the call that computes the gates too, which the oracle tests hold: they share nothing."""
    c = Case(*shape, seed=7, pad=3)
    x = torch.from_numpy(c.x).to(DEV).to(torch.bfloat16)
    n = c.t * c.spec.c_conv
    out = [Guarded(n * 2, 0x5B) for _ in range(2)]
    with_gates, alone = (g.view(torch.float16, (c.t, c.spec.c_conv)) for g in out)
    la, b = torch.full((c.t, c.hv), 7.0, device=DEV), torch.full((c.t, c.hv), 7.0, device=DEV)
    c.dl.conv_tree(x, f32_dev(c.ba), f32_dev(c.tail), with_gates, la, b, **c.more())
    c.dl.conv_tree(x, None, f32_dev(c.tail), alone, **c.more())
    sync(c.dl.lib)
    assert all(g.intact() for g in out)
    assert torch.equal(with_gates.view(torch.int16), alone.view(torch.int16))


def test_some_of_the_gates_are_refused():
    c = Case(1, 2, 64, [3, 4], "tree")
    x, ba, tail = torch.from_numpy(c.x).to(DEV).to(torch.bfloat16), f32_dev(c.ba), f32_dev(c.tail)
    la, b = torch.empty(c.t, 2, device=DEV), torch.empty(c.t, 2, device=DEV)
    for gates in ((ba, None, None), (None, la, b), (ba, la, None), (ba, None, b), (None, None, b)):
        with pytest.raises(ValueError):
            c.dl.conv_tree(x, gates[0], tail, c.qkv(), *gates[1:], **c.more())
    for over in (dict(qkv=c.qkv()[1:]), dict(conv_state=tail.cpu()), dict(cu=c.cu_dev[1:]), dict(tree=c.tree[1:])):
        with pytest.raises(ValueError):
            c.dl.conv_tree(**{**dict(qkvz=x, ba=None, conv_state=tail, qkv=c.qkv(), **c.more()), **over})
    sync(c.dl.lib)
