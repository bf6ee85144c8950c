"""States of drafted tokens at 16-byte places that are not 32-byte ones: the delta rule and the commit, in both directions.

The arithmetic does not depend on where a state lies, so the results equal, bit by bit, those of the same call on states
at a 32-byte place, which the oracle tests hold."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, f32_dev, sync
from test_gpu_drafts import Case

pytestmark = pytest.mark.gpu

SHAPES = [  # hk, hv, d, lens, kind: both kernels of the delta rule, each form of the commit, both sizes of heads
    (1, 2, 64, [9, 0, 3], "tree"), (2, 4, 128, [4], "chain"), (1, 2, 128, [64, 20], "tree"),
    (8, 64, 64, [8, 1, 5], "chain"), (16, 32, 128, [5, 2, 8, 1, 3, 0, 8, 4, 6, 7], "tree"),
]


class Place:
    """fp32 values ``off`` bytes behind a 32-byte place, between values that a stray store would change."""

    def __init__(self, a, off):
        self.n, self.off = a.size, off // 4
        self.raw = torch.full((self.n + 64,), 5.0, device=DEV)
        self.at = self.raw[16 + self.off:16 + self.off + self.n].view(a.shape)
        self.at.copy_(f32_dev(a))
        assert self.at.data_ptr() % 32 == off

    def intact(self):
        return bool((self.raw[:16 + self.off] == 5.0).all()) and bool((self.raw[16 + self.off + self.n:] == 5.0).all())


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_delta_tree(shape):
    c = Case(*shape, seed=13)
    out = []
    for off in (0, 16):
        state = Place(c.state, off)
        o, u = torch.empty(c.t, c.hv, c.d, dtype=torch.float16, device=DEV), torch.empty(c.t, c.hv, c.d, device=DEV)
        c.dl.delta_tree(c.qkv(), f32_dev(c.log_a), f32_dev(c.b), state.at, o, u, **c.more())
        sync(c.dl.lib)
        assert state.intact() and np.array_equal(state.at.cpu().numpy(), c.state)
        out.append((o, u))
    assert all(torch.equal(x, y) for x, y in zip(*out))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("offs", [(16, 0), (0, 16), (16, 16), (16, None)], ids=str)
def test_commit(shape, offs):
    """offs: of the state before and after (None: in place)."""
    c = Case(*shape, seed=14)
    rng = np.random.default_rng(1)
    u = (0.4 * rng.normal(size=(c.t, c.hv, c.d))).astype(np.float32)
    node = torch.tensor([rng.integers(-1, n) if n else -1 for n in c.lens], dtype=torch.int32, device=DEV)
    got = []
    for before, after in ((0, 0), offs):
        s_in = Place(c.state, before)
        s_out = s_in if after is None else Place(np.full_like(c.state, 7.0), after)
        c.dl.delta_commit(c.qkv(), f32_dev(c.log_a), f32_dev(u), node, s_in.at, s_out.at, **c.more())
        sync(c.dl.lib)
        assert s_in.intact() and s_out.intact()
        got.append(s_out.at.clone())
    assert torch.equal(*got)
