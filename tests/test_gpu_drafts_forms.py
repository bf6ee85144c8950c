"""The commit's form for batches against the oracle, and conv, commit and pages in the debug library, whose index checks
report any store outside its buffer."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, f32_dev, sync
from hybrid_gated_deltanet_q4k_gb300.api import KvPages
from oracle import drafts as OD
from test_gpu_drafts import Case, close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,kind", [([5, 2, 8, 1, 3, 0, 4, 6, 7, 33], "tree"), ([64, 2, 8, 1, 3, 8, 4, 6, 0, 5], "chain")])
def test_the_commit_of_a_batch(lens, kind):
    """32 heads of 128 and ten sequences, 320 heads in all: from 192 on a block takes 64 rows.  The tolerance is that of
    the commit's other tests: a step of 2^-23 of the sum of absolute values per token of the path, and four."""
    c = Case(16, 32, 128, lens, kind, seed=17, pad=1)
    rng = np.random.default_rng(4)
    u = (0.4 * rng.normal(size=(c.t, c.hv, c.d))).astype(np.float32)
    node = np.array([rng.integers(-1, n) if n else -1 for n in lens], np.int32)
    node[0] = lens[0] - 1
    state = torch.full((c.s, c.hv, c.d, c.d), 7.0, device=DEV)
    c.dl.delta_commit(c.qkv(), f32_dev(c.log_a), f32_dev(u), torch.from_numpy(node).to(DEV), f32_dev(c.state), state, **c.more())
    sync(c.dl.lib)
    for s, n in enumerate(lens):
        r = slice(c.cu[s], c.cu[s] + n)
        steps = len(OD.path(c.up[s], node[s])) + 4
        for h in range(c.hv):
            ref, e = OD.commit(c.k[r, h // 2].astype(np.float64), u[r, h].astype(np.float64), c.log_a[r, h].astype(np.float64), c.state[s, h],
                               c.up[s], node[s])
            close(state[s, h], ref, (steps if node[s] >= 0 else 0) * 2.0 ** -23 * e)


@pytest.mark.parametrize("shape", [(1, 3, 64, [3, 0, 8, 5], "tree"), (1, 2, 128, [64, 5], "chain"),
                                   (16, 32, 128, [5, 2, 8, 1, 3, 0, 4, 6, 7, 9], "tree")], ids=str)
def test_conv_and_commit_in_the_debug_library(shape):
    got = []
    for debug in (False, True):
        c = Case(*shape, seed=19, pad=2, debug=debug)
        rng = np.random.default_rng(5)
        u = (0.4 * rng.normal(size=(c.t, c.hv, c.d))).astype(np.float32)
        node = torch.tensor([rng.integers(-1, n) if n else -1 for n in c.lens], dtype=torch.int32, device=DEV)
        x, tail = torch.from_numpy(c.x).to(DEV).to(torch.bfloat16), f32_dev(c.tail)
        qkv = torch.zeros(c.t, c.spec.c_conv, dtype=torch.float16, device=DEV)
        la, b, state, after = torch.zeros(c.t, c.hv, device=DEV), torch.zeros(c.t, c.hv, device=DEV), f32_dev(c.state), torch.empty_like(tail)
        c.dl.conv_tree(x, f32_dev(c.ba), tail, qkv, la, b, **c.more())
        c.dl.delta_commit(c.qkv(), f32_dev(c.log_a), f32_dev(u), node, state, state, x, tail, after, **c.more())
        sync(c.dl.lib)
        got.append((qkv, la, b, state, after))
    assert all(torch.equal(x, y) for x, y in zip(*got))


@pytest.mark.parametrize("n,wide,most", [(5, 12, 20), (40, 60, 700), (256, 300, 30)])
def test_pages_in_the_debug_library(n, wide, most):
    """Extensions and trims, in one launch each and over all SMs."""
    got = []
    for debug in (False, True):
        rng = np.random.default_rng(n)
        ints = lambda a, t=np.int32: torch.from_numpy(np.ascontiguousarray(a, t)).to(DEV)  # noqa: E731
        d = KvPages.new(n, wide, n * wide // 2, 16, device=DEV, debug=debug)
        lens, seen = ints([0] * n), []
        for _ in range(4):
            new = rng.integers(0, most + 1, size=n)
            t = int(new.sum()) + 7
            after, cu, pos, slots = ints([0] * n), ints([0] * (n + 1)), ints([0] * t), ints([0] * t, np.int64)
            # a sequence whose row of the table is full would be reported: it gets nothing new
            new = np.where(lens.cpu().numpy() + new > 16 * wide, 0, new)
            d.extend(lens, ints(new), after, cu, pos, slots)
            sync(d.lib)
            lens = after // 2
            d.trim(lens)
            sync(d.lib)
            seen += [after, cu, pos, slots, d.n_blocks.clone(), d.n_free.clone(), d.free_pages[:int(d.n_free[0])].clone()]
        got.append(seen)
    assert all(torch.equal(x, y) for x, y in zip(*got))
