"""A step of drafted tokens in which a sequence finds no pages: it is as it was, and may try again."""
import numpy as np
import pytest
import torch

from examples import serve_drafts as SD
from gpu_util import DEV, sync

pytestmark = pytest.mark.gpu


def take(model, seqs, sizes, seed):
    """A step over trees of these sizes, the same for the same seed."""
    rng, gen = np.random.default_rng(seed), torch.Generator(device=DEV)
    gen.manual_seed(seed)
    tokens, tree, q = SD.draft(model, rng.integers(0, 500, size=len(sizes)), sizes, rng, gen)
    u, u_next = torch.rand(tokens.numel(), generator=gen, device=DEV), torch.rand(len(sizes), generator=gen, device=DEV)
    out = SD.step(model, seqs, tokens, torch.tensor(sizes, dtype=torch.int32, device=DEV), tree, 20, u, u_next, q)
    sync(model.lib)
    return out


def held(seqs, s):
    """What a sequence holds: states, length, pages, and its keys and values."""
    n = int(seqs.lens[s])
    k, v = (torch.empty(n, seqs.cache.struct.n_kv_heads, seqs.cache.struct.head_dim, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    seqs.cache.read(seqs.cache.slots(seqs.pages.block_table[s], 0, n), k, v)
    return seqs.state[s].clone(), seqs.conv[s].clone(), n, int(seqs.pages.n_blocks[s]), k, v


def same(a, b):
    return all(torch.equal(x, y) if isinstance(x, torch.Tensor) else x == y for x, y in zip(a, b))


@pytest.mark.parametrize("first", [4, 0])
def test_a_sequence_without_pages_is_left_out(first):
    """Three sequences and three pages of 16 tokens; the second, which holds some tokens or none, asks for 20 more."""
    model = SD.Model()
    seqs, ample = SD.Sequences(model, 3, 64, n_pages=3), SD.Sequences(model, 3, 64)
    sizes = [4, first, 4]
    for x in (seqs, ample):
        take(model, x, sizes, 1)
    assert same(held(seqs, 1), held(ample, 1))
    seqs.pages.trim(seqs.lens)
    before = held(seqs, 1)
    _, count, _, _ = take(model, seqs, [5, 20, 5], 2)
    assert count[1] == 0 and count[0] >= 1 and count[2] >= 1
    assert same(before, held(seqs, 1))
    # the third one ends, and the second tries again, as it would with pages enough
    seqs.lens[2] = 0
    seqs.state[2], seqs.conv[2] = 0, 0
    got, want = (take(model, x, [0, 20, 0], 3) for x in (seqs, ample))
    assert want[1][1] >= 1 and all(torch.equal(x, y) for x, y in zip(got, want))
    assert same(held(seqs, 1), held(ample, 1))
