"""Block tables, slots and the stack of free pages against the oracle: whole numbers, equal."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, Guarded, stream, sync
from hybrid_gated_deltanet_q4k_gb300 import lib as gl
from hybrid_gated_deltanet_q4k_gb300.api import KvPages
from oracle import drafts as OD

pytestmark = pytest.mark.gpu


def ints(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype)).to(DEV)


class Book:
    """Tables on the GPU and the oracle's, in step."""

    def __init__(self, n_seqs, wide, n_pages, page, seed=0, room=0):
        self.n, self.wide, self.page = n_seqs, wide, page
        order = np.random.default_rng(seed).permutation(n_pages).astype(np.int32)
        self.bufs = [Guarded(4 * x, 0x5B) for x in (n_seqs * (wide + room), n_seqs, n_pages, 1)]
        table, held, stack, free = (b.view(torch.int32, (-1,)) for b in self.bufs)
        held.zero_()
        stack.copy_(ints(order))
        free.fill_(n_pages)
        self.table = table.view(n_seqs, wide + room)[:, :wide]
        self.dev = KvPages(page, self.table, held, stack, free)
        self.host = OD.Pages([[None] * wide for _ in range(n_seqs)], [0] * n_seqs, order.tolist(), page)

    def extend(self, lens, new, most=None, words=None, in_place=False):
        t = int(np.sum(new)) if most is None else most
        out = [Guarded(4 * self.n, 0x5B), Guarded(4 * (self.n + 1), 0x5B), Guarded(4 * t, 0x5B), Guarded(8 * t, 0x5B)]
        before = ints(lens)
        after = before if in_place else out[0].view(torch.int32, (self.n,))
        cu, pos, slots = out[1].view(torch.int32, (self.n + 1,)), out[2].view(torch.int32, (t,)), out[3].view(torch.int64, (t,))
        tree = None if words is None else ints(np.concatenate([words, np.zeros(t - len(words), np.uint64)]).view(np.int64), np.int64)
        self.dev.extend(before, ints(new), after, cu, pos, slots, tree=tree)
        sync(self.dev.lib)
        assert all(b.intact() for b in out + self.bufs)
        depth = None
        if words is not None:
            ends = np.cumsum([0] + list(new))
            depth = [[bin(int(words[ends[s] + i]) & ((1 << i) - 1)).count("1") for i in range(m)] for s, m in enumerate(new)]
        want = self.host.extend(list(map(int, lens)), list(map(int, new)), depth)
        n = want[1][-1]
        assert after.tolist() == want[0] and cu.tolist() == want[1]
        assert pos.tolist() == want[2] + [0] * (t - n) and slots.tolist() == want[3] + [-1] * (t - n)
        self.same()
        return want[0], slots

    def trim(self, keep):
        self.dev.trim(ints(keep))
        sync(self.dev.lib)
        self.host.trim(list(map(int, keep)))
        self.same()

    def same(self):
        assert all(b.intact() for b in self.bufs)
        assert self.dev.n_blocks.tolist() == self.host.held
        free = int(self.dev.n_free[0])
        assert free == len(self.host.stack) and self.dev.free_pages[:free].tolist() == self.host.stack
        table = self.table.cpu().numpy()
        for s, h in enumerate(self.host.held):
            assert table[s, :h].tolist() == self.host.table[s][:h]


@pytest.mark.parametrize("n,page,most,wide", [(1, 16, 1, 4), (3, 64, 5, 8), (17, 16, 40, 30), (256, 32, 8, 20), (256, 16, 70, 300), (40, 128, 2000, 60)])
def test_many_steps(n, page, most, wide):
    """Extensions and trims of random lengths; with most = 2000 and with 256 times 300 columns, over all SMs."""
    rng = np.random.default_rng(n)
    b = Book(n, wide, n * wide // 2 + 1, page, seed=n, room=n % 3)
    lens = np.zeros(n, np.int64)
    for step in range(8):
        new = np.minimum(rng.integers(0, most + 1, size=n), wide * page - lens)
        pad = int(rng.integers(0, 50))
        after, _ = b.extend(lens, new, most=int(new.sum()) + pad, in_place=bool(step % 2))
        got = np.array(after) - lens
        lens = lens + np.where(got > 0, rng.integers(0, got + 1), 0)       # part of it is accepted
        if step == 5:
            lens[rng.random(n) < 0.5] = 0                                  # some end
        b.trim(lens)


def test_a_trim_restores_the_stack():
    b = Book(5, 10, 60, 16)
    b.extend([0] * 5, [20, 0, 33, 16, 1])
    before = b.dev.free_pages.clone(), b.dev.n_free.clone()
    b.extend([20, 0, 33, 16, 1], [9, 40, 0, 1, 64])
    b.trim([20, 0, 33, 16, 1])
    n = int(before[1][0])
    assert torch.equal(b.dev.n_free, before[1]) and torch.equal(b.dev.free_pages[:n], before[0][:n])


@pytest.mark.parametrize("tokens", [24, 3000])
def test_positions_of_trees(tokens):
    rng = np.random.default_rng(1)
    new = np.full(max(1, tokens // 24), 24)
    words = np.zeros(new.sum(), np.uint64)
    for s in range(len(new)):
        for i in range(24):
            up = words[24 * s + rng.integers(0, i)] if i else np.uint64(0)
            words[24 * s + i] = up | (np.uint64(1) << np.uint64(i))
    Book(len(new), 8, 8 * len(new), 16).extend(rng.integers(0, 90, size=len(new)), new, words=words)


def test_too_few_pages():
    """The first that finds too few gets none, nor does a later one that asks; one that asks for none goes on."""
    b = Book(5, 8, 6, 16)
    b.extend([0, 0, 0, 0, 0], [16, 10, 0, 16, 0])
    assert b.host.held == [1, 1, 0, 1, 0]
    after, slots = b.extend([16, 10, 0, 16, 0], [40, 6, 60, 1, 16])        # 3, 0, 4 (one page is left), 1, 1
    assert after == [56, 16, 0, 16, 0] and b.host.held == [4, 1, 0, 1, 0]
    b.trim([0, 0, 0, 0, 0])


def test_every_sequence_empty_and_no_rows():
    b = Book(3, 4, 9, 16)
    b.extend([0, 5, 0], [0, 0, 0], most=0)
    b.extend([0, 5, 0], [0, 0, 0], most=7)


BAD = {  # what is out of range, on tables of 2 sequences with 4 pages of 16 each
    "lens": dict(lens=[-5, 3]), "new": dict(new=[-1, 2]), "row": dict(lens=[60, 3], new=[5, 2]), "rows": dict(most=3),
    "held": dict(held=[9, 0]), "held_negative": dict(held=[-2, 0]), "free": dict(free=99), "free_negative": dict(free=-1),
    "page": dict(stack=[77] * 8), "page_negative": dict(stack=[-3] * 8),
}


@pytest.mark.parametrize("what", BAD)
def test_out_of_range_is_reported_and_harmless(what):
    bad = BAD[what]
    table, held = Guarded(4 * 8, 0), Guarded(8, 0)
    stack = ints(bad.get("stack", range(8)))
    d = KvPages(16, table.view(torch.int32, (2, 4)), held.view(torch.int32, (2,)), stack, ints([bad.get("free", 8)]))
    d.n_blocks.copy_(ints(bad.get("held", [0, 0])))
    t = bad.get("most", 10)
    out = [Guarded(8, 0), Guarded(12, 0), Guarded(4 * t, 0), Guarded(8 * t, 0)]
    after, cu = out[0].view(torch.int32, (2,)), out[1].view(torch.int32, (3,))
    pos, slots = out[2].view(torch.int32, (t,)), out[3].view(torch.int64, (t,))
    d.extend(ints(bad.get("lens", [0, 3])), ints(bad.get("new", [2, 4])), after, cu, pos, slots)
    assert d.lib.gdn_sync_status(stream(), check=False) == gl.GDN_EINDEX and "gdn_kv_extend" in d.lib.last_error()
    assert all(g.intact() for g in out + [table, held])
    assert cu[0] == 0 and (cu[1:] >= cu[:-1]).all() and cu[2] <= t
    assert (slots < 8 * 16).all() and (slots >= -1).all()
    if what in ("page", "page_negative"):
        assert (slots == -1).all()
    d.trim(ints([0, 0]))
    d.lib.gdn_sync_status(stream(), check=False)
    assert table.intact() and held.intact() and d.n_blocks.tolist() == [0, 0] and 0 <= int(d.n_free[0]) <= 8


def test_more_back_than_there_are_pages():
    """Tables that hold more than the cache has: the stack ends at its end."""
    stack = Guarded(4 * 3, 0)
    d = KvPages(16, ints([[0, 1, 2, 0], [1, 2, 0, 1]]), ints([4, 4]), stack.view(torch.int32, (3,)), ints([1]))
    d.trim(ints([0, 16]))
    assert d.lib.gdn_sync_status(stream(), check=False) == gl.GDN_EINDEX
    assert stack.intact() and int(d.n_free[0]) == 3 and d.n_blocks.tolist() == [0, 1]
    sync(d.lib)


def test_a_tree_of_more_than_64_tokens_is_reported():
    d = KvPages.new(1, 8, 8, 16)
    out = ints([0]), ints([0, 0]), ints([0] * 65), ints([0] * 65, np.int64)
    d.extend(ints([0]), ints([65]), *out, tree=torch.zeros(65, dtype=torch.int64, device=DEV))
    assert d.lib.gdn_sync_status(stream(), check=False) == gl.GDN_EINDEX
    sync(d.lib)


def test_replayed_with_other_lengths():
    """A captured step of trim and extension follows what its buffers hold."""
    n, page, wide = 12, 16, 700
    a, b = Book(n, wide, 9000, page, seed=1), Book(n, wide, 9000, page, seed=1)
    side, t = torch.cuda.Stream(), 4000
    lens, new, keep = ints([0] * n), ints([0] * n), ints([0] * n)
    after, cu, pos, slots = ints([0] * n), ints([0] * (n + 1)), ints([0] * t), ints([0] * t, np.int64)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            a.dev.trim(keep)
            a.dev.extend(lens, new, after, cu, pos, slots)
        rng = np.random.default_rng(0)
        held = np.zeros(n, np.int64)
        for _ in range(6):
            more = rng.integers(0, 300, size=n)
            for x, v in ((keep, held), (lens, held), (new, more)):
                x.copy_(ints(v))
            g.replay()
            side.synchronize()
            b.host.trim(held.tolist())
            want = b.host.extend(held.tolist(), more.tolist())
            m = want[1][-1]
            assert after.tolist() == want[0] and cu.tolist() == want[1]
            assert pos[:m].tolist() == want[2] and slots[:m].tolist() == want[3] and (slots[m:] == -1).all()
            held = held + rng.integers(0, more + 1)


def test_wrappers_refuse_what_does_not_fit():
    d = KvPages.new(3, 4, 12, 16)
    good = dict(lens=ints([0] * 3), n_new=ints([1] * 3), lens_out=ints([0] * 3), cu=ints([0] * 4), positions=ints([0] * 5), slots=ints([0] * 5, np.int64))
    d.extend(**good)
    for bad in (dict(lens=ints([0] * 4)), dict(n_new=good["n_new"].long()), dict(lens_out=good["lens_out"].cpu()), dict(cu=ints([0] * 3)),
                dict(slots=ints([0] * 4, np.int64)), dict(slots=ints([0] * 5)), dict(tree=torch.zeros(4, dtype=torch.int64, device=DEV)),
                dict(lens=ints([0] * 6)[::2])):
        with pytest.raises(ValueError):
            d.extend(**{**good, **bad})
    with pytest.raises(ValueError):
        d.trim(ints([0] * 2))
    with pytest.raises(ValueError):
        KvPages(16, d.block_table.t(), d.n_blocks, d.free_pages, d.n_free)
    with pytest.raises(gl.GdnError):
        KvPages(17, d.block_table, d.n_blocks, d.free_pages, d.n_free).trim(ints([0] * 3))
    sync(d.lib)
