"""Verification of drafted tokens against the oracle: whole numbers, equal."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, Guarded, stream, sync
from hybrid_gated_deltanet_q4k_gb300 import api
from hybrid_gated_deltanet_q4k_gb300 import lib as gl
from oracle import drafts as OD

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, lens, vocab, kind="q", dtype="f32", tree=True, seed=0, off=0, room=0, sharp=3.0, off_q=None):
        """off: elements that rows start behind a 16-byte place; room: elements between rows; off_q: q's own offset."""
        rng = np.random.default_rng(seed)
        self.lens, self.v, self.kind = list(lens), vocab, kind
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        t = int(self.cu[-1])
        self.t, self.max_new = t, max(1, max(lens))
        words = np.zeros(t, np.uint64)
        self.up = []
        for s, n in enumerate(lens):
            for i in range(n):
                up = words[self.cu[s] + (rng.integers(0, i) if tree else i - 1)] if i else np.uint64(0)
                words[self.cu[s] + i] = up | (np.uint64(1) << np.uint64(i))
            self.up.append(OD.parents(n, words[self.cu[s]:self.cu[s] + n]))
        self.tree = torch.from_numpy(words.view(np.int64)).to(DEV) if tree else None
        td = torch.float32 if dtype == "f32" else torch.bfloat16
        x = torch.from_numpy(sharp * rng.normal(size=(t, vocab))).float()
        y = x + torch.from_numpy(rng.normal(size=(t, vocab))).float()
        rounded = lambda a: a.to(td)  # noqa: E731
        self.p = rounded(x if kind == "greedy" else torch.softmax(x, 1))
        self.q = rounded(torch.softmax(y, 1)) if kind == "q" else None
        self.layout = [(off, room), (off if off_q is None else off_q, room)]
        src = (self.q if kind == "q" else self.p).float().numpy()
        self.tokens = np.zeros(t, np.int32)
        for s, n in enumerate(lens):
            for i in range(1, n):
                row = src[self.cu[s] + max(self.up[s][i], 0)].astype(np.float64)
                if kind == "greedy":
                    self.tokens[self.cu[s] + i] = OD._best(row) if rng.random() < 0.6 else rng.integers(vocab)
                else:
                    self.tokens[self.cu[s] + i] = rng.choice(vocab, p=row / row.sum())
        self.u = None if kind == "greedy" else rng.random(t).astype(np.float32)
        self.u_next = None if kind == "greedy" else rng.random(len(lens)).astype(np.float32)

    def place(self, x, off, room):
        """A device copy whose rows lie at the wanted places, between values that would win."""
        if x is None:
            return None
        ld = self.v + room
        raw = torch.full((self.t * ld + off + 16,), 9.0, dtype=x.dtype, device=DEV)
        view = raw[off:off + self.t * ld].view(self.t, ld)[:, :self.v]
        view.copy_(x)
        return view

    def run(self, debug=False, stream=None):
        dev = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
        s, t = len(self.lens), self.t
        bufs = [Guarded(4 * n, 0x5B) for n in (t, t, s, s, s)]
        out = [b.view(torch.int32, (n,)) for b, n in zip(bufs, (t, t, s, s, s))]
        api.verify(self.place(self.p, *self.layout[0]), dev(self.tokens), *out, u=dev(self.u), u_next=dev(self.u_next),
                   q=self.place(self.q, *self.layout[1]), cu=dev(self.cu), max_new=self.max_new, tree=self.tree, debug=debug)
        sync(gl.load(debug=debug))
        assert all(b.intact() for b in bufs)
        return [x.cpu().numpy() for x in out]

    def oracle(self):
        rows, ids = np.full(self.t, -1, np.int32), np.full(self.t, -1, np.int32)
        count, node, nxt = (np.zeros(len(self.lens), np.int32) for _ in range(3))
        p, q = self.p.float().numpy(), None if self.q is None else self.q.float().numpy()
        for s, n in enumerate(self.lens):
            a, b = self.cu[s], self.cu[s] + n
            keep, out, nx = OD.verify(p[a:b], None if q is None else q[a:b], self.tokens[a:b], self.up[s],
                                      None if self.u is None else self.u[a:b], None if self.u is None else self.u_next[s])
            rows[a:a + len(keep)] = a + np.array(keep, np.int32)
            ids[a:a + len(out)] = out
            count[s], node[s], nxt[s] = len(keep), keep[-1] if keep else -1, nx
        return [rows, ids, count, node, nxt]

    def check(self, **k):
        for got, want, name in zip(self.run(**k), self.oracle(), ("rows", "ids", "count", "node", "next")):
            assert np.array_equal(got, want), (name, got, want)


@pytest.mark.parametrize("kind", ["q", "certain", "greedy"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,vocab,tree", [([1], 1, False), ([5], 7, False), ([4, 0, 3], 33, True), ([64, 2, 31], 1000, True),
                                             ([8] * 20, 257, True), ([3] * 64, 4099, False), ([12, 9], 50001, True)])
def test_against_the_oracle(kind, dtype, lens, vocab, tree):
    Case(lens, vocab, kind, dtype, tree, seed=vocab + len(lens)).check()


@pytest.mark.parametrize("kind", ["q", "certain", "greedy"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off,room,off_q", [(1, 0, None), (3, 5, None), (0, 1, 2), (5, 3, 0), (7, 9, 1)])
@pytest.mark.parametrize("vocab", [2, 9, 8193])
def test_rows_at_any_place(kind, dtype, off, room, off_q, vocab):
    Case([6, 1, 9], vocab, kind, dtype, True, seed=off + vocab, off=off, room=room, off_q=off_q).check()


@pytest.mark.parametrize("sharp", [0.0, 0.3, 8.0])
@pytest.mark.parametrize("kind", ["q", "certain"])
def test_flat_and_sharp(sharp, kind):
    Case([20, 20, 20, 5], 777, kind, "f32", True, seed=int(10 * sharp), sharp=sharp).check()


def test_most_sequences():
    Case([2] * gl.GDN_MAX_SEQS, 1025, "q", "bf16", False, seed=1).check()


def test_q_equal_to_p_accepts_all():
    c = Case([6, 9], 100, "q", "f32", True, seed=3)
    c.p = c.q.clone()
    rows, ids, count, node, _ = c.run()
    for s in range(2):                                      # the first child of each token on the path
        here, n = 0, 1
        while here in c.up[s]:
            here, n = c.up[s].index(here), n + 1
        assert count[s] == n and node[s] == here
    c.check()


def test_random_numbers_at_the_ends():
    for u in (0.0, 1.0 - 2.0 ** -24, 2.0 ** -149):
        c = Case([7, 3], 500, "q", "f32", True, seed=4)
        c.u[:], c.u_next[:] = u, u
        c.check()


def test_nothing_left_of_the_residual():
    """p = q with a sum that rounding left below 1: a rejected draft leaves nothing, and the target's row is taken."""
    c = Case([2], 8, "q", "f32", False, seed=0)
    c.p = torch.tensor([[0.25, 0.25, 0.125, 0, 0, 0, 0.25, 0.0]] * 2)
    c.q = torch.tensor([[0.25, 0.25, 0.125, 0.5, 0, 0, 0.25, 0.0]] * 2)
    c.tokens[1], c.u[1], c.u_next[0] = 3, 0.5, 0.5
    rows, ids, count, node, nxt = c.run()
    assert count[0] == 1 and nxt[0] == 1                    # 0.4375 of 0.875 lies in token 1
    c.check()


def test_rows_without_probability_have_no_token():
    c = Case([2, 2], 40, "certain", "f32", False, seed=0)
    c.p[:2] = 0.0
    c.p[2] = float("nan")
    c.p[3, :] = -1.0
    rows, ids, count, node, nxt = c.run()
    assert list(count) == [1, 1] and list(nxt) == [-1, -1] and list(ids) == [-1] * 4


def test_nan_negative_and_large_entries():
    c = Case([10, 4], 300, "q", "f32", True, seed=6)
    c.p[:, 5], c.p[:, 17], c.q[:, 5], c.q[:, 40] = float("nan"), -0.5, float("nan"), -1.0
    c.p[3, 9] = float("inf")
    c.check()


def test_the_same_draft_twice_among_certain_siblings():
    c = Case([4], 20, "certain", "f32", False, seed=0)
    c.up = [[-1, 0, 0, 0]]
    c.tree = torch.tensor([1, 3, 5, 9], device=DEV)
    c.tokens[:], c.u[:] = [0, 7, 7, 7], 0.999
    c.check()


@pytest.mark.parametrize("row", ["ties", "all_nan", "all_-inf", "nan_first", "zeros"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_greedy_rows(row, dtype):
    """The lowest of equal ones; a NaN is never the largest."""
    c = Case([3, 1, 1], 1003, "greedy", dtype, False, seed=2)
    p = c.p
    if row == "ties":
        p[:, 100], p[:, 900], p[:, 1002] = 50.0, 50.0, 50.0
    elif row == "all_nan":
        p[:] = float("nan")
    elif row == "all_-inf":
        p[:] = float("-inf")
    elif row == "nan_first":
        p[:] = float("-inf")
        p[:, :3] = float("nan")
    else:
        p[:] = 0.0
        p[:, ::2] = -0.0
    want = {"ties": 100, "all_nan": 0, "all_-inf": 0, "nan_first": 3, "zeros": 0}[row]
    c.tokens[1:3] = want
    rows, ids, count, node, nxt = c.run()
    assert list(count) == [3, 1, 1] and list(nxt) == [want] * 3


@pytest.mark.parametrize("kind", ["q", "certain", "greedy"])
def test_tokens_outside_the_vocabulary_are_rejected(kind):
    c = Case([4, 3], 64, kind, "f32", False, seed=8)
    c.tokens[1], c.tokens[5] = 64, -1
    dev = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
    out = [torch.zeros(n, dtype=torch.int32, device=DEV) for n in (7, 7, 2, 2, 2)]
    api.verify(c.p.to(DEV), dev(c.tokens), *out, u=dev(c.u), u_next=dev(c.u_next), q=None if c.q is None else c.q.to(DEV), cu=dev(c.cu), max_new=4)
    assert gl.load().gdn_sync_status(stream(), check=False) == gl.GDN_EINDEX and "gdn_verify" in gl.load().last_error()
    assert out[2].tolist() == [1, 1]
    sync(gl.load())


def test_offsets_out_of_range_count_as_empty():
    c = Case([4, 3], 64, "q", "f32", False, seed=8)
    for cu in ([0, 9, 7], [0, 4, 2], [-3, 1, 4], [0, 4, 2 ** 30]):
        out = [torch.full((n,), 7, dtype=torch.int32, device=DEV) for n in (7, 7, 2, 2, 2)]
        api.verify(c.p.to(DEV), torch.from_numpy(c.tokens).to(DEV), *out, u=torch.from_numpy(c.u).to(DEV),
                   u_next=torch.from_numpy(c.u_next).to(DEV), q=c.q.to(DEV), cu=torch.tensor(cu, dtype=torch.int32, device=DEV), max_new=4)
        assert gl.load().gdn_sync_status(stream(), check=False) == gl.GDN_EINDEX
        assert (out[2] == 0).any() and (out[3][out[2] == 0] == -1).all() and (out[4][out[2] == 0] == -1).all()


@pytest.mark.parametrize("kind", ["q", "certain", "greedy"])
def test_without_offsets_every_sequence_has_max_new(kind):
    c = Case([6, 6, 6], 300, kind, "f32", True, seed=12)
    want = c.oracle()
    c.cu = None
    assert all(np.array_equal(x, y) for x, y in zip(c.run(), want))


def test_no_tokens_at_all():
    c = Case([0, 0], 10, "q", "f32", False, seed=0)
    rows, ids, count, node, nxt = c.run()
    assert list(count) == [0, 0] and list(node) == [-1, -1] and list(nxt) == [-1, -1]


def test_rows_behind_the_last_sequence_stay():
    c = Case([4, 3, 5], 64, "q", "f32", True, seed=9)
    want = c.oracle()
    c.lens, c.cu, c.u_next, c.max_new = c.lens[:2], c.cu[:3], c.u_next[:2], 8
    got = c.run()
    assert np.array_equal(got[0][:7], want[0][:7]) and (got[0][7:] == 0x5B5B5B5B).all() and (got[1][7:] == 0x5B5B5B5B).all()


def test_tokens_follow_the_target():
    """The first new token of many steps is distributed as the target's row, whatever the draft's (5 standard deviations)."""
    v, s, rounds = 6, 256, 40
    rng = np.random.default_rng(0)
    p, q = rng.dirichlet(np.ones(v)).astype(np.float32), rng.dirichlet(np.ones(v)).astype(np.float32)
    t = 4 * s
    P, Q = torch.from_numpy(np.tile(p, (t, 1))).to(DEV), torch.from_numpy(np.tile(q, (t, 1))).to(DEV)
    tree = torch.tensor([1, 3, 5, 9] * s, device=DEV)       # three siblings
    seen = np.zeros(v)
    for _ in range(rounds):
        tokens = torch.from_numpy(rng.choice(v, size=t, p=q.astype(np.float64) / q.astype(np.float64).sum()).astype(np.int32)).to(DEV)
        out = [torch.empty(n, dtype=torch.int32, device=DEV) for n in (t, t, s, s, s)]
        api.verify(P, tokens, *out, u=torch.from_numpy(rng.random(t).astype(np.float32)).to(DEV),
                   u_next=torch.from_numpy(rng.random(s).astype(np.float32)).to(DEV), q=Q, max_new=4, tree=tree)
        seen += np.bincount(out[1].view(s, 4)[:, 0].cpu().numpy(), minlength=v)
    n = s * rounds
    assert (np.abs(seen - n * p) <= 5 * np.sqrt(n * p * (1 - p))).all(), (seen / n, p)


def test_two_calls_at_once_and_replays():
    a, b = Case([9, 4], 20011, "q", "f32", True, seed=1), Case([5] * 30, 3001, "greedy", "bf16", True, seed=2)
    dev = lambda x: None if x is None else torch.from_numpy(x).to(DEV)  # noqa: E731
    runs = []
    for c in (a, b):
        s = len(c.lens)
        out = [torch.zeros(n, dtype=torch.int32, device=DEV) for n in (c.t, c.t, s, s, s)]
        kw = dict(u=dev(c.u), u_next=dev(c.u_next), q=None if c.q is None else c.q.to(DEV), cu=dev(c.cu), max_new=c.max_new, tree=c.tree)
        runs.append((c, c.p.to(DEV), dev(c.tokens), out, kw, torch.cuda.Stream()))
    torch.cuda.synchronize()
    graphs = []
    for c, p, tok, out, kw, st in runs:
        with torch.cuda.stream(st):
            api.verify(p, tok, *out, **kw)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                api.verify(p, tok, *out, **kw)
        graphs.append((g, st))
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, st), r in zip(graphs, runs):
            with torch.cuda.stream(st):
                for x in r[3]:
                    x.zero_()
                g.replay()
    torch.cuda.synchronize()
    for c, _, _, out, _, _ in runs:
        assert all(np.array_equal(x.cpu().numpy(), w) for x, w in zip(out, c.oracle()))


def test_the_debug_library_agrees():
    Case([9, 4, 0, 30], 3001, "q", "f32", True, seed=5).check(debug=True)


def test_wrapper_refuses_what_does_not_fit():
    c = Case([4, 3], 64, "q", "f32", True, seed=8)
    dev = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    i = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
    good = dict(p=c.p.to(DEV), tokens=dev(c.tokens), rows=i(7), ids=i(7), count=i(2), node=i(2), next=i(2), u=dev(c.u), u_next=dev(c.u_next),
                q=c.q.to(DEV), cu=dev(c.cu), max_new=4, tree=c.tree)
    api.verify(**good)
    for bad in (dict(p=good["p"].half()), dict(p=good["p"].t()), dict(q=good["q"].bfloat16()), dict(q=good["q"][:, :60]), dict(u=None),
                dict(tokens=i(6)), dict(rows=i(8)), dict(ids=good["ids"].long()), dict(count=i(3)), dict(node=i(1)), dict(cu=i(2)),
                dict(tree=good["tree"][:-1]), dict(u=good["u"].double()), dict(q=c.q), dict(next=i(4)[::2])):
        with pytest.raises(ValueError):
            api.verify(**{**good, **bad})
    with pytest.raises(gl.GdnError):
        api.verify(**{**good, "max_new": 65})
    sync(gl.load())
