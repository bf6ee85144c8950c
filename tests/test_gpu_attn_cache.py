"""gdn_attn_cache against fp64 attention over the values the cache holds.

Tolerance per element, from the arithmetic.  The cached values and q are the
same numbers on both sides.  The output is rounded to bf16 once: 2^-8 of the
value.  The probabilities may enter the second product rounded to its operand
type, bf16 over a bf16 cache (half a step: 2^-8 of each) and fp16 over 8-bit
codes (2^-11): relative to S = sum_j p_j |v_j|.  Scores are fp32 sums of D <=
256 products, whose error is below 256 * 2^-24 sum |q k| scale < 2e-4 here
(sum |q k| scale < 13 for unit rows), exp and the sums add less than 1e-5:
3e-4 S.
"""
import numpy as np
import pytest
import torch

from hybrid_gated_deltanet_q4k_gb300 import api
from hybrid_gated_deltanet_q4k_gb300 import lib as gl
from oracle import serving as OS

from gpu_util import DEV, Guarded, guarded, stream, sync

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "i8", "e4m3"]


@pytest.fixture(scope="module")
def L():
    return gl.load(build=True)


class Case:
    """Sequences with their pages scattered over a pool, its free places holding `junk` (bytes)."""

    def __init__(self, kind, d, page, hkv, ratio, lens, nq, tree=None, seed=0, junk=0x7F, gain=1.0, debug=False, spare=3,
                 widen=0):
        rng = np.random.default_rng(seed)
        self.rng, self.kind, self.d, self.hkv, self.hq = rng, kind, d, hkv, hkv * ratio
        self.lens, self.nq = list(lens), list(nq)
        self.cu = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
        T = int(self.cu[-1])
        per = [-(-n // page) for n in lens]
        n_pages = sum(per) + spare
        size = 2 if kind == "bf16" else 1
        dtype = api.KvCache.TYPES[kind][1]
        pools = [torch.full((n_pages, hkv, page, d * size), junk, dtype=torch.uint8, device=DEV).view(dtype) for _ in "kv"]
        # 0x7fffffff: a scale that is not a number, where no row was stored
        scales = [None if kind == "bf16" else
                  torch.full((n_pages, hkv, page), 0x7FFFFFFF, dtype=torch.int32, device=DEV).view(torch.float32) for _ in "kv"]
        self.cache = api.KvCache(kind, *pools, *scales, debug=debug)
        order = rng.permutation(n_pages)
        blocks = max(max(per), 1) + widen
        table = np.full((len(lens), blocks), -7, np.int32)
        at = 0
        self.k, self.v = [], []
        for s, n in enumerate(lens):
            table[s, :per[s]] = order[at:at + per[s]]
            at += per[s]
            k = rng.standard_normal((n, hkv, d), dtype=np.float32)
            v = rng.standard_normal((n, hkv, d), dtype=np.float32) + 0.25
            k, v = (torch.from_numpy(x).to(DEV).to(torch.bfloat16) for x in (k, v))
            sl = self.cache.slots(torch.from_numpy(table[s]).to(DEV), 0, n)
            self.cache.write(k, v, sl)
            self.k.append(self._value(k))
            self.v.append(self._value(v))
        self.table_host = table
        self.table = torch.from_numpy(table).to(DEV)
        self.q = torch.from_numpy(gain * rng.standard_normal((T, self.hq, d), dtype=np.float32)).to(DEV).to(torch.bfloat16)
        self.tree = None if tree is None else np.array(tree, np.uint64)
        self.max_q = max(nq)

    def _value(self, x):
        x = x.float().cpu().numpy()
        if self.kind == "bf16":
            return x.astype(np.float64)
        codes, s = OS.quantise_rows(x, self.kind)
        return codes * s[..., None].astype(np.float64)

    def visible(self, s):
        m, n = self.nq[s], self.lens[s]
        out = np.ones((m, n), bool)
        for i in range(m):
            w = (1 << (i + 1)) - 1 if self.tree is None else int(self.tree[self.cu[s] + i])
            for j in range(m):
                if n - m + j >= 0:
                    out[i, n - m + j] = (w >> j) & 1
        return out

    def run(self, L, o=None, cu=True, lens=None, table=None, st=None, ws=None, q=None, scale=0.0, max_q=None):
        T = int(self.cu[-1])
        o = torch.full((T, self.hq, self.d), 7.0, dtype=torch.bfloat16, device=DEV) if o is None else o
        ws = self.cache.new_attend_workspace(T, self.hq) if ws is None else ws
        self.dev = (torch.tensor(self.lens if lens is None else lens, dtype=torch.int32, device=DEV),
                    torch.from_numpy(self.cu).to(DEV) if cu else None,
                    None if self.tree is None else torch.from_numpy(self.tree.view(np.int64)).to(DEV))
        if st is not None:
            st.wait_stream(torch.cuda.current_stream())
        self.cache.attend(self.q if q is None else q, self.dev[0], self.table if table is None else table, o, ws,
                          cu_q=self.dev[1], max_q=self.max_q if max_q is None else max_q, tree=self.dev[2], scale=scale, stream=st)
        return o

    def check(self, got, scale=None, rows=None):
        got = got.double().cpu().numpy()
        for s in range(len(self.lens)):
            a, b = self.cu[s], self.cu[s + 1]
            if rows is not None and s not in rows:
                continue
            ref, spread = OS.attend(self.q[a:b].double().cpu().numpy(), self.k[s], self.v[s], self.visible(s),
                                    scale or self.d ** -0.5)
            tol = 2.0 ** -8 * np.abs(ref) + ((2.0 ** -8 if self.kind == "bf16" else 2.0 ** -11) + 3e-4) * spread
            err = np.abs(got[a:b] - ref)
            assert np.all(err <= tol), (s, float((err / np.maximum(tol, 1e-30)).max()))


def _tree(rng, nq, roots=0.1):
    words = []
    for n in nq:
        mine = []
        for i in range(n):
            up = mine[rng.integers(0, i)] if i and rng.random() > roots else 0
            mine.append(up | (1 << i))
        words += mine
    return words


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page,hkv,ratio,lens", [
    (16, 1, 1, [1]), (64, 4, 4, [777]), (16, 2, 8, [1, 2, 15, 16, 17, 300]), (32, 3, 3, [63, 64, 65, 500, 1]),
    (128, 1, 16, [127, 129, 1000]), (64, 2, 5, [2500]),
])
def test_one_token(L, kind, d, page, hkv, ratio, lens):
    c = Case(kind, d, page, hkv, ratio, lens, [1] * len(lens), seed=d + page)
    o = c.run(L)
    sync(L)
    c.check(o)
    assert torch.equal(o, c.run(L, cu=False))      # no offsets: one token each; and the same bits a second time
    sync(L)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,page,hkv,ratio,lens,nq", [
    (64, 16, 2, 4, [5, 70, 333], [2, 4, 3]), (128, 64, 2, 3, [64, 65, 900], [7, 1, 5]), (256, 32, 1, 8, [40, 700], [40, 33]),
    (256, 64, 2, 4, [1500, 64, 200], [64, 64, 17]), (128, 16, 1, 16, [130, 70], [64, 9]), (64, 128, 1, 5, [2000], [64]),
    (256, 64, 1, 1, [300], [64]), (128, 128, 1, 2, [129, 255], [2, 63]), (64, 64, 1, 16, [1100], [64]),
])
@pytest.mark.parametrize("masked", ["chain", "tree"])
def test_several_tokens(L, kind, d, page, hkv, ratio, lens, nq, masked):
    rng = np.random.default_rng(d + lens[0])
    c = Case(kind, d, page, hkv, ratio, lens, nq, tree=_tree(rng, nq) if masked == "tree" else None, seed=d + lens[-1], widen=2)
    o = c.run(L)
    sync(L)
    c.check(o)
    assert torch.equal(o, c.run(L))
    sync(L)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ratio", [1, 4, 16])
def test_rows_that_see_nothing(L, kind, ratio):
    """Tokens whose mask is empty and that have no context give zeros; bits past the sequence's tokens mean nothing."""
    nq, lens = [6, 5, 40], [6, 70, 40]
    tree = _tree(np.random.default_rng(0), nq)
    tree[0] = tree[3] = 0
    tree[4] = 1 << 63 | 1 << 6                     # only bits past the six tokens
    tree[7] = 0                                    # with context: sees the context alone
    tree[11 + 39] = 0
    tree[11 + 2] |= 0xFF << 50
    c = Case(kind, 128, 16, 2, ratio, lens, nq, tree=tree, seed=3)
    o = c.run(L)
    sync(L)
    c.check(o)
    assert not o[[0, 3, 4, 50]].any() and o[7].any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,nq,ratio", [(64, 9, 2), (128, 5, 4), (256, 3, 4), (256, 40, 4), (128, 60, 8)])
def test_what_is_not_seen_does_not_count(L, kind, d, nq, ratio):
    """Keys and values that are infinite or NaN reach only the tokens that see them."""
    lens = [100 + nq]
    tree = [1 << i for i in range(nq)]             # each token sees the context and itself
    c = Case(kind, d, 16, 2, ratio, lens, [nq], tree=tree, seed=d + nq)
    clean = c.run(L)
    sync(L)
    c.check(clean)
    bad = torch.ones(1, 2, d, dtype=torch.bfloat16, device=DEV)
    bad[0, :, 3] = float("inf")
    bad[0, :, 5] = float("-inf")
    nan = bad.clone()
    nan[0, :, 7] = float("nan")
    slots = c.cache.slots(c.table[0], 0, lens[0])
    c.cache.write(bad, bad, slots[-2:-1])
    c.cache.write(nan, nan, slots[-nq:-nq + 1])
    o = c.run(L)
    sync(L)
    hit = [0, nq - 2]
    keep = [i for i in range(nq) if i not in hit]
    assert bool(torch.isfinite(o[keep].float()).all())
    c.check_rows = keep
    got, ref = o[keep], clean[keep]
    # the same sums without the two keys that were masked before as well
    assert float((got.double() - ref.double()).abs().max()) <= 2.0 ** -6 * float(ref.double().abs().max())
    assert not bool(torch.isfinite(o[hit].float()).all(dim=-1).any())
    # values alone: the scores stay finite and so do the elements without a bad value
    if kind == "bf16":
        fine = torch.ones(1, 2, d, dtype=torch.bfloat16, device=DEV)
        c.cache.write(fine, bad, slots[-2:-1])
        c.cache.write(fine, nan, slots[-nq:-nq + 1])
        o = c.run(L)
        sync(L)
        assert bool(torch.isfinite(o[keep].float()).all())
        finite = torch.isfinite(o[hit].float())
        want = torch.ones_like(finite)
        want[:, :, [3, 5]] = False
        want[0, :, 7] = False
        assert torch.equal(finite, want)
        assert bool((o[hit][:, :, 3] == float("inf")).all()) and bool((o[hit][:, :, 5] == float("-inf")).all())


@pytest.mark.parametrize("kind", KINDS)
def test_large_scores_and_explicit_scale(L, kind):
    """A peaked softmax: the running maximum rises often, the largest score far above the others."""
    c = Case(kind, 128, 32, 2, 4, [900, 33], [3, 1], seed=8, gain=30.0)
    o = c.run(L, scale=0.02)
    sync(L)
    c.check(o, scale=0.02)
    o = c.run(L)
    sync(L)
    # scores up to some hundreds: their fp32 error is 2e-5 of them
    got = o.double().cpu().numpy()
    for s in range(2):
        a, b = c.cu[s], c.cu[s + 1]
        ref, spread = OS.attend(c.q[a:b].double().cpu().numpy(), c.k[s], c.v[s], c.visible(s), 128 ** -0.5)
        assert np.all(np.abs(got[a:b] - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 1e-2) * spread)


@pytest.mark.parametrize("kind", KINDS)
def test_tiny_and_huge_rows(L, kind):
    """Rows of very different sizes (8-bit scales from 1e-30 to 1e30) and a row of zeros keep their weights."""
    d, n = 128, 70
    c = Case(kind, d, 16, 1, 2, [n], [1], seed=9)
    rng = np.random.default_rng(4)
    k = torch.from_numpy(rng.standard_normal((n, 1, d), dtype=np.float32)).to(DEV).to(torch.bfloat16)
    v = torch.from_numpy((rng.standard_normal((n, 1, d)) * 10.0 ** rng.integers(-30, 30, (n, 1, 1))).astype(np.float32)).to(DEV).to(torch.bfloat16)
    v[5], k[6], v[11] = 0, 0, 1e-38
    c.cache.write(k, v, c.cache.slots(c.table[0], 0, n))
    c.k, c.v = [c._value(k)], [c._value(v)]
    o = c.run(L)
    sync(L)
    c.check(o)
    small = v.clone()
    small[:] = v * 1e-36
    c.cache.write(k, small, c.cache.slots(c.table[0], 0, n))
    c.v = [c._value(small)]
    q0 = c.run(L)
    sync(L)
    c.check(q0)
    tiny = torch.full_like(q0, 0)
    c.cache.write(k, torch.zeros_like(v), c.cache.slots(c.table[0], 0, n))
    assert torch.equal(c.run(L), tiny)
    sync(L)


@pytest.mark.parametrize("kind", KINDS)
def test_strides_streams_and_guards(L, kind):
    c = Case(kind, 128, 32, 2, 4, [200, 77, 150], [3, 1, 8], seed=10)
    T, w = int(c.cu[-1]), c.hq * c.d
    want = c.run(L)
    sync(L)
    c.check(want)
    wide = torch.zeros(T, w + 72, dtype=torch.bfloat16, device=DEV)
    wide[:, 8:8 + w] = c.q.reshape(T, w)
    go, out = guarded((T, w + 8), torch.bfloat16, init=torch.full((T, w + 8), 7.0, dtype=torch.bfloat16, device=DEV))
    n = c.cache.attend_workspace_bytes(T, c.hq)
    gw = Guarded(n)
    wide_table = torch.full((3, c.table.shape[1] + 5), -9, dtype=torch.int32, device=DEV)
    wide_table[:, 2:2 + c.table.shape[1]] = c.table
    st = torch.cuda.Stream()
    c.run(L, o=out[:, :w].view(T, c.hq, c.d), q=wide[:, 8:8 + w].view(T, c.hq, c.d), st=st, ws=gw.view(torch.uint8, (n,)),
          table=wide_table[:, 2:2 + c.table.shape[1]])
    st.synchronize()
    sync(L)
    assert go.intact() and gw.intact()
    assert torch.equal(out[:, :w].view(T, c.hq, c.d), want) and bool((out[:, w:] == 7.0).all())


def test_a_captured_call_replays_with_other_lengths(L):
    """Lengths, offsets, pages and masks are read when the graph runs, not when it is captured."""
    c = Case("i8", 256, 64, 4, 4, [500, 90], [4, 2], tree=_tree(np.random.default_rng(1), [4, 2]), seed=11)
    o = c.run(L)
    ws = c.cache.new_attend_workspace(6, c.hq)
    sync(L)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.cache.attend(c.q, c.dev[0], c.table, o, ws, cu_q=c.dev[1], max_q=4, tree=c.dev[2])
    o.zero_()
    g.replay()
    sync(L)
    c.check(o)
    c.lens = [131, 70]
    c.nq, c.cu = [2, 4], np.array([0, 2, 6], np.int32)
    c.dev[0].copy_(torch.tensor(c.lens))
    c.dev[1].copy_(torch.from_numpy(c.cu))
    c.tree = np.array(_tree(np.random.default_rng(2), c.nq), np.uint64)
    c.dev[2].copy_(torch.from_numpy(c.tree.view(np.int64)))
    c.k, c.v = [x[:n] for x, n in zip(c.k, c.lens)], [x[:n] for x, n in zip(c.v, c.lens)]
    g.replay()
    sync(L)
    c.check(o)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nq", [1, 40])
def test_indices_out_of_range_are_reported(L, kind, nq):
    """A page outside the cache counts as not seen, a length past the table is clamped, a sequence with bad offsets is
    left out; each is reported once and the next call is fine."""
    c = Case(kind, 128, 16, 2, 4, [100, 130], [nq, nq], seed=12)
    want = c.run(L)
    sync(L)
    for bad_page in (-1, c.cache.n_pages, 2 ** 31 - 1):
        t = c.table.clone()
        t[1, 2] = bad_page
        o = c.run(L, table=t)
        assert L.gdn_sync_status(stream(), check=False) == gl.GDN_EINDEX
        assert L.gdn_sync_status(stream(), check=False) == gl.GDN_OK
        assert torch.equal(o[:nq], want[:nq])
        see = np.r_[0:32, 48:130]
        ref, spread = OS.attend(c.q[nq:].double().cpu().numpy(), c.k[1][see], c.v[1][see], c.visible(1)[:, see], 128 ** -0.5)
        assert np.all(np.abs(o[nq:].double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 3e-4) * spread)
    o = c.run(L, lens=[-5, 130])
    assert L.gdn_sync_status(stream(), check=False) == gl.GDN_EINDEX
    assert not o[:nq].any() and torch.equal(o[nq:], want[nq:])
    if nq == 1:                                    # 2^31 - 1 becomes the table's 144, whose last 14 were never stored
        o = c.run(L, lens=[100, 2 ** 31 - 1])
        assert L.gdn_sync_status(stream(), check=False) == gl.GDN_EINDEX
        assert torch.equal(o[:nq], want[:nq])
    keep = c.cu.copy()
    for cu in ([0, nq, 2 * nq + 1], [0, -1, nq], [nq, 0, nq], [0, 2 ** 31 - 1, nq]):
        c.cu = np.array(cu, np.int32)
        o = torch.full_like(want, 7.0)
        c.cache.attend(c.q, c.dev[0].new_tensor([100, 130]), c.table, o, c.cache.new_attend_workspace(2 * nq, c.hq),
                       cu_q=torch.from_numpy(c.cu).to(DEV), max_q=nq)
        assert L.gdn_sync_status(stream(), check=False) == gl.GDN_EINDEX
        if cu[1] == nq:
            assert torch.equal(o[:nq], want[:nq]) and bool((o[nq:] == 7.0).all())
    c.cu = keep
    assert torch.equal(c.run(L), want)
    sync(L)


@pytest.mark.parametrize("kind", ["i8", "bf16"])
def test_many_sequences_of_every_length(L, kind):
    """256 sequences, from one token to some hundreds, some without a new token."""
    rng = np.random.default_rng(13)
    nq = rng.integers(0, 4, size=256)
    lens = np.maximum(rng.integers(1, 260, size=256), nq)
    c = Case(kind, 64, 32, 2, 4, lens.tolist(), nq.tolist(), seed=13)
    o = c.run(L)
    sync(L)
    c.check(o)


@pytest.mark.parametrize("kind,d,n,nq,ratio", [("bf16", 256, 40000, 1, 4), ("i8", 256, 70001, 2, 4), ("e4m3", 128, 50000, 64, 4),
                                               ("bf16", 256, 20011, 64, 4), ("i8", 64, 90000, 48, 8)])
def test_long_contexts(L, kind, d, n, nq, ratio):
    c = Case(kind, d, 64, 1, ratio, [n], [nq], tree=_tree(np.random.default_rng(3), [nq]), seed=14)
    o = c.run(L)
    sync(L)
    c.check(o)


@pytest.mark.parametrize("nq", [1, 40])
def test_pages_past_32_bits(L, nq):
    """Pages more than 2^32 bytes into the cache."""
    heads, page, d = 8, 128, 256
    n_pages = (1 << 32) // (heads * page * d) + 3
    cache = api.KvCache.new("i8", n_pages, heads, page, d)
    rng = np.random.default_rng(15)
    n = 200
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device=DEV)
    k, v = (torch.from_numpy(rng.standard_normal((n, heads, d), dtype=np.float32)).to(DEV).to(torch.bfloat16) for _ in "kv")
    cache.write(k, v, cache.slots(table[0], 0, n))
    small = Case("i8", d, page, heads, 1, [n], [nq], seed=15)
    small.k, small.v = [small._value(k)], [small._value(v)]
    small.cache, small.table = cache, table
    o = small.run(L)
    sync(L)
    small.check(o)


def test_debug_library_gives_the_same_bits():
    gl.load(build=True)
    outs = []
    for debug in (False, True):
        c = Case("e4m3", 128, 32, 2, 4, [400, 61], [20, 1], seed=16, debug=debug)
        o = c.run(c.cache.lib)
        assert c.cache.lib.gdn_sync_status(stream(), check=False) == gl.GDN_OK
        outs.append(o)
    assert torch.equal(*outs)


def test_attend_wrapper_refuses(L):
    c = Case("i8", 64, 16, 2, 2, [20], [2], seed=17)
    c.run(L)
    sync(L)
    lens, cu, _ = c.dev
    ws = c.cache.new_attend_workspace(2, 4)
    o = torch.empty_like(c.q)
    for bad in [lambda: c.cache.attend(c.q, lens.long(), c.table, o, ws, cu_q=cu, max_q=2),
                lambda: c.cache.attend(c.q, lens, c.table.long(), o, ws, cu_q=cu, max_q=2),
                lambda: c.cache.attend(c.q, lens, c.table, o[:1], ws, cu_q=cu, max_q=2),
                lambda: c.cache.attend(c.q.float(), lens, c.table, o, ws, cu_q=cu, max_q=2),
                lambda: c.cache.attend(c.q, lens, c.table, o, ws, cu_q=cu[:1], max_q=2),
                lambda: c.cache.attend(c.q, lens, c.table, o, ws, cu_q=cu, max_q=2, tree=lens)]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gl.GdnError):
        c.cache.attend(c.q, lens, c.table, o, ws, max_q=1)
