"""gdn_attn_cache over values, scales and scores of every size, in both of its kernels.

A token of a few heads takes the kernel for few rows, forty tokens or more the one for many.  The tolerance is
the one of the cache attention's other tests: 2^-8 of the value for the output's rounding, 2^-8 (bf16 cache) or
2^-11 (codes) of S = sum_j p_j |v_j| for the probabilities' rounding, 3e-4 S for scores in fp32.  Over codes a
probability times its value scale is an fp16 number that is lifted to 2^11 or more for the largest one, so what is
rounded below fp16's normal numbers or lost is 2^-25 at most: 2^-36 of the largest product of a probability and a
row's amax, for each key.
"""
import numpy as np
import pytest
import torch

from hybrid_gated_deltanet_q4k_gb300 import lib as gl
from oracle import serving as OS

from gpu_util import DEV, stream, sync
from test_gpu_attn_cache import Case, _tree

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "i8", "e4m3"]
FEW, MANY = 1, 40       # new tokens


@pytest.fixture(scope="module")
def L():
    return gl.load(build=True)


def _bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(DEV).to(torch.bfloat16)


def _store(c, s, k=None, v=None):
    """Other keys or values (bf16 [n][heads][d]) for sequence s of the case, and what the cache then holds."""
    n = c.lens[s]
    k = _bf16(c.rng.standard_normal((n, c.hkv, c.d))) if k is None else k
    v = _bf16(c.rng.standard_normal((n, c.hkv, c.d)) + 0.25) if v is None else v
    c.cache.write(k, v, c.cache.slots(c.table[s], 0, n))
    c.k[s], c.v[s] = c._value(k), c._value(v)


def _check(c, got, scores=3e-4, lost=2.0 ** -36, weights=None):
    """c.check with the errors of the scores and of the probabilities as given, and what fp16 loses."""
    weights = weights or (2.0 ** -8 if c.kind == "bf16" else 2.0 ** -11)
    got = got.double().cpu().numpy()
    for s in range(len(c.lens)):
        a, b = c.cu[s], c.cu[s + 1]
        q = c.q[a:b].double().cpu().numpy()
        see = c.visible(s)
        ref, spread = OS.attend(q, c.k[s], c.v[s], see, c.d ** -0.5)
        tol = 2.0 ** -8 * np.abs(ref) + (weights + scores) * spread
        if c.kind != "bf16":
            amax = np.abs(c.v[s]).max(axis=-1, keepdims=True)     # [n][hkv][1]
            top = np.zeros(ref.shape[:2])
            for h in range(c.hq):
                g = h // (c.hq // c.hkv)
                x = np.where(see, c.d ** -0.5 * (q[:, h] @ c.k[s][:, g].T), -np.inf)
                p = np.exp(x - x.max(axis=1, keepdims=True))
                top[:, h] = (p / p.sum(axis=1, keepdims=True) * amax[:, g, 0]).max(axis=1)
            tol = tol + lost * c.lens[s] * top[..., None]
        err = np.abs(got[a:b] - ref)
        assert np.all(err <= tol), (s, float((err / np.maximum(tol, 1e-300)).max()))


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("d,nq", [(64, MANY), (128, MANY), (256, MANY), (128, FEW)])
def test_scales_of_every_key_reach_their_own_scores(L, kind, d, nq):
    """Keys and values whose scales differ from one row to the next by up to 2^6 and 2^16, over many tiles."""
    c = Case(kind, d, 32, 2, 2, [1500], [nq], seed=d + nq)
    size = lambda lo, hi: np.exp2(c.rng.integers(lo, hi, size=(1500, 2, 1), endpoint=True))  # noqa: E731
    x = c.rng.standard_normal((2, 1500, 2, d))
    _store(c, 0, _bf16(x[0] * size(-3, 3)), _bf16(x[1] * size(-8, 8)))
    o = c.run(L)
    sync(L)
    _check(c, o, scores=8 * 3e-4)          # keys up to 2^3 times as large: their scores' errors too
    assert torch.equal(o, c.run(L))
    sync(L)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nq", [FEW, MANY])
@pytest.mark.parametrize("zeros,n,hkv", [(256, 1300, 1), (2048, 2500, 1), (20000, 20700, 1), (2048, 2300, 160), (300, 300, 2)])
def test_values_of_zero_ahead_of_others(L, kind, nq, zeros, n, hkv):
    """Tokens whose values (and keys) are zero, more than a tile of them, ahead of ordinary ones: within one piece of a
    run (160 heads: a run takes whole pairs) and over many runs."""
    c = Case(kind, 64, 64, hkv, 1, [n], [nq], seed=zeros + nq)
    k, v = (c.rng.standard_normal((n, hkv, 64)) for _ in "kv")
    k[:zeros] = v[:zeros] = 0.0
    _store(c, 0, _bf16(k), _bf16(v + 0.5 * (v != 0)))
    o = c.run(L)
    sync(L)
    _check(c, o)
    assert bool(o.any()) == (n > zeros)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nq", [FEW, MANY])
@pytest.mark.parametrize("score", [25.0, 45.0])
@pytest.mark.parametrize("where", ["first", "amid", "last"])
def test_values_of_zero_that_score_above_all_others(L, kind, nq, score, where):
    """Tokens whose values are zero and whose scores are 25 and 45 above the others': the sum is theirs, the result is what
    little the others have of it."""
    n, zeros, d = 2600, 1000, 64
    c = Case(kind, d, 64, 1, 1, [n], [nq], seed=int(score))
    k, v = (c.rng.standard_normal((n, 1, d)) for _ in "kv")
    k[..., 0] = 0.0                          # the first element carries the difference alone
    at = {"first": 0, "amid": 777, "last": n - nq - zeros}[where]
    k[at:at + zeros], v[at:at + zeros] = 0.0, 0.0
    k[at:at + zeros, 0, 0] = score * d ** 0.5
    c.q[..., 0] = 1.0
    _store(c, 0, _bf16(k), _bf16(v))
    o = c.run(L)
    sync(L)
    _check(c, o)
    assert bool(o.any())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nq", [FEW, MANY])
def test_rows_of_every_size(L, kind, d, nq):
    """Values from 1e-30 to 1e30 in one sequence, small ones alone, and every value near 2^-100."""
    n = 400
    c = Case(kind, d, 16, 1, 2, [n], [nq], seed=19)
    x = c.rng.standard_normal((n, 1, d))
    v = x * 10.0 ** c.rng.integers(-30, 30, (n, 1, 1))
    v[5], v[11] = 0, 1e-38
    for y in (v, v * 1e-36, x * 2.0 ** 60, x * 2.0 ** -60, x * 2.0 ** -70):
        _store(c, 0, v=_bf16(y))
        o = c.run(L)
        sync(L)
        _check(c, o)
    # a scale below 2^-80 counts as that for the running maximum: at 2^-85 the largest product may be 2^-14 of what it is
    # otherwise (amax / 448 > 2^-94), at 2^-100 2^-29
    _store(c, 0, v=_bf16(x * 2.0 ** -85))
    o = c.run(L)
    sync(L)
    _check(c, o, lost=2.0 ** -22)
    _store(c, 0, v=_bf16(x * 2.0 ** -100))
    o = c.run(L)
    sync(L)
    # (the kernel for few rows multiplies what fp16 loses in bf16)
    _check(c, o, lost=2.0 ** -36 if nq == FEW else 2.0 ** -7, weights=2.0 ** -8)
    assert bool(o.any())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nq", [FEW, MANY])
@pytest.mark.parametrize("power", [-118, -60, 60, 110, 118])
def test_queries_of_every_size(L, kind, nq, power):
    """Queries of 2^power over keys of 2^-power: the scores are those of ordinary rows."""
    c = Case(kind, 128, 32, 2, 2, [300], [nq], seed=20)
    plain = c.q.clone()
    k = c.rng.standard_normal((300, 2, 128))
    _store(c, 0, k=_bf16(k * 2.0 ** -power))
    c.q = (plain.double() * 2.0 ** power).to(torch.bfloat16)
    o = c.run(L)
    sync(L)
    _check(c, o)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,n,nq", [(64, 900, 50), (128, 2100, 64), (256, 1300, 41)])
def test_peaked_rows_of_many_tokens(L, kind, d, n, nq):
    """The running maximum rises often, by more than its margin, and the accumulator is scaled again each time."""
    c = Case(kind, d, 32, 1, 4, [n], [nq], tree=_tree(np.random.default_rng(5), [nq]), seed=21, gain=30.0)
    k = c.rng.standard_normal((n, 1, d)) * np.linspace(0.2, 1.0, n)[:, None, None]      # later keys count for more
    _store(c, 0, k=_bf16(k))
    o = c.run(L)
    sync(L)
    _check(c, o, scores=1e-2)              # scores up to some hundreds: their fp32 error is 2e-5 of them


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nq,ratio,hkv,n", [(1, 8, 16, 40000), (4, 4, 8, 9001), (64, 2, 1, 40000), (64, 2, 1, 16500)])
def test_every_key_counts_once(L, kind, nq, ratio, hkv, n):
    """Each row has two keys that take all of its weight, one of them at or beside a border of blocks and runs: a tile
    that is left out, or counted twice, changes the row by a sixth of the values or more."""
    d = 128
    rows = nq * ratio                       # of a key/value head; row r looks along its own axis r % 128
    assert rows <= d
    c = Case(kind, d, 64, hkv, ratio, [n], [nq], tree=[1 << i for i in range(nq)], seed=22)
    ctx = n - nq
    edges = np.unique(np.clip(np.concatenate([np.arange(0, n, 128) + e for e in (-1, 0, 1, 15, 16, 63, 64)]), 0, ctx - 2))
    places = c.rng.permutation(edges)[:hkv * rows].reshape(hkv, -1) if len(edges) >= hkv * rows else None
    assert places is not None
    other = ctx - 1                          # the second key of every row
    k = np.zeros((n, hkv, d))
    k[other] = 64.0
    for h in range(hkv):
        for r in range(rows):
            k[places[h, r], h, r] += 64.0
    v = c.rng.choice([-1.0, 1.0], size=(n, hkv, d)) * c.rng.uniform(0.5, 1.0, (n, hkv, d))
    q = np.zeros((nq, hkv * ratio, d), np.float32)
    for h in range(hkv):
        for r in range(rows):
            q[r // ratio, h * ratio + r % ratio, r] = 8.0      # a score of 8 * 64 / sqrt(128) = 45; the others 0
    _store(c, 0, _bf16(k), _bf16(v))
    c.q = _bf16(q)
    o = c.run(L)
    sync(L)
    got = o.double().cpu().numpy()
    for h in range(hkv):
        for r in range(rows):
            want = (c.v[0][places[h, r], h] + c.v[0][other, h]) / 2
            err = np.abs(got[r // ratio, h * ratio + r % ratio] - want)
            # the rest: 40000 e^-45 of weight; the output's and the probabilities' rounding
            assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -8), (h, r, places[h, r], err.max())
