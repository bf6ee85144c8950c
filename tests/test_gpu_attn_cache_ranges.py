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
