"""Verification where c0, the sum of the residuals so far, is large: rows that sum to nearly 8 and a dozen rejected siblings.

The last sibling x has u = 0, so it stays exactly if p(x) > c0 q(x).  c0 follows from the rejections before it in exact
arithmetic (a rejected sibling takes the residual's sum, here a sum of dyadic numbers), and p(x) is one of the two fp32
numbers around c0 q(x), chosen where it lies within 2^-18 q(x) of it: what c0 loses where its upper part is rounded to
24 bits.  The kernel's sums of 2^-44 are off by 2^-45 per number and row, 2^-38 in all."""
from fractions import Fraction as F

import numpy as np
import pytest
import torch

from gpu_util import DEV, sync
from hybrid_gated_deltanet_q4k_gb300 import api
from hybrid_gated_deltanet_q4k_gb300 import lib as gl
from oracle import drafts as OD

pytestmark = pytest.mark.gpu

HEAVY, X, DRAFT, VOCAB = 8, 8, 9, 40


def rows(n, stays, siblings):
    """Row and draft's row in which sibling X stays, or just does not; None where it is not within 2^-18 q of c0 q."""
    heavy, q = np.float32(0.96 + n * 2.0 ** -20), F(3, 1024)
    p_x = np.float32(0.2)
    for _ in range(20):                                     # p(x) is in the sums itself
        c0, z = F(0), F(1)
        for _ in range(siblings):
            c0 += z
            z = HEAVY * F(float(heavy)) + max(F(0), F(float(p_x)) - c0 * q)
        near = np.float32(float(c0 * q))
        want = near if (F(float(near)) > c0 * q) == stays else np.nextafter(near, np.float32(1 if stays else 0))
        if want == p_x:
            break
        p_x = want
    gap = F(float(p_x)) - c0 * q
    if (gap > 0) != stays or not F(1, 2 ** 30) * q < abs(gap) < F(9, 10) * F(1, 2 ** 18) * q or not 64 < c0 < 128:
        return None
    if int(c0 * 2 ** 18) % 4 != (3 if stays else 1):        # rounded to 24 bits: up where it stays, down where it does not
        return None
    P, Q = np.zeros(VOCAB, np.float32), np.zeros(VOCAB, np.float32)
    P[:HEAVY], P[X], Q[X], Q[DRAFT] = heavy, p_x, float(q), 2.0 ** -10
    return P, Q


@pytest.mark.parametrize("stays", [True, False])
@pytest.mark.parametrize("siblings", [11, 14])
def test_a_sibling_at_the_border_after_many_rejections(stays, siblings):
    P, Q = next(r for r in (rows(n, stays, siblings) for n in range(20000)) if r is not None)
    t = siblings + 2                                        # the root, the rejected ones, x
    up = [-1] + [0] * (siblings + 1)
    tree = torch.tensor([1] + [1 | 1 << i for i in range(1, t)], device=DEV)
    tokens = np.array([0] + [DRAFT] * siblings + [X], np.int32)
    u = np.array([0.5] * (t - 1) + [0.0], np.float32)
    out = [torch.empty(n, dtype=torch.int32, device=DEV) for n in (t, t, 1, 1, 1)]
    p, q = np.tile(P, (t, 1)), np.tile(Q, (t, 1))
    api.verify(torch.from_numpy(p).to(DEV), torch.from_numpy(tokens).to(DEV), *out, u=torch.from_numpy(u).to(DEV),
               u_next=torch.tensor([0.3], device=DEV), q=torch.from_numpy(q).to(DEV), max_new=t, tree=tree)
    sync(gl.load())
    keep, ids, nxt = OD.verify(p, q, tokens, up, u, np.float32(0.3))
    assert (len(keep) == 2) == stays
    assert out[2].tolist() == [len(keep)] and out[3].tolist() == [keep[-1]] and out[4].tolist() == [nxt]
    assert out[1].tolist() == ids + [-1] * (t - len(ids))
