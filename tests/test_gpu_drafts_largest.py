"""A token whose u is next to the largest fp32 number: what does not descend from it has its own results.

u_2 = b v = 3.4028e38 in one row, above 2^128 - 2^116, from where the nearest number of 11 bits is infinite.  Tolerances are
those of the delta rule's other tests (2^-18 of the sums of absolute values, half a step of fp16)."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, f32_dev, stream
from hybrid_gated_deltanet_q4k_gb300 import lib as gl
from oracle import drafts as OD
from test_gpu_drafts import Case, f16_bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,hk,hv,d,more", [(12, 1, 2, 64, 1), (30, 1, 2, 128, 0), (7, 16, 64, 64, 3)])
def test_u_near_the_largest_number_stays_on_its_branch(n, hk, hv, d, more):
    c = Case(hk, hv, d, [n] * (1 + more), "tree", seed=21)
    c.state[0, 0, 5], c.v[2, 0, 5], c.b[2, 0] = 0.0, 2.0 ** 15, 3.4028e38 / 2 ** 15
    for i in OD.path(c.up[0], 2)[:-1]:
        c.v[i, 0, 5] = 0.0                                  # row 5 holds nothing before token 2
    with np.errstate(all="ignore"):
        ru, ro, eu, eo = c.oracle_delta()
    o, u = torch.empty(c.t, hv, d, dtype=torch.float16, device=DEV), torch.empty(c.t, hv, d, device=DEV)
    c.dl.delta_tree(c.qkv(), f32_dev(c.log_a), f32_dev(c.b), f32_dev(c.state), o, u, **c.more())
    assert c.dl.lib.gdn_sync_status(stream(), check=False) == gl.GDN_ERANGE
    assert abs(ru[2, 0, 5] - 3.4028e38) < 1e33 and abs(float(u[2, 0, 5]) - 3.4028e38) <= 2.0 ** -18 * 3.4028e38
    fine = np.ones(c.t, bool)
    fine[[i for i in range(n) if 2 in OD.path(c.up[0], i)]] = False
    got_u, got_o = u.double().cpu().numpy()[fine], o.double().cpu().numpy()[fine]
    assert fine[3:n].any() and np.isfinite(ro[fine]).all()
    assert (np.abs(got_u - ru[fine]) <= 2.0 ** -18 * eu[fine]).all()
    assert (np.abs(got_o - ro[fine]) <= 2.0 ** -18 * eo[fine] + f16_bound(ro[fine])).all()
