"""The cache attention's bounded waits: a copy that never comes surfaces as GDN_ETIMEOUT, and the next call is fine.

The first copy of every CTA is withheld and the limit is 1 ms; nothing faults.  What the call leaves in o and the
workspace means nothing, but it stays inside them.
"""
import ctypes

import numpy as np
import pytest
import torch

from hybrid_gated_deltanet_q4k_gb300 import lib as gl

from gpu_util import Guarded, guarded, stream, sync
from test_gpu_attn_cache import Case, _tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return gl.load(build=True)


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nq", [[1, 1, 1], [40, 1, 17]], ids=["few", "many"])
def test_a_wait_runs_out_then_the_next_call_is_fine(L, kind, d, nq):
    lens = [3000, 70, 900]
    c = Case(kind, d, 32, 2, 2, lens, nq, tree=_tree(np.random.default_rng(0), nq), seed=23)
    want = c.run(L)
    sync(L)
    c.check(want)
    T, nbytes = int(c.cu[-1]), c.cache.attend_workspace_bytes(int(c.cu[-1]), c.hq)
    go, o = guarded((T, c.hq, d), torch.bfloat16)
    gw = Guarded(nbytes)
    lens_d, cu, tree = c.dev
    args = (ctypes.byref(c.cache.struct), gl.ptr(c.q), c.hq * d, gl.ptr(cu), T, max(nq), gl.ptr(tree), gl.ptr(c.table),
            c.table.shape[1], c.table.shape[1], gl.ptr(lens_d), len(lens), c.hq, 0.0, gl.ptr(o), c.hq * d,
            gl.ptr(gw.view(torch.uint8, (nbytes,))), nbytes)
    assert L.gdn_test_attn_cache_wait_timeout(*args, 10, stream(), check=False) == gl.GDN_EINVAL    # limit below 1 us
    assert L.gdn_test_attn_cache_wait_timeout(*args, 200_000_000, stream(), check=False) == gl.GDN_EINVAL
    for _ in range(2):
        L.gdn_test_attn_cache_wait_timeout(*args, 1_000_000, stream())
        assert L.gdn_sync_status(stream(), check=False) == gl.GDN_ETIMEOUT
        assert "cache attention" in L.last_error()
        assert L.gdn_sync_status(stream(), check=False) == gl.GDN_OK
        assert go.intact() and gw.intact()
        assert torch.equal(c.run(L), want)
        sync(L)
