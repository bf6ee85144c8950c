"""Slots given twice in one store, which the contract excludes: they disturb no other slot."""
import numpy as np
import pytest
import torch

from hybrid_gated_deltanet_q4k_gb300 import lib as gl

from gpu_util import DEV, sync
from test_gpu_kv_cache import _bytes, _guarded_cache, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return gl.load(build=True)


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("n,heads,d", [(40, 2, 64), (700, 3, 256)])
def test_a_slot_given_twice_disturbs_no_other(L, kind, n, heads, d):
    rng = np.random.default_rng(n)
    page = 32
    n_pages = -(-n // page) + 2
    k, v = _rows(rng, n, heads, d), _rows(rng, n, heads, d)
    slots = rng.permutation(n_pages * page)[:n].astype(np.int64)
    twice = slots.copy()
    twice[n // 2] = twice[1]                 # in one block of the store, and in two far apart
    twice[-1] = twice[-2]
    free = [slots[n // 2], slots[-1]]        # what these tokens' own slots would have been
    shared = [slots[1], slots[-2]]
    caches = []
    for s in (slots, twice):
        guards, cache = _guarded_cache(kind, n_pages, heads, page, d)
        cache.write(k, v, torch.from_numpy(s).to(DEV))
        sync(L)
        assert all(g.intact() for g in guards)
        caches.append(cache)
    keep = np.setdiff1d(np.arange(n_pages * page), free + shared)
    for name in ("k", "v") if kind == "bf16" else ("k", "v", "k_scale", "v_scale"):
        a, b = (_bytes(getattr(c, name)).reshape(n_pages, heads, page, -1).transpose(0, 2, 1, 3).reshape(n_pages * page, -1)
                for c in caches)
        assert np.array_equal(a[keep], b[keep])
        assert bool((b[free] == 0x5A).all())  # nothing was stored there
