"""gdn_rope over enough rows that a thread takes two or four of them, against the fp64 formula.

A block has 256 / (head_dim / 16) rows for each that a thread takes; a thread takes four where that leaves 608 blocks,
two where two do.  The tolerance is that of the small cases: 2^-8 of the value and 1e-6 amp (|a| + |b|).
"""
import numpy as np
import pytest
import torch

from hybrid_gated_deltanet_q4k_gb300 import api
from hybrid_gated_deltanet_q4k_gb300 import lib as gl
from oracle import serving as OS

from gpu_util import DEV, guarded, sync
from test_gpu_rope import _bf16, _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return gl.load(build=True)


def _rows_per_thread(n, heads, d):
    per = 256 // (d // 16)
    return next(k for k in (4, 2, 1) if k == 1 or -(-n * heads // (per * k)) >= 608)


CASES = [   # rows a thread, n, hq, hk, d, table
    (1, 971, 16, 4, 256, dict(rot=64, base=1e7)),
    (2, 1001, 16, 4, 256, dict(rot=64, base=1e7)),
    (4, 2501, 16, 4, 256, dict(rot=64, base=1e7)),
    (2, 1103, 32, 8, 128, dict(rot=128, base=1e6, layout="interleaved", scaling="parts", factor=8.0, orig_len=32768)),
    (4, 5001, 32, 8, 128, dict(rot=128, base=1e6, layout="interleaved", scaling="parts", factor=8.0, orig_len=32768)),
    (4, 4999, 33, 0, 64, dict(rot=32, base=1e4, scaling="linear", factor=2.0)),
    (2, 20011, 1, 1, 128, dict(rot=128, base=1e6)),
    (4, 777, 12, 13, 512, dict(rot=256, base=1e6, layout="interleaved")),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("form", ["out", "in_place", "fused", "sixteen"])
def test_many_rows_match_the_formula(L, case, form):
    """"sixteen": rows that start on 16 bytes and not on 32."""
    per, n, hq, hk, d, kw = case
    assert _rows_per_thread(n, hq + hk, d) == per
    rng = np.random.default_rng(n + d)
    t = api.RopeTable(**kw)
    freq = OS.rope_frequencies(**{k: v for k, v in kw.items() if k != "layout"})
    pos = rng.integers(0, 1000000, size=n).astype(np.int32)
    pos[:2], pos[-1] = (0, 1), 1000000
    p = torch.from_numpy(pos).to(DEV)
    if form in ("fused", "sixteen"):
        pad = 8 if form == "sixteen" else 0
        x = _bf16(rng, n, (hq + 2 * hk) * d + 2 * pad)
        q = x[:, pad:pad + hq * d].view(n, hq, d)
        k = x[:, pad + hq * d:pad + (hq + hk) * d].view(n, hk, d) if hk else None
    else:
        q, k = _bf16(rng, n, hq, d), _bf16(rng, n, hk, d) if hk else None
    q0, k0 = q.clone(), k.clone() if hk else None
    if form == "in_place":
        t.apply(p, q, k)
        sync(L)
        qo, ko = q, k
    else:
        gq, qo = guarded((n, hq, d), torch.bfloat16)
        gk, ko = guarded((n, max(hk, 1), d), torch.bfloat16)
        t.apply(p, q, k, qo, ko if hk else None)
        sync(L)
        assert gq.intact() and gk.intact() and torch.equal(q, q0)
    _check(qo, q0, pos, t.table, freq, kw.get("layout", "half"))
    if hk:
        _check(ko, k0, pos, t.table, freq, kw.get("layout", "half"))
