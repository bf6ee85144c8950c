"""gdn_rope against the fp64 formula.

Tolerance per element, from the arithmetic: the output is rounded to bf16 once
(half a step: 2^-8 of the value); before that the angle is off by less than
4e-7 (a 24-bit fraction of half a turn, and sincospif), the sine and cosine by
2 units of 2^-24, and the two products and their sum by 3 of 2^-24, each
relative to |a| + |b|: below 1e-6 amp (|a| + |b|) together.
"""
import numpy as np
import pytest
import torch

from hybrid_gated_deltanet_q4k_gb300 import api
from hybrid_gated_deltanet_q4k_gb300 import lib as gl
from oracle import serving as OS

from gpu_util import DEV, guarded, stream, sync

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return gl.load(build=True)


def _bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).to(DEV).to(torch.bfloat16)


def _check(got, x, pos, table, freq, layout):
    x, got = x.double().cpu().numpy(), got.double().cpu().numpy()
    amp, rot, half = table.amp, table.rot, table.rot // 2
    ref = OS.rope(x, pos, freq, layout, amp)
    if layout == "half":
        pair = np.abs(x[..., :half]) + np.abs(x[..., half:rot])
        pair = np.concatenate([pair, pair], -1)
    else:
        pair = np.repeat(np.abs(x[..., 0:rot:2]) + np.abs(x[..., 1:rot:2]), 2, -1)
    assert np.array_equal(got[..., rot:], x[..., rot:])
    assert np.all(np.abs(got - ref)[..., :rot] <= 2.0 ** -8 * np.abs(ref[..., :rot]) + 1e-6 * amp * pair)


CASES = [   # n, hq, hk, d, table, lowest and highest position
    (1, 16, 4, 256, dict(rot=64, base=1e7), 0, 40000),
    (300, 16, 4, 256, dict(rot=64, base=1e7), 0, 262144),
    (7, 3, 1, 128, dict(rot=128, base=1e6, layout="interleaved", scaling="parts", factor=8.0, orig_len=32768), 0, 2000000),
    (65, 5, 5, 64, dict(rot=32, layout="interleaved", base=1e4), -50, 50),
    (33, 2, 1, 128, dict(rot=128, base=5e5, scaling="linear", factor=4.0), 2 ** 31 - 40, 2 ** 31 - 1),
    (9, 4, 0, 96, dict(rot=96), 0, 100),
    (5, 3, 2, 66, dict(rot=18, layout="half"), 0, 9000),              # nothing a multiple of a vector
    (5, 3, 2, 130, dict(rot=34, layout="interleaved"), -(2 ** 31), 2 ** 31 - 1),
    (3, 1, 1, 2, dict(rot=2), 0, 7),
    (2, 2, 2, 512, dict(rot=256, base=1e6), 0, 500000),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("form", ["out", "in_place", "fused", "offset"])
def test_rope_matches_the_formula(L, case, form):
    n, hq, hk, d, kw, lo, hi = case
    rng = np.random.default_rng(n + d)
    t = api.RopeTable(**kw)
    freq = OS.rope_frequencies(**{k: v for k, v in kw.items() if k in ("rot", "base", "scaling", "factor", "orig_len")}
                               if "base" in kw else dict(kw_base(kw)))
    pos = rng.integers(lo, hi, size=n, endpoint=True).astype(np.int32)
    pos[0], pos[-1] = lo, hi
    if form in ("fused", "offset"):         # columns of one projection; "offset": not 16-byte aligned
        extra = 3 if form == "offset" else 0
        x = _bf16(rng, n, (hq + 2 * hk) * d + 2 * extra)
        q = x[:, extra:extra + hq * d].view(n, hq, d)
        k = x[:, extra + hq * d:extra + (hq + hk) * d].view(n, hk, d) if hk else None
        keep = x.clone()
    else:
        q, k = _bf16(rng, n, hq, d), _bf16(rng, n, hk, d) if hk else None
    q0, k0 = q.clone(), k.clone() if hk else None
    p = torch.from_numpy(pos).to(DEV)
    if form == "out" or form == "offset":
        gq, qo = guarded((n, hq, d), torch.bfloat16)
        gk, ko = guarded((n, max(hk, 1), d), torch.bfloat16)
        t.apply(p, q, k, qo, ko if hk else None)
        sync(L)
        assert gq.intact() and gk.intact()
        assert torch.equal(q, q0)
    else:
        t.apply(p, q, k)
        sync(L)
        qo, ko = q, k
        if form == "fused" and hk:
            assert torch.equal(x[:, (hq + hk) * d:], keep[:, (hq + hk) * d:])
    _check(qo, q0, pos, t.table, freq, kw.get("layout", "half"))
    if hk:
        _check(ko, k0, pos, t.table, freq, kw.get("layout", "half"))


def kw_base(kw):
    return {"base": 10000.0, **{k: v for k, v in kw.items() if k in ("rot", "scaling", "factor", "orig_len")}}


def test_rope_keeps_relative_angles_and_specials(L):
    """Turning by p and then by -p gives the input back (two roundings); infinities and NaN stay in their pair."""
    rng = np.random.default_rng(1)
    n, d = 40, 128
    t = api.RopeTable(128, base=1e6)
    p = torch.arange(1000, 1000 + n, dtype=torch.int32, device=DEV)
    q = _bf16(rng, n, 4, d)
    y, z = torch.empty_like(q), torch.empty_like(q)
    t.apply(p, q, None, y)
    t.apply(-p, y, None, z)
    sync(L)
    pair = (q[..., :64].abs() + q[..., 64:].abs()).repeat(1, 1, 2).double()
    assert bool(((z.double() - q.double()).abs() <= 3 * 2.0 ** -8 * pair).all())
    q[3, 1, 5] = float("inf")
    q[4, 2, 64 + 7] = float("nan")
    t.apply(p, q, None, z)
    sync(L)
    bad = ~torch.isfinite(z)
    want = torch.zeros_like(bad)
    want[3, 1, [5, 69]] = True
    want[4, 2, [7, 71]] = True
    assert torch.equal(bad, want)
    assert torch.equal(z[~want], y[~want])


def test_rope_on_another_stream_and_in_a_graph(L):
    rng = np.random.default_rng(2)
    n = 50
    t = api.RopeTable(64, base=1e7)
    q, k = _bf16(rng, n, 16, 256), _bf16(rng, n, 4, 256)
    p = torch.arange(n, dtype=torch.int32, device=DEV)
    want_q, want_k = torch.empty_like(q), torch.empty_like(k)
    t.apply(p, q, k, want_q, want_k)
    sync(L)
    side = torch.cuda.Stream()
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    side.wait_stream(torch.cuda.current_stream())
    t.apply(p, q, k, qo, ko, stream=side)
    side.synchronize()
    assert torch.equal(qo, want_q) and torch.equal(ko, want_k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t.apply(p, q, k, qo, ko)
    p.add_(7)
    g.replay()
    t.apply(p, q, k, want_q, want_k)
    sync(L)
    assert torch.equal(qo, want_q) and torch.equal(ko, want_k)


def test_rope_wrapper_refuses(L):
    t = api.RopeTable(64)
    q = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device=DEV)
    p = torch.zeros(4, dtype=torch.int32, device=DEV)
    for bad in [lambda: t.apply(p[:3], q), lambda: t.apply(p.long(), q), lambda: t.apply(p, q.float()),
                lambda: t.apply(p, q.transpose(0, 1)), lambda: t.apply(p, q, q[:3]), lambda: t.apply(p, q, None, q[:, :1]),
                lambda: api.RopeTable(64, layout="other")]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gl.GdnError):
        t.apply(p, q[..., :32].contiguous())
    assert stream() is not None
