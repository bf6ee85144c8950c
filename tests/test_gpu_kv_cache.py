"""gdn_kv_write and gdn_kv_read against the definition of a cached row.

Codes and scales are compared for equality: every step (the scale's division,
each quotient, its rounding) is an IEEE fp32 operation on both sides.  A value
read back is code * scale in fp32 rounded to bf16 once: the fp32 product is
formed the same way here, so it too is compared for equality.
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


def _guarded_cache(kind, n_pages, heads, page, d, debug=False):
    size = 2 if kind == "bf16" else 1
    dtype = api.KvCache.TYPES[kind][1]
    guards, parts = [], []
    for _ in "kv":
        g = Guarded(n_pages * heads * page * d * size, fill_inside=0x5A)
        guards.append(g)
        parts.append(g.view(dtype, (n_pages, heads, page, d)))
    for _ in "kv":
        if kind == "bf16":
            parts.append(None)
        else:
            g = Guarded(n_pages * heads * page * 4, fill_inside=0x5A)
            guards.append(g)
            parts.append(g.view(torch.float32, (n_pages, heads, page)))
    return guards, api.KvCache(kind, *parts, debug=debug)


def _bytes(t):
    return t.view(torch.uint8).cpu().numpy()


def _rows(rng, n, heads, d):
    x = rng.standard_normal((n, heads, d), dtype=np.float32) * np.exp(2 * rng.standard_normal((n, heads, 1))).astype(np.float32)
    x[0, 0] = 0.0
    if n > 1:
        x[1, 0] *= 1e-38                      # subnormal scale
        x[1, -1, :] = 3.0                      # every element the largest
    if n > 2:
        x[2, 0, 1:] = 0.0
        x[2, -1, ::2] = -0.5 * x[2, -1, 1]     # quotients next to a border
    return torch.from_numpy(x).to(DEV).to(torch.bfloat16)


def _expected(x, kind):
    """Codes as stored bytes' values and scales."""
    codes, scale = OS.quantise_rows(x.float().cpu().numpy(), kind)
    return codes, scale


def _values(cache, side):
    """The code values of the whole cache [slots][heads][d] and its scales [slots][heads]."""
    c = getattr(cache, side)
    v = c.float() if c.dtype != torch.float8_e4m3fn else c.view(torch.uint8).view(torch.float8_e4m3fn).float()
    v = v.transpose(1, 2).reshape(-1, cache.n_kv_heads, cache.head_dim).cpu().numpy()
    s = getattr(cache, side + "_scale")
    return v, None if s is None else s.transpose(1, 2).reshape(-1, cache.n_kv_heads).cpu().numpy()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,heads,page,form", [(1, 1, 16, "plain"), (3, 4, 64, "plain"), (77, 2, 32, "fused"),
                                               (130, 5, 128, "offset"), (41, 3, 16, "picked")])
def test_store_and_fetch(L, kind, d, n, heads, page, form):
    rng = np.random.default_rng(n + d)
    n_pages = -(-n // page) + 2
    nr = n if form != "picked" else 2 * n + 5
    k, v = _rows(rng, nr, heads, d), _rows(rng, nr, heads, d)
    if form in ("fused", "offset"):
        pad = 5 if form == "offset" else 0
        x = torch.zeros(nr, 2 * heads * d + 2 * pad, dtype=torch.bfloat16, device=DEV)
        x[:, pad:pad + heads * d] = k.reshape(nr, -1)
        x[:, pad + heads * d:pad + 2 * heads * d] = v.reshape(nr, -1)
        k, v = x[:, pad:pad + heads * d].view(nr, heads, d), x[:, pad + heads * d:pad + 2 * heads * d].view(nr, heads, d)
    rows = np.sort(rng.permutation(nr)[:n]) if form == "picked" else np.arange(n)
    slots = rng.permutation(n_pages * page)[:n].astype(np.int64)
    if n > 10:
        slots[7] = -1                          # this token goes nowhere
    guards, cache = _guarded_cache(kind, n_pages, heads, page, d)
    before = [_bytes(cache.k).copy(), _bytes(cache.v).copy()]
    sl = torch.from_numpy(slots).to(DEV)
    cache.write(k, v, sl, rows=torch.from_numpy(rows.astype(np.int32)).to(DEV) if form == "picked" else None)
    sync(L)
    assert all(g.intact() for g in guards)
    used = slots >= 0
    for i, (side, x) in enumerate((("k", k), ("v", v))):
        got, scale = _values(cache, side)
        picked = x[torch.from_numpy(rows).to(DEV)][torch.from_numpy(used).to(DEV)]
        if kind == "bf16":
            assert np.array_equal(got[slots[used]], picked.float().cpu().numpy())
        else:
            codes, s = _expected(picked, kind)
            assert np.array_equal(scale[slots[used]], s)
            assert np.array_equal(got[slots[used]], codes)
        # what no token went to is untouched
        size = 2 if kind == "bf16" else 1
        after = _bytes(getattr(cache, side)).reshape(n_pages, heads, page, d * size).transpose(0, 2, 1, 3).reshape(n_pages * page, -1)
        old = before[i].reshape(n_pages, heads, page, d * size).transpose(0, 2, 1, 3).reshape(n_pages * page, -1)
        free = np.setdiff1d(np.arange(n_pages * page), slots)
        assert np.array_equal(after[free], old[free])
    # read back, with the unstored token as zeros, contiguous and into strided rows
    for pad in (0, 8, 3):
        w = heads * d + pad
        gk, ko = guarded((n, w), torch.bfloat16, init=torch.full((n, w), 7.0, dtype=torch.bfloat16, device=DEV))
        gv, vo = guarded((n, w), torch.bfloat16, init=torch.full((n, w), 7.0, dtype=torch.bfloat16, device=DEV))
        cache.read(sl, ko[:, :heads * d].view(n, heads, d), vo[:, :heads * d].view(n, heads, d))
        sync(L)
        assert gk.intact() and gv.intact()
        for side, out in (("k", ko), ("v", vo)):
            got, scale = _values(cache, side)
            val = torch.from_numpy(got if scale is None else got * scale[..., None]).to(torch.bfloat16)
            want = torch.zeros(n, heads, d, dtype=torch.bfloat16)
            want[used] = val[torch.from_numpy(slots[used])]
            assert torch.equal(out[:, :heads * d].view(n, heads, d).cpu(), want)
            assert bool((out[:, heads * d:] == 7.0).all())


@pytest.mark.parametrize("kind", KINDS)
def test_rows_that_are_not_finite(L, kind):
    """A NaN takes code 0 and no part in the scale; an infinity makes the row's scale infinite and every code 0
    (so the row reads back as NaN); a bf16 cache keeps both as they are."""
    x = torch.ones(3, 1, 64, dtype=torch.bfloat16, device=DEV)
    x[0, 0, 3] = float("nan")
    x[1, 0, 4] = float("-inf")
    cache = api.KvCache.new(kind, 1, 1, 16, 64)
    sl = torch.arange(3, device=DEV)
    cache.write(x, x, sl)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    cache.read(sl, ko, vo)
    sync(L)
    if kind == "bf16":
        assert torch.equal(ko.view(torch.int16), x.view(torch.int16))
        return
    got, scale = _values(cache, "k")
    codes, s = OS.quantise_rows(x.float().cpu().numpy(), kind)
    assert np.array_equal(got[:3], codes) and np.array_equal(scale[:3], s)
    assert got[0, 0, 3] == 0 and np.isinf(scale[1, 0]) and not got[1].any()
    assert bool(torch.isnan(ko[1]).all()) and bool(torch.isfinite(ko[[0, 2]]).all())


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("size", [-40, 0, 55])
def test_every_quotient_of_two_mantissas(L, kind, size):
    """Rows whose largest element has each of the 128 mantissas, over elements of every mantissa and of 18 exponents
    from the largest one down: every quotient that a row of bf16 can have, but for powers of two."""
    big = np.arange(128, 256, dtype=np.float64)
    x = np.zeros((128, 18, 256), np.float64)
    x[:, :, :128] = np.minimum(np.arange(128, 256) * np.exp2(-np.arange(18.0))[:, None], big[:, None, None])
    x[:, :, 128:] = -x[:, :, :128]
    x[:, :, 0] = big[:, None]
    x = torch.from_numpy((x * 2.0 ** size).reshape(-1, 2, 256).astype(np.float32)).to(DEV).to(torch.bfloat16)
    n = x.shape[0]
    cache = api.KvCache.new(kind, n // 16, 2, 16, 256)
    cache.write(x, x, torch.arange(n, device=DEV))
    sync(L)
    codes, scale = _expected(x, kind)
    for side in "kv":
        got, s = _values(cache, side)
        assert np.array_equal(s, scale) and np.array_equal(got, codes)


@pytest.mark.parametrize("kind", KINDS)
def test_indices_out_of_range_are_skipped_and_reported(L, kind):
    heads, page, d, n = 2, 16, 128, 4
    x = torch.ones(n, heads, d, dtype=torch.bfloat16, device=DEV)
    guards, cache = _guarded_cache(kind, 2, heads, page, d)
    before = _bytes(cache.k).copy()
    ko, vo = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    for slots, rows in [([32, -1, -1, -1], None), ([1 << 60, -5, -1, -1], None), ([0, -1, -1, -1], [4, 0, 0, 0]),
                        ([0, -1, -1, -1], [-1, 0, 0, 0])]:
        sl = torch.tensor(slots, dtype=torch.int64, device=DEV)
        cache.write(x, x, sl, rows=None if rows is None else torch.tensor(rows, dtype=torch.int32, device=DEV))
        assert L.gdn_sync_status(stream(), check=False) == gl.GDN_EINDEX
        assert L.gdn_sync_status(stream(), check=False) == gl.GDN_OK
        assert np.array_equal(_bytes(cache.k), before) and all(g.intact() for g in guards)
    cache.read(torch.tensor([32, -1, 1 << 40, -9], dtype=torch.int64, device=DEV), ko, vo)
    assert L.gdn_sync_status(stream(), check=False) == gl.GDN_EINDEX
    assert not ko.any() and not vo.any()


def test_slots_past_32_bits(L):
    """A cache of more than 2^32 bytes a side: the last page's rows land where they belong."""
    heads, page, d = 8, 128, 256
    n_pages = (1 << 32) // (heads * page * d) + 3
    cache = api.KvCache.new("i8", n_pages, heads, page, d)
    rng = np.random.default_rng(5)
    x = _rows(rng, 4, heads, d)
    slots = torch.tensor([n_pages * page - 1, 0, (n_pages - 1) * page, n_pages * page - 2], device=DEV)
    cache.write(x, x, slots)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    cache.read(slots, ko, vo)
    sync(L)
    codes, s = OS.quantise_rows(x.float().cpu().numpy(), "i8")
    assert np.array_equal(cache.k[-1, :, page - 1].cpu().numpy(), codes[0])
    want = torch.from_numpy(codes.astype(np.float32) * s[..., None]).to(torch.bfloat16)
    assert torch.equal(ko.cpu(), want) and torch.equal(vo.cpu(), want)
    assert not cache.k[1].any()


def test_store_in_a_graph_and_on_another_stream(L):
    rng = np.random.default_rng(6)
    x = _rows(rng, 20, 4, 128)
    cache, other = api.KvCache.new("e4m3", 4, 4, 16, 128), api.KvCache.new("e4m3", 4, 4, 16, 128)
    sl = torch.arange(20, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.write(x, x, sl)
    sl.add_(30)
    g.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other.write(x, x, sl, stream=side)
    side.synchronize()
    sync(L)
    assert torch.equal(cache.k.view(torch.uint8), other.k.view(torch.uint8)) and torch.equal(cache.v_scale, other.v_scale)
    assert cache.k.view(torch.uint8).any()


def test_cache_wrapper_refuses(L):
    cache = api.KvCache.new("i8", 2, 2, 16, 64)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    sl = torch.arange(3, device=DEV)
    for bad in [lambda: cache.write(x, x[:2], sl), lambda: cache.write(x.float(), x, sl), lambda: cache.write(x, x, sl.int()),
                lambda: cache.write(x[:, :1], x[:, :1], sl), lambda: cache.read(sl[:2], x, x),
                lambda: cache.write(x, x, sl, rows=sl), lambda: api.KvCache("i8", cache.k, cache.v),
                lambda: api.KvCache("i4", cache.k, cache.v), lambda: api.KvCache("bf16", cache.k, cache.v),
                lambda: api.KvCache("i8", cache.k[:, :1], cache.v[:, :1], cache.k_scale, cache.v_scale)]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gl.GdnError):
        cache.write(x[:2], x[:2], sl)          # three tokens of two rows
