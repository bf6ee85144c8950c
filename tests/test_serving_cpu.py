"""CPU checks of the full-attention serving entry points: the rotation table
against its formula, the oracle's code rounding, and every refusal before a GPU
is touched."""
import ctypes
import math

import numpy as np
import pytest

from hybrid_gated_deltanet_q4k_gb300 import api
from hybrid_gated_deltanet_q4k_gb300 import lib as gl
from oracle import serving as OS


@pytest.fixture(scope="module")
def L():
    return gl.load(build=True)


@pytest.mark.parametrize("kw", [
    dict(rot=64, base=1e7), dict(rot=2, base=1e4), dict(rot=256, base=1e6, scaling="linear", factor=4.0),
    dict(rot=128, base=1e6, scaling="parts", factor=8.0, orig_len=32768, layout="interleaved"),
    dict(rot=18, base=5e5, scaling="parts", factor=2.0, orig_len=1, fast=8.0, slow=0.5),
])
def test_rope_table_holds_the_formula(L, kw):
    t = api.RopeTable(**kw).table
    args = {k: v for k, v in kw.items() if k != "layout"}
    f = OS.rope_frequencies(**args)
    got = np.array([t.step[i] for i in range(kw["rot"] // 2)], np.float64) * 2.0 ** -64 * 2 * math.pi
    assert np.all(np.abs(got - f) <= 4 * 2.0 ** -53 * f + 2.0 ** -63 * 2 * math.pi)
    assert all(t.step[i] == 0 for i in range(kw["rot"] // 2, gl.GDN_ROPE_MAX_PAIRS))
    amp = 0.1 * math.log(kw["factor"]) + 1 if kw.get("scaling") == "parts" else 1.0
    assert t.amp == np.float32(amp) and t.rot == kw["rot"]
    assert api.RopeTable(**kw, amp=0.5).table.amp == 0.5


@pytest.mark.parametrize("args", [
    (0, 0, 1e4, 0, 1.0, 0, 32.0, 1.0, 0.0), (63, 0, 1e4, 0, 1.0, 0, 32.0, 1.0, 0.0), (258, 0, 1e4, 0, 1.0, 0, 32.0, 1.0, 0.0),
    (64, 2, 1e4, 0, 1.0, 0, 32.0, 1.0, 0.0), (64, 0, 1.0, 0, 1.0, 0, 32.0, 1.0, 0.0),
    (64, 0, math.inf, 0, 1.0, 0, 32.0, 1.0, 0.0), (64, 0, math.nan, 0, 1.0, 0, 32.0, 1.0, 0.0),
    (64, 0, 1e4, 3, 1.0, 0, 32.0, 1.0, 0.0), (64, 0, 1e4, 1, 0.5, 0, 32.0, 1.0, 0.0), (64, 0, 1e4, 1, math.nan, 0, 32.0, 1.0, 0.0),
    (64, 0, 1e4, 2, 2.0, 0, 32.0, 1.0, 0.0), (64, 0, 1e4, 2, 2.0, 100, 1.0, 1.0, 0.0), (64, 0, 1e4, 2, 2.0, 100, 32.0, 0.0, 0.0),
    (64, 0, 1e4, 0, 1.0, 0, 32.0, 1.0, -1.0),
])
def test_rope_make_refuses(L, args):
    t = gl.GdnRopeTable()
    assert L.gdn_rope_make(*args, ctypes.byref(t), check=False) == gl.GDN_EINVAL
    assert "gdn_rope_make" in L.last_error()
    assert t.rot == 0


A = 0x10000   # an aligned address that no check reads


def test_rope_refuses(L):
    t = api.RopeTable(64)._ref
    ok = [t, A, 4, 128, A, 512, 4, A, 512, A, 256, 2, A, 256, 0]
    for i, bad in [(0, None), (1, 0), (1, A + 2), (2, -1), (2, 1 << 31), (3, 63), (3, 62), (3, 514), (4, 0), (4, A + 1),
                   (5, 511), (6, 0), (6, 257), (7, 0), (8, 511), (9, 0), (10, 255), (11, -1), (11, 257), (12, 0), (13, 100)]:
        args = list(ok)
        args[i] = bad
        assert L.gdn_rope(*args, check=False) == gl.GDN_EINVAL, (i, bad)
    in_place = list(ok)
    in_place[8] = 520                      # in place with another stride
    assert L.gdn_rope(*in_place, check=False) == gl.GDN_EINVAL
    raw = gl.GdnRopeTable()                # not from gdn_rope_make
    assert L.gdn_rope(ctypes.byref(raw), *ok[1:], check=False) == gl.GDN_EINVAL
    empty = list(ok)
    empty[2] = 0
    assert L.gdn_rope(*empty, check=False) == gl.GDN_OK


def _cache(**kw):
    c = gl.GdnKvCache()
    base = dict(dtype=gl.GDN_KV_I8, n_kv_heads=4, head_dim=128, page_tokens=64, n_pages=10, k=A, v=A, k_scale=A, v_scale=A)
    for name, value in {**base, **kw}.items():
        setattr(c, name, value)
    return c


BAD_CACHES = [dict(dtype=3), dict(n_kv_heads=0), dict(n_kv_heads=257), dict(head_dim=96), dict(page_tokens=8),
              dict(page_tokens=48), dict(n_pages=0), dict(n_pages=1 << 30), dict(k=0), dict(v=0), dict(k=A + 64), dict(k_scale=0),
              dict(v_scale=0), dict(v_scale=A + 8), dict(dtype=gl.GDN_KV_BF16), dict(dtype=gl.GDN_KV_BF16, k_scale=0)]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_cache_descriptor_refusals(L, kw):
    c = ctypes.byref(_cache(**kw))
    assert L.gdn_kv_write(c, A, 512, A, 512, 4, 0, A, 4, 0, check=False) == gl.GDN_EINVAL
    assert L.gdn_kv_read(c, A, 4, A, 512, A, 512, 0, check=False) == gl.GDN_EINVAL
    assert L.gdn_attn_cache_workspace_size(c, 4, 8) == 0
    assert L.gdn_attn_cache(c, A, 1024, 0, 4, 1, 0, A, 8, 8, A, 4, 8, 0.0, A, 1024, A, 1 << 30, 0, check=False) == gl.GDN_EINVAL
    assert "gdn_attn_cache" in L.last_error()


def test_store_and_fetch_refuse(L):
    c = ctypes.byref(_cache())
    ok = [c, A, 512, A, 512, 4, 0, A, 4, 0]
    for i, bad in [(0, None), (1, 0), (1, A + 1), (2, 511), (3, 0), (4, 0), (5, -1), (5, 3), (6, A + 2), (7, 0), (7, A + 4),
                   (8, -1), (8, 1 << 31)]:
        args = list(ok)
        args[i] = bad
        assert L.gdn_kv_write(*args, check=False) == gl.GDN_EINVAL, (i, bad)
    assert L.gdn_kv_write(c, A, 512, A, 512, 4, 0, A, 0, 0, check=False) == gl.GDN_OK
    ok = [c, A, 4, A, 512, A, 512, 0]
    for i, bad in [(0, None), (1, 0), (1, A + 4), (2, -1), (2, 1 << 31), (3, 0), (3, A + 1), (4, 511), (5, 0), (6, 1)]:
        args = list(ok)
        args[i] = bad
        assert L.gdn_kv_read(*args, check=False) == gl.GDN_EINVAL, (i, bad)
    assert L.gdn_kv_read(c, A, 0, A, 512, A, 512, 0, check=False) == gl.GDN_OK


def test_attention_refuses(L):
    c = ctypes.byref(_cache())
    need = L.gdn_attn_cache_workspace_size(c, 8, 8)
    assert need > 0
    ok = [c, A, 1024, A, 8, 2, 0, A, 8, 8, A, 4, 8, 0.0, A, 1024, A, need, 0]
    for i, bad in [(0, None), (1, 0), (1, A + 8), (2, 1016), (2, 1028), (3, A + 2), (4, -1), (4, 9), (5, 0), (5, 65), (6, A + 4),
                   (7, 0), (7, A + 2), (8, 7), (9, 0), (9, 1 << 26), (10, 0), (10, A + 1), (11, 0), (11, 257), (12, 0), (12, 6),
                   (12, 68), (13, math.nan), (13, math.inf), (14, 0), (14, A + 2), (15, 1020), (16, 0), (16, A + 128)]:
        args = list(ok)
        args[i] = bad
        if (i, bad) == (9, 1 << 26):
            args[8] = bad
        assert L.gdn_attn_cache(*args, check=False) == gl.GDN_EINVAL, (i, bad)
    args = list(ok)
    args[3] = 0                            # no offsets: max_q tokens for each sequence
    args[4] = 7
    assert L.gdn_attn_cache(*args, check=False) == gl.GDN_EINVAL
    args = list(ok)
    args[17] = need - 1
    assert L.gdn_attn_cache(*args, check=False) == gl.GDN_ENOMEM
    args = list(ok)
    args[4] = 0
    assert L.gdn_attn_cache(*args, check=False) == gl.GDN_OK
    for n, h in [(0, 8), (64 * 256 + 1, 8), (8, 6), (8, 68), (8, 0)]:
        assert L.gdn_attn_cache_workspace_size(c, n, h) == 0


def test_oracle_code_rounding():
    """e4m3 rounding against the list of all its values: nearest, ties to the even code."""
    vals = []
    for b in range(127):
        e, m = b >> 3, b & 7
        vals.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    vals = np.array(vals)
    rng = np.random.default_rng(0)
    mids = (vals[1:] + vals[:-1]) / 2
    x = np.concatenate([rng.uniform(0, 448, 2000), np.exp(rng.uniform(-8, 6, 2000)), vals, mids, mids * (1 + 1e-6)])
    x = np.minimum(x, 448.0)
    x = np.concatenate([[448.0], x, -x]).astype(np.float32)
    codes, scale = OS.quantise_rows(x[None], "e4m3")
    assert scale[0] == 1.0
    for xi, ci in zip(x.astype(np.float64), codes[0]):
        d = np.abs(vals - abs(xi))
        best = np.flatnonzero(d == d.min())
        want = vals[best[0]] if len(best) == 1 else vals[best[best % 2 == 0][0]]
        assert abs(ci) == want and (ci == 0 or (ci > 0) == (xi > 0))
    assert np.array_equal(OS.quantise_rows(np.zeros((2, 8)), "i8")[0], np.zeros((2, 8)))


def test_header_structs_match(tmp_path):
    import os
    import shutil
    import subprocess
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    lines = []
    for name, cls in (("gdn_rope_table", gl.GdnRopeTable), ("gdn_kv_cache", gl.GdnKvCache)):
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_]
    for name in ("GDN_KV_BF16", "GDN_KV_I8", "GDN_KV_E4M3", "GDN_MAX_NEW", "GDN_ROPE_HALF", "GDN_ROPE_INTERLEAVED",
                 "GDN_ROPE_PLAIN", "GDN_ROPE_LINEAR", "GDN_ROPE_PARTS", "GDN_ROPE_MAX_PAIRS"):
        lines.append(f'printf("{name} %zu\\n", (size_t){name});')
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gdn.h"\nint main(void) {\n' + "\n".join(lines)
                   + "\nreturn 0;\n}\n")
    subprocess.run([gcc, "-std=c99", "-I", inc, str(src), "-o", str(tmp_path / "s")], check=True)
    out = subprocess.run([str(tmp_path / "s")], check=True, capture_output=True, text=True).stdout.splitlines()
    got = {k: int(v) for k, v in (line.split() for line in out)}
    for name, cls in (("gdn_rope_table", gl.GdnRopeTable), ("gdn_kv_cache", gl.GdnKvCache)):
        assert got[name] == ctypes.sizeof(cls)
        for f in cls._fields_:
            assert got[f"{name}.{f[0]}"] == getattr(cls, f[0]).offset
    for name, v in got.items():
        if name.startswith("GDN_"):
            assert getattr(gl, name) == v
