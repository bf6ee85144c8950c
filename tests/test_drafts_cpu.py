"""Drafted tokens without a GPU: the oracle against closed forms, and every refusal of the calls."""
import ctypes

import numpy as np
import pytest
import torch

from hybrid_gated_deltanet_q4k_gb300 import api
from hybrid_gated_deltanet_q4k_gb300 import lib as gl
from hybrid_gated_deltanet_q4k_gb300 import synth
from oracle import drafts as OD

A = 0x10000          # an aligned address that no check dereferences


@pytest.fixture(scope="module")
def L():
    return gl.load(build=True)


def _layer(**over):
    spec = synth.SPECS["tiny_f32"]
    s = gl.make_layer_struct(spec, {k: None for k in ("w_in", "w_out", "conv_w", "A_log", "dt_bias", "norm_w")})
    for name in ("w_in", "w_out", "conv_w", "A_log", "dt_bias", "norm_w"):
        setattr(s, name, A)
    for k, v in over.items():
        setattr(s, k, v)
    return s


def test_a_branch_equals_its_path_alone():
    """What the tree's tokens give is what each path gives as a chain, and the commit is the state at its end."""
    rng = np.random.default_rng(0)
    n, d = 9, 8
    up = [-1, 0, 0, 1, 1, 2, 4, 6, 2]
    q, k, v = rng.normal(size=(3, n, d)) * 0.4
    la, b, s0 = -rng.random(n), rng.random(n), rng.normal(size=(d, d))
    u, o, _, _ = OD.delta(q, k, v, la, b, s0, up)
    for i in range(n):
        p = OD.path(up, i)
        uc, oc, _, _ = OD.delta(q[p], k[p], v[p], la[p], b[p], s0, list(range(-1, len(p) - 1)))
        assert np.allclose(u[i], uc[-1], rtol=1e-12, atol=1e-12) and np.allclose(o[i], oc[-1], rtol=1e-12, atol=1e-12)
        s, _ = OD.commit(k, u, la, s0, up, i)
        assert np.allclose(s @ q[i], o[i], rtol=1e-12, atol=1e-12)


def test_the_residual_telescopes():
    """max(0, p - (Z0 + Z1 + ..) q) is the residual taken and normalised time after time."""
    rng = np.random.default_rng(1)
    p, q = rng.dirichlet(np.ones(50)), rng.dirichlet(np.ones(50))
    r, c0, z = p.copy(), 0.0, 1.0
    for _ in range(4):
        r = np.maximum(r - q, 0)
        r /= r.sum()
        c0 += z
        z = np.maximum(p - c0 * q, 0).sum()
        assert np.allclose(np.maximum(p - c0 * q, 0) / z, r, rtol=1e-9, atol=1e-15)


def test_words_give_parents():
    assert OD.parents(3) == [-1, 0, 1]
    assert OD.parents(4, [1, 3, 5, 0b1101]) == [-1, 0, 0, 2]      # bits from the token itself on do not matter
    assert OD.parents(2, [0, (1 << 64) - 1]) == [-1, 0]


# ---------------------------------------------------------------- refusals of the C entry points

def _conv(L, s=None, **o):
    a = dict(qkvz=A, ld=512, ba=A, ld_ba=4, state=A, cu=A, n=8, most=4, tree=0, seqs=2, qkv=A, la=A, b=A)
    a.update(o)
    s = s or _layer()
    return L.gdn_conv_tree(ctypes.byref(s), a["qkvz"], a["ld"], a["ba"], a["ld_ba"], a["state"], a["cu"], a["n"], a["most"], a["tree"],
                           a["seqs"], a["qkv"], a["la"], a["b"], 0, check=False)


def _delta(L, s=None, **o):
    a = dict(qkv=A, la=A, b=A, state=A, cu=A, n=8, most=4, tree=0, seqs=2, o=A, delta=A)
    a.update(o)
    s = s or _layer()
    return L.gdn_delta_tree(ctypes.byref(s), a["qkv"], a["la"], a["b"], a["state"], a["cu"], a["n"], a["most"], a["tree"], a["seqs"],
                            a["o"], a["delta"], 0, check=False)


def _commit(L, s=None, **o):
    a = dict(qkv=A, la=A, delta=A, cu=A, n=8, most=4, tree=0, seqs=2, node=A, i=A, o=A, qkvz=A, ld=512, ci=A, co=A)
    a.update(o)
    s = s or _layer()
    return L.gdn_delta_commit(ctypes.byref(s), a["qkv"], a["la"], a["delta"], a["cu"], a["n"], a["most"], a["tree"], a["seqs"], a["node"],
                              a["i"], a["o"], a["qkvz"], a["ld"], a["ci"], a["co"], 0, check=False)


def _verify(L, **o):
    a = dict(dtype=0, p=A, ld_p=100, q=A, ld_q=100, vocab=100, tokens=A, cu=A, n=8, most=4, tree=0, seqs=2, u=A, u_next=A, rows=A, ids=A,
             count=A, node=A, next=A)
    a.update(o)
    return L.gdn_verify(*a.values(), 0, check=False)


def _pages(**o):
    a = dict(page_tokens=16, max_blocks=10, n_pages=40, block_table=A, ld_table=10, n_blocks=A, free_pages=A, n_free=A)
    a.update(o)
    return gl.GdnKvPages(*a.values())


def _extend(L, pages=None, **o):
    a = dict(lens=A, new=A, seqs=2, tree=0, most=8, after=A, cu=A, pos=A, slots=A)
    a.update(o)
    p = pages or _pages()
    return L.gdn_kv_extend(ctypes.byref(p), *a.values(), 0, check=False)


DRAFTS = [dict(seqs=0), dict(seqs=gl.GDN_MAX_SEQS + 1), dict(most=0), dict(most=gl.GDN_MAX_NEW + 1), dict(n=-1), dict(n=9),
          dict(cu=0, n=7), dict(cu=A + 2), dict(tree=A + 4)]


@pytest.mark.parametrize("bad", DRAFTS + [dict(qkvz=0), dict(qkvz=A + 4), dict(ld=383), dict(ld=514), dict(state=0), dict(state=A + 1),
                                          dict(qkv=0), dict(qkv=A + 8), dict(ba=0), dict(ba=A + 2), dict(ld_ba=3), dict(la=0), dict(b=0)])
def test_conv_tree_refuses(L, bad):
    assert _conv(L, **bad) == gl.GDN_EINVAL and L.last_error()


@pytest.mark.parametrize("bad", DRAFTS + [dict(qkv=0), dict(la=0), dict(b=0), dict(state=0), dict(o=0), dict(delta=0), dict(qkv=A + 8),
                                          dict(state=A + 8), dict(o=A + 8), dict(delta=A + 8), dict(la=A + 2), dict(b=A + 1)])
def test_delta_tree_refuses(L, bad):
    assert _delta(L, **bad) == gl.GDN_EINVAL and L.last_error()


@pytest.mark.parametrize("bad", DRAFTS + [dict(node=0), dict(node=A + 2), dict(i=0), dict(o=0), dict(i=A + 8), dict(o=A + 4), dict(qkv=0),
                                          dict(la=0), dict(delta=0), dict(ld=383), dict(ci=0), dict(co=0), dict(ci=A + 2),
                                          dict(qkvz=0), dict(qkvz=A + 1)])
def test_commit_refuses(L, bad):
    assert _commit(L, **bad) == gl.GDN_EINVAL and L.last_error()


@pytest.mark.parametrize("bad", DRAFTS + [dict(dtype=2), dict(dtype=-1), dict(vocab=0), dict(vocab=1 << 29), dict(ld_p=99), dict(ld_q=99),
                                          dict(p=0), dict(p=A + 2), dict(q=A + 2), dict(tokens=0), dict(rows=0), dict(ids=0), dict(count=0),
                                          dict(node=0), dict(next=0), dict(u=0), dict(u_next=0), dict(u=0, u_next=0), dict(count=A + 2)])
def test_verify_refuses(L, bad):
    assert _verify(L, **bad) == gl.GDN_EINVAL and L.last_error()


@pytest.mark.parametrize("bad", [dict(seqs=0), dict(seqs=257), dict(most=-1), dict(most=1 << 31), dict(lens=0), dict(new=0), dict(after=0),
                                 dict(cu=0), dict(pos=0), dict(slots=0), dict(slots=A + 4), dict(tree=A + 4), dict(lens=A + 2)])
def test_extend_refuses(L, bad):
    assert _extend(L, **bad) == gl.GDN_EINVAL and L.last_error()


@pytest.mark.parametrize("bad", [dict(page_tokens=8), dict(page_tokens=48), dict(max_blocks=0), dict(max_blocks=1 << 27), dict(ld_table=9),
                                 dict(n_pages=0), dict(n_pages=1 << 31), dict(block_table=0), dict(n_blocks=0), dict(free_pages=0), dict(n_free=0),
                                 dict(n_free=A + 2)])
def test_pages_are_checked(L, bad):
    assert _extend(L, _pages(**bad)) == gl.GDN_EINVAL and L.last_error()
    p = _pages(**bad)
    assert L.gdn_kv_trim(ctypes.byref(p), A, 2, 0, check=False) == gl.GDN_EINVAL


def test_null_structs_and_keep(L):
    assert L.gdn_kv_extend(0, A, A, 1, 0, 1, A, A, A, A, 0, check=False) == gl.GDN_EINVAL
    p = _pages()
    assert L.gdn_kv_trim(ctypes.byref(p), 0, 2, 0, check=False) == gl.GDN_EINVAL
    assert L.gdn_delta_tree(0, A, A, A, A, A, 1, 1, 0, 1, A, A, 0, check=False) == gl.GDN_EINVAL


def test_no_tokens_is_nothing_to_do(L):
    """No launch is made, so this needs no GPU."""
    assert _conv(L, n=0, qkvz=0, qkv=0, state=0) == gl.GDN_OK
    assert _delta(L, n=0, qkv=0, o=0, delta=0, state=0) == gl.GDN_OK


def test_the_layer_is_checked(L):
    bad = _layer(n_v_heads=3)
    assert _conv(L, bad) == gl.GDN_EINVAL and _delta(L, bad) == gl.GDN_EINVAL and _commit(L, bad) == gl.GDN_EINVAL


def test_pages_struct_layout():
    """Field offsets as the header's struct has them on both machines (natural alignment)."""
    off = {f: getattr(gl.GdnKvPages, f).offset for f, _ in gl.GdnKvPages._fields_}
    assert off == dict(page_tokens=0, max_blocks=4, n_pages=8, block_table=16, ld_table=24, n_blocks=32, free_pages=40, n_free=48)
    assert ctypes.sizeof(gl.GdnKvPages) == 56


# ---------------------------------------------------------------- refusals of the wrappers

def test_wrappers_refuse_host_memory(L):
    f32, i32 = torch.zeros(8, 4), torch.zeros(8, dtype=torch.int32)
    one = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="p"):
        api.verify(f32, i32, i32, i32, one, one, one, max_new=4)
    with pytest.raises(ValueError, match="CUDA device"):
        api.KvPages(16, torch.zeros(2, 4, dtype=torch.int32), one, i32, torch.zeros(1, dtype=torch.int32))
    dl = api.DeviceLayer.__new__(api.DeviceLayer)
    dl.lib, dl._dll, dl._sizes, dl._struct = L, L.dll, (384, 2, 64), _layer()
    st, t = torch.zeros(2, 2, 64, 64), 3
    qkv, g, o, u = torch.zeros(t, 384, dtype=torch.float16), torch.zeros(t, 2), torch.zeros(t, 2, 64, dtype=torch.float16), torch.zeros(t, 2, 64)
    with pytest.raises(ValueError, match="CUDA device"):
        dl.delta_tree(qkv, g, g, st, o, u)
    with pytest.raises(ValueError, match="CUDA device"):
        dl.delta_commit(qkv, g, u, one, st, st)
    with pytest.raises(ValueError, match="qkvz"):
        dl.conv_tree(torch.zeros(t, 384, dtype=torch.bfloat16), g, torch.zeros(2, 384, 3), qkv, g, g)


def test_a_call_is_on_its_memory_s_device(monkeypatch):
    """Tensors of another device than the stream's are refused, with the current stream and with a given one."""
    monkeypatch.setattr(gl, "_raw_stream", lambda device: 100 + device)
    monkeypatch.setattr(gl, "_current_device", lambda: 1, raising=False)
    assert gl.stream_on(1) == 101
    with pytest.raises(ValueError, match="cuda:0"):
        gl.stream_on(0)

    class Stream:
        device_index, cuda_stream = 0, 7
    assert gl.stream_on(0, Stream) == 7
    with pytest.raises(ValueError, match="cuda:1"):
        gl.stream_on(1, Stream)
