"""gdn_sync_status where several error words are set: a result that is not valid is reported before an index that
was skipped."""
import ctypes
import time

import numpy as np
import pytest
import torch

from hybrid_gated_deltanet_q4k_gb300 import api, synth
from hybrid_gated_deltanet_q4k_gb300 import lib as gl

from gpu_util import DEV, f16_dev, f32_dev, stream
from test_gpu_stages import CONV_SPECS, DELTA_SPECS, _delta_inputs, _layer, bf16_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return gl.load(build=True)


def _skip_a_slot(L):
    """A cache write whose slot lies past the cache: skipped, GDN_EINDEX."""
    cache = api.KvCache.new("i8", 2, 2, 16, 64)
    x = torch.ones(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    cache.write(x, x, torch.tensor([99], device=DEV))
    torch.cuda.synchronize()


def _skip_a_length(L):
    """A length below zero: clamped, GDN_EINDEX."""
    cache = api.KvCache.new("i8", 2, 2, 16, 64)
    q = torch.ones(1, 4, 64, dtype=torch.bfloat16, device=DEV)
    cache.attend(q, torch.tensor([-3], dtype=torch.int32, device=DEV), torch.zeros(1, 2, dtype=torch.int32, device=DEV),
                 torch.empty_like(q), cache.new_attend_workspace(1, 4))
    torch.cuda.synchronize()


def _delta_wait(L):
    spec = DELTA_SPECS[0]
    _, dev, s = _layer(spec, L)
    n = 200
    qkv, _, _, _, la, b = _delta_inputs(spec, n, np.random.default_rng(91))
    nbytes = L.gdn_delta_rule_scratch_size(ctypes.byref(s), n)
    scratch = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    keep = (f16_dev(qkv), f32_dev(la), f32_dev(b))
    L.gdn_test_delta_wait_timeout(ctypes.byref(s), *map(gl.ptr, keep), n, gl.ptr(scratch), nbytes, 1_000_000, stream())
    torch.cuda.synchronize()


def _conv_range(L):
    spec = CONV_SPECS[2]
    layer, dev, s = _layer(spec, L)
    n, nb = 70, 2 * spec.c_qk + 2 * spec.c_v
    wsum = np.asarray(layer["conv_w"], np.float64).reshape(spec.c_conv, -1)[2 * spec.c_qk + np.arange(spec.c_v)].sum(axis=1)
    c = int(np.argmax(np.abs(wsum)))
    x = np.zeros((n, nb), np.float32)
    x[:, 2 * spec.c_qk + c] = 3.0e6 * np.sign(wsum[c])
    keep = (bf16_dev(synth._to_bf16_bits(x)), f32_dev(np.zeros((spec.c_conv, 3))), f32_dev(np.zeros((n, 2 * spec.n_v_heads))))
    qkv = torch.empty(n, spec.c_conv, dtype=torch.float16, device=DEV)
    la = torch.empty(n, spec.n_v_heads, dtype=torch.float32, device=DEV)
    bb = torch.empty_like(la)
    L.gdn_conv(ctypes.byref(s), gl.ptr(keep[0]), nb, n, gl.ptr(keep[1]), gl.ptr(keep[2]), 2 * spec.n_v_heads, gl.ptr(qkv), gl.ptr(la),
               gl.ptr(bb), stream())
    torch.cuda.synchronize()


@pytest.mark.parametrize("skip", [_skip_a_slot, _skip_a_length])
@pytest.mark.parametrize("failure,code", [(_delta_wait, "GDN_ETIMEOUT"), (_conv_range, "GDN_ERANGE")])
@pytest.mark.parametrize("skip_first", [True, False])
def test_a_failure_is_reported_before_a_skipped_index(L, skip, failure, code, skip_first):
    for call in (skip, failure) if skip_first else (failure, skip):
        call(L)
    assert L.gdn_sync_status(stream(), check=False) == getattr(gl, code)
    assert "index" in L.last_error() or "skipped" in L.last_error()      # the other is named beside it
    assert L.gdn_sync_status(stream(), check=False) == gl.GDN_OK         # one call reports and clears both
    skip(L)
    assert L.gdn_sync_status(stream(), check=False) == gl.GDN_EINDEX


@pytest.mark.parametrize("nq", [1, 40])
def test_a_wait_that_ran_out_is_reported_before_a_length_of_the_same_launch(L, nq):
    cache = api.KvCache.new("i8", 40, 2, 16, 64)
    q = torch.ones(2 * nq, 4, 64, dtype=torch.bfloat16, device=DEV)
    o, ws = torch.empty_like(q), cache.new_attend_workspace(2 * nq, 4)
    lens = torch.tensor([-3, 300], dtype=torch.int32, device=DEV)
    table = torch.arange(40, dtype=torch.int32, device=DEV).view(2, 20)
    args = (ctypes.byref(cache.struct), gl.ptr(q), 256, 0, 2 * nq, nq, 0, gl.ptr(table), 20, 20, gl.ptr(lens), 2, 4, 0.0, gl.ptr(o), 256,
            gl.ptr(ws), ws.numel())
    L.gdn_test_attn_cache_wait_timeout(*args, 1_000_000, stream())
    assert L.gdn_sync_status(stream(), check=False) == gl.GDN_ETIMEOUT
    assert "length" in L.last_error()
    assert L.gdn_sync_status(stream(), check=False) == gl.GDN_OK
    L.gdn_attn_cache(*args, stream())
    assert L.gdn_sync_status(stream(), check=False) == gl.GDN_EINDEX


def test_the_words_are_read_in_one_go(L):
    """gdn_sync_status is called after every step, and a copy for each word made it as long as fifteen of them: a launch
    and a copy take as long as two or three."""
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    at = stream()
    call, copy = [], []
    for _ in range(300):
        t = time.perf_counter()
        L.gdn_sync_status(at)
        call.append(time.perf_counter() - t)
        t = time.perf_counter()
        word.cpu()
        copy.append(time.perf_counter() - t)
    assert np.median(call) < 6 * np.median(copy)
