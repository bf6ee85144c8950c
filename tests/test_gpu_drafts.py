"""Conv, delta rule and commit over drafted tokens against the oracle.

Tolerances, element by element.  fp16 results are off by half a step, 2^-11 of the value (2^-25 where it is
subnormal).  Everything before is fp32 and proportional to the sums of absolute values that the oracle gives:
a product with the state keeps 22 bits of it (2^-21 with the truncation of the second part), 128 terms are
added in at most 16 steps of 2^-23 each, and a token's errors pass to its descendants with the same
coefficients, which those sums hold already: 2^-18 of them covers both.  The conv has four terms, an
exponential and a reciprocal of a few ulp and a norm: 2^-19.
"""
import numpy as np
import pytest
import torch

from gpu_util import DEV, Guarded, f16_dev, f16_round, f32_dev, stream, sync
from hybrid_gated_deltanet_q4k_gb300 import lib as gl
from hybrid_gated_deltanet_q4k_gb300 import synth
from hybrid_gated_deltanet_q4k_gb300.api import DeviceLayer
from oracle import drafts as OD

pytestmark = pytest.mark.gpu

EPS = 1e-6


def layer(hk, hv, d, rng, debug=False):
    spec = synth.LayerSpec("drafts", 256, hk, hv, d, d, 1, "f32", 0, "softplus_normal")
    p = {"w_in": np.zeros((spec.r_in, 256), np.float32), "w_out": np.zeros((256, spec.c_v), np.float32),
         "conv_w": (0.5 * rng.normal(size=(spec.c_conv, 4))).astype(np.float32), "A_log": rng.normal(size=hv).astype(np.float32),
         "dt_bias": rng.normal(size=hv).astype(np.float32), "norm_w": np.ones(d, np.float32)}
    return spec, p, DeviceLayer(spec, p, device=DEV, eps_l2=EPS, debug=debug)


def trees(lens, rng, kind):
    """Mask words of each sequence's tree, and None for chains."""
    if kind == "chain":
        return None
    out = []
    for n in lens:
        w = np.zeros(n, np.uint64)
        for i in range(n):
            up = {"tree": rng.integers(0, i) if i else -1, "star": 0 if i else -1, "roots": -1 if i % 3 == 0 else i - 1}[kind]
            w[i] = (w[up] if up >= 0 else np.uint64(0)) | (np.uint64(1) << np.uint64(i))
            if rng.random() < 0.5 and i < 63:
                w[i] |= np.uint64(1) << np.uint64(63)       # bits from the token on are not looked at
        # a later token must not inherit the odd bit as an ancestor's
        out.append(w & ((np.uint64(1) << np.arange(1, n + 1, dtype=np.uint64)) - np.uint64(1) | np.uint64(1 << 63)) if n < 64 else w)
    return out


class Case:
    """Inputs of one call, on the host and the GPU."""

    def __init__(self, hk, hv, d, lens, kind, seed=0, pad=0, debug=False):
        rng = np.random.default_rng(seed)
        self.spec, self.p, self.dl = layer(hk, hv, d, rng, debug)
        self.hk, self.hv, self.d, self.lens = hk, hv, d, list(lens)
        self.cu = np.concatenate([[0], np.cumsum(lens)])
        self.t, self.s, c = int(self.cu[-1]) + pad, len(lens), self.spec.c_conv
        words = trees(lens, rng, kind)
        self.up = [OD.parents(n, None if words is None else words[i]) for i, n in enumerate(lens)]
        self.tree = None
        if words is not None:
            flat = np.concatenate([np.concatenate(words) if self.cu[-1] else np.zeros(0, np.uint64), np.zeros(pad, np.uint64)])
            self.tree = torch.from_numpy(flat.view(np.int64)).to(DEV)
        self.cu_dev = torch.from_numpy(self.cu.astype(np.int32)).to(DEV)
        self.max_new = min(64, max(1, max(lens)) + pad)     # n_tokens is at most as many for each sequence
        unit = lambda x: x / np.sqrt((x ** 2).sum(-1, keepdims=True) + EPS)  # noqa: E731
        self.q = f16_round(unit(rng.normal(size=(self.t, hk, d))) * d ** -0.5)
        self.k = f16_round(unit(rng.normal(size=(self.t, hk, d)) + 0.5))
        self.v = f16_round(0.5 * rng.normal(size=(self.t, hv, d)))
        self.log_a = (-np.logaddexp(0, rng.normal(size=(self.t, hv)))).astype(np.float32)
        self.b = (1 / (1 + np.exp(-rng.normal(size=(self.t, hv))))).astype(np.float32)
        self.state = (0.3 * rng.normal(size=(self.s, hv, d, d))).astype(np.float32)
        self.x = (rng.normal(size=(self.t, c + hv * d + 8))).astype(np.float32)
        self.x = torch.from_numpy(self.x).to(torch.bfloat16).float().numpy()
        self.tail = rng.normal(size=(self.s, c, 3)).astype(np.float32)
        self.ba = rng.normal(size=(self.t, 2 * hv)).astype(np.float32)

    def more(self):
        return dict(cu=self.cu_dev, max_new=self.max_new, tree=self.tree)

    def qkv(self):
        w, t = self.d, self.t
        return f16_dev(np.concatenate([self.q.reshape(t, self.hk * w), self.k.reshape(t, self.hk * w), self.v.reshape(t, self.hv * w)], axis=1))

    def run_delta(self):
        o, u = Guarded(self.t * self.hv * self.d * 2, 0x5B), Guarded(self.t * self.hv * self.d * 4, 0x5B)
        shape = (self.t, self.hv, self.d)
        ov, uv = o.view(torch.float16, shape), u.view(torch.float32, shape)
        state = f32_dev(self.state)
        self.dl.delta_tree(self.qkv(), f32_dev(self.log_a), f32_dev(self.b), state, ov, uv, **self.more())
        sync(self.dl.lib)
        assert o.intact() and u.intact() and torch.equal(state.cpu(), torch.from_numpy(self.state))
        return ov, uv

    def oracle_delta(self):
        out = [np.zeros((self.t, self.hv, self.d)) for _ in range(4)]
        for s, n in enumerate(self.lens):
            r = slice(self.cu[s], self.cu[s] + n)
            for h in range(self.hv):
                g = h // (self.hv // self.hk)
                for x, y in zip(out, OD.delta(self.q[r, g].astype(np.float64), self.k[r, g].astype(np.float64), self.v[r, h].astype(np.float64),
                                              self.log_a[r, h].astype(np.float64), self.b[r, h].astype(np.float64), self.state[s, h], self.up[s])):
                    x[r, h] = y
        return out


def close(got, ref, bound):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    worst = np.abs(got - ref) - bound
    assert np.isfinite(got).all() and worst.max() <= 0, (float(worst.max()), np.unravel_index(worst.argmax(), worst.shape))


def f16_bound(ref):
    return np.maximum(np.abs(ref) * 2.0 ** -11, 2.0 ** -25)


SHAPES = [  # hk, hv, d, lens, kind
    (1, 1, 64, [1], "chain"), (2, 4, 128, [4], "chain"), (1, 3, 64, [3, 0, 8, 5], "chain"), (2, 2, 128, [8, 1, 7], "tree"),
    (1, 2, 128, [9], "chain"), (1, 2, 64, [17, 33, 0, 2], "tree"), (1, 1, 128, [64, 5], "chain"), (2, 4, 64, [64, 63, 16], "tree"),
    (1, 2, 128, [40, 24], "star"), (1, 8, 64, [31, 15], "roots"), (4, 32, 64, [8, 3, 6, 1, 7, 0, 5, 8], "tree"),
    (16, 32, 128, [5, 2, 8, 1, 3, 8, 4, 6], "chain"),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_delta_tree(shape):
    c = Case(*shape, seed=len(shape[3]))
    o, u = c.run_delta()
    ru, ro, eu, eo = c.oracle_delta()
    close(u, ru, 2.0 ** -18 * eu)
    close(o, ro, 2.0 ** -18 * eo + f16_bound(ro))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_conv_tree(shape):
    c = Case(*shape, seed=7, pad=3)
    spec, t = c.spec, c.t
    x = torch.from_numpy(c.x).to(DEV).to(torch.bfloat16)
    out, la, b = Guarded(t * spec.c_conv * 2, 0x5B), Guarded(t * c.hv * 4, 0x5B), Guarded(t * c.hv * 4, 0x5B)
    tail = f32_dev(c.tail)
    for view in (x, x[:, :spec.c_conv].contiguous(), x[:, 4:]):       # rows at 16-byte and at 8-byte places
        c.dl.conv_tree(view, f32_dev(c.ba), tail, out.view(torch.float16, (t, spec.c_conv)), la.view(torch.float32, (t, c.hv)),
                       b.view(torch.float32, (t, c.hv)), **c.more())
        sync(c.dl.lib)
        assert out.intact() and la.intact() and b.intact() and torch.equal(tail.cpu(), torch.from_numpy(c.tail))
        raw, n = view.float().cpu().numpy()[:, :spec.c_conv], int(c.cu[-1])
        ry, ey = np.zeros((n, spec.c_conv)), np.zeros((n, spec.c_conv))
        for s, m in enumerate(c.lens):
            r = slice(c.cu[s], c.cu[s] + m)
            if m:
                ry[r], ey[r] = OD.conv(raw[r], c.tail[s], c.up[s], c.p["conv_w"].astype(np.float64), 2 * c.hk, c.d, c.hk, EPS, c.d ** -0.5)
        close(out.view(torch.float16, (t, spec.c_conv))[:n], ry, f16_bound(ry) + 2.0 ** -19 * (np.abs(ry) + ey))
        rla, rb = OD.gates(c.ba[:n, :c.hv], c.ba[:n, c.hv:], c.p["A_log"], c.p["dt_bias"])
        close(la.view(torch.float32, (t, c.hv))[:n], rla, 2.0 ** -20 * np.abs(rla) + 1e-12)
        close(b.view(torch.float32, (t, c.hv))[:n], rb, 2.0 ** -20 * rb)
        for buf, dtype, w in ((out, torch.float16, spec.c_conv), (la, torch.float32, c.hv), (b, torch.float32, c.hv)):
            assert (buf.view(dtype, (t, w))[n:].contiguous().view(torch.uint8) == 0x5B).all()      # rows behind the last sequence


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("in_place", [False, True])
def test_commit(shape, in_place):
    c = Case(*shape, seed=11, pad=2)
    rng = np.random.default_rng(3)
    u = (0.4 * rng.normal(size=(c.t, c.hv, c.d))).astype(np.float32)
    node = np.array([rng.integers(-1, n) if n else -1 for n in c.lens], np.int32)
    node[0] = c.lens[0] - 1
    x = torch.from_numpy(c.x).to(DEV).to(torch.bfloat16)
    s_in, t_in = f32_dev(c.state), f32_dev(c.tail)
    s_out, t_out = (s_in, t_in) if in_place else (torch.full_like(s_in, 7.0), torch.full_like(t_in, 7.0))
    c.dl.delta_commit(c.qkv(), f32_dev(c.log_a), f32_dev(u), torch.from_numpy(node).to(DEV), s_in, s_out, x, t_in, t_out, **c.more())
    sync(c.dl.lib)
    for s, n in enumerate(c.lens):
        r = slice(c.cu[s], c.cu[s] + n)
        assert np.array_equal(t_out[s].cpu().numpy(), OD.conv_commit(c.x[r, :c.spec.c_conv], c.tail[s], c.up[s], node[s]))
        steps = len(OD.path(c.up[s], node[s])) + 4
        for h in range(c.hv):
            ref, e = OD.commit(c.k[r, h // (c.hv // c.hk)].astype(np.float64), u[r, h].astype(np.float64), c.log_a[r, h].astype(np.float64),
                               c.state[s, h], c.up[s], node[s])
            if node[s] < 0:
                assert np.array_equal(s_out[s, h].cpu().numpy(), c.state[s, h])
            else:
                close(s_out[s, h], ref, steps * 2.0 ** -23 * e)


def test_a_commit_without_tokens_passes_the_states_through():
    c = Case(1, 2, 64, [0, 0], "chain", seed=1)
    state, tail = torch.full((2, 2, 64, 64), 7.0, device=DEV), torch.full((2, c.spec.c_conv, 3), 7.0, device=DEV)
    x = torch.empty(0, c.spec.c_conv, dtype=torch.bfloat16, device=DEV)
    c.dl.delta_commit(c.qkv(), f32_dev(c.log_a), torch.empty(0, 2, 64, device=DEV), torch.tensor([-1, -1], dtype=torch.int32, device=DEV),
                      f32_dev(c.state), state, x, f32_dev(c.tail), tail, **c.more())
    sync(c.dl.lib)
    assert np.array_equal(state.cpu().numpy(), c.state) and np.array_equal(tail.cpu().numpy(), c.tail)
    # and the other calls have nothing to do
    none = torch.empty(0, 2, 64, device=DEV)
    c.dl.delta_tree(c.qkv(), f32_dev(c.log_a), f32_dev(c.b), f32_dev(c.state), none.half(), none, **c.more())
    c.dl.conv_tree(x, torch.empty(0, 4, device=DEV), f32_dev(c.tail), c.qkv(), f32_dev(c.log_a), f32_dev(c.b), **c.more())
    sync(c.dl.lib)


def test_a_step_is_tokens_one_after_another():
    """Drafts, their commit and the next drafts: as the oracle's chain of all accepted tokens."""
    c = Case(2, 4, 128, [6, 6], "tree", seed=5)
    o, u = c.run_delta()
    node = np.array([5, 3], np.int32)
    state = torch.empty(c.s, c.hv, c.d, c.d, device=DEV)
    c.dl.delta_commit(c.qkv(), f32_dev(c.log_a), u, torch.from_numpy(node).to(DEV), f32_dev(c.state), state, **c.more())
    o2, u2 = torch.empty_like(o), torch.empty_like(u)
    c.dl.delta_tree(c.qkv(), f32_dev(c.log_a), f32_dev(c.b), state, o2, u2, **c.more())
    sync(c.dl.lib)
    for s in range(2):
        first = OD.path(c.up[s], node[s])
        for i in range(6):
            p = [c.cu[s] + j for j in first + OD.path(c.up[s], i)]
            for h in range(c.hv):
                g = h // 2
                ru, ro, eu, eo = OD.delta(c.q[p, g].astype(np.float64), c.k[p, g].astype(np.float64), c.v[p, h].astype(np.float64),
                                          c.log_a[p, h].astype(np.float64), c.b[p, h].astype(np.float64), c.state[s, h], list(range(-1, len(p) - 1)))
                close(o2[c.cu[s] + i, h], ro[-1], 2.0 ** -17 * eo[-1] + f16_bound(ro[-1]))


def test_a_chain_is_the_delta_rule():
    """The same tokens through gdn_delta_rule (its operands are fp16, its tolerance a relative L2 of 4e-3)."""
    c = Case(2, 4, 128, [64], "chain", seed=9)
    o, _ = c.run_delta()
    L, st = c.dl.lib, c.dl.struct()
    import ctypes
    scratch = torch.empty(L.gdn_delta_rule_scratch_size(ctypes.byref(st), 64), dtype=torch.uint8, device=DEV)
    o2, s2 = torch.empty_like(o), torch.empty(c.hv, c.d, c.d, device=DEV)
    qkv, la, b, s0 = c.qkv(), f32_dev(c.log_a), f32_dev(c.b), f32_dev(c.state)
    L.gdn_delta_rule(ctypes.byref(st), gl.ptr(qkv), gl.ptr(la), gl.ptr(b), 64, gl.ptr(s0), gl.ptr(s2), gl.ptr(o2), gl.ptr(scratch),
                     scratch.numel(), stream())
    sync(L)
    assert float((o.float() - o2.float()).norm() / o2.float().norm()) <= 4e-3


@pytest.mark.parametrize("n,hv,more", [(7, 2, 1), (20, 2, 1), (7, 64, 3)])       # the last: many heads of few tokens
@pytest.mark.parametrize("what", ["v", "k", "q", "b", "log_a", "state_row"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_on_its_branch(n, hv, more, what, value):
    """Token 2's branch does not reach the tokens that do not descend from it; a state row reaches its own row alone."""
    c = Case(hv // 2 if hv == 2 else 16, hv, 64, [n] * (1 + more), "tree", seed=21)
    if what == "state_row":
        c.state[0, 1, 5, 9] = value
    elif what == "log_a":
        if value != value:
            c.log_a[2, 0] = value
        else:
            c.log_a[2, 0] = -value                          # a = 0: all of it stays finite
    elif what == "b":
        c.b[2, 0] = value
    else:
        getattr(c, what)[2, 0, 3] = value
    with np.errstate(all="ignore"):
        ru, ro, eu, eo = c.oracle_delta()
    o, u = c.run_delta_unchecked()
    hurt = np.zeros(ru.shape, bool)
    if what == "state_row":
        hurt[:n, 1, 5] = True
    else:
        for i in range(n):
            if 2 in (OD.path(c.up[0], i) if what != "q" else [i]):
                hurt[i] = True
    fine = ~hurt
    got_u, got_o = u.double().cpu().numpy(), o.double().cpu().numpy()
    assert np.isfinite(ru[fine]).all()
    assert (np.abs(got_u[fine] - ru[fine]) <= 2.0 ** -18 * eu[fine]).all()
    assert (np.abs(got_o[fine] - ro[fine]) <= 2.0 ** -18 * eo[fine] + f16_bound(ro[fine])).all()
    # and what the oracle has as not a number does not come back as one
    assert not np.isfinite(got_o[np.isnan(ro)]).any()


def _unchecked(self):
    shape = (self.t, self.hv, self.d)
    o, u = torch.empty(shape, dtype=torch.float16, device=DEV), torch.empty(shape, device=DEV)
    self.dl.delta_tree(self.qkv(), f32_dev(self.log_a), f32_dev(self.b), f32_dev(self.state), o, u, **self.more())
    assert self.dl.lib.gdn_sync_status(stream(), check=False) in (gl.GDN_OK, gl.GDN_ERANGE)
    return o, u


Case.run_delta_unchecked = _unchecked


def test_decays_of_any_size():
    """log a from -1e-6 to -1e5 and -inf (a = 0): nothing overflows, and what follows an a of 0 has forgotten."""
    c = Case(1, 2, 128, [30, 8], "chain", seed=2)
    rng = np.random.default_rng(0)
    c.log_a = (-10.0 ** rng.uniform(-6, 5, size=c.log_a.shape)).astype(np.float32)
    c.log_a[4] = -np.inf
    o, u = c.run_delta()
    ru, ro, eu, eo = c.oracle_delta()
    close(u, ru, 2.0 ** -18 * eu)
    close(o, ro, 2.0 ** -18 * eo + f16_bound(ro))


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1e8, 1e30])
@pytest.mark.parametrize("n,hv,seqs", [(8, 1, 1), (12, 1, 1), (8, 64, 3)])
def test_states_of_any_size(scale, n, hv, seqs):
    c = Case(min(hv, 8), hv, 128 if hv == 1 else 64, [n] * seqs, "chain", seed=4)
    c.state *= np.float32(scale)
    c.v *= 0
    o, u = c.run_delta_unchecked()
    ru, ro, eu, eo = c.oracle_delta()
    close(u, ru, 2.0 ** -18 * eu)


def test_over_fp16_is_reported():
    c = Case(1, 1, 64, [3], "chain")
    c.state[:] = 3e6
    shape = (c.t, 1, 64)
    c.dl.delta_tree(c.qkv(), f32_dev(c.log_a), f32_dev(c.b), f32_dev(c.state), torch.empty(shape, dtype=torch.float16, device=DEV),
                    torch.empty(shape, device=DEV), **c.more())
    assert c.dl.lib.gdn_sync_status(stream(), check=False) == gl.GDN_ERANGE
    sync(c.dl.lib)


@pytest.mark.parametrize("cu", [[0, 9, 12], [0, 5, 3], [-1, 4, 8], [0, 4, 20], [0, 2 ** 30, 8]])
def test_offsets_out_of_range_leave_the_sequence_out(cu):
    """Each call reports them and works on the others."""
    c = Case(1, 2, 64, [4, 8], "tree", seed=1)
    c.max_new = 8
    c.cu_dev = torch.tensor(cu, dtype=torch.int32, device=DEV)
    shape = (c.t, c.hv, c.d)
    o, u = torch.full(shape, 7.0, dtype=torch.float16, device=DEV), torch.full(shape, 7.0, device=DEV)
    L = c.dl.lib
    c.dl.delta_tree(c.qkv(), f32_dev(c.log_a), f32_dev(c.b), f32_dev(c.state), o, u, **c.more())
    assert L.gdn_sync_status(stream(), check=False) == gl.GDN_EINDEX and "gdn_delta_tree" in L.last_error()
    x = torch.from_numpy(c.x).to(DEV).to(torch.bfloat16)
    qkv, la, b = c.qkv(), f32_dev(c.log_a), f32_dev(c.b)
    c.dl.conv_tree(x, f32_dev(c.ba), f32_dev(c.tail), qkv, la, b, **c.more())
    assert L.gdn_sync_status(stream(), check=False) == gl.GDN_EINDEX
    out = torch.full((2, c.hv, c.d, c.d), 7.0, device=DEV)
    c.dl.delta_commit(c.qkv(), f32_dev(c.log_a), f32_dev(u.cpu().numpy()), torch.tensor([-1, -1], dtype=torch.int32, device=DEV),
                      f32_dev(c.state), out, **c.more())
    assert L.gdn_sync_status(stream(), check=False) == gl.GDN_EINDEX
    assert torch.equal(out.cpu(), torch.from_numpy(c.state))
    sync(L)


@pytest.mark.parametrize("node", [[4, 0], [-2, 0], [2 ** 31 - 1, 0], [0, 0]])
def test_a_node_outside_its_sequence_counts_as_none(node):
    c = Case(1, 2, 64, [4, 0], "chain", seed=1)
    out = torch.full((2, c.hv, c.d, c.d), 7.0, device=DEV)
    u = torch.zeros(c.t, c.hv, c.d, device=DEV)
    c.dl.delta_commit(c.qkv(), f32_dev(c.log_a), u, torch.tensor(node, dtype=torch.int32, device=DEV), f32_dev(c.state), out, **c.more())
    assert c.dl.lib.gdn_sync_status(stream(), check=False) == gl.GDN_EINDEX
    assert torch.equal(out[1].cpu(), torch.from_numpy(c.state[1]))
    if node[0]:
        assert torch.equal(out[0].cpu(), torch.from_numpy(c.state[0]))


@pytest.mark.parametrize("hk,hv,lens", [(1, 2, [5, 5, 5]), (16, 64, [7, 7, 7]), (1, 1, [64])])
def test_without_offsets_every_sequence_has_max_new(hk, hv, lens):
    c = Case(hk, hv, 64, lens, "chain", seed=6)
    o, u = c.run_delta()
    c.cu_dev = None
    o2, u2 = c.run_delta()
    assert torch.equal(o, o2) and torch.equal(u, u2)


@pytest.mark.parametrize("lens,kind", [([8, 3], "chain"), ([20, 9], "tree")])
def test_replayed_on_another_stream_with_other_inputs(lens, kind):
    """A captured step follows what its buffers hold, other lengths among it, and gives what the calls give."""
    a, b = Case(1, 4, 64, lens, kind, seed=1), Case(1, 4, 64, lens[::-1], kind, seed=2)
    side = torch.cuda.Stream()
    buf = dict(qkv=a.qkv(), la=f32_dev(a.log_a), b=f32_dev(a.b), state=f32_dev(a.state), cu=a.cu_dev.clone(),
               tree=None if a.tree is None else a.tree.clone(), node=torch.tensor([2, 1], dtype=torch.int32, device=DEV))
    shape = (a.t, a.hv, a.d)
    o, u = torch.empty(shape, dtype=torch.float16, device=DEV), torch.empty(shape, device=DEV)
    after = torch.empty_like(buf["state"])

    def step():
        more = dict(cu=buf["cu"], max_new=a.max_new, tree=buf["tree"])
        a.dl.delta_tree(buf["qkv"], buf["la"], buf["b"], buf["state"], o, u, **more)
        a.dl.delta_commit(buf["qkv"], buf["la"], u, buf["node"], buf["state"], after, **more)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
        for c in (b, a):
            buf["qkv"].copy_(c.qkv())
            buf["la"].copy_(f32_dev(c.log_a))
            buf["b"].copy_(f32_dev(c.b))
            buf["state"].copy_(f32_dev(c.state))
            buf["cu"].copy_(c.cu_dev)
            if buf["tree"] is not None:
                buf["tree"].copy_(c.tree)
            g.replay()
            side.synchronize()
            got = [x.clone() for x in (o, u, after)]
            o.zero_(), u.zero_(), after.zero_()
            step()
            side.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(got, (o, u, after)))


def test_the_debug_library_agrees():
    for lens, kind in (([5, 8], "tree"), ([30, 2], "tree")):
        a, b = Case(1, 2, 64, lens, kind, seed=3), Case(1, 2, 64, lens, kind, seed=3, debug=True)
        (o, u), (o2, u2) = a.run_delta(), b.run_delta()
        assert torch.equal(o, o2) and torch.equal(u, u2)


@pytest.mark.parametrize("over", [dict(qkv=1), dict(o=1), dict(cu=1), dict(tree=1), dict(log_a=1), dict(state=1)])
def test_wrappers_refuse_what_does_not_fit(over):
    c = Case(1, 2, 64, [3, 4], "tree")
    a = dict(qkv=c.qkv(), log_a=f32_dev(c.log_a), b=f32_dev(c.b), state=f32_dev(c.state),
             o=torch.empty(c.t, 2, 64, dtype=torch.float16, device=DEV), delta=torch.empty(c.t, 2, 64, device=DEV), **c.more())
    name = next(iter(over))
    for bad in (a[name][:-1], a[name].cpu(), a[name].to(torch.float64)):
        if name == "qkv" and bad.shape[0] != c.t:           # fewer tokens: the other tensors are too long
            name = "qkv"
        with pytest.raises(ValueError):
            c.dl.delta_tree(**{**a, name: bad})
    with pytest.raises(ValueError):
        c.dl.delta_tree(**{**a, name: a[name].repeat(2, *[1] * (a[name].dim() - 1))[::2]})
