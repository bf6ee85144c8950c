"""A hybrid model's drafted tokens decided on the GPU: a GDN layer, an attention layer, and the step around them.

Per round, for all sequences at once and without a number read back to the host: the last round's spare pages go
back and the new tokens get theirs (``KvPages.trim``, ``extend``); the GDN layer runs over the drafted trees
(``conv_tree``, ``delta_tree`` between its projections) and so does the attention layer (``RopeTable.apply``,
``KvCache.write``, ``attend``); the drafts are verified against the target's probabilities (``verify``); the state
moves to the accepted token (``delta_commit``) and the accepted keys and values to their final slots
(``KvCache.write`` with ``rows``).  A sequence that found no pages is left out on the GPU too, and is as it was.

Random weights stand for the model, and a model without its layers drafts for it.  The example also checks itself:
every accepted token is decoded again, one at a time (``decode``), and the probabilities are compared.

    python examples/serve_drafts.py
"""
from __future__ import annotations

import ctypes
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np
import torch

from hybrid_gated_deltanet_q4k_gb300 import api, synth
from hybrid_gated_deltanet_q4k_gb300 import lib as gl
from hybrid_gated_deltanet_q4k_gb300.api import DeviceLayer, KvCache, KvPages, RopeTable


class Model:
    """Embedding, one GDN layer (fp32 weights), one attention layer and the head; a layer adds half as much as there is."""

    def __init__(self, vocab=500, hq=4, hkv=2, d=64, seed=0, device="cuda"):
        self.spec = synth.SPECS["tiny_f32"]
        self.gdn = DeviceLayer(self.spec, synth.make_layer(self.spec, seed), device=device)
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen, device=device)  # noqa: E731
        h = self.spec.hidden
        self.embed, self.w_head = rand(vocab, h), 0.15 * rand(h, vocab)
        self.w_qkv, self.w_o = 0.05 * rand(h, (hq + 2 * hkv) * d), 0.05 * rand(hq * d, h)
        self.hq, self.hkv, self.d, self.device, self.lib = hq, hkv, d, device, self.gdn.lib
        self.rope = RopeTable(d, base=1e6)

    def new(self, *shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def head(self, x):
        return torch.softmax(x @ self.w_head, dim=1)

    @staticmethod
    def add(x, y):
        return x + y * (0.5 * x.norm(dim=1, keepdim=True) / y.norm(dim=1, keepdim=True))

    def gdn_drafts(self, x, state, conv, **tokens):
        """The GDN layer over drafted tokens: y, and what the commit needs."""
        sp, L, st = self.spec, self.lib, gl.stream_handle()
        t, s = x.shape[0], self.gdn.struct()
        n_bf16 = sp.r_in - 2 * sp.n_v_heads
        qkvz, ba = self.new(t, n_bf16, dtype=torch.bfloat16), self.new(t, 2 * sp.n_v_heads)
        L.gdn_gemm_f32(gl.ptr(x), gl.ptr(self.gdn.dev["w_in"]), t, sp.r_in, sp.hidden, gl.ptr(qkvz), n_bf16, n_bf16, gl.ptr(ba),
                       2 * sp.n_v_heads, st)
        qkv, log_a, b = self.new(t, sp.c_conv, dtype=torch.float16), self.new(t, sp.n_v_heads), self.new(t, sp.n_v_heads)
        self.gdn.conv_tree(qkvz, ba, conv, qkv, log_a, b, **tokens)
        o, delta = self.new(t, sp.n_v_heads, sp.dv, dtype=torch.float16), self.new(t, sp.n_v_heads, sp.dv)
        self.gdn.delta_tree(qkv, log_a, b, state, o, delta, **tokens)
        normed, y = self.new(t, sp.c_v), self.new(t, sp.hidden)
        L.gdn_gated_norm(ctypes.byref(s), gl.ptr(o), gl.ptr(qkvz) + 2 * sp.c_conv, n_bf16, t, 0, 0, gl.ptr(normed), st)
        L.gdn_gemm_f32(gl.ptr(normed), gl.ptr(self.gdn.dev["w_out"]), t, sp.hidden, sp.c_v, 0, 0, 0, gl.ptr(y), sp.hidden, st)
        return y, (qkv, log_a, delta, qkvz)

    def attention(self, x, positions, slots, cache, lens, table, cu, max_new, tree):
        """The attention layer over drafted tokens: y, and their keys and values."""
        t, wq, wk = x.shape[0], self.hq * self.d, self.hkv * self.d
        qkv = (x @ self.w_qkv).to(torch.bfloat16)
        q, k, v = (qkv[:, a:b].view(t, -1, self.d) for a, b in ((0, wq), (wq, wq + wk), (wq + wk, wq + 2 * wk)))
        self.rope.apply(positions, q, k)
        cache.write(k, v, slots)
        o = self.new(t, self.hq, self.d, dtype=torch.bfloat16)
        cache.attend(q, lens, table, o, cache.new_attend_workspace(t, self.hq), cu_q=cu, max_q=max_new, tree=tree)
        return o.view(t, -1).float() @ self.w_o, k, v


class Sequences:
    """States, cache and pages of several sequences, on the GPU."""

    def __init__(self, model, n, tokens, page=16, n_pages=None):
        """n_pages: of the pool, where it is to have fewer than all sequences may come to need."""
        sp = model.spec
        self.state = torch.zeros(n, sp.n_v_heads, sp.dv, sp.dk, device=model.device)
        self.conv = torch.zeros(n, sp.c_conv, 3, device=model.device)
        blocks = -(-tokens // page)
        n_pages = n * blocks if n_pages is None else n_pages
        self.cache = KvCache.new("bf16", n_pages, model.hkv, page, model.d, device=model.device)
        self.pages = KvPages.new(n, blocks, n_pages, page, device=model.device)
        self.lens = torch.zeros(n, dtype=torch.int32, device=model.device)


def step(model, seqs, tokens, n_new, tree, max_new, u, u_next, draft_p):
    """One round over the tokens [T] of all sequences (the last certain one of each, then its drafts).  Returns the new
    tokens, how many each sequence has (0: it found no pages and may try again), the target's probabilities and the
    accepted rows."""
    t, n = tokens.numel(), n_new.numel()
    ints = lambda k, dtype=torch.int32: torch.empty(k, dtype=dtype, device=model.device)  # noqa: E731
    after, cu, positions, slots = ints(n), ints(n + 1), ints(t), ints(t, torch.int64)
    seqs.pages.trim(seqs.lens)
    seqs.pages.extend(seqs.lens, n_new, after, cu, positions, slots, tree=tree)
    starved = (after == seqs.lens) & (n_new > 0)            # these have tokens but no slots: nothing of them may stay
    more = dict(cu=cu, max_new=max_new, tree=tree)
    x = model.embed[tokens.long()]
    y, (qkv, log_a, delta, qkvz) = model.gdn_drafts(x, seqs.state, seqs.conv, **more)
    x = model.add(x, y)
    y, k, v = model.attention(x, positions, slots, seqs.cache, after.masked_fill(starved, 0), seqs.pages.block_table, **more)
    p = model.head(model.add(x, y))
    rows, ids, count, node, nxt = ints(t), ints(t), ints(n), ints(n), ints(n)
    api.verify(p, tokens, rows, ids, count, node, nxt, u=u, u_next=u_next, q=draft_p, **more)
    node.masked_fill_(starved, -1)
    count.masked_fill_(starved, 0)
    model.gdn.delta_commit(qkv, log_a, delta, node, seqs.state, seqs.state, qkvz, seqs.conv, seqs.conv, **more)
    seqs.cache.write(k, v, torch.where(rows < 0, torch.full_like(slots, -1), slots), rows=rows)
    seqs.lens += count
    return ids, count, p, rows


def decode(model, seqs, tokens):
    """One certain token of each sequence by the one-token calls: the target's probabilities after it."""
    n = tokens.numel()
    after, cu = torch.empty_like(seqs.lens), torch.empty(n + 1, dtype=torch.int32, device=model.device)
    positions, slots = torch.empty_like(seqs.lens), torch.empty(n, dtype=torch.int64, device=model.device)
    seqs.pages.extend(seqs.lens, torch.ones_like(seqs.lens), after, cu, positions, slots)
    x = model.embed[tokens.long()]
    y = torch.empty_like(x)
    model.gdn.decode(x, seqs.state, seqs.conv, y, model.gdn.new_decode_workspace(n))
    x = model.add(x, y)
    y, _, _ = model.attention(x, positions, slots, seqs.cache, after, seqs.pages.block_table, None, 1, None)
    seqs.lens.copy_(after)
    return model.head(model.add(x, y))


def draft(model, last, sizes, rng, gen):
    """Trees drafted by the model without its layers: tokens, mask words, and its probabilities after each token."""
    tokens, words, parents = [], [], []
    for s, n in enumerate(sizes):
        first = len(tokens)
        for i in range(n):
            up = -1 if i == 0 else int(rng.integers(0, i))
            parents.append(first + up if i else -1)
            words.append((words[first + up] if i else 0) | 1 << i)
            tokens.append(int(last[s]) if i == 0 else -1)
    device = model.device
    out = torch.tensor(tokens, dtype=torch.int32, device=device)
    for i, up in enumerate(parents):
        if up >= 0:                                         # one child after another, each drawn for itself
            out[i] = torch.multinomial(model.head(model.embed[out[up:up + 1].long()]), 1, generator=gen)[0, 0]
    return out, torch.tensor(np.array(words, np.uint64).view(np.int64), device=device), model.head(model.embed[out.long()])


def serve(n=3, rounds=4, largest=8, seed=0):
    """The largest relative difference of the probabilities after an accepted token, drafted and one at a time; and the
    number of new tokens per sequence and round."""
    model = Model(seed=seed)
    rng, gen = np.random.default_rng(seed), torch.Generator(device=model.device)
    gen.manual_seed(seed)
    seqs, check = Sequences(model, n, 16 * rounds * largest), Sequences(model, n, 16 * rounds * largest)
    last = rng.integers(0, model.embed.shape[0], size=n)
    worst, total = 0.0, 0
    for _ in range(rounds):
        sizes = rng.integers(1, largest + 1, size=n)
        tokens, tree, draft_p = draft(model, last, sizes, rng, gen)
        u, u_next = torch.rand(tokens.numel(), generator=gen, device=model.device), torch.rand(n, generator=gen, device=model.device)
        ids, count, p, rows = step(model, seqs, tokens, torch.tensor(sizes, dtype=torch.int32, device=model.device), tree, largest, u,
                                   u_next, draft_p)
        # the accepted tokens again, one at a time; sequences with fewer of them wait
        counts, ends = count.tolist(), np.concatenate([[0], np.cumsum(sizes)])
        for d in range(max(counts)):
            held = [x.clone() for x in (check.state, check.conv, check.lens)]
            at = [int(rows[ends[s] + min(d, counts[s] - 1)]) for s in range(n)]
            q = decode(model, check, tokens[torch.tensor(at, device=model.device)])
            for s in range(n):
                if d < counts[s]:
                    worst = max(worst, float((p[at[s]] - q[s]).norm() / q[s].norm()))
                else:
                    for now, was in zip((check.state, check.conv, check.lens), held):
                        now[s] = was[s]
            check.pages.trim(check.lens)
        assert torch.equal(check.lens, seqs.lens)
        last = [int(ids[ends[s] + counts[s] - 1]) for s in range(n)]
        total += sum(counts)
    model.lib.gdn_sync_status(gl.stream_handle())
    state = float((seqs.state - check.state).norm() / check.state.norm())
    return worst, state, total / (n * rounds)


if __name__ == "__main__":
    p, state, rate = serve()
    print(f"{rate:.2f} tokens a round; probabilities differ from single decoding by {p:.1e}, the states by {state:.1e}")
