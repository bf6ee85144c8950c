"""One full-attention layer served end to end: prompt, drafted trees, an extension of the held prompt.

Per sequence: the prompt's queries and keys are rotated (``RopeTable.apply``), attended
(``gdn_attn_prefill``) and stored (``KvCache.write``).  Each round then drafts a tree of tokens, rotates
them at their depths, stores them past the end, attends all trees in one call (``KvCache.attend`` with
mask words) and moves the accepted path to its final slots (``KvCache.write`` with ``rows``).  At the
end a prefix is read back (``KvCache.read``) and extended.

Random tables stand for the layer's projections, so the example also checks itself: the accepted tokens
are decoded again one at a time, and the extension is computed both by the prefill and over the cache.

    python examples/serve_attention.py [bf16|i8|e4m3]
"""
from __future__ import annotations

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np
import torch

from hybrid_gated_deltanet_q4k_gb300 import lib as gl
from hybrid_gated_deltanet_q4k_gb300.api import KvCache, RopeTable


class Layer:
    """A layer's projections (a table of q | k | v rows per token id), its positions and its cache."""

    def __init__(self, kind, n_pages, hq=16, hkv=4, d=256, rot=64, page=64, vocab=512, seed=0, device="cuda"):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        self.hq, self.hkv, self.d, self.device = hq, hkv, d, device
        self.table = torch.randn(vocab, (hq + 2 * hkv) * d, generator=gen, device=device).to(torch.bfloat16)
        self.rope = RopeTable(rot, base=1e7)
        self.cache = KvCache.new(kind, n_pages, hkv, page, d, device=device)
        self.lib = self.cache.lib

    def project(self, ids, positions):
        """Rotated q and k and v of the tokens (v a view of the fused rows)."""
        n, wq, wk = len(ids), self.hq * self.d, self.hkv * self.d
        qkv = self.table[torch.as_tensor(ids, device=self.device)]
        q = torch.empty(n, self.hq, self.d, dtype=torch.bfloat16, device=self.device)
        k = torch.empty(n, self.hkv, self.d, dtype=torch.bfloat16, device=self.device)
        pos = torch.as_tensor(positions, dtype=torch.int32, device=self.device)
        self.rope.apply(pos, qkv[:, :wq].view(n, self.hq, self.d), qkv[:, wq:wq + wk].view(n, self.hkv, self.d), q, k)
        return q, k, qkv[:, wq + wk:].view(n, self.hkv, self.d)

    def prefill(self, q, k, v):
        """Causal attention of q over k and v, q's tokens the last of them."""
        v, o = v.contiguous(), torch.empty_like(q)
        nbytes = self.lib.gdn_attn_workspace_size(k.shape[0], self.hkv, self.d)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self.lib.gdn_attn_prefill(gl.ptr(q), gl.ptr(k), gl.ptr(v), q.shape[0], k.shape[0], self.hq, self.hkv, self.d, 0.0,
                                  gl.ptr(o), gl.ptr(ws), nbytes, gl.stream_handle(None))
        return o

    def attend(self, q, lens, pages, cu=None, max_q=1, tree=None):
        o = torch.empty_like(q)
        ints = lambda x: None if x is None else torch.as_tensor(x, dtype=torch.int32, device=self.device)  # noqa: E731
        self.cache.attend(q, ints(lens), pages, o, self.cache.new_attend_workspace(q.shape[0], self.hq), cu_q=ints(cu),
                          max_q=max_q, tree=tree)
        return o


def draft(rng, nodes):
    """Parents (-1: the sequence's last token), depths and mask words of a random tree."""
    parent = np.array([rng.integers(-1, i) if i else -1 for i in range(nodes)])
    depth, words = np.zeros(nodes, np.int64), np.zeros(nodes, np.uint64)
    for i, p in enumerate(parent):
        depth[i] = 0 if p < 0 else depth[p] + 1
        words[i] = (np.uint64(0) if p < 0 else words[p]) | (np.uint64(1) << np.uint64(i))
    return parent, depth, words


def difference(a, b):
    a, b = a.double(), b.double()
    return float((a - b).norm() / b.norm())


def worse(a, b):
    """The larger difference; one that is no number stays (max() would drop it)."""
    return a if b <= a or a != a else b


def serve(kind="e4m3", prompts=(1000, 77, 333), rounds=3, nodes=12, extension=40, seed=0, least=1, **layer):
    """Relative differences: of accepted tokens against single decoding, and of the extension.  Trees have from
    ``least`` to ``nodes`` tokens."""
    rng = np.random.default_rng(seed)
    page = layer.get("page", 64)
    blocks = -(-(max(prompts) + rounds * nodes + extension + nodes) // page)
    # the sequences' pages and as many for the check, in any order
    lay = Layer(kind, 2 * blocks * len(prompts), seed=seed, **layer)
    order = torch.as_tensor(rng.permutation(lay.cache.n_pages), dtype=torch.int32, device=lay.device).view(2, len(prompts), blocks)
    pages, check = order[0], order[1]
    vocab = lay.table.shape[0]

    lens = list(prompts)
    for s, n in enumerate(prompts):
        q, k, v = lay.project(rng.integers(0, vocab, n), np.arange(n))
        lay.prefill(q, k, v)
        for table in (pages, check):
            lay.cache.write(k, v, lay.cache.slots(table[s], 0, n))

    worst_tree = 0.0
    for _ in range(rounds):
        trees = [draft(rng, int(rng.integers(least, nodes + 1))) for _ in lens]
        ids = [rng.integers(0, vocab, len(t[0])) for t in trees]
        cu = np.concatenate([[0], np.cumsum([len(i) for i in ids])])
        q, k, v = lay.project(np.concatenate(ids), np.concatenate([n + t[1] for n, t in zip(lens, trees)]))
        lay.cache.write(k, v, torch.cat([lay.cache.slots(pages[s], n, len(ids[s])) for s, n in enumerate(lens)]))
        words = torch.from_numpy(np.concatenate([t[2] for t in trees]).view(np.int64)).to(lay.device)
        o = lay.attend(q, [n + len(i) for n, i in zip(lens, ids)], pages, cu, nodes, words)
        # accept the path to the deepest node: its tokens go to the slots that follow the sequence
        for s, (parent, depth, _) in enumerate(trees):
            path = [int(depth.argmax())]
            while parent[path[0]] >= 0:
                path.insert(0, int(parent[path[0]]))
            rows = torch.as_tensor(path, device=lay.device) + int(cu[s])
            lay.cache.write(k, v, lay.cache.slots(pages[s], lens[s], len(path)), rows=rows.to(torch.int32))
            for j, r in enumerate(path):
                q1, k1, v1 = lay.project(ids[s][r:r + 1], [lens[s] + j])
                lay.cache.write(k1, v1, lay.cache.slots(check[s], lens[s] + j, 1))
                one = lay.attend(q1, [lens[s] + j + 1], check[s:s + 1])
                worst_tree = worse(worst_tree, difference(o[int(cu[s]) + r], one[0]))
            lens[s] += len(path)

    # the first sequence comes back from the cache and is extended
    n = lens[0]
    held_k, held_v = (torch.empty(n, lay.hkv, lay.d, dtype=torch.bfloat16, device=lay.device) for _ in "kv")
    lay.cache.read(lay.cache.slots(pages[0], 0, n), held_k, held_v)
    q, k, v = lay.project(rng.integers(0, vocab, extension), n + np.arange(extension))
    lay.cache.write(k, v, lay.cache.slots(pages[0], n, extension))
    new_k, new_v = torch.empty_like(k), torch.empty_like(k)
    lay.cache.read(lay.cache.slots(pages[0], n, extension), new_k, new_v)
    by_prefill = lay.prefill(q, torch.cat([held_k, new_k]), torch.cat([held_v, new_v]))
    by_cache = lay.attend(q, [n + extension], pages[:1], max_q=extension)
    lay.lib.gdn_sync_status(gl.stream_handle(None))
    return worst_tree, difference(by_cache, by_prefill)


if __name__ == "__main__":
    for kind in sys.argv[1:] or ["bf16", "i8", "e4m3"]:
        tree, ext = serve(kind)
        print(f"{kind}: drafted trees differ from single tokens by {tree:.1e}, the extension from its prefill by {ext:.1e}")
