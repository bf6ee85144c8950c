"""User-facing wrappers: a GDN layer resident on the GPU, prefilled through the C ABI, and the
rotary table and paged key/value cache that serve the full-attention layers.

Weights are encoded to Q4_K on the host by the library's ``q4k_pack`` (or kept
fp32 for an F32 layer) and uploaded once; ``prefill`` enqueues one
``gdn_prefill`` call.  PyTorch only provides device memory and the stream.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import lib as gl


def pack_q4k(w: np.ndarray) -> np.ndarray:
    """Host Q4_K encoding through the library (``q4k_pack``)."""
    w = np.ascontiguousarray(w, np.float32)
    out = np.zeros((w.shape[0], w.shape[1] // 256 * 144), np.uint8)
    gl.load().q4k_pack(gl.ptr(w), w.shape[0], w.shape[1], gl.ptr(out))
    return out


def pack_q6k(w: np.ndarray) -> np.ndarray:
    """Host Q6_K encoding through the library (``q6k_pack``)."""
    w = np.ascontiguousarray(w, np.float32)
    out = np.zeros((w.shape[0], w.shape[1] // 256 * 210), np.uint8)
    gl.load().q6k_pack(gl.ptr(w), w.shape[0], w.shape[1], gl.ptr(out))
    return out


class DeviceLayer:
    """One GDN layer's parameters in device memory, in the layouts ``gdn_layer`` names."""

    def __init__(self, spec, params: dict, device: str = "cuda", eps_l2: float = 1e-6, eps_rms: float = 1e-6,
                 q_scale: float | None = None, blocks: dict | None = None, q6k: tuple = (), debug: bool = False):
        """q6k: names of the matrices ("w_in", "w_out") to hold in Q6_K instead of Q4_K.
        debug: run on the library's debug variant (index-checked kernels)."""
        self.spec = spec
        self.device = device
        self.lib = gl.load(debug=debug)
        self.q6k_mask = (1 if "w_in" in q6k else 0) | (2 if "w_out" in q6k else 0)
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
        if spec.wtype == "q4k":
            enc = {k: (pack_q6k if k in q6k else pack_q4k) for k in ("w_in", "w_out")}
            b_in = blocks["w_in"] if blocks else enc["w_in"](params["w_in"])
            b_out = blocks["w_out"] if blocks else enc["w_out"](params["w_out"])
            self.host_blocks = {"w_in": b_in, "w_out": b_out}
            self.dev = {"w_in": t(b_in), "w_out": t(b_out)}
        else:
            self.dev = {"w_in": t(params["w_in"].astype(np.float32)), "w_out": t(params["w_out"].astype(np.float32))}
        for k in ("conv_w", "A_log", "dt_bias", "norm_w"):
            self.dev[k] = t(params[k].astype(np.float32))
        self.eps_l2, self.eps_rms = eps_l2, eps_rms
        self.q_scale = spec.dk ** -0.5 if q_scale is None else q_scale

    def struct(self, gate_log_a=None, gate_b=None) -> gl.GdnLayer:
        L = gl.make_layer_struct(self.spec, self.dev, self.eps_l2, self.eps_rms, self.q_scale, gate_log_a, gate_b)
        L.q6k_mask = self.q6k_mask
        return L

    def workspace_bytes(self, ubatch_tokens: int) -> int:
        s = self.struct()
        return self.lib.gdn_workspace_size(ctypes.byref(s), int(ubatch_tokens))

    def new_workspace(self, ubatch_tokens: int) -> torch.Tensor:
        return torch.empty(self.workspace_bytes(ubatch_tokens), dtype=torch.uint8, device=self.device)

    def new_state(self) -> tuple:
        sp = self.spec
        state = torch.zeros(sp.n_v_heads, sp.dv, sp.dk, dtype=torch.float32, device=self.device)
        conv = torch.zeros(sp.c_conv, 3, dtype=torch.float32, device=self.device)
        return state, conv

    def prefill(self, x: torch.Tensor, state_in, state_out, conv_state, y, workspace, gate_log_a=None, gate_b=None,
                stream=None, check=True) -> int:
        """Enqueue gdn_prefill over x's rows; returns the status (raises if check and it is not 0)."""
        s = self.struct(gate_log_a, gate_b)
        return self.lib.gdn_prefill(ctypes.byref(s), gl.ptr(x), x.shape[0], gl.ptr(state_in), gl.ptr(state_out),
                                    gl.ptr(conv_state), gl.ptr(y), gl.ptr(workspace), workspace.numel(),
                                    gl.stream_handle(stream), check=check)

    def host_workspace_bytes(self, pass_tokens: int, gates: bool = False) -> int:
        """Device workspace of ``prefill_host`` for passes of ``pass_tokens`` (with or without drawn gates)."""
        s = self.struct()
        if gates:                   # only whether gates are drawn matters for the size
            s.gate_log_a = s.gate_b = 16
        return self.lib.gdn_host_workspace_size(ctypes.byref(s), int(pass_tokens))

    def new_host_workspace(self, pass_tokens: int, gates: bool = False) -> torch.Tensor:
        return torch.empty(self.host_workspace_bytes(pass_tokens, gates), dtype=torch.uint8, device=self.device)

    def prefill_host(self, x_host: torch.Tensor, state_in, state_out, conv_state, y_host: torch.Tensor, workspace,
                     pass_tokens: int = 0, gate_log_a=None, gate_b=None, stream=None, check=True) -> int:
        """Enqueue gdn_prefill_host: x_host, y_host (and the gates, if given) are pinned host tensors."""
        s = self.struct(gate_log_a, gate_b)
        return self.lib.gdn_prefill_host(ctypes.byref(s), gl.ptr(x_host), x_host.shape[0], gl.ptr(state_in),
                                         gl.ptr(state_out), gl.ptr(conv_state), gl.ptr(y_host), int(pass_tokens),
                                         gl.ptr(workspace), workspace.numel(), gl.stream_handle(stream), check=check)

    def batch_workspace_bytes(self, n_tokens: int, n_seqs: int) -> int:
        s = self.struct()
        return self.lib.gdn_batch_workspace_size(ctypes.byref(s), int(n_tokens), int(n_seqs))

    def new_batch_workspace(self, n_tokens: int, n_seqs: int) -> torch.Tensor:
        return torch.empty(self.batch_workspace_bytes(n_tokens, n_seqs), dtype=torch.uint8, device=self.device)

    def new_batch_state(self, n_seqs: int) -> tuple:
        sp = self.spec
        state = torch.zeros(n_seqs, sp.n_v_heads, sp.dv, sp.dk, dtype=torch.float32, device=self.device)
        conv = torch.zeros(n_seqs, sp.c_conv, 3, dtype=torch.float32, device=self.device)
        return state, conv

    def prefill_batch(self, x: torch.Tensor, cu_seqlens, state_in, state_out, conv_state, y, workspace,
                      gate_log_a=None, gate_b=None, stream=None, check=True) -> int:
        """Enqueue gdn_prefill_batch: x holds the sequences' tokens back to back, cu_seqlens (host, n_seqs + 1)
        their offsets; states [n_seqs][Hv][dv][dk] and conv tails [n_seqs][C_conv][3] are per sequence."""
        cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int64))
        s = self.struct(gate_log_a, gate_b)
        return self.lib.gdn_prefill_batch(ctypes.byref(s), gl.ptr(x), gl.ptr(cu), len(cu) - 1, gl.ptr(state_in),
                                          gl.ptr(state_out), gl.ptr(conv_state), gl.ptr(y), gl.ptr(workspace),
                                          workspace.numel(), gl.stream_handle(stream), check=check)

    def decode_workspace_bytes(self, n_seqs: int) -> int:
        s = self.struct()
        return self.lib.gdn_decode_workspace_size(ctypes.byref(s), int(n_seqs))

    def new_decode_workspace(self, n_seqs: int) -> torch.Tensor:
        return torch.empty(self.decode_workspace_bytes(n_seqs), dtype=torch.uint8, device=self.device)

    def decode(self, x: torch.Tensor, state, conv_state, y, workspace, gate_log_a=None, gate_b=None, stream=None,
               check=True) -> int:
        """Enqueue gdn_decode: one token per sequence (x [n_seqs][H]), states [n_seqs][Hv][dv][dk] and
        conv tails [n_seqs][C_conv][3] updated in place."""
        s = self.struct(gate_log_a, gate_b)
        return self.lib.gdn_decode(ctypes.byref(s), gl.ptr(x), x.shape[0], gl.ptr(state), gl.ptr(conv_state),
                                   gl.ptr(y), gl.ptr(workspace), workspace.numel(), gl.stream_handle(stream),
                                   check=check)

    def prefill_ckpt(self, x: torch.Tensor, state_in, state_out, conv_state, y, workspace, ckpt_every: int,
                     ckpt_state, ckpt_conv, gate_log_a=None, gate_b=None, stream=None, check=True) -> int:
        """Enqueue gdn_prefill_ckpt: as prefill, plus snapshots of the state [N // every][Hv][dv][dk] and conv
        state [N // every][C_conv][3] every ckpt_every tokens."""
        s = self.struct(gate_log_a, gate_b)
        return self.lib.gdn_prefill_ckpt(ctypes.byref(s), gl.ptr(x), x.shape[0], gl.ptr(state_in), gl.ptr(state_out),
                                         gl.ptr(conv_state), gl.ptr(y), int(ckpt_every), gl.ptr(ckpt_state),
                                         gl.ptr(ckpt_conv), gl.ptr(workspace), workspace.numel(),
                                         gl.stream_handle(stream), check=check)


def _heads(t: torch.Tensor, name: str, device: int, width=None) -> int:
    """Elements between the tokens of a bf16 tensor [tokens][heads][head_dim] on ``device`` (-1: host memory, which
    a kernel must not be given) whose heads are contiguous (and whose heads and head_dim are ``width``, if given)."""
    shape = t.shape
    if t.dtype is not torch.bfloat16 or len(shape) != 3 or device < 0 or t.get_device() != device:
        raise ValueError(f"{name}: a bf16 tensor [tokens][heads][head_dim] on the device of the others is required")
    n, h, d = shape
    if width is not None and (h, d) != width:
        raise ValueError(f"{name}: [tokens][{width[0]}][{width[1]}] is required")
    sn, sh, sd = t.stride()
    if n and ((d > 1 and sd != 1) or (h > 1 and sh != d)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return sn if n > 1 else h * d


def _vector(t: torch.Tensor, dtype: torch.dtype, n: int, name: str, device: int):
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name}: {n} contiguous {dtype} on device cuda:{device} are required")


class RopeTable:
    """Rotary positions of one attention layer: the table of ``gdn_rope_make`` and the call on it.

    layout "half" pairs x[i] with x[i + rot/2], "interleaved" x[2i] with x[2i + 1]; scaling "none",
    "linear" (positions divided by factor) or "parts" (slow pairs divided, fast ones kept, for a model
    trained on orig_len tokens)."""

    LAYOUTS = {"half": gl.GDN_ROPE_HALF, "interleaved": gl.GDN_ROPE_INTERLEAVED}
    SCALINGS = {"none": gl.GDN_ROPE_PLAIN, "linear": gl.GDN_ROPE_LINEAR, "parts": gl.GDN_ROPE_PARTS}

    def __init__(self, rot: int, base: float = 10000.0, layout: str = "half", scaling: str = "none", factor: float = 1.0,
                 orig_len: int = 0, fast: float = 32.0, slow: float = 1.0, amp: float = 0.0, debug: bool = False):
        self.lib = gl.load(debug=debug)
        self.table = gl.GdnRopeTable()
        if layout not in self.LAYOUTS or scaling not in self.SCALINGS:
            raise ValueError(f"layout {layout!r} or scaling {scaling!r} unknown")
        self.lib.gdn_rope_make(rot, self.LAYOUTS[layout], base, self.SCALINGS[scaling], factor, orig_len, fast, slow, amp,
                               ctypes.byref(self.table))
        self._ref = ctypes.byref(self.table)

    def apply(self, positions: torch.Tensor, q: torch.Tensor, k: torch.Tensor | None = None,
              q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None, check=True) -> int:
        """Enqueue gdn_rope on q [n][Hq][d] and k [n][Hk][d] (bf16; slices of a fused projection are fine),
        positions int32 [n]; into q_out and k_out, or in place without them."""
        n, hq, d = q.shape
        q_out = q if q_out is None else q_out
        dev = q.get_device()
        ld_q, ld_qo = _heads(q, "q", dev), _heads(q_out, "q_out", dev)
        _vector(positions, torch.int32, n, "positions", dev)
        if q_out.shape != q.shape:
            raise ValueError("q_out: the shape of q is required")
        hk = ld_k = ld_ko = 0
        if k is not None:
            k_out = k if k_out is None else k_out
            ld_k, ld_ko, hk = _heads(k, "k", dev), _heads(k_out, "k_out", dev), k.shape[1]
            if k.shape[0] != n or k.shape[2] != d or k_out.shape != k.shape:
                raise ValueError("k and k_out: as many tokens of the same head size as q are required")
        return self.lib.gdn_rope(self._ref, gl.ptr(positions), n, d, gl.ptr(q), ld_q, hq, gl.ptr(q_out), ld_qo, gl.ptr(k),
                                 ld_k, hk, gl.ptr(k_out) if hk else 0, ld_ko, gl.stream_handle(stream), check=check)


class KvCache:
    """A paged key/value cache of one full-attention layer in device memory.

    k and v [n_pages][n_kv_heads][page_tokens][head_dim] (bf16, int8 or float8_e4m3fn) and, for the 8-bit
    types, k_scale and v_scale fp32 [n_pages][n_kv_heads][page_tokens]; ``KvCache.new`` makes them.  Token
    slot s is row s % page_tokens of page s // page_tokens."""

    TYPES = {"bf16": (gl.GDN_KV_BF16, torch.bfloat16), "i8": (gl.GDN_KV_I8, torch.int8),
             "e4m3": (gl.GDN_KV_E4M3, torch.float8_e4m3fn)}

    def __init__(self, kind: str, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None, debug: bool = False):
        if kind not in self.TYPES:
            raise ValueError(f"cache type {kind!r} unknown")
        code, dtype = self.TYPES[kind]
        if k.dim() != 4 or k.shape != v.shape or k.dtype != dtype or v.dtype != dtype or not (
                k.is_contiguous() and v.is_contiguous()):
            raise ValueError(f"k and v: contiguous {dtype} [n_pages][n_kv_heads][page_tokens][head_dim] are required")
        scales = (k_scale, v_scale)
        if kind == "bf16":
            if scales != (None, None):
                raise ValueError("a bf16 cache has no scales")
        elif any(s is None or s.shape != k.shape[:3] or s.dtype != torch.float32 or not s.is_contiguous() for s in scales):
            raise ValueError("k_scale and v_scale: contiguous fp32 [n_pages][n_kv_heads][page_tokens] are required")
        self._device = k.get_device()
        if self._device < 0 or any(t is not None and t.get_device() != self._device for t in (v, *scales)):
            raise ValueError("the pages and their scales: memory of one CUDA device is required")
        self.lib = gl.load(debug=debug)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.n_kv_heads, self.page_tokens, self.head_dim = k.shape
        c = gl.GdnKvCache()
        c.dtype, c.n_kv_heads, c.head_dim, c.page_tokens, c.n_pages = (code, self.n_kv_heads, self.head_dim,
                                                                       self.page_tokens, self.n_pages)
        c.k, c.v, c.k_scale, c.v_scale = gl.ptr(k), gl.ptr(v), gl.ptr(k_scale), gl.ptr(v_scale)
        self.struct = c
        self._ref = ctypes.byref(c)
        self._width = (self.n_kv_heads, self.head_dim)

    @classmethod
    def new(cls, kind: str, n_pages: int, n_kv_heads: int, page_tokens: int, head_dim: int, device: str = "cuda",
            debug: bool = False) -> "KvCache":
        if kind not in cls.TYPES:
            raise ValueError(f"cache type {kind!r} unknown")
        shape, dtype = (n_pages, n_kv_heads, page_tokens, head_dim), cls.TYPES[kind][1]
        size = torch.empty((), dtype=dtype).element_size()
        pages = [torch.zeros(shape[:3] + (head_dim * size,), dtype=torch.uint8, device=device).view(dtype) for _ in "kv"]
        scales = [None if kind == "bf16" else torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in "kv"]
        return cls(kind, *pages, *scales, debug=debug)

    def slots(self, pages: torch.Tensor, first: int, n: int) -> torch.Tensor:
        """Slots (int64) of tokens first .. first + n - 1 of a sequence whose block table row is ``pages``."""
        if first < 0 or n < 0 or first + n > pages.numel() * self.page_tokens:
            raise ValueError(f"tokens {first} .. {first + n - 1} lie outside the {pages.numel()} pages")
        t = torch.arange(first, first + n, device=pages.device)
        return pages[t // self.page_tokens].long() * self.page_tokens + t % self.page_tokens

    def write(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, rows: torch.Tensor | None = None, stream=None,
              check=True) -> int:
        """Enqueue gdn_kv_write: rows of k and v (bf16 [n][n_kv_heads][head_dim]) into slots (int64, no slot
        twice, a negative one for a token that is not stored); with rows (int32), token t is row rows[t]: the
        accepted tokens of a drafted tree."""
        ld_k, ld_v = _heads(k, "k", self._device, self._width), _heads(v, "v", self._device, self._width)
        n = slots.numel()
        _vector(slots, torch.int64, n, "slots", self._device)
        if v.shape[0] != k.shape[0]:
            raise ValueError("k and v: the same number of rows is required")
        if rows is not None:
            _vector(rows, torch.int32, n, "rows", self._device)
        return self.lib.gdn_kv_write(self._ref, gl.ptr(k), ld_k, gl.ptr(v), ld_v, k.shape[0], gl.ptr(rows), gl.ptr(slots), n,
                                     gl.stream_handle(stream), check=check)

    def read(self, slots: torch.Tensor, k: torch.Tensor, v: torch.Tensor, stream=None, check=True) -> int:
        """Enqueue gdn_kv_read: the values of the slots (int64) into k and v (bf16 [n][n_kv_heads][head_dim])."""
        ld_k, ld_v = _heads(k, "k", self._device, self._width), _heads(v, "v", self._device, self._width)
        n = slots.numel()
        _vector(slots, torch.int64, n, "slots", self._device)
        if k.shape[0] != n or v.shape[0] != n:
            raise ValueError(f"k and v: {n} rows are required")
        return self.lib.gdn_kv_read(self._ref, gl.ptr(slots), n, gl.ptr(k), ld_k, gl.ptr(v), ld_v, gl.stream_handle(stream),
                                    check=check)

    def attend_workspace_bytes(self, n_tokens: int, n_q_heads: int) -> int:
        return self.lib.gdn_attn_cache_workspace_size(self._ref, int(n_tokens), int(n_q_heads))

    def new_attend_workspace(self, n_tokens: int, n_q_heads: int) -> torch.Tensor:
        return torch.empty(self.attend_workspace_bytes(n_tokens, n_q_heads), dtype=torch.uint8, device=self.k.device)

    def attend(self, q: torch.Tensor, lens: torch.Tensor, block_table: torch.Tensor, o: torch.Tensor,
               workspace: torch.Tensor, cu_q: torch.Tensor | None = None, max_q: int = 1, tree: torch.Tensor | None = None,
               scale: float = 0.0, stream=None, check=True) -> int:
        """Enqueue gdn_attn_cache: the new tokens q [T][Hq][head_dim] (bf16) of the sequences over their cached
        tokens.  lens int32 [n_seqs] counts the cached tokens, the new ones (already written) among them;
        block_table int32 [n_seqs][blocks]; cu_q int32 [n_seqs + 1] the new tokens' offsets (None: max_q
        each); tree int64 [T] mask words (None: a chain)."""
        ld_q, ld_o = _heads(q, "q", self._device), _heads(o, "o", self._device)
        n, hq, d = q.shape
        if o.shape != q.shape or d != self.head_dim:
            raise ValueError(f"q and o: [tokens][heads][{self.head_dim}] of one shape are required")
        s = lens.numel()
        _vector(lens, torch.int32, s, "lens", self._device)
        if block_table.dtype != torch.int32 or block_table.get_device() != self._device or block_table.dim() != 2 or \
                block_table.shape[0] != s or (
                block_table.shape[1] > 1 and block_table.stride(1) != 1) or (s > 1 and block_table.stride(0) < block_table.shape[1]):
            raise ValueError(f"block_table: int32 [{s}][blocks] on the cache's device is required")
        if workspace.get_device() != self._device or not workspace.is_contiguous():
            raise ValueError("workspace: contiguous memory of the cache's device is required")
        if cu_q is not None:
            _vector(cu_q, torch.int32, s + 1, "cu_q", self._device)
        if tree is not None:
            _vector(tree, torch.int64, n, "tree", self._device)
        ld_table = block_table.stride(0) if s > 1 else block_table.shape[1]
        return self.lib.gdn_attn_cache(self._ref, gl.ptr(q), ld_q, gl.ptr(cu_q), n, max_q, gl.ptr(tree), gl.ptr(block_table),
                                       ld_table, block_table.shape[1], gl.ptr(lens), s, hq, scale, gl.ptr(o), ld_o, gl.ptr(workspace),
                                       workspace.numel(), gl.stream_handle(stream), check=check)
