"""Measured cases of the full-attention serving operators.

Rotary positions of queries and keys (``rope``), the quantised paged key/value
cache written and read back (``store``, ``fetch``), and attention of one token,
a short chain or a tree of drafted tokens over that cache (``attend``), each in
a plain form (elementary torch operations in fp32) and through the framework's
public calls.  The sizes are the hybrid layer's full attention (16 query heads
over 4 key/value heads of 256, prompts of 32768 tokens) and generic ones.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = ("bf16", "i8", "e4m3")
CODE_MAX = {"i8": 127.0, "e4m3": 448.0}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token of one sequence: latency alone
        dict(name="rope_one_token", op="rope", n=1, hq=16, hkv=4, d=256, rot=64, layout="half", base=1e7, scaling="none",
             factor=1.0, orig=0, far=20000, fused=0),
        # a whole prompt of the hybrid model's full-attention layer, a quarter of each head rotated
        dict(name="rope_prompt", op="rope", n=32768, hq=16, hkv=4, d=256, rot=64, layout="half", base=1e7,
             scaling="none", factor=1.0, orig=0, far=32768, fused=0),
        # a piece of a very long document with positions scaled by parts, read out of a fused q|k|v projection
        dict(name="rope_far_pairs", op="rope", n=5001, hq=32, hkv=8, d=128, rot=128, layout="interleaved", base=1e6,
             scaling="parts", factor=8.0, orig=131072, far=1000000, fused=1),
        # the accepted tokens of 24 drafted trees go to their final slots
        dict(name="store_accepted", op="store", type="i8", n=97, rows=768, hkv=4, d=256, page=64, fused=1),
        # a prompt's keys and values enter the cache
        dict(name="store_prompt", op="store", type="e4m3", n=32768, rows=0, hkv=4, d=256, page=64, fused=0),
        # a short held prefix comes back for a prompt that extends it
        dict(name="fetch_prefix", op="fetch", type="e4m3", n=777, hkv=8, d=128, page=16),
        # a long held prompt comes back
        dict(name="fetch_prompt", op="fetch", type="i8", n=100003, hkv=4, d=256, page=64),
        # one user, one token, a short conversation: latency alone
        dict(name="attend_short", op="attend", type="bf16", seqs=1, lo=777, hi=777, qlo=1, qhi=1, tree=0, hq=16, hkv=4,
             d=256, page=64),
        # one user, one token, a very long document
        dict(name="attend_long", op="attend", type="i8", seqs=1, lo=131072, hi=131072, qlo=1, qhi=1, tree=0, hq=16,
             hkv=4, d=256, page=64),
        # a serving batch, one token each, every length from one token to 16 thousand
        dict(name="attend_batch", op="attend", type="e4m3", seqs=48, lo=1, hi=16384, qlo=1, qhi=1, tree=0, hq=16, hkv=4,
             d=256, page=64),
        # chains of up to four drafted tokens, heads of 128, small pages
        dict(name="attend_chain", op="attend", type="i8", seqs=16, lo=300, hi=12000, qlo=1, qhi=4, tree=0, hq=32, hkv=8,
             d=128, page=16),
        # trees of drafted tokens over an unquantised cache
        dict(name="attend_tree", op="attend", type="bf16", seqs=6, lo=4000, hi=24000, qlo=24, qhi=64, tree=1, hq=16,
             hkv=4, d=256, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    """Nanoseconds of a pass at 6.7 TB/s and 1.9 PFLOP/s, one after the other."""
    w = work(case)
    return w["bytes"] / 6.7e3 + w["flops"] / 1.9e6


def draw(rng):
    case = _draw(rng)
    while _cost(case) > 110e3:                        # the largest listed one takes 123e3
        for key in ("n", "lo", "hi", "rows"):
            if case.get(key):
                case[key] = max(1, case[key] * 2 // 3)
        if case.get("rows"):
            case["rows"] = max(case["rows"], case["n"])
    return case


def _draw(rng):
    op = rng.choice(["rope", "store", "fetch", "attend", "attend", "attend"])
    d, hkv = rng.choice([(64, 8), (64, 2), (128, 8), (128, 2), (128, 1), (256, 4), (256, 1), (256, 2)])
    ratio = rng.choice([1, 2, 3, 4, 5, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        rot = rng.choice([d, d // 2, d // 4, d // 4 + 2])
        far = _log(rng, 40000, 2000000)
        scaling = rng.choice(["none", "linear", "parts"])
        return dict(op=op, n=_log(rng, 1, 32768), hq=hkv * min(ratio, 4), hkv=hkv, d=d, rot=rot,
                    layout=rng.choice(["half", "interleaved"]), base=rng.choice([1e4, 1e6, 1e7]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                    orig=rng.choice([8192, 32768]) if scaling == "parts" else 0, far=far, fused=rng.randint(0, 1))
    kind = rng.choice(TYPES)
    if op == "store":
        n = _log(rng, 1, 32768)
        return dict(op=op, type=kind, n=n, rows=n + rng.randint(0, 3 * n) if rng.random() < 0.4 else 0, hkv=hkv, d=d,
                    page=page, fused=rng.randint(0, 1))
    if op == "fetch":
        return dict(op=op, type=kind, n=_log(rng, 1, 100000), hkv=hkv, d=d, page=page)
    tree = rng.randint(0, 1)
    qhi = rng.randint(2, 64) if tree else rng.choice([1, 1, 1, 2, 4, 7])
    seqs = _log(rng, 1, 48)
    hi = min(_log(rng, 1, 131072), max(64, 300000 // seqs))
    return dict(op=op, type=kind, seqs=seqs, lo=max(1, _log(rng, 1, max(2, hi)) if hi > 1 else 1), hi=hi,
                qlo=rng.randint(1, qhi), qhi=qhi, tree=tree, hq=hkv * ratio, hkv=hkv, d=d, page=page)


# ---------------------------------------------------------------- inputs

def _lengths(case):
    """Per sequence: tokens in the cache (the new ones among them) and new tokens."""
    s, lo, hi = case["seqs"], min(case["lo"], case["hi"]), case["hi"]
    r = np.random.default_rng(1000 * s + 7 * hi + case["d"])
    nq = r.integers(case["qlo"], case["qhi"] + 1, size=s)
    lens = r.integers(lo, hi + 1, size=s)
    lens[0] = hi
    return np.maximum(lens, nq), nq


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _rows(gen, n, heads, d):
    """bf16 rows whose channels differ in size, as those of keys and values do."""
    gain = torch.exp(0.5 * torch.randn(heads, d, generator=gen, device=DEV))
    return (torch.randn(n, heads, d, generator=gen, device=DEV) * gain).to(torch.bfloat16)


def _random_pool(gen, case, n_pages):
    """Key and value pages [n_pages][heads][page][d] and their row scales, as a running server's pool holds them."""
    out = {}
    for side in ("k", "v"):
        shape = (n_pages, case["hkv"], case["page"], case["d"])
        scales = torch.zeros(shape[:3], dtype=torch.float32, device=DEV) if case["type"] != "bf16" else None
        dtype = {"bf16": torch.bfloat16, "i8": torch.int8, "e4m3": torch.float8_e4m3fn}[case["type"]]
        codes = torch.empty(shape, dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype, device=DEV)
        gain = torch.exp(0.5 * torch.randn(1, case["hkv"], 1, case["d"], generator=gen, device=DEV))
        step = max(1, (64 << 20) // (shape[1] * shape[2] * shape[3]))
        for p in range(0, n_pages, step):
            x = (torch.randn((min(step, n_pages - p),) + shape[1:], generator=gen, device=DEV) * gain).to(torch.bfloat16)
            if case["type"] == "bf16":
                codes[p:p + step] = x
            else:
                q, s = _quantise(x.float(), case["type"])
                codes[p:p + step] = q.view(torch.uint8) if case["type"] == "e4m3" else q
                scales[p:p + step] = s
        out[side] = codes.view(dtype)
        out[side + "_scale"] = scales
    return out


def _empty_pool(case, n_pages):
    dtype = {"bf16": torch.bfloat16, "i8": torch.int8, "e4m3": torch.float8_e4m3fn}[case["type"]]
    shape = (n_pages, case["hkv"], case["page"], case["d"])
    out = {}
    for side in ("k", "v"):
        out[side] = torch.zeros(shape, dtype=torch.uint8 if case["type"] == "e4m3" else dtype, device=DEV).view(dtype)
        out[side + "_scale"] = None if case["type"] == "bf16" else torch.zeros(shape[:3], dtype=torch.float32, device=DEV)
    return out


def _slots(gen, n, page, n_pages):
    """Slots of n consecutive tokens whose pages lie anywhere in the pool."""
    pages = torch.randperm(n_pages, generator=gen, device=DEV)
    t = torch.arange(n, device=DEV)
    return pages[t // page] * page + t % page


def _inputs(case, seed):
    gen = _gen(seed)
    st = {"case": case}
    d = case["d"]
    if case["op"] == "rope":
        n, hq, hkv = case["n"], case["hq"], case["hkv"]
        if case["fused"]:
            # q | k | v columns of one projection
            qkv = torch.randn(n, (hq + 2 * hkv) * d, generator=gen, device=DEV).to(torch.bfloat16)
            st["q"] = qkv[:, :hq * d].view(n, hq, d)
            st["k"] = qkv[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
        else:
            st["q"], st["k"] = _rows(gen, n, hq, d), _rows(gen, n, hkv, d)
        first = int(torch.randint(max(1, case["far"] - n + 1), (1,), generator=gen, device=DEV))
        st["pos"] = (first + torch.arange(n, device=DEV)).to(torch.int32)
    elif case["op"] == "store":
        n, hkv = case["n"], case["hkv"]
        nr = case["rows"] or n
        if case["fused"]:
            kv = torch.randn(nr, 2 * hkv * d, generator=gen, device=DEV).to(torch.bfloat16)
            st["k"], st["v"] = kv[:, :hkv * d].view(nr, hkv, d), kv[:, hkv * d:].view(nr, hkv, d)
        else:
            st["k"], st["v"] = _rows(gen, nr, hkv, d), _rows(gen, nr, hkv, d)
        st["rows"] = None
        if case["rows"]:
            st["rows"] = torch.sort(torch.randperm(nr, generator=gen, device=DEV)[:n]).values.to(torch.int32)
        n_pages = -(-n // case["page"]) + 3
        st["slots"] = _slots(gen, n, case["page"], n_pages)
        st["pool"] = _empty_pool(case, n_pages)
    elif case["op"] == "fetch":
        n_pages = -(-case["n"] // case["page"]) + 3
        st["pool"] = _random_pool(gen, case, n_pages)
        st["slots"] = _slots(gen, case["n"], case["page"], n_pages)
    else:
        lens, nq = _lengths(case)
        per = -(-lens // case["page"])
        n_pages = int(per.sum()) + 3
        st["pool"] = _random_pool(gen, case, n_pages)
        order = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
        table = torch.zeros(case["seqs"], int(per.max()), dtype=torch.int32, device=DEV)
        at = 0
        for s in range(case["seqs"]):
            table[s, :per[s]] = order[at:at + per[s]]
            at += int(per[s])
        cu = np.concatenate([[0], np.cumsum(nq)])
        st["table"] = table
        st["lens"] = torch.from_numpy(lens.astype(np.int32)).to(DEV)
        st["cu"] = torch.from_numpy(cu.astype(np.int32)).to(DEV)
        st["host"] = (lens.tolist(), nq.tolist(), cu.tolist())
        st["q"] = (1.5 * torch.randn(int(cu[-1]), case["hq"], d, generator=gen, device=DEV)).to(torch.bfloat16)
        st["tree"] = None
        if case["tree"]:
            # each node hangs on a random earlier one; it sees itself and its ancestors
            rng = np.random.default_rng(seed)
            words = np.zeros(int(cu[-1]), np.uint64)
            for s in range(case["seqs"]):
                for i in range(int(nq[s])):
                    up = words[cu[s] + rng.integers(0, i)] if i and rng.random() < 0.9 else np.uint64(0)
                    words[cu[s] + i] = up | (np.uint64(1) << np.uint64(i))
            st["tree"] = torch.from_numpy(words.view(np.int64)).to(DEV)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    d = case["d"]
    if case["op"] == "rope":
        st["q_out"] = torch.empty(case["n"], case["hq"], d, dtype=torch.bfloat16, device=DEV)
        st["k_out"] = torch.empty(case["n"], case["hkv"], d, dtype=torch.bfloat16, device=DEV)
    elif case["op"] in ("store", "fetch"):
        st["k_out"] = torch.empty(case["n"], case["hkv"], d, dtype=torch.bfloat16, device=DEV)
        st["v_out"] = torch.empty_like(st["k_out"])
    else:
        st["o"] = torch.empty_like(st["q"])
    if own:
        from hybrid_gated_deltanet_q4k_gb300 import api
        if case["op"] == "rope":
            st["rope"] = api.RopeTable(case["rot"], base=case["base"], layout=case["layout"], scaling=case["scaling"],
                                       factor=case["factor"], orig_len=case["orig"])
        else:
            st["cache"] = api.KvCache(case["type"], st["pool"]["k"], st["pool"]["v"], st["pool"]["k_scale"],
                                      st["pool"]["v_scale"])
            if case["op"] == "attend":
                st["ws"] = st["cache"].new_attend_workspace(st["q"].shape[0], case["hq"])
    else:
        if case["op"] == "rope":
            st["freq"] = torch.from_numpy(_frequencies(case)).to(DEV)
        elif case["op"] == "attend":
            lens, nq, cu = st["host"]
            st["pages"] = [st["table"][s, :-(-lens[s] // case["page"])].long() for s in range(case["seqs"])]
    return st


# ---------------------------------------------------------------- the plain forms

def _frequencies(case):
    """Radians per position of each pair (fp64)."""
    f = case["base"] ** (-2.0 * np.arange(case["rot"] // 2, dtype=np.float64) / case["rot"])
    if case["scaling"] == "linear":
        f = f / case["factor"]
    elif case["scaling"] == "parts":
        turns = case["orig"] * f / (2 * np.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        f = f * keep + f / case["factor"] * (1.0 - keep)
    return f


def _amplitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "parts" else 1.0


def _rotate(x, cos, sin, rot, layout):
    x = x.float()
    c, s = cos[:, None, :], sin[:, None, :]
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * s, a * s + b * c], dim=-1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)
    return torch.cat([y, x[..., rot:]], dim=-1).to(torch.bfloat16)


def _quantise(x, kind):
    """Codes and fp32 scale of each row: scale = amax / code maximum, code = x / scale rounded, all in fp32."""
    top = torch.tensor(CODE_MAX[kind], dtype=torch.float32, device=x.device)
    scale = x.abs().amax(dim=-1) / top
    y = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x))
    y = torch.minimum(torch.maximum(y, -top), top)
    if kind == "i8":
        return torch.round(y).to(torch.int8), scale
    return y.to(torch.float8_e4m3fn), scale


def _pool_rows(pool, page, off):
    """fp32 key and value rows [n][heads][d] at (page, offset)."""
    out = []
    for side in ("k", "v"):
        codes = pool[side]
        if codes.dtype == torch.float8_e4m3fn:
            x = codes.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn).float()
        else:
            x = codes[page, :, off].float()
        if pool[side + "_scale"] is not None:
            x = x * pool[side + "_scale"][page, :, off][..., None]
        out.append(x)
    return out


def _plain_store(st):
    case, pool = st["case"], st["pool"]
    page, off = st["slots"] // case["page"], st["slots"] % case["page"]
    for side in ("k", "v"):
        x = st[side] if st["rows"] is None else st[side][st["rows"].long()]
        if case["type"] == "bf16":
            pool[side][page, :, off] = x
        else:
            q, s = _quantise(x.float(), case["type"])
            if case["type"] == "e4m3":
                pool[side].view(torch.uint8)[page, :, off] = q.view(torch.uint8)
            else:
                pool[side][page, :, off] = q
            pool[side + "_scale"][page, :, off] = s


def _plain_fetch(st):
    page, off = st["slots"] // st["case"]["page"], st["slots"] % st["case"]["page"]
    k, v = _pool_rows(st["pool"], page, off)
    return {"k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16)}


def _plain_attend(st):
    case, pool = st["case"], st["pool"]
    lens, nq, cu = st["host"]
    ratio, d = case["hq"] // case["hkv"], case["d"]
    outs = []
    for s in range(case["seqs"]):
        n, m = lens[s], nq[s]
        kv = []
        for side in ("k", "v"):
            x = pool[side]
            x = (x.view(torch.uint8)[st["pages"][s]].view(x.dtype) if x.dtype == torch.float8_e4m3fn
                 else x[st["pages"][s]]).float()
            if pool[side + "_scale"] is not None:
                x = x * pool[side + "_scale"][st["pages"][s]][..., None]
            kv.append(x.transpose(0, 1).reshape(case["hkv"], -1, d)[:, :n])
        q = st["q"][cu[s]:cu[s] + m].float().view(m, case["hkv"], ratio, d).permute(1, 0, 2, 3).reshape(case["hkv"], -1, d)
        score = torch.matmul(q, kv[0].transpose(1, 2)).view(case["hkv"], m, ratio, n) * d ** -0.5
        j = torch.arange(m, device=DEV)
        if st["tree"] is None:
            seen = j[None, :] <= j[:, None]
        else:
            seen = (st["tree"][cu[s]:cu[s] + m, None] >> j[None, :]) & 1 == 1
        seen = torch.cat([torch.ones(m, n - m, dtype=torch.bool, device=DEV), seen], dim=1)
        score = score.masked_fill(~seen[None, :, None, :], float("-inf"))
        score = score - score.amax(dim=-1, keepdim=True)
        p = torch.exp(score)
        p = (p / p.sum(dim=-1, keepdim=True)).view(case["hkv"], m * ratio, n)
        o = torch.matmul(p, kv[1]).view(case["hkv"], m, ratio, d).permute(1, 0, 2, 3).reshape(m, case["hq"], d)
        outs.append(o.to(torch.bfloat16))
    return {"o": torch.cat(outs)}


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        if op == "rope":
            st["rope"].apply(st["pos"], st["q"], st["k"], st["q_out"], st["k_out"])
            return {"q": st["q_out"], "k": st["k_out"]}
        cache = st["cache"]
        if op == "attend":
            cache.attend(st["q"], st["lens"], st["table"], st["o"], st["ws"], cu_q=st["cu"], max_q=case["qhi"],
                         tree=st["tree"])
            return {"o": st["o"]}
        if op == "store":
            cache.write(st["k"], st["v"], st["slots"], rows=st["rows"])
        cache.read(st["slots"], st["k_out"], st["v_out"])
        return {"k": st["k_out"], "v": st["v_out"]}
    if op == "rope":
        angle = st["pos"].double()[:, None] * st["freq"][None, :]
        amp = _amplitude(case)
        cos, sin = (torch.cos(angle) * amp).float(), (torch.sin(angle) * amp).float()
        return {"q": _rotate(st["q"], cos, sin, case["rot"], case["layout"]),
                "k": _rotate(st["k"], cos, sin, case["rot"], case["layout"])}
    if op == "attend":
        return _plain_attend(st)
    if op == "store":
        _plain_store(st)
    return _plain_fetch(st)


# ---------------------------------------------------------------- work

def work(case):
    d = case["d"]
    if case["op"] == "rope":
        heads = case["hq"] + case["hkv"]
        return {"bytes": 2 * case["n"] * heads * d * 2 + 4 * case["n"], "flops": 3 * case["n"] * heads * case["rot"]}
    size = 2 if case["type"] == "bf16" else 1
    row = d * size + (0 if size == 2 else 4)          # a cached row of one head, with its scale
    if case["op"] in ("store", "fetch"):
        n = 2 * case["n"] * case["hkv"]
        moves = 2 if case["op"] == "store" else 1     # written and read back, or read
        return {"bytes": n * (moves * row + moves * 2 * d) + 8 * case["n"], "flops": moves * n * d}
    lens, nq = _lengths(case)
    keys = int((lens.astype(np.int64) * case["hkv"]).sum())
    pairs = int((lens.astype(np.int64) * nq).sum()) * case["hq"]
    return {"bytes": 2 * keys * row + 2 * int(nq.sum()) * case["hq"] * d * 2, "flops": 4 * pairs * d}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_frequency(case, i):
    f = math.pow(case["base"], -2.0 * i / case["rot"])
    if case["scaling"] == "linear":
        return f / case["factor"]
    if case["scaling"] == "parts":
        turns = case["orig"] * f / (2.0 * math.pi)
        w = 0.0 if turns <= 1.0 else 1.0 if turns >= 32.0 else (turns - 1.0) / 31.0
        return w * f + (1.0 - w) * f / case["factor"]
    return f


def _exact_rope(case, st):
    """Each pair as a complex number times amp e^(i pos f)."""
    half = case["rot"] // 2
    f = torch.tensor([_exact_frequency(case, i) for i in range(half)], dtype=torch.float64, device=DEV)
    amp = 1.0 + 0.1 * math.log(case["factor"]) if case["scaling"] == "parts" else 1.0
    turn = torch.polar(torch.full((case["n"], half), amp, dtype=torch.float64, device=DEV),
                       st["pos"].to(torch.float64).outer(f))
    out = {}
    for name in ("q", "k"):
        y = st[name].to(torch.float64).clone()
        first = torch.arange(half, device=DEV) * (1 if case["layout"] == "half" else 2)
        second = first + (half if case["layout"] == "half" else 1)
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None, :]
        y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
    return out


def _exact_values(x, kind):
    """What a stored row stands for: the scale is an fp32 number and each quotient is rounded to fp32 by definition."""
    x = x.to(torch.float64)
    if kind == "bf16":
        return x
    top = 127.0 if kind == "i8" else 448.0
    scale = (x.abs().max(dim=-1, keepdim=True).values / top).to(torch.float32).to(torch.float64)
    y = (x / scale.clamp_min(1e-300)).to(torch.float32).to(torch.float64)
    if kind == "i8":
        code = torch.clamp(torch.round(y), -127.0, 127.0)
    else:
        # 3 fraction bits, the smallest normal number 2^-6
        _, e = torch.frexp(torch.clamp(y, -448.0, 448.0))
        step = torch.exp2(torch.clamp(e - 1, min=-6).to(torch.float64) - 3.0)
        code = torch.round(torch.clamp(y, -448.0, 448.0) / step) * step
    return code * scale


def _exact_pool(case, pool, side, slots):
    """Rows [n][heads][d] of the pool in 64 bits."""
    flat = pool[side].transpose(1, 2).reshape(-1, case["hkv"], case["d"]) if case["type"] != "e4m3" else \
        pool[side].view(torch.uint8).transpose(1, 2).reshape(-1, case["hkv"], case["d"])
    x = flat[slots]
    if case["type"] == "e4m3":
        b = x.to(torch.int64)
        e, m = (b >> 3) & 15, (b & 7).to(torch.float64)
        mag = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2((e - 10).to(torch.float64)))
        x = torch.where(b >= 128, -mag, mag)
    x = x.to(torch.float64)
    if case["type"] != "bf16":
        x = x * pool[side + "_scale"].transpose(1, 2).reshape(-1, case["hkv"])[slots].to(torch.float64)[..., None]
    return x


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, st)
    if case["op"] == "store":
        pick = (lambda x: x) if st["rows"] is None else (lambda x: x[st["rows"].to(torch.int64)])
        return {side: _exact_values(pick(st[side]), case["type"]) for side in ("k", "v")}
    if case["op"] == "fetch":
        return {side: _exact_pool(case, st["pool"], side, st["slots"]) for side in ("k", "v")}
    lens, nq, cu = st["host"]
    ratio = case["hq"] // case["hkv"]
    out = torch.empty(cu[-1], case["hq"], case["d"], dtype=torch.float64, device=DEV)
    for s in range(case["seqs"]):
        t = torch.arange(lens[s], device=DEV)
        slots = st["table"][s].to(torch.int64)[t // case["page"]] * case["page"] + t % case["page"]
        k, v = (_exact_pool(case, st["pool"], side, slots) for side in ("k", "v"))
        ctx = lens[s] - nq[s]
        hidden = torch.zeros(nq[s], lens[s], dtype=torch.bool, device=DEV)
        for i in range(nq[s]):
            word = (1 << (i + 1)) - 1 if st["tree"] is None else int(st["tree"][cu[s] + i]) & (2 ** 64 - 1)
            hidden[i, ctx:] = torch.tensor([not (word >> j) & 1 for j in range(nq[s])], device=DEV)
        for h in range(case["hq"]):
            a = st["q"][cu[s]:cu[s + 1], h].to(torch.float64) @ k[:, h // ratio].t() / math.sqrt(case["d"])
            a[hidden] = -math.inf
            out[cu[s]:cu[s + 1], h] = torch.softmax(a, dim=-1) @ v[:, h // ratio]
    return {"o": out}
