"""Measured cases of the operators that decide drafted tokens.

The short conv and the gated delta rule over a chain or tree of drafted tokens
(``conv``, ``delta``), the move of the held state to the accepted token
(``commit``), the verification of the drafts against the target's probabilities
(``verify``), and the block tables and slots of the tokens (``plan``), each in a
plain form (elementary torch operations) and through the framework's public
calls.  The heads are those of the hybrid model's GDN layers (16 query/key heads
and 32 value heads of 128) and generic ones.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one user, a chain of three drafts: latency alone
        dict(name="conv_one", op="conv", seqs=1, lo=4, hi=4, tree=0, hk=16, hv=32, d=128),
        # trees of a full serving batch
        dict(name="conv_trees", op="conv", seqs=48, lo=20, hi=64, tree=1, hk=16, hv=32, d=128),
        # one user, a chain of three drafts: latency alone
        dict(name="delta_one", op="delta", seqs=1, lo=4, hi=4, tree=0, hk=16, hv=32, d=128),
        # a serving batch, each with a short chain of its own length
        dict(name="delta_chains", op="delta", seqs=64, lo=1, hi=8, tree=0, hk=16, hv=32, d=128),
        # large trees of a smaller batch
        dict(name="delta_trees", op="delta", seqs=24, lo=24, hi=64, tree=1, hk=16, hv=32, d=128),
        # one user's accepted chain
        dict(name="commit_one", op="commit", seqs=1, lo=4, hi=4, tree=0, hk=16, hv=32, d=128),
        # the accepted paths of a serving batch's trees
        dict(name="commit_batch", op="commit", seqs=64, lo=1, hi=32, tree=1, hk=16, hv=32, d=128),
        # one user, a chain of drafts that came with their draft model's probabilities
        dict(name="verify_one", op="verify", seqs=1, lo=5, hi=5, tree=0, vocab=150001, type="f32", q=1, greedy=0),
        # a serving batch, chains, the likeliest token is the answer
        dict(name="verify_greedy", op="verify", seqs=32, lo=1, hi=6, tree=0, vocab=128000, type="bf16", q=0, greedy=1),
        # trees sampled from a draft model, several children tried at a node
        dict(name="verify_trees", op="verify", seqs=16, lo=12, hi=32, tree=1, vocab=150001, type="f32", q=1, greedy=0),
        # the tables of a step of drafted trees
        dict(name="plan_step", op="plan", seqs=64, lo=1, hi=32, tree=1, held=20000, page=64, short=0),
        # the tables of a batch of new prompts
        dict(name="plan_prompts", op="plan", seqs=256, lo=1, hi=8192, tree=0, held=3000, page=16, short=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    """Nanoseconds of a pass at 6.7 TB/s and, for the products in 32 bits, 60 TFLOP/s, one after the other."""
    w = work(case)
    return w["bytes"] / 6.7e3 + w["flops"] / 60e3


def draw(rng):
    case = _draw(rng)
    top = max(_cost(c) for c in listed() if c["op"] == case["op"])
    while _cost(case) > top:
        if case["seqs"] > 1:
            case["seqs"] = case["seqs"] * 2 // 3
        else:
            case["hi"] = max(1, case["hi"] * 2 // 3)
            case["lo"] = min(case["lo"], case["hi"])
    return case


def _draw(rng):
    op = rng.choice(["conv", "delta", "delta", "commit", "verify", "verify", "plan"])
    tree = rng.randint(0, 1)
    hi = rng.randint(2, 64) if tree else _log(rng, 1, 24)
    lo = rng.randint(0 if rng.random() < 0.3 else 1, hi)
    seqs = _log(rng, 1, 64)
    if op in ("conv", "delta", "commit"):
        hk = rng.choice([1, 2, 4, 8, 16])
        return dict(op=op, seqs=seqs, lo=lo, hi=hi, tree=tree, hk=hk, hv=hk * rng.choice([1, 2, 3, 4]), d=rng.choice([64, 128, 128]))
    if op == "verify":
        vocab = _log(rng, 1000, 260000)
        seqs = max(1, min(seqs, 60000000 // (vocab * hi)))
        greedy = int(rng.random() < 0.3)
        return dict(op=op, seqs=seqs, lo=lo, hi=hi, tree=tree, vocab=vocab, type=rng.choice(["f32", "bf16"]),
                    q=0 if greedy else rng.randint(0, 1), greedy=greedy)
    if not tree:
        hi = _log(rng, 1, 8192)
        lo = rng.randint(0, hi)
    return dict(op=op, seqs=_log(rng, 1, 256), lo=lo, hi=hi, tree=tree, held=_log(rng, 1, 100000), page=rng.choice([16, 32, 64, 128]),
                short=int(rng.random() < 0.25))


# ---------------------------------------------------------------- inputs

def _rng(case, more=0):
    """The sizes of a case's sequences belong to the case."""
    return np.random.default_rng([case["seqs"], case["lo"], case["hi"], case["tree"], more])


def _lengths(case):
    n = _rng(case).integers(case["lo"], case["hi"] + 1, size=case["seqs"])
    n[0] = case["hi"]
    return n


def _words(n, rng):
    """Mask words of trees whose nodes hang on random earlier ones; the first token of a sequence is the root."""
    out = np.zeros(int(n.sum()), np.uint64)
    at = 0
    for m in n.tolist():
        for i in range(m):
            up = out[at + rng.integers(0, i)] if i else np.uint64(0)
            out[at + i] = up | (np.uint64(1) << np.uint64(i))
        at += m
    return out


def _paths(case, st):
    """Per token: its index in its sequence and its parent's (-1: none)."""
    local = torch.arange(st["total"], device=DEV) - st["first"]
    if st["tree"] is None:
        return local, local - 1
    bit = torch.arange(64, device=DEV)
    up = ((st["tree"][:, None] >> bit) & 1 == 1) & (bit < local[:, None])
    return local, torch.where(up, bit, torch.full_like(bit, -1)).amax(dim=1)


def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) & 0x7FFFFFFF)
    rng = np.random.default_rng(int(seed) & 0x7FFFFFFF)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)  # noqa: E731
    ints = lambda a, t=np.int32: torch.from_numpy(np.ascontiguousarray(a, dtype=t)).to(DEV)  # noqa: E731
    n = _lengths(case)
    cu = np.concatenate([[0], np.cumsum(n)])
    s, t = case["seqs"], int(cu[-1])
    st = {"case": case, "n": n, "total": t, "cu": ints(cu)}
    st["first"] = ints(np.repeat(cu[:-1], n), np.int64)       # a token's sequence and that one's first token
    st["seq"] = ints(np.repeat(np.arange(s), n), np.int64)
    st["tree"] = torch.from_numpy(_words(n, rng).view(np.int64)).to(DEV) if case["tree"] else None
    if case["op"] in ("conv", "delta", "commit"):
        hk, hv, d = case["hk"], case["hv"], case["d"]
        c = (2 * hk + hv) * d
        st["qkvz"] = rand(t, c + hv * d).to(torch.bfloat16)
        st["tail"] = rand(s, c, 3).to(torch.bfloat16).float()
        if case["op"] == "conv":
            st["ba"] = rand(t, 2 * hv)
            st["conv_w"] = 0.5 * rand(c, 4)
            st["A_log"], st["dt"] = 0.3 * rand(hv), 0.3 * rand(hv)
            return st
        norm = lambda x: x / torch.sqrt((x * x).sum(dim=-1, keepdim=True) + EPS)  # noqa: E731
        # keys of one sequence share a direction, as those of neighbouring tokens do
        q = norm(rand(t, hk, d)) * d ** -0.5
        k = norm(rand(t, hk, d) + 0.7 * rand(s, hk, d)[st["seq"]])
        st["qkv"] = torch.cat([q.flatten(1), k.flatten(1), 0.5 * rand(t, hv * d)], dim=1).to(torch.float16)
        u = rand(t, hv)
        st["log_a"] = -(torch.clamp(u, min=0) + torch.log1p(torch.exp(-u.abs())))
        st["b"] = torch.sigmoid(rand(t, hv))
        st["state"] = 0.3 * rand(s, hv, d, d)
        if case["op"] == "commit":
            st["delta"] = 0.4 * rand(t, hv, d)
            # deeper nodes are accepted as well as the root; some sequences keep their state
            node = np.minimum(rng.integers(-1, 8, size=s) if s > 1 else np.array([2]), n - 1)
            st["node"] = ints(node)
    elif case["op"] == "verify":
        v = case["vocab"]
        dtype = torch.float32 if case["type"] == "f32" else torch.bfloat16
        x = 3.0 * rand(t, v)
        if case["greedy"]:
            st["p"], st["q"] = x.to(dtype), None
        else:
            st["p"] = torch.softmax(x, dim=1).to(dtype)
            st["q"] = torch.softmax(x.add_(rand(t, v)), dim=1).to(dtype) if case["q"] else None
        st["u"] = torch.rand(t, generator=gen, device=DEV)
        st["u_next"] = torch.rand(s, generator=gen, device=DEV)
        # a draft comes from the draft's probabilities at its parent, or guesses the target's
        _, up = _paths(case, st)
        row = (st["first"] + up).clamp(min=0)
        if case["greedy"]:
            best = _first(x.to(dtype) == x.to(dtype).amax(dim=1, keepdim=True))[row]
            guess = torch.randint(v, (t,), generator=gen, device=DEV)
            tokens = torch.where(torch.rand(t, generator=gen, device=DEV) < 0.6, best, guess)
        else:
            src = st["q"] if case["q"] else st["p"]
            tokens = torch.multinomial(src[row].float(), 1, generator=gen)[:, 0]
        st["tokens"] = tokens.to(torch.int32)
    else:
        page = case["page"]
        lens = _rng(case, 1).integers(0, case["held"] + 1, size=s)
        blocks = -(-(lens + n) // page)
        had = np.minimum(-(-lens // page) + rng.integers(0, 3, size=s), blocks)    # some of the last step's pages are left over
        n_pages = int(blocks.sum()) + 5
        wide = int(blocks.max()) + 2
        order = rng.permutation(n_pages).astype(np.int32)
        table = np.full((s, wide), -1, np.int32)
        at = 0
        for i in range(s):
            table[i, :had[i]] = order[at:at + had[i]]
            at += had[i]
        free = n_pages - at
        if case["short"]:
            free //= 2                                      # the last sequences find no pages
        stack = np.full(n_pages, -1, np.int32)
        stack[:free] = order[at:at + free]
        st.update(lens=ints(lens), n_new=ints(n), table=ints(table), n_blocks=ints(had), stack=ints(stack), n_free=ints([free]),
                  room=t if case["tree"] else t + t // 7 + 3, pages=n_pages)
    return st


def _layer(case, st):
    from hybrid_gated_deltanet_q4k_gb300 import synth
    from hybrid_gated_deltanet_q4k_gb300.api import DeviceLayer
    spec = synth.LayerSpec("drafts", 256, case["hk"], case["hv"], case["d"], case["d"], 1, "f32", 0, "softplus_normal")
    host = lambda x, shape: np.zeros(shape, np.float32) if x is None else x.cpu().numpy()  # noqa: E731
    params = {"w_in": np.zeros((spec.r_in, 256), np.float32), "w_out": np.zeros((256, spec.c_v), np.float32),
              "conv_w": host(st.get("conv_w"), (spec.c_conv, 4)), "A_log": host(st.get("A_log"), spec.n_v_heads),
              "dt_bias": host(st.get("dt"), spec.n_v_heads), "norm_w": np.ones(spec.dv, np.float32)}
    return DeviceLayer(spec, params, device=DEV, eps_l2=EPS)


def prepare(case, seed):
    st = _inputs(case, seed)
    t, s = st["total"], case["seqs"]
    new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
    if case["op"] == "conv":
        st["out"] = {"qkv": new(st["tail"].shape[1] * t, torch.float16).view(t, -1), "log_a": new((t, case["hv"]), torch.float32),
                     "b": new((t, case["hv"]), torch.float32)}
    elif case["op"] == "delta":
        st["out"] = {"o": new((t, case["hv"], case["d"]), torch.float16), "delta": new((t, case["hv"], case["d"]), torch.float32)}
    elif case["op"] == "commit":
        st["out"] = {"state": torch.empty_like(st["state"]), "tail": torch.empty_like(st["tail"])}
    elif case["op"] == "verify":
        st["out"] = {"rows": new(t, torch.int32), "ids": new(t, torch.int32), "count": new(s, torch.int32),
                     "node": new(s, torch.int32), "next": new(s, torch.int32)}
    else:
        st["out"] = {"lens": new(s, torch.int32), "cu": new(s + 1, torch.int32), "positions": new(st["room"], torch.int32),
                     "slots": new(st["room"], torch.int64)}
    if own:
        if case["op"] in ("conv", "delta", "commit"):
            st["layer"] = _layer(case, st)
        elif case["op"] == "verify":
            from hybrid_gated_deltanet_q4k_gb300 import api
            st["verify"] = api.verify
        else:
            from hybrid_gated_deltanet_q4k_gb300.api import KvPages
            st["book"] = KvPages(case["page"], st["table"], st["n_blocks"], st["stack"], st["n_free"])
    return st


# ---------------------------------------------------------------- the plain forms

def _padded(st, x, fill=0):
    """Rows [T] laid out as [seqs][most tokens]."""
    out = torch.full((st["case"]["seqs"], int(st["n"].max())) + x.shape[1:], fill, dtype=x.dtype, device=DEV)
    out[st["seq"], torch.arange(st["total"], device=DEV) - st["first"]] = x
    return out


def _ancestors(st):
    """[seqs][m][m]: 1 where j is a proper ancestor of i."""
    m = int(st["n"].max())
    j = torch.arange(m, device=DEV)
    earlier = (j[None, :] < j[:, None]).double()
    if st["tree"] is None:
        return earlier.expand(st["case"]["seqs"], m, m)
    return ((_padded(st, st["tree"])[:, :, None] >> j) & 1).double() * earlier


def _heads(st, part):
    """q, k or v of the tokens as [seqs][value heads][m][d] in 32 bits."""
    case = st["case"]
    hk, hv, d = case["hk"], case["hv"], case["d"]
    lo, h = {"q": (0, hk), "k": (hk, hk), "v": (2 * hk, hv)}[part]
    x = _padded(st, st["qkv"][:, lo * d:(lo + h) * d].float().view(-1, h, d)).transpose(1, 2)
    return x if part == "v" else x.repeat_interleave(hv // hk, dim=1)


def _taps(case, st):
    """Raw inputs [T][channels][4] of each token's conv, oldest first."""
    _, up = _paths(case, st)
    c = st["tail"].shape[1]
    x = torch.cat([st["qkvz"][:, :c].float(), st["tail"].transpose(1, 2).reshape(-1, c)])
    at, taps = torch.arange(st["total"], device=DEV), []
    before = torch.zeros_like(at)                              # steps taken past the sequence's first token
    for _ in range(4):
        row = torch.where(before > 0, st["total"] + 3 * st["seq"] + 3 - before, at)
        taps.insert(0, x[row])
        nxt = torch.where(before > 0, at, up[at] + st["first"])
        before = torch.where((before > 0) | (up[at] < 0), before + 1, before)
        at = torch.where(before > 0, at, nxt)
    return torch.stack(taps, dim=-1)


def _plain_conv(case, st):
    hk, hv, d = case["hk"], case["hv"], case["d"]
    u = (_taps(case, st) * st["conv_w"]).sum(dim=-1)
    y = (u / (1 + torch.exp(-u))).view(-1, 2 * hk + hv, d)
    r = torch.sqrt((y[:, :2 * hk] ** 2).sum(dim=-1, keepdim=True) + EPS)
    qk = y[:, :2 * hk] / r
    out = torch.cat([qk[:, :hk] * d ** -0.5, qk[:, hk:], y[:, 2 * hk:]], dim=1)
    w = st["ba"][:, hv:] + st["dt"]
    soft = torch.clamp(w, min=0) + torch.log1p(torch.exp(-w.abs()))
    return {"qkv": out.flatten(1).to(torch.float16), "log_a": -torch.exp(st["A_log"]) * soft, "b": 1 / (1 + torch.exp(-st["ba"][:, :hv]))}


def _plain_delta(case, st):
    q, k, v = _heads(st, "q"), _heads(st, "k"), _heads(st, "v")
    anc = _ancestors(st)[:, None]
    m = anc.shape[-1]
    g = torch.matmul(anc + torch.eye(m, device=DEV, dtype=torch.float64), _padded(st, st["log_a"]).double().transpose(1, 2)[..., None])
    decay = torch.exp(torch.where(anc > 0, g - g.transpose(2, 3), torch.zeros_like(g))).float() * anc.float()
    grow, b = torch.exp(g).float(), _padded(st, st["b"]).transpose(1, 2)[..., None]
    held = st["state"].transpose(2, 3)
    u = b * (v - grow * torch.matmul(k, held))
    mix = b * decay * torch.matmul(k, k.transpose(2, 3))
    for i in range(1, m):                                       # a node needs its ancestors' results
        u[:, :, i] -= torch.matmul(mix[:, :, i:i + 1, :i], u[:, :, :i])[:, :, 0]
    o = grow * torch.matmul(q, held) + torch.matmul((decay + torch.eye(m, device=DEV)) * torch.matmul(q, k.transpose(2, 3)), u)
    at = torch.arange(st["total"], device=DEV) - st["first"]
    return {"o": o[st["seq"], :, at].to(torch.float16), "delta": u[st["seq"], :, at]}


def _plain_commit(case, st):
    node = st["node"].long()
    path = _ancestors(st)
    m = path.shape[-1]
    path = (path + torch.eye(m, device=DEV, dtype=torch.float64))[torch.arange(case["seqs"], device=DEV), node.clamp(min=0)] * (node >= 0)[:, None]
    la = _padded(st, st["log_a"]).double().transpose(1, 2) * path[:, None]
    # the decay from a node on the path to its end: what lies after it
    after = la.sum(dim=2, keepdim=True) - torch.cumsum(la, dim=2)
    w = (torch.exp(after) * path[:, None]).float()
    grow = torch.exp(la.sum(dim=2)).float()[..., None, None]
    u = _padded(st, st["delta"]).transpose(1, 2)
    state = grow * st["state"] + torch.matmul((u * w[..., None]).transpose(2, 3), _heads(st, "k"))
    taps = torch.cat([_taps(case, st), torch.zeros(1, st["tail"].shape[1], 4, device=DEV)])
    last = torch.where(node >= 0, st["cu"][:-1].long() + node, torch.full_like(node, st["total"]))
    return {"state": state, "tail": torch.where(node[:, None, None] >= 0, taps[last][..., 1:], st["tail"])}


def _first(hit):
    """The lowest index of a row where `hit` holds (the row's length if nowhere)."""
    at = torch.arange(hit.shape[1], device=DEV)
    return torch.where(hit, at, torch.full_like(at, hit.shape[1])).amin(dim=1)


def _plain_verify(case, st):
    s, t, v = case["seqs"], st["total"], case["vocab"]
    n = st["cu"][1:] - st["cu"][:-1]
    _, up = _paths(case, st)
    up, tok = _padded(st, up, -2), _padded(st, st["tokens"].long())
    draw_u = _padded(st, st["u"]).double()
    first, each = st["cu"][:-1].long(), torch.arange(s, device=DEV)
    some = n > 0
    cur, depth = torch.zeros(s, dtype=torch.long, device=DEV), torch.zeros(s, dtype=torch.long, device=DEV)
    last = max(t - 1, 0)
    rows = torch.full((s, up.shape[1]), -1, dtype=torch.long, device=DEV)
    ids = rows.clone()
    rows[:, 0] = first
    row_of = lambda c: (first + c).clamp(max=last)  # noqa: E731
    c0, z = torch.zeros(s, dtype=torch.float64, device=DEV), torch.ones(s, dtype=torch.float64, device=DEV)
    gone = torch.zeros(s, v, dtype=torch.bool, device=DEV)      # tokens that were rejected at the current node
    pick = lambda m: m[row_of(cur)]  # noqa: E731
    weight = lambda: torch.clamp(pick(st["p"]).double() - (c0[:, None] * pick(st["q"]).double() if st["q"] is not None  # noqa: E731
                                                           else gone * 2.0), min=0)
    if case["greedy"]:
        best = _first(st["p"].float() == st["p"].float().amax(dim=1, keepdim=True))
    for i in range(1, up.shape[1]):                              # each node's fate depends on those before it
        asked = up[:, i] == cur
        x = tok[:, i]
        if case["greedy"]:
            ok = best[row_of(cur)] == x
        else:
            p = st["p"][row_of(cur), x].double()
            if st["q"] is not None:
                ok = (c0 + draw_u[:, i] * z) * st["q"][row_of(cur), x].double() < p
            else:
                ok = draw_u[:, i] * z < torch.where(gone[each, x], torch.zeros_like(p), p)
            no = asked & ~ok
            c0 = torch.where(no, c0 + z, c0)
            gone[each, x] |= no
            z = torch.where(no, weight().sum(dim=1), z)
        yes = asked & ok
        cur, depth = torch.where(yes, i, cur), depth + yes
        ids[each, (depth - 1).clamp(min=0)] = torch.where(yes, x, ids[each, (depth - 1).clamp(min=0)])
        rows[each, depth] = torch.where(yes, first + i, rows[each, depth])
        c0, z = torch.where(yes, torch.zeros_like(c0), c0), torch.where(yes, torch.ones_like(z), z)
        gone &= ~yes[:, None]
    if case["greedy"]:
        nxt = best[row_of(cur)]
    else:
        w = weight()
        w = torch.where(w.sum(dim=1, keepdim=True) > 0, w, torch.clamp(pick(st["p"]).double(), min=0))
        run_sum = torch.cumsum(w, dim=1)
        nxt = _first(run_sum > st["u_next"].double()[:, None] * run_sum[:, -1:])
    ids[each, depth] = nxt
    at = torch.arange(t, device=DEV) - st["first"]
    pack = lambda m: torch.where(m[st["seq"], at] < 0, -1, m[st["seq"], at]).to(torch.int32)  # noqa: E731
    none = torch.full_like(cur, -1)
    return {"rows": pack(rows), "ids": pack(ids), "count": torch.where(some, depth + 1, 0).to(torch.int32),
            "node": torch.where(some, cur, none).to(torch.int32), "next": torch.where(some, nxt, none).to(torch.int32)}


def _plain_plan(case, st):
    page, wide, n_pages = case["page"], st["table"].shape[1], st["pages"]
    lens, new = st["lens"].long(), st["n_new"].long()
    col = torch.arange(wide, device=DEV)
    # what the sequences hold past their lengths goes back on the stack, the first of it on top
    keep = torch.minimum(st["n_blocks"].long(), -(-lens // page))
    back = (col >= keep[:, None]) & (col < st["n_blocks"].long()[:, None])
    rank, some = torch.cumsum(back.flatten().long(), 0) - 1, back.sum()
    stack = torch.cat([st["stack"], st["stack"][:1]])            # the last place takes what has no other
    stack[torch.where(back.flatten(), st["n_free"].long() + some - 1 - rank, n_pages)] = st["table"].flatten()
    free = st["n_free"].long() + some
    # pages for the new tokens, in the order of the sequences, from the top
    need = torch.clamp(-(-(lens + new) // page) - keep, min=0)
    upto = torch.cumsum(need, 0)
    got = (need == 0) | (upto <= free)
    need = torch.where(got, need, 0)
    blocks = keep + need
    add = (col >= keep[:, None]) & (col < blocks[:, None])
    rank = (upto - need)[:, None] + col - keep[:, None]
    table = torch.where(add, stack[torch.where(add, free - 1 - rank, 0)], st["table"])
    st["table"].copy_(table)
    st["stack"].copy_(stack[:-1])
    st["n_blocks"].copy_(blocks)
    st["n_free"].copy_(free - need.sum())
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(new, 0)])
    tok = torch.arange(st["room"], device=DEV)
    seq = (torch.searchsorted(cu, tok, right=True) - 1).clamp(max=case["seqs"] - 1)
    i = tok - cu[seq]
    pos = lens[seq] + i
    slot = table[seq, (pos // page).clamp(max=wide - 1)].long() * page + pos % page
    if st["tree"] is not None:
        depth = _depth(st)
        pos = lens[seq] + depth
    live = tok < cu[-1]
    return {"lens": torch.where(got, lens + new, lens).to(torch.int32), "cu": cu.to(torch.int32),
            "positions": torch.where(live, pos, 0).to(torch.int32), "slots": torch.where(live & got[seq], slot, -1),
            "table": st["table"], "n_blocks": st["n_blocks"], "n_free": st["n_free"]}


def _depth(st):
    local = torch.arange(st["total"], device=DEV) - st["first"]
    bit = torch.arange(64, device=DEV)
    return (((st["tree"][:, None] >> bit) & 1 == 1) & (bit < local[:, None])).sum(dim=1)


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"conv": _plain_conv, "delta": _plain_delta, "commit": _plain_commit, "verify": _plain_verify,
                "plan": _plain_plan}[op](case, st)
    out, more = st["out"], dict(cu=st["cu"], max_new=case["hi"], tree=st["tree"])
    if op == "conv":
        st["layer"].conv_tree(st["qkvz"], st["ba"], st["tail"], out["qkv"], out["log_a"], out["b"], **more)
    elif op == "delta":
        st["layer"].delta_tree(st["qkv"], st["log_a"], st["b"], st["state"], out["o"], out["delta"], **more)
    elif op == "commit":
        st["layer"].delta_commit(st["qkv"], st["log_a"], st["delta"], st["node"], st["state"], out["state"], st["qkvz"], st["tail"],
                                 out["tail"], **more)
    elif op == "verify":
        u, u_next = (None, None) if case["greedy"] else (st["u"], st["u_next"])
        st["verify"](st["p"], st["tokens"], out["rows"], out["ids"], out["count"], out["node"], out["next"], u=u, u_next=u_next, q=st["q"],
                     **more)
    else:
        st["book"].trim(st["lens"])
        st["book"].extend(st["lens"], st["n_new"], out["lens"], out["cu"], out["positions"], out["slots"], tree=st["tree"])
        return {**out, "table": st["table"], "n_blocks": st["n_blocks"], "n_free": st["n_free"]}
    return out


# ---------------------------------------------------------------- work

def work(case):
    n = _lengths(case).astype(np.int64)
    s, t = case["seqs"], int(n.sum())
    if case["op"] in ("conv", "delta", "commit"):
        hk, hv, d = case["hk"], case["hv"], case["d"]
        c = (2 * hk + hv) * d
        if case["op"] == "conv":
            return {"bytes": t * (4 * c + 16 * hv) + s * c * 12 + c * 16, "flops": t * c * 14}
        state = s * hv * d * d
        if case["op"] == "delta":
            pairs = int((n * n).sum()) * hv
            return {"bytes": 4 * state + t * (2 * c + 8 * hv + 6 * hv * d), "flops": 4 * t * hv * d * d + 4 * pairs * d}
        return {"bytes": 8 * state + s * c * 24, "flops": 4 * state}
    if case["op"] == "verify":
        # the row that the next token comes from, of each sequence
        size = 4 if case["type"] == "f32" else 2
        return {"bytes": s * case["vocab"] * size * (1 + case["q"]) + 16 * t + 16 * s, "flops": 3 * s * case["vocab"]}
    return {"bytes": 12 * t + 4 * (int((n / case["page"]).sum()) + 6 * s), "flops": 4 * t}


# ---------------------------------------------------------------- the definition in 64 bits

def _host_paths(case, st):
    """Parents by sequence, from the mask words on the host."""
    words = None if st["tree"] is None else st["tree"].cpu().numpy().view(np.uint64)
    out, at = [], 0
    for m in st["n"].tolist():
        out.append([i - 1 if words is None else (int(words[at + i]) & ((1 << i) - 1)).bit_length() - 1 for i in range(m)])
        at += m
    return out


def _exact_tail(st, parents, s, node):
    """The last three raw inputs [channels][3] of a sequence up to `node`, oldest first."""
    at, c, out = int(st["cu"][s]), st["tail"].shape[1], []
    while node >= 0 and len(out) < 3:
        out.insert(0, st["qkvz"][at + node, :c].double())
        node = parents[s][node]
    old = st["tail"][s].double()
    return torch.stack([old[:, len(out) + j] for j in range(3 - len(out))] + out, dim=1)


def _exact_conv(case, st):
    hk, hv, d = case["hk"], case["hv"], case["d"]
    parents = _host_paths(case, st)
    c, w = st["tail"].shape[1], st["conv_w"].double()
    rows = []
    for s, up in enumerate(parents):
        for i, p in enumerate(up):
            x = torch.cat([_exact_tail(st, parents, s, p), st["qkvz"][int(st["cu"][s]) + i, :c].double()[:, None]], dim=1)
            y = torch.einsum("cj,cj->c", x, w)
            y = (y * torch.sigmoid(y)).view(-1, d)
            size = torch.sqrt(torch.einsum("hd,hd->h", y, y) + EPS)[:, None]
            y = torch.cat([y[:hk] / size[:hk] / math.sqrt(d), y[hk:2 * hk] / size[hk:2 * hk], y[2 * hk:]])
            rows.append(y.flatten())
    beta, alpha = st["ba"].double()[:, :hv], st["ba"].double()[:, hv:]
    return {"qkv": torch.stack(rows), "log_a": -st["A_log"].double().exp() * torch.logaddexp(alpha + st["dt"].double(), torch.zeros_like(alpha)),
            "b": torch.sigmoid(beta)}


def _exact_delta(case, st):
    """Each node's state from its parent's, one token after another."""
    hk, hv, d = case["hk"], case["hv"], case["d"]
    x = st["qkv"].double()
    o, u = (torch.empty(st["total"], hv, d, dtype=torch.float64, device=DEV) for _ in range(2))
    share = torch.arange(hv, device=DEV) // (hv // hk)
    for s, up in enumerate(_host_paths(case, st)):
        at, states = int(st["cu"][s]), []
        for i, p in enumerate(up):
            row = x[at + i].view(-1, d)
            q, k, v = row[:hk][share], row[hk:2 * hk][share], row[2 * hk:]
            prev = (states[p] if p >= 0 else st["state"][s].double()) * st["log_a"][at + i].double().exp()[:, None, None]
            u[at + i] = st["b"][at + i].double()[:, None] * (v - torch.einsum("hij,hj->hi", prev, k))
            states.append(prev + torch.einsum("hi,hj->hij", u[at + i], k))
            o[at + i] = torch.einsum("hij,hj->hi", states[-1], q)
    return {"o": o, "delta": u}


def _exact_commit(case, st):
    hk, hv, d = case["hk"], case["hv"], case["d"]
    parents, nodes = _host_paths(case, st), st["node"].tolist()
    share = torch.arange(hv, device=DEV) // (hv // hk)
    state, tail = [], []
    for s, node in enumerate(nodes):
        at, path = int(st["cu"][s]), []
        tail.append(_exact_tail(st, parents, s, node))
        while node >= 0:
            path.insert(0, node)
            node = parents[s][node]
        now = st["state"][s].double()
        for i in path:
            k = st["qkv"][at + i].double().view(-1, d)[hk:2 * hk][share]
            now = now * st["log_a"][at + i].double().exp()[:, None, None] + torch.einsum("hi,hj->hij", st["delta"][at + i].double(), k)
        state.append(now)
    return {"state": torch.stack(state), "tail": torch.stack(tail)}


def _exact_verify(case, st):
    """One sequence after another; the residual is taken and divided by its sum after each rejection."""
    rows, ids, count, node, nxt = [], [], [], [], []
    tokens, u, u_next = st["tokens"].tolist(), st["u"].tolist(), st["u_next"].tolist()
    for s, up in enumerate(_host_paths(case, st)):
        at, here, path, out = int(st["cu"][s]), 0, [], []
        if up:
            path, r = [0], st["p"][at].double()
            for i in range(1, len(up)):
                x = tokens[at + i]
                if up[i] != here:
                    continue
                if case["greedy"]:
                    ok = int((r == r.max()).nonzero()[0]) == x
                elif case["q"]:
                    ok = u[at + i] * float(st["q"][at + here, x]) < float(r[x])
                else:
                    ok = u[at + i] < float(r[x])
                if ok:
                    here, r = i, st["p"][at + i].double()
                    path.append(i)
                    out.append(x)
                elif not case["greedy"]:
                    if case["q"]:
                        r = (r - st["q"][at + here].double()).clamp(min=0)
                    else:
                        r = r.clone()
                        r[x] = 0
                    r = r / r.sum() if float(r.sum()) > 0 else r
            if case["greedy"]:
                out.append(int((r == r.max()).nonzero()[0]))
            else:
                r = r if float(r.sum()) > 0 else st["p"][at + here].double()
                run_sum = torch.cumsum(r, 0)
                out.append(int((run_sum > u_next[s] * run_sum[-1]).nonzero()[0]))
        rest = [-1] * (len(up) - len(path))
        rows += [at + i for i in path] + rest
        ids += out + rest
        count.append(len(path))
        node.append(path[-1] if path else -1)
        nxt.append(out[-1] if out else -1)
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    return {"rows": ints(rows), "ids": ints(ids), "count": ints(count), "node": ints(node), "next": ints(nxt)}


def _exact_plan(case, st):
    """One sequence after another, on the host."""
    page = case["page"]
    lens, new, had, table = (st[k].tolist() for k in ("lens", "n_new", "n_blocks", "table"))
    stack = st["stack"].tolist()[:int(st["n_free"])]
    back = []
    for s, n in enumerate(lens):
        keep = min(had[s], -(-n // page))
        back += table[s][keep:had[s]]
        had[s] = keep
    stack += back[::-1]
    parents = _host_paths(case, st) if case["tree"] else None
    cu, after, positions, slots, asked, free = [0], [], [], [], 0, len(stack)
    for s, n in enumerate(lens):
        need = max(0, -(-(n + new[s]) // page) - had[s])
        asked += need
        ok = need == 0 or asked <= free
        for _ in range(need if ok else 0):
            table[s][had[s]] = stack.pop()
            had[s] += 1
        i = np.arange(new[s])
        depth = []
        for p in parents[s] if parents else []:
            depth.append(depth[p] + 1 if p >= 0 else 0)
        positions.append(n + np.array(depth if parents else i, dtype=np.int64))
        slots.append(np.array(table[s], dtype=np.int64)[(n + i) // page] * page + (n + i) % page if ok else np.full(new[s], -1))
        cu.append(cu[-1] + new[s])
        after.append(n + new[s] if ok else n)
    fill = st["room"] - cu[-1]
    ints = lambda a, t=torch.int32: torch.as_tensor(np.asarray(a)).to(t).to(DEV)  # noqa: E731
    return {"lens": ints(after), "cu": ints(cu), "positions": ints(np.concatenate(positions + [np.zeros(fill, np.int64)])),
            "slots": ints(np.concatenate(slots + [np.full(fill, -1)]), torch.int64), "table": ints(table), "n_blocks": ints(had),
            "n_free": ints([len(stack)])}


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "conv":
        return _exact_conv(case, st)
    if case["op"] == "delta":
        return _exact_delta(case, st)
    if case["op"] == "commit":
        return _exact_commit(case, st)
    return _exact_verify(case, st) if case["op"] == "verify" else _exact_plan(case, st)
