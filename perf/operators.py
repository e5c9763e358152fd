"""Cases and plain forms of the operators over the paged K/V cache and the logits.

Five operators carry a sequence past one greedy token per step:

  append   K and V of any number of new tokens into the paged pools, rotated
           by their positions on the way (Q rotated alongside)
  attn     attention of those tokens over the pools: a tree of drafted tokens
           (a bit mask per token) or a causal run, split over long contexts
  commit   the accepted path of a drafted tree moved to the head of its slots,
           in every layer
  select   one step of beam search: the best continuations over beams x
           vocabulary
  reorder  the beams' block tables and open pages following their parents

`own` False computes them in elementary torch operations; True calls the
package.  Pools are bf16 [layers][pages][n_kv][page][d]; slot s of sequence b
is row s % page of page table[b][s // page].
"""
import math
import random

import torch

own = False

DEV = "cuda"
ROPE_BASE = 500000.0


# ------------------------------------------------------------------- cases

def listed():
    full = {"n_q": 32, "n_kv": 4, "d": 128, "page": 64}
    return [
        # the eight drafted tokens of one sequence at 8K context: latency
        {"name": "append_b1_t8", "op": "append", "batch": 1, "new": 8, "ctx_lo": 8192, "ctx_hi": 8192, "fp32": True,
         "tree": True, **full, "mix": 1},
        # a prompt's chunk on its way into the cache, BF16 projections: bandwidth
        {"name": "append_chunk_16k", "op": "append", "batch": 2, "new": 8192, "ctx_lo": 0, "ctx_hi": 4096,
         "fp32": False, "tree": False, **full, "mix": 2},
        # verifying eight drafted tokens of one sequence at 8K context: latency, K/V split over the SMs
        {"name": "attn_tree_b1_t8_8k", "op": "attn", "batch": 1, "new": 8, "ctx_lo": 8192, "ctx_hi": 8192,
         "window": 0, "tree": True, **full, "mix": 3},
        # continuous batching: 32 ragged contexts, trees of up to 16 tokens: bandwidth
        {"name": "attn_tree_b32_t16", "op": "attn", "batch": 32, "new": 16, "ctx_lo": 512, "ctx_hi": 32768,
         "window": 0, "tree": True, **full, "mix": 4},
        # a prompt's chunk over what the cache holds already: the tensor cores
        {"name": "attn_chunk_2k_8k", "op": "attn", "batch": 1, "new": 2048, "ctx_lo": 8192, "ctx_hi": 8192,
         "window": 0, "tree": False, **full, "mix": 5},
        # the dense model's sliding layers: heads of 64, window 512, odd lengths, a few tokens each
        {"name": "attn_window_b13_t5_d64", "op": "attn", "batch": 13, "new": 5, "ctx_lo": 37, "ctx_hi": 4001,
         "window": 512, "tree": True, "n_q": 16, "n_kv": 2, "d": 64, "page": 64, "mix": 6},
        # the accepted paths of a batch of trees, all 48 layers
        {"name": "commit_b32_t16", "op": "commit", "batch": 32, "new": 16, "ctx_lo": 64, "ctx_hi": 512, "depth": 5,
         "layers": 48, **full, "mix": 7},
        # one sequence of the eight-layer model
        {"name": "commit_b1_t8", "op": "commit", "batch": 1, "new": 8, "ctx_lo": 1024, "ctx_hi": 1024, "depth": 4,
         "layers": 8, "n_q": 16, "n_kv": 2, "d": 64, "page": 64, "mix": 8},
        # four beams of one request: latency
        {"name": "select_r1_w4", "op": "select", "requests": 1, "beams": 4, "out": 4, "vocab": 32768, "mix": 9},
        # a serving batch, twice as many candidates as beams: bandwidth
        {"name": "select_r64_w8", "op": "select", "requests": 64, "beams": 8, "out": 16, "vocab": 65536, "mix": 10},
        # four beams of one request, eight layers
        {"name": "reorder_r1_w4", "op": "reorder", "requests": 1, "beams": 4, "distinct": 2, "ctx_lo": 1000,
         "ctx_hi": 1000, "layers": 8, "n_q": 16, "n_kv": 2, "d": 64, "page": 64, "mix": 11},
        # sixteen requests, all 48 layers
        {"name": "reorder_r16_w8", "op": "reorder", "requests": 16, "beams": 8, "distinct": 4, "ctx_lo": 64,
         "ctx_hi": 320, "layers": 48, **full, "mix": 12},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "commit", "select", "reorder"])
    heads = rng.choice([{"n_q": 32, "n_kv": 4, "d": 128}, {"n_q": 16, "n_kv": 2, "d": 64}, {"n_q": 4, "n_kv": 2, "d": 64},
                        {"n_q": 24, "n_kv": 4, "d": 128}])
    c = {"op": op, **heads, "page": rng.choice([16, 64]), "mix": rng.randrange(1, 1 << 20)}
    if op == "append":
        c["batch"] = _log(rng, 1, 64)
        c["tree"] = rng.random() < 0.5
        c["fp32"] = rng.random() < 0.5
        c["new"] = _log(rng, 1, 200 if c["tree"] else max(1, (10000 if c["fp32"] else 15000) // c["batch"]))
        c["new"] = min(c["new"], 10000 // c["batch"])
        c["ctx_lo"], c["ctx_hi"] = rng.choice([0, 17]), _log(rng, 64, 8000)
    elif op == "attn":
        c["tree"] = rng.random() < 0.6
        c["batch"] = _log(rng, 1, 32)
        c["new"] = min(_log(rng, 1, 130) if c["tree"] else _log(rng, 1, 2048), 8192 // c["batch"])
        most = 400_000 // c["batch"] if c["new"] <= 16 else int(1.8e7 / (c["batch"] * c["new"]))
        c["ctx_hi"] = _log(rng, 40, max(64, min(32768, most)))
        c["ctx_lo"] = rng.randrange(0, 40)
        c["window"] = rng.choice([0, 0, 512, 4096])
    elif op == "commit":
        c["batch"] = _log(rng, 1, 32)
        c["new"] = _log(rng, 1, 64)
        c["depth"] = min(c["new"], rng.randrange(1, 8))
        c["ctx_lo"], c["ctx_hi"] = rng.randrange(0, 60), _log(rng, 64, 500)
        c["layers"] = rng.choice([1, 2, 8, 48])
    elif op == "select":
        c = {"op": op, "requests": _log(rng, 1, 64), "beams": rng.randrange(1, 9), "vocab": _log(rng, 1024, 65536),
             "mix": c["mix"]}
        c["out"] = rng.randrange(1, 2 * c["beams"] + 1)
    else:
        c["requests"], c["beams"] = _log(rng, 1, 16), rng.randrange(2, 9)
        c["distinct"] = rng.randrange((c["beams"] + 1) // 2, c["beams"] + 1)
        c["ctx_lo"], c["ctx_hi"] = rng.randrange(1, 60), _log(rng, 64, 320)
        c["layers"] = rng.choice([1, 2, 8, 48])
    return c


def _spread(case, n, lo, hi, what):
    """n whole numbers of [lo, hi], the case's own; the last one is hi."""
    r = random.Random("%s %d" % (what, case["mix"]))
    return [r.randint(lo, hi) for _ in range(n - 1)] + [hi]


def _new(case):
    return _spread(case, case["batch"], max(1, case["new"] // 2), case["new"], "new")


def _ctx(case, n):
    return _spread(case, n, case["ctx_lo"], case["ctx_hi"], "ctx")


def _accepted(case):
    return _spread(case, case["batch"], min(1, case["depth"]), case["depth"], "depth")


# ------------------------------------------------------------------- inputs

def _paged(case, g, rows, slots, layers):
    """Pools of `layers` whose tables give each of `rows` rows pages for slots[r] slots, in shuffled order."""
    page, need = case["page"], [-(-s // case["page"]) for s in slots]
    total = sum(need) + 3
    ids = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    width = max(need) + 1
    tables = torch.zeros(rows, width, dtype=torch.int32, device=DEV)
    at = 0
    for r in range(rows):
        tables[r, :need[r]] = ids[at:at + need[r]]
        at += need[r]
    shape = (layers, total, case["n_kv"], page, case["d"])
    k, v = (torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    return k, v, tables


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _tree(case, seed, counts):
    """Random trees in an order with parents first: ancestors as bit words, and each token's depth."""
    r = random.Random("tree %d %d" % (case["mix"], seed))
    words = -(-max(counts) // 64)
    masks, depths = [], []
    for n in counts:
        own_mask, own_depth = [], []
        for i in range(n):
            p = r.randint(max(-1, i - 5), i - 1) if i else -1
            own_mask.append((own_mask[p] if p >= 0 else 0) | (1 << i))
            own_depth.append(own_depth[p] + 1 if p >= 0 else 0)
        masks += own_mask
        depths += own_depth
    low = (1 << 64) - 1
    signed = [[(w := (m >> (64 * j)) & low) - (1 << 64 if w >> 63 else 0) for j in range(words)] for m in masks]
    return torch.tensor(signed, dtype=torch.int64, device=DEV), depths


def _fixed(n, m):
    """How many tokens at the head of an accepted path of m of n drafted ones stay where they are."""
    return max(min(1, m), 2 * m - n)


def _path(case, seed, n, m):
    """An accepted path: ascending, and no token that moves lies where another one lands, so that a pass may be
    repeated."""
    r = random.Random("path %d %d %d %d" % (case["mix"], seed, n, m))
    return list(range(_fixed(n, m))) + sorted(r.sample(range(m, n), m - _fixed(n, m)))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"case": case, "op": case["op"]}
    if case["op"] == "select":
        R, W, V = case["requests"], case["beams"], case["vocab"]
        # logits of a language model: a few tokens stand out of a broad field
        st["logits"] = torch.randn(R * W, V, generator=g, device=DEV) * 2.5
        st["scores"] = -20 * torch.rand(R, W, generator=g, device=DEV) - 1
        st["finished"] = (torch.rand(R, W, generator=g, device=DEV) < 0.1).to(torch.uint8)
        st["eos"] = 2
        n = case["out"]
        st["out_scores"] = torch.empty(R, n, device=DEV)
        st["out_parents"], st["out_tokens"] = (torch.empty(R, n, dtype=torch.int32, device=DEV) for _ in range(2))
        if own:
            import moe_decode_megakernel_gb300 as mk
            st["workspace"] = torch.empty(mk.beam_select_workspace_bytes(R, W, V, n), dtype=torch.uint8, device=DEV)
        return st
    d = case["d"]
    if case["op"] == "reorder":
        R, W, page = case["requests"], case["beams"], case["page"]
        lens = _ctx(case, R)
        st["lens"] = _ints(lens)
        # each beam of a request: the full pages in common, an open page and two more of its own
        full = [n // page for n in lens]
        width = max(full) + 4
        ids = torch.randperm(sum(full) + R * W * 3, generator=g, device=DEV).to(torch.int32)
        tables, at = torch.zeros(R * W, width, dtype=torch.int32, device=DEV), 0
        for r in range(R):
            tables[r * W:(r + 1) * W, :full[r]] = ids[at:at + full[r]]
            at += full[r]
            tables[r * W:(r + 1) * W, full[r]:full[r] + 3] = ids[at:at + 3 * W].view(W, 3)
            at += 3 * W
        shape = (case["layers"], ids.numel(), case["n_kv"], page, d)
        st["k"], st["v"] = (torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
        st["tables"], st["tables_out"] = tables, torch.empty_like(tables)
        r = random.Random("parents %d %d" % (case["mix"], seed))
        parents = []
        for _ in range(R):
            alive = r.sample(range(W), case["distinct"])
            row = alive + [r.choice(alive) for _ in range(W - len(alive))]
            r.shuffle(row)
            parents.append(row)
        st["parents"] = _ints(parents)
    else:
        new, ctx = _new(case), _ctx(case, case["batch"])
        B, T = case["batch"], sum(new)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        st["cu"], st["ctx"] = _ints(cu), _ints(ctx)
        st["k"], st["v"], st["tables"] = _paged(case, g, B, [a + b for a, b in zip(ctx, new)], case.get("layers", 1))
        if case["op"] == "commit":
            m = _accepted(case)
            m = [min(a, n) for a, n in zip(m, new)]
            st["path_lens"] = _ints(m)
            paths = [_path(case, seed + 7 * b, n, a) for b, (n, a) in enumerate(zip(new, m))]
            st["path"] = _ints([p + [0] * (case["depth"] - len(p)) for p in paths])
            st["new_lens"] = torch.empty(B, dtype=torch.int32, device=DEV)
        else:
            st["mask"] = st["positions"] = None
            if case["tree"]:
                st["mask"], depth = _tree(case, seed, new)
                at = [c for c, n in zip(ctx, new) for _ in range(n)]
                st["positions"] = _ints([a + b for a, b in zip(at, depth)])
            if case["op"] == "append":
                dt = torch.float32 if case["fp32"] else torch.bfloat16
                st["qkv"] = torch.randn(T, (case["n_q"] + 2 * case["n_kv"]) * d, generator=g, device=DEV, dtype=dt)
                st["q_out"] = torch.empty(T, case["n_q"], d, dtype=torch.bfloat16, device=DEV)
            else:
                # queries that single some of the keys out
                st["q"] = (2 * torch.randn(T, case["n_q"], d, generator=g, device=DEV)).to(torch.bfloat16)
                st["out"] = torch.empty_like(st["q"])
                st["lse"] = torch.empty(T, case["n_q"], device=DEV)
    st["status"] = torch.zeros(8, dtype=torch.int32, device=DEV)
    if own:  # the handle of the cache and the scratch that a program keeps with it
        import moe_decode_megakernel_gb300 as mk
        st["cache"] = mk.KvCache(st["k"], st["v"], ROPE_BASE)
        if case["op"] == "attn":
            need = mk.tree_attn_workspace_bytes(st["cache"])
            st["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------- passes

def run(st):
    return _OPS[st["op"]](st)


def _split(st):
    """Q, K and V heads of the fused projection's rows, as views."""
    c = st["case"]
    q, k, v = st["qkv"].view(-1, c["n_q"] + 2 * c["n_kv"], c["d"]).split((c["n_q"], c["n_kv"], c["n_kv"]), 1)
    return q, k, v


def _owner(cu, T):
    """The sequence of each token, and the token's index in it."""
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    return b, t - cu.long()[b]


def _rotated(x, pos):
    """Pairs (2i, 2i + 1) turned by pos * base^(-2i / d); angles and product in 64 bits."""
    d = x.shape[-1]
    inv = ROPE_BASE ** (-torch.arange(0, d, 2, device=DEV, dtype=torch.float64) / d)
    a = (pos.double()[:, None] * inv)[:, None, :]
    cos, sin = torch.cos(a).float(), torch.sin(a).float()
    x = x.float()
    e, o = x[..., 0::2], x[..., 1::2]
    return torch.stack((e * cos - o * sin, e * sin + o * cos), -1).flatten(-2)


def _append(st):
    c = st["case"]
    q, k, v = _split(st)
    if own:
        import moe_decode_megakernel_gb300 as mk
        mk.kv_append(st["cache"], 0, k, v, st["cu"], st["ctx"], st["tables"], q=q, q_out=st["q_out"],
                     positions=st["positions"], status=st["status"])
    else:
        b, i = _owner(st["cu"], q.shape[0])
        slot = st["ctx"].long()[b] + i
        pos = slot if st["positions"] is None else st["positions"].long()
        page = st["tables"].long()[b, slot // c["page"]]
        st["k"][0][page, :, slot % c["page"]] = _rotated(k, pos).to(torch.bfloat16)
        st["v"][0][page, :, slot % c["page"]] = v.to(torch.bfloat16)
        st["q_out"].copy_(_rotated(q, pos))
    return st["q_out"], st["k"], st["v"]


def _attn(st):
    c = st["case"]
    scale = 1 / math.sqrt(c["d"])
    if own:
        import moe_decode_megakernel_gb300 as mk
        mk.tree_attn(st["cache"], 0, st["q"], st["out"], st["cu"], st["ctx"], st["tables"], st["workspace"],
                     tree_mask=st["mask"], positions=st["positions"], window=c["window"], scale=scale, lse=st["lse"],
                     status=st["status"])
        return st["out"], st["lse"]
    G, B, n_max, P = c["n_q"] // c["n_kv"], c["batch"], c["new"], c["page"]
    S = c["ctx_hi"] + n_max
    T = st["q"].shape[0]
    b, i = _owner(st["cu"], T)
    ctx, n = st["ctx"].long(), (st["cu"][1:] - st["cu"][:-1]).long()
    s = torch.arange(S, device=DEV)
    # the pages of every sequence side by side, padded to the longest
    page = st["tables"].long()[:, torch.clamp(s // P, max=st["tables"].shape[1] - 1)]
    keys, vals = (x[0][page, :, s % P].float() for x in (st["k"], st["v"]))
    q = torch.zeros(B, n_max, c["n_q"], c["d"], device=DEV)
    q[b, i] = st["q"].float()
    q = q.view(B, n_max, c["n_kv"], G, c["d"])
    see = torch.zeros(B, n_max, S, dtype=torch.bool, device=DEV)
    pos = ctx[b] + i if st["positions"] is None else st["positions"].long()
    at = s[None] - ctx[b][:, None]  # each slot as an index among the token's fellows
    if st["mask"] is None:
        seen = at <= i[:, None]
    else:
        word = torch.gather(st["mask"], 1, torch.clamp(at, 0, 64 * st["mask"].shape[1] - 1) // 64)
        seen = (at < 0) | (((word >> (torch.clamp(at, min=0) % 64)) & 1) == 1) & (at < n[b][:, None])
    if c["window"]:
        slot_pos = s.expand(B, S).clone()
        if st["positions"] is not None:
            slot_pos[b, ctx[b] + i] = pos
        seen &= pos[:, None] - slot_pos[b] < c["window"]
    see[b, i] = seen
    w = torch.einsum("bthgd,bshd->bhgts", q, keys) * scale
    w = w.masked_fill(~see[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True).clamp(min=-3e38)
    w = torch.exp(w - top)
    total = w.sum(-1, keepdim=True)
    out = torch.einsum("bhgts,bshd->bthgd", w, vals) / total.clamp(min=1e-38).permute(0, 3, 1, 2, 4)
    lse = (torch.log(total) + top)[..., 0].permute(0, 3, 1, 2)
    st["out"].copy_(out.reshape(B, n_max, c["n_q"], c["d"])[b, i])
    st["lse"].copy_(lse.reshape(B, n_max, c["n_q"])[b, i])
    return st["out"], st["lse"]


def _commit(st):
    c = st["case"]
    if own:
        import moe_decode_megakernel_gb300 as mk
        mk.kv_commit(st["cache"], st["ctx"], st["path"], st["path_lens"], st["tables"], new_lens=st["new_lens"],
                     status=st["status"])
    else:
        P = c["page"]
        j = torch.arange(c["depth"], device=DEV)
        b, j = torch.nonzero(j[None] < st["path_lens"][:, None], as_tuple=True)
        src, dst = st["ctx"].long()[b] + st["path"].long()[b, j], st["ctx"].long()[b] + j
        t = st["tables"].long()
        k, v = (x[:, t[b, src // P], :, src % P] for x in (st["k"], st["v"]))
        st["k"][:, t[b, dst // P], :, dst % P] = k
        st["v"][:, t[b, dst // P], :, dst % P] = v
        st["new_lens"].copy_(st["ctx"] + st["path_lens"])
    return st["new_lens"], st["k"], st["v"]


def _select(st):
    c = st["case"]
    if own:
        import moe_decode_megakernel_gb300 as mk
        mk.beam_select(st["logits"], st["scores"], st["out_scores"], st["out_parents"], st["out_tokens"],
                       st["workspace"], finished=st["finished"], eos=st["eos"])
    else:
        R, W, V = c["requests"], c["beams"], c["vocab"]
        x = st["logits"].view(R, W, V).double()
        cand = st["scores"].double()[..., None] + (x - torch.logsumexp(x, -1, keepdim=True))
        only = torch.full_like(cand, -math.inf)
        only[..., st["eos"]] = st["scores"].double()
        cand = torch.where(st["finished"].bool()[..., None], only, cand).view(R, W * V)
        best, at = torch.sort(cand, dim=-1, descending=True, stable=True)
        st["out_scores"].copy_(best[:, :c["out"]])
        st["out_parents"].copy_(at[:, :c["out"]] // V)
        st["out_tokens"].copy_(at[:, :c["out"]] % V)
    return st["out_scores"], st["out_parents"], st["out_tokens"]


def _reorder(st):
    c = st["case"]
    if own:
        import moe_decode_megakernel_gb300 as mk
        mk.beam_reorder(st["cache"], st["lens"], st["parents"], st["tables"], st["tables_out"], status=st["status"])
    else:
        R, W, P = c["requests"], c["beams"], c["page"]
        par, lens = st["parents"].long(), st["lens"].long()
        old = st["tables"].long().view(R, W, -1)
        j = torch.arange(old.shape[-1], device=DEV)
        full = (lens // P)[:, None, None]
        moved = torch.gather(old, 1, par[..., None].expand_as(old))
        new = torch.where(j < full, moved, old)
        # a parent's first child keeps its open page, the k-th other child takes the k-th childless beam's
        eye = torch.arange(W, device=DEV)
        first = ((par[:, None, :] == par[:, :, None]) & (eye[None] < eye[:, None])).sum(-1) == 0
        alive = (par[:, None, :] == eye[None, :, None]).any(-1)
        rank_extra = (~first).long().cumsum(-1) - 1
        dead = torch.argsort(alive.long(), dim=-1, stable=True)  # childless beams first, ascending
        giver = torch.where(first, par, torch.gather(dead, 1, rank_extra.clamp(min=0)))
        opened = torch.gather(old, 2, full.expand(R, W, 1))[..., 0]
        page = torch.gather(opened, 1, giver)
        is_open = (lens % P > 0)[:, None]
        st["tables_out"].copy_(torch.where((j == full) & is_open[..., None], page[..., None], new).view(R * W, -1))
        r, i, s = torch.nonzero((~first & is_open)[..., None] & (torch.arange(P, device=DEV) < (lens % P)[:, None, None]),
                                as_tuple=True)
        src, dst = opened[r, par[r, i]], page[r, i]
        st["k"][:, dst, :, s] = st["k"][:, src, :, s]
        st["v"][:, dst, :, s] = st["v"][:, src, :, s]
    return st["tables_out"], st["k"], st["v"]


_OPS = {"append": _append, "attn": _attn, "commit": _commit, "select": _select, "reorder": _reorder}


# ------------------------------------------------------------------- what a pass needs

def work(case):
    op = case["op"]
    if op == "select":
        rows = case["requests"] * case["beams"]
        return {"bytes": 4 * rows * case["vocab"] + 5 * rows + 12 * case["requests"] * case["out"],
                "flops": 4 * rows * case["vocab"]}
    row = 2 * case["n_kv"] * case["d"] * 2  # one token's K and V of one layer
    if op == "reorder":
        used = sum(n % case["page"] for n in _ctx(case, case["requests"]))
        pages = sum(n // case["page"] + 1 for n in _ctx(case, case["requests"]))
        moved = (case["beams"] - case["distinct"]) * used * case["layers"]
        return {"bytes": 2 * moved * row + 8 * pages * case["beams"] + 4 * case["requests"] * (case["beams"] + 1),
                "flops": 0}
    new, ctx, B = _new(case), _ctx(case, case["batch"]), case["batch"]
    T = sum(new)
    if op == "commit":
        moved = sum(min(a, n) - _fixed(n, min(a, n)) for a, n in zip(_accepted(case), new))
        return {"bytes": 2 * moved * row * case["layers"] + 4 * B * (case["depth"] + 3), "flops": 0}
    heads = case["n_q"] + 2 * case["n_kv"]
    if op == "append":
        wide = 4 if case["fp32"] else 2
        return {"bytes": T * heads * case["d"] * (wide + 2) + 4 * T + 12 * B,
                "flops": 3 * T * (case["n_q"] + case["n_kv"]) * case["d"]}
    read = pairs = 0
    for n, a in zip(new, ctx):
        back = case["window"] or a + n
        read += min(a, back - 1) + n
        pairs += sum(min(a + i + 1, back) for i in range(n)) if not case["tree"] else n * (min(a, back) + min(n, 4))
    return {"bytes": read * row + T * case["n_q"] * (4 * case["d"] + 4) + 4 * (T + 2 * B),
            "flops": 4 * pairs * case["n_q"] * case["d"]}


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "commit": _exact_commit, "select": _exact_select,
            "reorder": _exact_reorder}[case["op"]](case, st)


def _turn(x, pos):
    """x [heads][d] as complex numbers times e^(i pos theta)."""
    d = x.shape[-1]
    theta = torch.exp(torch.arange(d // 2, device=DEV, dtype=torch.float64) * (-2 * math.log(ROPE_BASE) / d))
    z = torch.view_as_complex(x.double().reshape(*x.shape[:-1], d // 2, 2))
    turned = z * torch.polar(torch.ones_like(theta), (pos * theta) % (2 * math.pi))
    return torch.view_as_real(turned).reshape(x.shape)


def _exact_append(case, st):
    q, k, v = _split(st)
    new, ctx = _new(case), _ctx(case, case["batch"])
    if sum(new) > 2500:
        return None
    at = st["positions"].tolist() if st["positions"] is not None else None
    tables = st["tables"].tolist()
    q_out, ks, vs = torch.empty(q.shape, dtype=torch.float64, device=DEV), st["k"].double(), st["v"].double()
    t = 0
    for b in range(case["batch"]):
        for i in range(new[b]):
            s = ctx[b] + i
            p = at[t] if at else s
            page, row = tables[b][s // case["page"]], s % case["page"]
            q_out[t], ks[0, page, :, row], vs[0, page, :, row] = _turn(q[t], p), _turn(k[t], p), v[t].double()
            t += 1
    return q_out, ks, vs


def _exact_attn(case, st):
    new, ctx, P, W = _new(case), _ctx(case, case["batch"]), case["page"], case["window"]
    G = case["n_q"] // case["n_kv"]
    out, lse = [], []
    t = 0
    for b in range(case["batch"]):
        n, c = new[b], ctx[b]
        pages = st["tables"][b, :-(-(c + n) // P)].long()
        k, v = (x[0, pages].double().transpose(0, 1).reshape(case["n_kv"], -1, case["d"])[:, :c + n] for x in (st["k"], st["v"]))
        q = st["q"][t:t + n].double().view(n, case["n_kv"], G, case["d"])
        see = torch.ones(n, c + n, dtype=torch.bool, device=DEV)
        if case["tree"]:
            bits = [[(m >> j) & 1 for j in range(n)] for m in
                    (sum((w & ((1 << 64) - 1)) << (64 * e) for e, w in enumerate(row)) for row in st["mask"][t:t + n].tolist())]
            see[:, c:] = torch.tensor(bits, device=DEV).bool()
            mine = st["positions"][t:t + n].long()
        else:
            see[:, c:] = torch.tril(torch.ones(n, n, device=DEV)).bool()
            mine = torch.arange(c, c + n, device=DEV)
        if W:
            there = torch.cat((torch.arange(c, device=DEV), mine))
            see &= (mine[:, None] - there[None]) < W
        for h in range(case["n_kv"]):
            s = (q[:, h].reshape(n * G, -1) @ k[h].T).view(n, G, -1) / math.sqrt(case["d"])
            s = torch.where(see[:, None], s, torch.full_like(s, -math.inf))
            total = torch.logsumexp(s, -1)
            p = torch.exp(s - total[..., None])
            out.append((p.view(n * G, -1) @ v[h]).view(n, G, case["d"]))
            lse.append(total)
        t += n
    H = case["n_kv"]
    outs = [torch.cat(out[b * H:(b + 1) * H], 1) for b in range(case["batch"])]
    lses = [torch.cat(lse[b * H:(b + 1) * H], 1) for b in range(case["batch"])]
    return torch.cat(outs), torch.cat(lses)


def _exact_commit(case, st):
    P, tables, paths = case["page"], st["tables"].tolist(), st["path"].tolist()
    lens = [a + m for a, m in zip(_ctx(case, case["batch"]), st["path_lens"].tolist())]
    k, v = st["k"].clone(), st["v"].clone()
    for b, a in enumerate(_ctx(case, case["batch"])):
        for j, s in enumerate(paths[b][:lens[b] - a]):
            to, frm = a + j, a + s
            for new, old in ((k, st["k"]), (v, st["v"])):
                new[:, tables[b][to // P], :, to % P] = old[:, tables[b][frm // P], :, frm % P]
    return _ints(lens), k.double(), v.double()


def _exact_select(case, st):
    W, V, n = case["beams"], case["vocab"], case["out"]
    scores, parents, tokens = [], [], []
    for r in range(case["requests"]):
        found = []
        for w in range(W):
            cum = float(st["scores"][r, w])
            if int(st["finished"][r, w]):
                found.append((-cum, w, st["eos"]))
                continue
            x = st["logits"][r * W + w].double()
            top = x.max()
            x = x - (top + torch.log(torch.exp(x - top).sum()))
            best = torch.topk(x, min(V, n)).values[-1]
            at = torch.nonzero(x >= best)[:, 0]
            found += [(-(cum + a), w, b) for a, b in zip(x[at].tolist(), at.tolist())]
        found.sort()
        scores.append([-f[0] for f in found[:n]])
        parents.append([f[1] for f in found[:n]])
        tokens.append([f[2] for f in found[:n]])
        if len(found) < n:
            return None
    return torch.tensor(scores, dtype=torch.float64, device=DEV), _ints(parents), _ints(tokens)


def _exact_reorder(case, st):
    R, W, P = case["requests"], case["beams"], case["page"]
    old, par, lens = st["tables"].tolist(), st["parents"].tolist(), _ctx(case, R)
    new, k, v = [], st["k"].clone(), st["v"].clone()
    for r in range(R):
        full, used = divmod(lens[r], P)
        spare = [b for b in range(W) if b not in par[r]]
        taken = set()
        for i, p in enumerate(par[r]):
            row = old[r * W + p][:full] + old[r * W + i][full:]
            if used:
                src = old[r * W + p][full]
                row[full] = src
                if p in taken:
                    row[full] = old[r * W + spare.pop(0)][full]
                    for x in (k, v):
                        x[:, row[full], :, :used] = x[:, src, :, :used]
                taken.add(p)
            new.append(row)
    return _ints(new), k.double(), v.double()
