"""Cases that measure tree drafting over the paged cache and the cache's eviction.

A drafter may propose a tree of tokens instead of a chain.  Its nodes are verified in
one pass over the cache (``tree_verify_attn``), a path through it is accepted from given
random numbers (``spec_accept_tree``), and that path's keys and values go to the cache
(``kv_append_path``).  A rollout that outgrows its cache keeps the tokens that attention
has used: their weights are accumulated (``kv_weights_update``) and the rest is dropped
(``kv_evict``).  Each case runs one of these, in its plain form (elementary torch
operations in 32 bits, or in 64 where whole numbers need them, rounded once at the end)
or, where ``own`` is true, through the library.

The formulas:

* a tree of T nodes is parents [T]: node 0 is the root (-1), node v's parent is before it,
  -2 is no node.  Node v sees the whole cache, its ancestors and itself:
  o = softmax(scale * q . k) v over these, lse the log-sum-exp of the scaled logits; no
  node has o = 0 and lse = -inf.
* acceptance: with whole weights w(x) = floor(2^40 q(x)) of the row behind the current
  node and R their sum, its children are tried in order: child c with token x is taken
  when floor(u_acc[c] * R) < w(x); otherwise R falls by w(x) and w(x) becomes 0.  Where no
  child is taken, the last token is the smallest x whose running sum of w is above
  floor(u_res * R).
* weights of the cache's tokens: decay * w + the sum over query rows r that see the token of
  exp(scale * q_r . k - lse_r); tokens as new as the queries start from 0.
* eviction: each KV head keeps the first and the newest tokens and, of the others, those of
  the largest weights (the lower position among equals) up to a budget, moved in order
  to other pages, with the pages' key minima and maxima.
"""
import math

import torch

own = False

N_VOCAB = 151936


# ------------------------------------------------------------------ the cases

def listed():
    q8b = {"h_q": 32, "h_kv": 8, "d": 128}
    return [
        # one user's short conversation, a small tree: latency counts
        {"name": "tree_one", "op": "tree", **q8b, "batch": 1, "t": 8, "ps": 16, "len_lo": 1003, "len_hi": 1003, "shape": "wide"},
        # one long sequence and a large odd tree
        {"name": "tree_long", "op": "tree", **q8b, "batch": 1, "t": 61, "ps": 16, "len_lo": 131001, "len_hi": 131001, "shape": "random"},
        # the rollouts' batch with a tree of the size of a draft round and its alternatives
        {"name": "tree_round", "op": "tree", **q8b, "batch": 64, "t": 15, "ps": 16, "len_lo": 8192, "len_hi": 16384, "shape": "random"},
        # the same with large trees
        {"name": "tree_batch", "op": "tree", **q8b, "batch": 64, "t": 64, "ps": 32, "len_lo": 8192, "len_hi": 16384, "shape": "wide"},
        # one user's walk through a small tree
        {"name": "accept_one", "op": "accept", "batch": 1, "t": 8, "n_vocab": N_VOCAB, "shape": "wide"},
        # the batch's walks through trees of a draft round's size
        {"name": "accept_batch", "op": "accept", "batch": 64, "t": 31, "n_vocab": N_VOCAB, "shape": "random"},
        # one user's accepted path
        {"name": "append_path_one", "op": "append_path", **q8b, "batch": 1, "t": 8, "ps": 16, "len_lo": 1003, "len_hi": 1003},
        # many sequences' paths through large trees
        {"name": "append_path_batch", "op": "append_path", **q8b, "batch": 256, "t": 64, "ps": 16, "len_lo": 0, "len_hi": 2048},
        # one sequence's step
        {"name": "weights_one", "op": "weights", **q8b, "batch": 1, "t": 1, "ps": 16, "len_lo": 4099, "len_hi": 4099, "sparse": 0},
        # the batch's accepted paths of up to seven nodes
        {"name": "weights_batch", "op": "weights", **q8b, "batch": 64, "t": 7, "ps": 16, "len_lo": 8192, "len_hi": 16384, "sparse": 0},
        # a long sequence cut to an eighth
        {"name": "evict_one", "op": "evict", **q8b, "batch": 1, "ps": 16, "len_lo": 65521, "len_hi": 65521, "budget": 8192},
        # the rollouts' batch cut to the tokens of a quarter of its longest sequence
        {"name": "evict_batch", "op": "evict", **q8b, "batch": 64, "ps": 16, "len_lo": 8192, "len_hi": 16384, "budget": 4096},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "accept", "append_path", "weights", "evict"])
    shape = rng.choice(["chain", "wide", "random"])
    if op == "accept":
        batch, t = _spread(rng, 1, 64), _spread(rng, 1, 64)
        return {"op": op, "batch": batch, "t": t, "n_vocab": _spread(rng, 500, min(N_VOCAB, 280000000 // (batch * t))), "shape": shape}
    h_q, h_kv = rng.choice([(32, 8), (16, 8), (4, 2), (8, 1), (28, 4), (8, 8), (6, 2)])
    batch = _spread(rng, 1, 64)
    case = {"op": op, "h_q": h_q, "h_kv": h_kv, "d": rng.choice([64, 128]), "batch": batch, "ps": rng.choice([16, 32, 64])}
    if op == "append_path":
        hi = _spread(rng, 1, 4000)
        return {**case, "t": _spread(rng, 1, 64), "len_lo": rng.randint(0, hi), "len_hi": hi}
    hi = _spread(rng, 40, min(131072, 500000 // batch))
    lo = rng.choice([0, hi // 2, hi])
    if op == "tree":
        return {**case, "t": _spread(rng, 1, 64), "len_lo": lo, "len_hi": hi, "shape": shape}
    if op == "weights":
        sparse = _spread(rng, 1, max(2, hi // 64)) if rng.random() < 0.3 else 0
        t = 1 if sparse else _spread(rng, 1, 16)
        return {**case, "t": t, "len_lo": max(lo, t), "len_hi": hi, "sparse": sparse}
    return {**case, "len_lo": lo, "len_hi": hi, "budget": max(16, int(hi * rng.uniform(0.1, 0.9)))}


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """The sequences' lengths: evenly spaced over the case's range (their order comes from the seed)."""
    b, lo, hi = case["batch"], case["len_lo"], case["len_hi"]
    return [hi if b == 1 else lo + (hi - lo) * i // (b - 1) for i in range(b)]


def _paging(case, gen, room=0):
    """Lengths in a drawn order, and a page table over drawn physical pages, with room for so many tokens more (-1 behind a sequence's last page)."""
    ps, lens = case["ps"], torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    lens = lens[torch.randperm(lens.numel(), generator=gen, device="cuda")]
    pages = (lens + room + ps - 1) // ps
    max_pages = max(1, -(-(case["len_hi"] + room) // ps))
    used = torch.arange(max_pages, device="cuda")[None] < pages[:, None]
    table = torch.full(used.shape, -1, dtype=torch.int32, device="cuda")
    n_phys = sum(-(-(n + room) // ps) for n in _lengths(case))
    table[used] = torch.randperm(n_phys, generator=gen, device="cuda").to(torch.int32)
    return lens, table, n_phys


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _cache(case, gen, n_phys):
    shape = (max(1, n_phys), case["h_kv"], case["ps"], case["d"])
    return tuple(torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))


def _parents(case, gen):
    """A tree for every sequence, int32 [batch][t]; those of every third sequence have fewer nodes."""
    b, t = case["batch"], case["t"]
    at = torch.arange(t, device="cuda")[None]
    if case["shape"] == "chain":
        parent = (at - 1).repeat(b, 1)
    elif case["shape"] == "wide":
        parent = torch.div(at - 1, 3, rounding_mode="floor").repeat(b, 1)
    else:
        back = 1 + torch.floor(4 * torch.rand((b, t), generator=gen, device="cuda")).long()
        parent = (at - back).clamp(min=0)
    parent[:, 0] = -1
    few = torch.where(torch.arange(b, device="cuda") % 3 == 2, (t + 1) // 2, t)
    return torch.where(at < few[:, None], parent, -2).to(torch.int32).contiguous()


def _paths(case, gen):
    """Accepted nodes of every sequence, in ascending order behind the root, int32 [batch][t] (-1 behind the last), and their number."""
    b, t = case["batch"], case["t"]
    most = min(t, 8)
    count = torch.randint(1, most + 1, (b,), generator=gen, device="cuda")
    order = torch.rand((b, t), generator=gen, device="cuda")
    order[:, 0] = -1.0
    rank = order.argsort(dim=1).argsort(dim=1)
    taken = torch.where(rank < count[:, None], torch.arange(t, device="cuda")[None], t)
    path = taken.sort(dim=1).values
    return torch.where(path == t, -1, path).to(torch.int32).contiguous(), count.to(torch.int32)


def _fused(case, gen):
    """q, k and v rows [batch][t] of one projection's buffer; queries and keys are turned into buffers of their own."""
    b, t, h_q, h_kv, d = case["batch"], case["t"], case["h_q"], case["h_kv"], case["d"]
    q, k, v = torch.split(_normal(gen, b, t, h_q + 2 * h_kv, d), [h_q, h_kv, h_kv], dim=2)
    return q.contiguous(), k.contiguous(), v


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s, op = dict(case), case["op"]
    b, t = case["batch"], case.get("t", 1)
    if op == "accept":
        n = case["n_vocab"]
        s["parents"] = _parents(case, gen)
        logits = torch.randn((b, t, n), generator=gen, device="cuda")
        peaks = torch.randint(0, n, (b, t, 16), generator=gen, device="cuda")  # the few tokens that a model prefers
        logits.scatter_add_(2, peaks, 8 + 8 * torch.rand((b, t, 16), generator=gen, device="cuda"))
        s["q_target"] = torch.softmax(logits, dim=2)
        del logits
        top = s["q_target"].topk(8, dim=2).indices  # a good drafter proposes what the target prefers
        parent = s["parents"].long()
        earlier = torch.ones((t, t), dtype=torch.bool, device="cuda").tril(-1)
        rank = ((parent[:, :, None] == parent[:, None, :]) & earlier).sum(dim=2).clamp(max=7)
        s["draft"] = torch.gather(top.flatten(1), 1, (parent.clamp(min=0) * 8 + rank)).to(torch.int32).contiguous()
        s["u_acc"] = torch.rand((b, t), generator=gen, device="cuda")
        s["u_res"] = torch.rand((b,), generator=gen, device="cuda")
        s["n_path"] = torch.empty((b,), dtype=torch.int32, device="cuda")
        s["path"], s["tokens"] = (torch.empty((b, t), dtype=torch.int32, device="cuda") for _ in range(2))
        return s
    h_q, h_kv, d, ps = case["h_q"], case["h_kv"], case["d"], case["ps"]
    s["lens"], s["table"], n_phys = _paging(case, gen, t if op == "append_path" else 0)
    max_pages = s["table"].shape[1]
    s["n_src"] = n_phys
    if op == "evict":  # free pages for what stays
        spare = sum(-(-min(n, case["budget"]) // ps) for n in _lengths(case))
        new_pages = (s["lens"].clamp(max=case["budget"]) + ps - 1) // ps
        used = torch.arange(max_pages, device="cuda")[None] < new_pages[:, None]
        s["dst_table"] = torch.full_like(s["table"], -1)
        s["dst_table"][used] = n_phys + torch.randperm(spare, generator=gen, device="cuda").to(torch.int32)
        n_phys += spare
    s["K"], s["V"] = _cache(case, gen, n_phys)
    s["dims"] = (b, h_q, h_kv, d, ps, max_pages, max(1, n_phys))
    s["summ"] = torch.zeros((b, h_kv, max_pages, 2, d), dtype=torch.bfloat16, device="cuda")
    s["new_lens"] = torch.zeros_like(s["lens"])
    if op == "tree":
        s["q"], s["k"], s["v"] = _fused(case, gen)
        s["parents"] = _parents(case, gen)
        s["o"] = torch.empty((b, t, h_q, d), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((b, t, h_q), device="cuda")
        s["ws"] = torch.zeros(128 << 20, dtype=torch.uint8, device="cuda")
    elif op == "append_path":
        _, s["k"], s["v"] = _fused(case, gen)
        s["path"], s["n_path"] = _paths(case, gen)
    elif op == "weights":
        s["q"] = _normal(gen, b, t, h_q, d)
        s["w"] = torch.rand((b, h_kv, max_pages * ps), generator=gen, device="cuda")
        s["w_out"] = torch.zeros_like(s["w"])
        if case["sparse"]:
            pages, most = (s["lens"] + ps - 1) // ps, min(case["sparse"], max_pages)
            order = torch.rand((b, h_kv, max_pages), generator=gen, device="cuda")
            order.masked_fill_(torch.arange(max_pages, device="cuda") >= pages[:, None, None], -1.0)
            s["nsel"] = pages.clamp(max=most)[:, None].expand(b, h_kv).to(torch.int32).contiguous()
            past = torch.arange(most, device="cuda") >= s["nsel"][:, :, None]
            s["sel"] = order.topk(most, dim=2).indices.masked_fill(past, 1 << 30).sort(dim=2).values.to(torch.int32).contiguous()
        else:
            s["path"], s["n_path"] = _paths(case, gen)
        s["lse"] = torch.zeros((b, t, h_q), device="cuda")
        z = _logits(s).masked_fill_(~_seen(s), -math.inf)  # what the attention of these queries gives
        lse = torch.logsumexp(z, dim=-1)
        del z
        s["lse"] = lse.unflatten(2, (t, h_q // h_kv)).transpose(1, 2).flatten(2, 3).contiguous()
        if not case["sparse"]:  # the rows of a path lie at their nodes
            at = s["path"].long().clamp(min=0)[:, :, None].expand(-1, -1, h_q)
            s["lse"] = torch.full_like(s["lse"], -math.inf).scatter_reduce_(1, at, s["lse"], "amax")
    else:
        w = torch.exp(2 * torch.randn((b, h_kv, max_pages * ps), generator=gen, device="cuda"))
        s["w"] = w * (torch.rand(w.shape, generator=gen, device="cuda") > 0.2)  # some tokens have never been looked at
        s["w_out"] = torch.zeros_like(s["w"])
        s["kept"] = torch.full((b, h_kv, case["budget"]), -1, dtype=torch.int32, device="cuda")
    return s


def _evict_rule(case):
    """First and newest tokens that always stay."""
    return min(4, case["budget"] // 4), case["budget"] // 8


# ------------------------------------------------------------------ plain forms

def _gathered(s, cache):
    """fp32 [batch][h_kv][max_pages * ps][d] of a paged cache."""
    x = cache[s["table"].clamp(min=0).long()]  # [b][pages][h][ps][d]
    return x.transpose(1, 2).flatten(2, 3).float()


def _ancestors(parents):
    """[batch][t][t]: whether node v sees node u (its ancestors and itself); no row and no column of what is no node."""
    t = parents.shape[1]
    node = parents > -2
    at = torch.arange(t, device=parents.device)
    step = ((parents[:, :, None] == at) | (at[:, None] == at)).float() * node[:, :, None]
    for _ in range(max(1, math.ceil(math.log2(max(t, 2))))):  # paths of one edge, two, four ...
        step = ((step @ step) > 0).float()
    return step > 0


def _rows(x, h_kv):
    """[b][t][h_q][..] -> [b][h_kv][t * g][..]."""
    b, t, h_q = x.shape[:3]
    return x.unflatten(2, (h_kv, h_q // h_kv)).transpose(1, 2).flatten(2, 3)


def _plain_tree(s):
    b, t, h, g, d = s["batch"], s["t"], s["h_kv"], s["h_q"] // s["h_kv"], s["d"]
    keys = torch.cat([_gathered(s, s["K"]), s["k"].transpose(1, 2).float()], dim=2)
    z = torch.matmul(_rows(s["q"], h).float(), keys.transpose(2, 3)) / math.sqrt(d)
    del keys
    n = z.shape[3] - t
    sees = _ancestors(s["parents"])
    cached = (torch.arange(n, device="cuda") < s["lens"][:, None])[:, None] & sees.any(dim=2)[:, :, None]
    visible = torch.cat([cached, sees], dim=2).repeat_interleave(g, dim=1)[:, None]  # [b][1][t * g][n + t]
    z.masked_fill_(~visible, -math.inf)
    m = z.amax(dim=-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(z - m)
    del z
    total = p.sum(dim=-1, keepdim=True)
    values = torch.cat([_gathered(s, s["V"]), s["v"].transpose(1, 2).float()], dim=2)
    o = torch.matmul(p, values) / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, m + torch.log(total), -math.inf)
    back = lambda x: x.unflatten(2, (t, g)).transpose(1, 2).flatten(2, 3).contiguous()
    return back(o.to(torch.bfloat16)), back(lse).squeeze(-1)


def _floor_of(u, total):
    """floor(u * total), exactly, for u of 24 bits after the point and whole totals below 2^62."""
    k = (u.double() * 16777216.0).long()
    high, low = total >> 24, total & 16777215
    return k * high + (k * low >> 24)


def _plain_accept(s):
    b, t = s["batch"], s["t"]
    parent = s["parents"].long()
    w = (s["q_target"].double().clamp(max=1.0) * 1099511627776.0).long()  # [b][t][n]
    total = w.sum(dim=2)
    up = parent.clamp(min=0)
    mine = torch.gather(w.flatten(1), 1, up * s["n_vocab"] + s["draft"].long())  # a node's weight in its parent's row
    at = torch.arange(t, device="cuda")
    sibling = (parent[:, :, None] == parent[:, None, :]) & (at[:, None] > at)  # [v][u]: u is tried before v
    same = sibling & (s["draft"][:, :, None] == s["draft"][:, None, :])
    mine = torch.where(same.any(dim=2) | (parent < 0), 0, mine)  # a token that was tried weighs nothing
    left = torch.gather(total, 1, up) - (sibling * mine[:, None, :]).sum(dim=2)
    passes = _floor_of(s["u_acc"], left) < mine
    taken = passes & ~(sibling & passes[:, None, :]).any(dim=2)
    taken |= parent == -1
    sees = _ancestors(s["parents"])
    on = (parent > -2) & ~(sees & ~taken[:, None, :]).any(dim=2)  # every node up to the root is taken
    count = on.sum(dim=1)
    order = torch.where(on, at, t).sort(dim=1).values
    last = order.gather(1, (count - 1)[:, None])  # the node where the walk ends
    row = w.gather(1, last[:, :, None].expand(-1, -1, w.shape[2]))[:, 0]
    tried = parent == last
    row.scatter_reduce_(1, s["draft"].long(), torch.where(tried, 0, 1 << 60), "amin")
    running = row.cumsum(dim=1)
    drawn = torch.searchsorted(running, _floor_of(s["u_res"], running[:, -1])[:, None], right=True)
    path = torch.where(order == t, -1, order)
    following = torch.gather(s["draft"].long(), 1, path.roll(-1, dims=1).clamp(min=0))
    tokens = torch.where(at < (count - 1)[:, None], following, torch.where(at == (count - 1)[:, None], drawn, -1))
    return count.to(torch.int32), path.to(torch.int32), tokens.to(torch.int32)


def _page_bounds(keys, valid):
    """Minima and maxima [..][2][d] of pages of keys [..][ps][d] over their valid tokens."""
    low = torch.where(valid[..., None], keys, math.inf).amin(dim=-2)
    high = torch.where(valid[..., None], keys, -math.inf).amax(dim=-2)
    return torch.stack([low, high], dim=-2).to(torch.bfloat16)


def _plain_append_path(s):
    ps, t = s["ps"], s["t"]
    new_lens = s["lens"] + s["n_path"]
    b, i = (torch.arange(t, device="cuda") < s["n_path"][:, None]).nonzero(as_tuple=True)
    pos = s["lens"].long()[b] + i
    phys, slot, node = s["table"][b, pos // ps].long(), pos % ps, s["path"].long()[b, i]
    s["K"][phys, :, slot] = s["k"][b, node]
    s["V"][phys, :, slot] = s["v"][b, node]
    page = torch.arange(s["table"].shape[1], device="cuda")
    b, p = ((page >= s["lens"][:, None] // ps) & (page * ps < new_lens[:, None])).nonzero(as_tuple=True)
    valid = (p[:, None] * ps + torch.arange(ps, device="cuda")) < new_lens[b][:, None]
    s["summ"][b, :, p] = _page_bounds(s["K"][s["table"][b, p].long()], valid[:, None].expand(-1, s["h_kv"], -1))
    s["new_lens"].copy_(new_lens)
    return s["K"], s["V"], s["summ"], s["new_lens"]


def _picked(s, x):
    """Rows [b][t][..] of x at the nodes of the path (as they are where there is none)."""
    if "path" not in s:
        return x
    at = s["path"].long().clamp(min=0).reshape(s["batch"], s["t"], *[1] * (x.dim() - 2))
    return torch.gather(x, 1, at.expand(-1, -1, *x.shape[2:]))


def _logits(s):
    """Scaled logits [b][h_kv][t * g][n] of the path's queries."""
    q = _rows(_picked(s, s["q"]), s["h_kv"]).float()
    return torch.matmul(q, _gathered(s, s["K"]).transpose(2, 3)) / math.sqrt(s["d"])


def _seen(s):
    """Which tokens each query sees [b][1 or h_kv][t * g][n]: those up to its own, of the selected pages."""
    b, t, g, ps = s["batch"], s["t"], s["h_q"] // s["h_kv"], s["ps"]
    n = s["table"].shape[1] * ps
    count = s["n_path"] if "path" in s else torch.full_like(s["lens"], t)
    i = torch.arange(t, device="cuda")
    last = torch.where(i < count[:, None], (s["lens"] - count)[:, None] + i, -1)  # [b][t]
    seen = (torch.arange(n, device="cuda") <= last[:, :, None]).repeat_interleave(g, dim=1)[:, None]
    if s["sparse"]:
        pages = torch.zeros((b, s["h_kv"], n // ps + 1), dtype=torch.bool, device="cuda")
        pages.scatter_(2, s["sel"].long().clamp(max=n // ps), True)
        seen = seen & pages[:, :, :n // ps].repeat_interleave(ps, dim=2)[:, :, None]
    return seen


def _plain_weights(s):
    p = torch.exp(_logits(s) - _rows(_picked(s, s["lse"])[..., None], s["h_kv"])).masked_fill_(~_seen(s), 0.0)
    count = s["n_path"] if "path" in s else torch.full_like(s["lens"], s["t"])
    at = torch.arange(s["w"].shape[2], device="cuda")
    old = torch.where(at < (s["lens"] - count)[:, None, None], s["w"] * 0.9, 0.0)
    s["w_out"].copy_(torch.where(at < s["lens"][:, None, None], old + p.sum(dim=2), s["w_out"]))
    return s["w_out"]


def _plain_evict(s):
    b, h, ps, budget = s["batch"], s["h_kv"], s["ps"], s["budget"]
    sink, recent = _evict_rule(s)
    lens, new = s["lens"][:, None, None], s["lens"].clamp(max=budget)
    at = torch.arange(s["w"].shape[2], device="cuda")
    key = s["w"].masked_fill((at < sink) | (at >= lens - recent), math.inf).masked_fill_(at >= lens, -1.0)
    order = key.sort(dim=2, descending=True, stable=True).indices[:, :, :budget]
    past = torch.arange(order.shape[2], device="cuda") >= new[:, None, None]
    kept = order.masked_fill(past, 1 << 30).sort(dim=2).values.masked_fill(past, -1)
    s["kept"][:, :, :kept.shape[2]] = kept.to(torch.int32)
    i, hh, j = (~past).expand(b, h, -1).nonzero(as_tuple=True)
    src = kept[i, hh, j]
    to, slot = s["dst_table"][i, j // ps].long(), j % ps
    s["K"][to, hh, slot] = s["K"][s["table"][i, src // ps].long(), hh, src % ps]
    s["V"][to, hh, slot] = s["V"][s["table"][i, src // ps].long(), hh, src % ps]
    s["w_out"][i, hh, j] = s["w"][i, hh, src]
    i, p = (torch.arange(s["table"].shape[1], device="cuda") * ps < new[:, None]).nonzero(as_tuple=True)
    valid = (p[:, None] * ps + torch.arange(ps, device="cuda")) < new[i][:, None]
    s["summ"][i, :, p] = _page_bounds(s["K"][s["dst_table"][i, p].long()], valid[:, None].expand(-1, h, -1))
    s["new_lens"].copy_(new)
    return s["K"][s["n_src"]:], s["V"][s["n_src"]:], s["w_out"], s["kept"], s["summ"], s["new_lens"]


_PLAIN = {"tree": _plain_tree, "accept": _plain_accept, "append_path": _plain_append_path, "weights": _plain_weights, "evict": _plain_evict}


# ------------------------------------------------------------------ the library's calls

def _own(s):
    import sparse_attention_decode_pages_gb300 as spd
    op = s["op"]
    if op == "accept":
        spd.spec_accept_tree(s["q_target"], s["draft"], s["parents"], s["u_acc"], s["u_res"], s["n_path"], s["path"], s["tokens"])
        return s["n_path"], s["path"], s["tokens"]
    dims = spd.dims_of(*s["dims"])
    if op == "tree":
        spd.tree_verify_attn(dims, s["t"], s["q"], s["K"], s["V"], s["table"], s["lens"], s["k"], s["v"], s["parents"], s["o"], s["ws"], lse=s["lse"])
        return s["o"], s["lse"]
    if op == "append_path":
        spd.kv_append_path(dims, s["t"], s["K"], s["V"], s["table"], s["lens"], s["k"], s["v"], s["path"], s["n_path"], s["summ"], s["new_lens"])
        return s["K"], s["V"], s["summ"], s["new_lens"]
    if op == "weights":
        spd.kv_weights_update(dims, s["t"], s["q"], s["lse"], s["K"], s["table"], s["lens"], s["w_out"], w_in=s["w"], decay=0.9, path=s.get("path"),
                              n_path=s.get("n_path"), sel=s.get("sel"), nsel=s.get("nsel"))
        return s["w_out"]
    sink, recent = _evict_rule(s)
    spd.kv_evict(dims, s["budget"], sink, recent, s["K"], s["V"], s["table"], s["lens"], s["w"], s["dst_table"], s["kept"], s["w_out"], s["summ"], s["new_lens"])
    return s["K"][s["n_src"]:], s["V"][s["n_src"]:], s["w_out"], s["kept"], s["summ"], s["new_lens"]


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, b, t = case["op"], case["batch"], case.get("t", 1)
    if op == "accept":  # a walk ends after about two nodes behind the root: three rows
        n = b * min(t, 3) * case["n_vocab"]
        return {"bytes": 4 * n + b * t * 20, "flops": 3 * n}
    h_q, h_kv, d, ps, lens = case["h_q"], case["h_kv"], case["d"], case["ps"], _lengths(case)
    row = 2 * h_kv * d  # bytes of one token's keys, or values
    if op == "tree":
        tokens = sum(lens)
        return {"bytes": 2 * tokens * row + b * t * (2 * row + h_q * (4 * d + 4)), "flops": 4 * (tokens + b * t) * t * h_q * d}
    if op == "append_path":  # paths of (1 + min(t, 8)) / 2 nodes, one page each
        new = b * (1 + min(t, 8)) / 2
        return {"bytes": new * 4 * row + b * row * (2 + ps / 2), "flops": b * h_kv * ps * d}
    if op == "weights":
        tokens = sum(min(n, case["sparse"] * ps) if case["sparse"] else n for n in lens)
        rows = t if case["sparse"] else (1 + min(t, 8)) / 2
        return {"bytes": tokens * row + sum(lens) * h_kv * 8 + b * rows * h_q * (2 * d + 4), "flops": 2 * tokens * rows * h_q * d}
    kept = sum(min(n, case["budget"]) for n in lens)
    return {"bytes": sum(lens) * h_kv * 4 + kept * (4 * row + 8 * h_kv + 2 * row / ps), "flops": kept * 2 * h_kv * d + sum(lens) * h_kv * 4}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_tree(s):
    b, t, h, g, d, ps = s["batch"], s["t"], s["h_kv"], s["h_q"] // s["h_kv"], s["d"], s["ps"]
    o = torch.zeros((b, t, h, g, d), dtype=torch.float64, device="cuda")
    lse = torch.full((b, t, h, g), -math.inf, dtype=torch.float64, device="cuda")
    for i, (n, parent) in enumerate(zip(s["lens"].tolist(), s["parents"].tolist())):
        at = torch.arange(n, device="cuda")
        phys, slot = s["table"][i].long()[at // ps], at % ps
        keys = torch.cat([s["K"][phys, :, slot], s["k"][i]]).double()  # [n + t][h][d]
        values = torch.cat([s["V"][phys, :, slot], s["v"][i]]).double()
        for first in range(0, t, 16):
            nodes = range(first, min(t, first + 16))
            seen = torch.zeros((len(nodes), n + t), dtype=torch.bool)
            for k, v in enumerate(nodes):
                if parent[v] > -2:
                    seen[k, :n] = True
                while v >= 0 and parent[v] > -2:
                    seen[k, n + v] = True
                    v = parent[v]
            z = torch.einsum("thgd,nhd->thgn", s["q"][i, first:first + 16].reshape(-1, h, g, d).double(), keys) * d ** -0.5
            z = torch.where(seen.cuda()[:, None, None], z, -math.inf)
            total = torch.logsumexp(z, dim=-1)
            lse[i, first:first + 16] = total
            p = torch.where(total[..., None] > -math.inf, torch.exp(z - total[..., None]), 0.0)
            o[i, first:first + 16] = torch.einsum("thgn,nhd->thgd", p, values)
    return o.flatten(2, 3), lse.flatten(2, 3)


def _exact_accept(s):
    b, t = s["batch"], s["t"]
    count, path, tokens = [], [], []
    for i, (parent, draft, u) in enumerate(zip(s["parents"].tolist(), s["draft"].tolist(), s["u_acc"].tolist())):
        node, way, said = 0, [0], []
        while True:
            w = torch.floor(s["q_target"][i, node].double().clamp(0, 1) * 2.0 ** 40).long()
            left, nxt = int(w.sum()), None
            for c in range(node + 1, t):
                if parent[c] != node:
                    continue
                x = int(w[draft[c]])
                if int(u[c] * 2 ** 24) * left >> 24 < x:
                    nxt = c
                    break
                left -= x
                w[draft[c]] = 0
            if nxt is None:
                break
            said.append(draft[nxt])
            way.append(nxt)
            node = nxt
        mark = int(s["u_res"][i].item() * 2 ** 24) * left >> 24
        said.append(int((w.cumsum(0) <= mark).sum()))
        count.append(len(way))
        path.append(way + [-1] * (t - len(way)))
        tokens.append(said + [-1] * (t - len(said)))
    return tuple(torch.tensor(x, dtype=torch.int32) for x in (count, path, tokens))


def _exact_append_path(s):
    K, V, summ = s["K"].clone(), s["V"].clone(), s["summ"].clone()
    ps, new = s["ps"], (s["lens"] + s["n_path"]).tolist()
    for i, (n, end) in enumerate(zip(s["lens"].tolist(), new)):
        rows = s["path"][i, :end - n].long()
        at = torch.arange(n, end, device="cuda")
        phys, slot = s["table"][i].long()[at // ps], at % ps
        K[phys, :, slot], V[phys, :, slot] = s["k"][i, rows], s["v"][i, rows]
        for p in range(n // ps, -(-end // ps)):
            keys = K[s["table"][i, p].long(), :, :min(ps, end - p * ps)].double()
            summ[i, :, p, 0], summ[i, :, p, 1] = keys.amin(1).to(summ.dtype), keys.amax(1).to(summ.dtype)
    return K, V, summ, torch.tensor(new, dtype=torch.int32)


def _exact_weights(s):
    w, ps, g, t = s["w_out"].double(), s["ps"], s["h_q"] // s["h_kv"], s["t"]
    for i, n in enumerate(s["lens"].tolist()):
        rows = list(range(t)) if "path" not in s else s["path"][i, :int(s["n_path"][i])].tolist()
        fresh = n - len(rows)
        w[i, :, :fresh] = s["w"][i, :, :fresh].double() * 0.9
        w[i, :, fresh:n] = 0.0
        at = torch.arange(n, device="cuda")
        keys = s["K"][s["table"][i].long()[at // ps], :, at % ps].double()  # [n][h][d]
        for j, r in enumerate(rows):
            q = s["q"][i, r].unflatten(0, (s["h_kv"], g)).double()
            p = torch.exp(torch.einsum("hgd,nhd->hgn", q, keys) * s["d"] ** -0.5 - s["lse"][i, r].double().unflatten(0, (s["h_kv"], g))[..., None])
            p[..., fresh + j + 1:] = 0.0
            if s["sparse"]:
                for hh in range(s["h_kv"]):
                    chosen = s["sel"][i, hh, :int(s["nsel"][i, hh])]
                    p[hh] *= torch.isin(at // ps, chosen)
            w[i, :, :n] += p.sum(dim=1)
    return w


def _exact_evict(s):
    ps, (sink, recent) = s["ps"], _evict_rule(s)
    K, V, w_out, kept, summ = s["K"].clone(), s["V"].clone(), s["w_out"].double(), s["kept"].clone(), s["summ"].clone()
    new = s["lens"].clamp(max=s["budget"])
    for i, (n, m) in enumerate(zip(s["lens"].tolist(), new.tolist())):
        for hh in range(s["h_kv"]):
            always = torch.zeros(n, dtype=torch.bool, device="cuda")
            always[:sink], always[max(0, n - recent):] = True, True
            w = s["w"][i, hh, :n].double()
            rest = torch.argsort(-w[~always], stable=True)[:m - int(always.sum())]
            stay = torch.cat([always.nonzero()[:, 0], (~always).nonzero()[:, 0][rest]]).sort().values if m < n else torch.arange(n, device="cuda")
            src, to = s["table"][i].long()[stay // ps], s["dst_table"][i].long()[torch.arange(m, device="cuda") // ps]
            slot = torch.arange(m, device="cuda") % ps
            K[to, hh, slot], V[to, hh, slot] = s["K"][src, hh, stay % ps], s["V"][src, hh, stay % ps]
            w_out[i, hh, :m], kept[i, hh, :m] = w[stay], stay.to(torch.int32)
        for p in range(-(-m // ps)):
            keys = K[s["dst_table"][i, p].long(), :, :min(ps, m - p * ps)]
            summ[i, :, p, 0], summ[i, :, p, 1] = keys.amin(1), keys.amax(1)
    return K[s["n_src"]:], V[s["n_src"]:], w_out, kept, summ, new


def exact(case, seed):
    s = prepare(case, seed)
    form = {"tree": _exact_tree, "accept": _exact_accept, "append_path": _exact_append_path, "weights": _exact_weights, "evict": _exact_evict}
    return form[case["op"]](s)
