"""Cases that measure the operators around the paged attention of a rollout step.

A decode or verification step of a rollout normalises and rotates its queries and
keys (``qk_norm_rope``), or does so on the way into the paged cache
(``kv_append_rope``); the cache may be held in 4 bits (``kv4_append``,
``kv4_sparse_decode_attn``, ``kv4_dense_verify_attn``); and what the model answers
is scored from its logits (``token_logprobs``).  Each case runs one of these, in its
plain form (elementary torch operations in 32 bits, rounded once at the end) or,
where ``own`` is true, through the library.

The formulas:

* norm and rotation of one head row x of D channels: y = x / sqrt(mean(x^2) + eps) * w,
  then channels (i, i + R/2), or (2i, 2i + 1) where interleaved, of the first R
  turn by the position's angle: (a, b) -> (a cos - b sin, b cos + a sin).
* 4-bit storage of a row of D channels, in groups of 16: scale s = e4m3(amax / (6 * 2^e)),
  codes c = e2m1(x / (s * 2^e)) (ties to even, saturating); the value is c * s * 2^e.
* attention: softmax(scale * q . k) v over the visible tokens; lse is the natural
  log-sum-exp of the scaled logits.
* log probabilities: z = logits * inv_temperature, lse = log sum exp z,
  logprob = z[target] - lse, entropy = lse - sum p z, and the K largest logits.
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 1000000.0  # rotary base of the Qwen3 shapes
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
N_VOCAB = 151936


# ------------------------------------------------------------------ the cases

def listed():
    q8b = {"h_q": 32, "h_kv": 8, "d": 128}
    q17b = {"h_q": 16, "h_kv": 8, "d": 128}
    return [
        # one token of one sequence: what a single user waits for in every layer
        {"name": "qk_one_token", "op": "qk_norm_rope", **q8b, "rows": 1, "packed": True, "norm": True, "rot": 128, "interleaved": False, "n_pos": 32768},
        # a long prompt's queries and keys, views of one fused projection
        {"name": "qk_prompt", "op": "qk_norm_rope", **q8b, "rows": 16381, "packed": True, "norm": True, "rot": 128, "interleaved": False, "n_pos": 32768},
        # the cache update of one decode step at the batch of the rollouts
        {"name": "append_rope_step", "op": "kv_append_rope", **q8b, "batch": 64, "t": 1, "ps": 16, "len_lo": 1024, "len_hi": 2048, "packed": True, "norm": True, "rot": 128, "interleaved": False},
        # a prompt's chunk written to the cache of four sequences, half of the channels rotated
        {"name": "append_rope_chunk", "op": "kv_append_rope", **q17b, "batch": 4, "t": 4095, "ps": 32, "len_lo": 4095, "len_hi": 8192, "packed": True, "norm": True, "rot": 64, "interleaved": True},
        # the 4-bit cache update of one decode step
        {"name": "kv4_append_step", "op": "kv4_append", **q8b, "batch": 64, "t": 1, "ps": 16, "len_lo": 1024, "len_hi": 2048},
        # prompt chunks quantised into the 4-bit cache
        {"name": "kv4_append_chunk", "op": "kv4_append", **q8b, "batch": 8, "t": 2039, "ps": 32, "len_lo": 2039, "len_hi": 4096},
        # sparse decode of the rollouts' batch: 64 pages of each sequence
        {"name": "kv4_sparse_batch", "op": "kv4_sparse", **q8b, "batch": 64, "ps": 16, "len_lo": 8192, "len_hi": 16384, "pages": 64},
        # the long tail of a rollout: few long sequences, a sixteenth of their pages
        {"name": "kv4_sparse_tail", "op": "kv4_sparse", **q8b, "batch": 8, "ps": 32, "len_lo": 65536, "len_hi": 131072, "pages": 256},
        # verification of seven drafted positions over the whole cache
        {"name": "kv4_verify_batch", "op": "kv4_dense", **q8b, "batch": 64, "t": 7, "ps": 16, "len_lo": 8192, "len_hi": 16384},
        # dense decode of one long sequence
        {"name": "kv4_dense_one", "op": "kv4_dense", **q8b, "batch": 1, "t": 1, "ps": 16, "len_lo": 131001, "len_hi": 131001},
        # the log probabilities of one sampled token
        {"name": "logprobs_one", "op": "logprobs", "rows": 1, "n_vocab": N_VOCAB, "dtype": "bf16", "top": 20},
        # those of a verified round: 64 sequences of seven positions
        {"name": "logprobs_round", "op": "logprobs", "rows": 448, "n_vocab": N_VOCAB, "dtype": "fp32", "top": 8},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk_norm_rope", "kv_append_rope", "kv4_append", "kv4_sparse", "kv4_dense", "logprobs"])
    h_q, h_kv = rng.choice([(32, 8), (16, 8), (4, 2), (8, 1), (28, 4), (8, 8)])
    d = rng.choice([64, 128])
    heads = {"h_q": h_q, "h_kv": h_kv, "d": d}
    rope = {"packed": rng.random() < 0.5, "norm": rng.random() < 0.7, "rot": rng.choice([d, d // 2, 16]), "interleaved": rng.random() < 0.4}
    ps = rng.choice([16, 32, 64])
    if op == "qk_norm_rope":
        return {"op": op, **heads, "rows": _spread(rng, 1, 16000), **rope, "n_pos": _spread(rng, 64, 131072)}
    if op in ("kv_append_rope", "kv4_append"):
        batch = _spread(rng, 1, 64)
        t = _spread(rng, 1, min(4000, 16000 // batch)) if rng.random() < 0.7 else 1
        hi = t + _spread(rng, 1, 2000)
        case = {"op": op, **heads, "batch": batch, "t": t, "ps": ps, "len_lo": rng.randint(t, hi), "len_hi": hi}
        return {**case, **rope} if op == "kv_append_rope" else case
    if op == "kv4_sparse":
        batch = _spread(rng, 1, 64)
        hi = _spread(rng, 40, min(131072, 1000000 // batch))
        pages = min(-(-hi // ps), _spread(rng, 1, 512))
        return {"op": op, **heads, "batch": batch, "ps": ps, "len_lo": rng.randint(hi // 2, hi), "len_hi": hi, "pages": pages}
    if op == "kv4_dense":
        batch = _spread(rng, 1, 64)
        t = _spread(rng, 1, min(16, 64 * h_kv // h_q))
        hi = _spread(rng, 40, min(131072, 500000 // batch))
        return {"op": op, **heads, "batch": batch, "t": t, "ps": ps, "len_lo": rng.randint(hi // 2, hi), "len_hi": hi}
    return {"op": op, "rows": _spread(rng, 1, 440), "n_vocab": _spread(rng, 500, N_VOCAB), "dtype": rng.choice(["bf16", "fp32"]), "top": rng.randint(1, 32)}


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """The sequences' lengths: evenly spaced over the case's range (their order comes from the seed)."""
    b, lo, hi = case["batch"], case["len_lo"], case["len_hi"]
    return [hi if b == 1 else lo + (hi - lo) * i // (b - 1) for i in range(b)]


def _paging(case, gen):
    """Lengths in a drawn order, and a page table over drawn physical pages (-1 behind a sequence's last page)."""
    ps, lens = case["ps"], torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    lens = lens[torch.randperm(lens.numel(), generator=gen, device="cuda")]
    pages = (lens + ps - 1) // ps
    max_pages = -(-case["len_hi"] // ps)
    used = torch.arange(max_pages, device="cuda")[None] < pages[:, None]
    table = torch.full(used.shape, -1, dtype=torch.int32, device="cuda")
    n_phys = sum(-(-n // ps) for n in _lengths(case))
    table[used] = torch.randperm(n_phys, generator=gen, device="cuda").to(torch.int32)
    return lens, table, n_phys


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _rope_table(n_pos, rot):
    """fp32 [n_pos][2][rot / 2]: the cosines and sines of position * theta^(-2i / rot), from 64 bits."""
    freq = THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.stack([angle.cos(), angle.sin()], dim=1).float().contiguous()


def _projection(case, gen, rows):
    """q, k and v rows of one projection: views of one buffer where packed, buffers of their own otherwise."""
    h_q, h_kv, d = case["h_q"], case["h_kv"], case["d"]
    if case.get("packed"):
        return torch.split(_normal(gen, rows, h_q + 2 * h_kv, d), [h_q, h_kv, h_kv], dim=1)
    return _normal(gen, rows, h_q, d), _normal(gen, rows, h_kv, d), _normal(gen, rows, h_kv, d)


def _weights(case, gen):
    if not case["norm"]:
        return None, None
    return tuple((1 + 0.2 * torch.randn(case["d"], generator=gen, device="cuda")).to(torch.bfloat16) for _ in range(2))


def _quantised_cache(case, n_phys, gen):
    """A 4-bit cache [n_phys][h_kv][2][ps * d * 9 / 16] of normal keys and values, quantised as the append does."""
    h, ps, d = case["h_kv"], case["ps"], case["d"]
    x = torch.randn((n_phys, h, 2, ps, d), generator=gen, device="cuda", dtype=torch.bfloat16)
    codes, scales = _quantise(x)
    return torch.cat([codes.flatten(3), scales.flatten(3)], dim=3).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s, op = dict(case), case["op"]
    if op == "logprobs":
        rows, n = case["rows"], case["n_vocab"]
        logits = torch.randn((rows, n), generator=gen, device="cuda") * 2.5
        peaks = torch.randint(0, n, (rows, 16), generator=gen, device="cuda")  # the few tokens that a model prefers
        logits.scatter_add_(1, peaks, 4 + 6 * torch.rand((rows, 16), generator=gen, device="cuda"))
        targets = peaks[:, 0].to(torch.int32)
        targets[torch.rand(rows, generator=gen, device="cuda") < 0.1] = -1  # behind a round's last token
        logits[:, n - n // 512:] = -math.inf  # a padded vocabulary
        s["logits"] = logits.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        s["targets"] = targets
        s["inv_temperature"] = 1.25
        s["out"] = [torch.empty(rows, device="cuda") for _ in range(3)]
        s["top_ids"] = torch.empty((rows, case["top"]), dtype=torch.int32, device="cuda")
        s["top_logprobs"] = torch.empty((rows, case["top"]), device="cuda")
        s["ws"] = torch.zeros(16 << 20, dtype=torch.uint8, device="cuda")
        return s
    h_q, h_kv, d = case["h_q"], case["h_kv"], case["d"]
    if op == "qk_norm_rope":
        s["q"], s["k"], _ = _projection(case, gen, case["rows"])
        s["positions"] = torch.randint(0, case["n_pos"], (case["rows"],), generator=gen, device="cuda", dtype=torch.int32)
        s["rope"] = _rope_table(case["n_pos"], case["rot"])
        s["q_weight"], s["k_weight"] = _weights(case, gen)
        s["q_out"] = torch.empty((case["rows"], h_q, d), dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty((case["rows"], h_kv, d), dtype=torch.bfloat16, device="cuda")
        return s
    s["lens"], s["table"], s["n_phys"] = _paging(case, gen)
    batch, t, ps = case["batch"], case.get("t", 1), case["ps"]
    s["dims"] = (batch, h_q, h_kv, d, ps, s["table"].shape[1], s["n_phys"])
    if op == "kv_append_rope":
        s["q"], s["k"], s["v"] = (x.unflatten(0, (batch, t)) for x in _projection(case, gen, batch * t))
        s["rope"] = _rope_table(case["len_hi"], case["rot"])
        s["q_weight"], s["k_weight"] = _weights(case, gen)
        s["K"], s["V"] = _normal(gen, s["n_phys"], h_kv, ps, d), _normal(gen, s["n_phys"], h_kv, ps, d)
        s["q_out"] = torch.empty((batch, t, h_q, d), dtype=torch.bfloat16, device="cuda")
        s["summ"] = torch.zeros((batch, h_kv, s["table"].shape[1], 2, d), dtype=torch.bfloat16, device="cuda")
        return s
    s["kv4"] = _quantised_cache(case, s["n_phys"], gen)
    if op == "kv4_append":
        s["k"], s["v"] = _normal(gen, batch, t, h_kv, d), _normal(gen, batch, t, h_kv, d)
        s["summ"] = torch.zeros((batch, h_kv, s["table"].shape[1], 2, d), dtype=torch.bfloat16, device="cuda")
        s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        return s
    rows = (batch, h_q) if op == "kv4_sparse" else (batch, t, h_q)
    s["q"] = _normal(gen, *rows, d)
    s["o"] = torch.empty((*rows, d), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty(rows, device="cuda")
    s["ws"] = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    if op == "kv4_sparse":
        pages = (s["lens"] + ps - 1) // ps
        order = torch.rand((batch, h_kv, s["table"].shape[1]), generator=gen, device="cuda")
        at = torch.arange(order.shape[2], device="cuda")
        order.masked_fill_(at >= pages[:, None, None], -1.0)  # no page behind the last one
        order.masked_fill_(at == 0, 2.0)  # the sink page and the newest one are always taken
        order.masked_fill_(at == pages[:, None, None] - 1, 2.0)
        s["nsel"] = pages.clamp(max=case["pages"])[:, None].expand(batch, h_kv).to(torch.int32).contiguous()
        top = order.topk(case["pages"], dim=2).indices
        past = at[:case["pages"]] >= s["nsel"][:, :, None]
        s["sel"] = top.masked_fill(past, 1 << 30).sort(dim=2).values.to(torch.int32).contiguous()
    return s


# ------------------------------------------------------------------ plain forms

def _norm_rope(x, weight, cos, sin, rot, interleaved):
    """x [rows][heads][d] normalised and turned, in 32 bits; cos and sin [rows][rot / 2]."""
    y = x.float()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(dim=-1, keepdim=True) + EPS) * weight.float()
    cos, sin = cos[:, None], sin[:, None]
    turned, rest = y[..., :rot], y[..., rot:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = turned[..., :rot // 2], turned[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _quantise(x):
    """Packed e2m1 codes [..][d / 2] (even channel in the low bits) and e4m3 scale bytes [..][d / 16] of x [..][d]."""
    g = x.float().unflatten(-1, (-1, 16))
    scale = (g.abs().amax(dim=-1) / 6).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    a = torch.where(s > 0, g.abs() / s, torch.zeros_like(g))
    c = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    c = (c + 8 * torch.signbit(g).to(torch.uint8)).flatten(-2)
    return c[..., 0::2] + 16 * c[..., 1::2], scale.view(torch.uint8)


def _values(codes, scales):
    """The fp32 values of packed codes [..][d / 2] and scale bytes [..][d / 16]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    return lut[c.int()] * scales.view(torch.float8_e4m3fn).float().repeat_interleave(16, dim=-1)


def _tile_values(tiles, ps, d):
    """fp32 [..][ps][d] of tiles [..][ps * d * 9 / 16]."""
    n = ps * d // 2
    return _values(tiles[..., :n].unflatten(-1, (ps, d // 2)), tiles[..., n:].unflatten(-1, (ps, d // 16)))


def _new_slots(s):
    """For the t newest tokens of every sequence: positions, physical pages and slots, each [batch][t]."""
    pos = (s["lens"] - s["t"])[:, None] + torch.arange(s["t"], device="cuda", dtype=torch.int32)
    page = torch.gather(s["table"], 1, (pos // s["ps"]).long())
    return pos.long(), page.long(), (pos % s["ps"]).long()


def _refresh(s, key_pages):
    """Rewrites the summaries of the pages that hold the t newest tokens. key_pages(physical) gives the pages' keys [n][h][ps][d]."""
    ps, first = s["ps"], (s["lens"] - s["t"])[:, None]
    page = torch.arange(s["table"].shape[1], device="cuda")[None]
    touched = (page >= first // ps) & (page * ps < s["lens"][:, None])
    b, p = touched.nonzero(as_tuple=True)
    keys = key_pages(s["table"][b, p].long())
    valid = (p[:, None] * ps + torch.arange(ps, device="cuda"))[:, :] < s["lens"][b][:, None]
    valid = valid[:, None, :, None]
    low = torch.where(valid, keys, math.inf).amin(dim=2)
    high = torch.where(valid, keys, -math.inf).amax(dim=2)
    s["summ"][b, :, p] = torch.stack([low, high], dim=2).to(torch.bfloat16)


def _plain_qk(s):
    table = s["rope"][s["positions"].long()]
    turn = lambda x, w: _norm_rope(x, w, table[:, 0], table[:, 1], s["rot"], s["interleaved"]).to(torch.bfloat16)
    return turn(s["q"], s["q_weight"]), turn(s["k"], s["k_weight"])


def _plain_append_rope(s):
    pos, page, slot = _new_slots(s)
    table = s["rope"][pos.flatten()]
    turn = lambda x, w: _norm_rope(x.flatten(0, 1), w, table[:, 0], table[:, 1], s["rot"], s["interleaved"]).to(torch.bfloat16)
    q = turn(s["q"], s["q_weight"]).unflatten(0, (s["batch"], s["t"]))
    s["K"][page.flatten(), :, slot.flatten()] = turn(s["k"], s["k_weight"])
    s["V"][page.flatten(), :, slot.flatten()] = s["v"].flatten(0, 1)
    _refresh(s, lambda phys: s["K"][phys])
    return q, s["K"], s["V"], s["summ"]


def _plain_kv4_append(s):
    _, page, slot = _new_slots(s)
    ps, d = s["ps"], s["d"]
    codes, scales = _quantise(torch.stack([s["k"], s["v"]], dim=3))  # [batch][t][h][2][..]
    n = ps * d // 2
    s["kv4"][..., :n].unflatten(-1, (ps, d // 2))[page.flatten(), :, :, slot.flatten()] = codes.flatten(0, 1)
    s["kv4"][..., n:].unflatten(-1, (ps, d // 16))[page.flatten(), :, :, slot.flatten()] = scales.flatten(0, 1)
    _refresh(s, lambda phys: _tile_values(s["kv4"][phys, :, 0], ps, d))
    back = _values(codes, scales).to(torch.bfloat16)
    return back[:, :, :, 0], back[:, :, :, 1], s["summ"]


def _attend(q, keys, values, visible):
    """q [b][h][r][d], keys and values [b][h][n][d], visible [b][h][r][n] -> o [b][h][r][d], lse [b][h][r]."""
    z = torch.einsum("bhrd,bhnd->bhrn", q.float(), keys) / math.sqrt(q.shape[-1])
    z = z.masked_fill_(~visible, -math.inf)
    m = z.amax(dim=-1, keepdim=True)
    p = torch.exp(z - m)
    total = p.sum(dim=-1, keepdim=True)
    o = torch.einsum("bhrn,bhnd->bhrd", p, values) / total
    return o.to(torch.bfloat16), (m + torch.log(total)).squeeze(-1)


def _plain_sparse(s):
    b, h, ps, d, g = s["batch"], s["h_kv"], s["ps"], s["d"], s["h_q"] // s["h_kv"]
    given = torch.arange(s["pages"], device="cuda") < s["nsel"][:, :, None]
    page = torch.where(given, s["sel"], 0).long()
    phys = torch.gather(s["table"][:, None].expand(b, h, -1), 2, page).long()
    tiles = s["kv4"][phys, torch.arange(h, device="cuda")[None, :, None]]  # [b][h][pages][2][..]
    kv = _tile_values(tiles, ps, d)
    pos = page[..., None] * ps + torch.arange(ps, device="cuda")
    visible = given[..., None] & (pos < s["lens"][:, None, None, None])
    o, lse = _attend(s["q"].unflatten(1, (h, g)), kv[:, :, :, 0].flatten(2, 3), kv[:, :, :, 1].flatten(2, 3), visible.flatten(2)[:, :, None])
    return o.flatten(1, 2), lse.flatten(1, 2)


def _plain_dense(s):
    b, t, h, ps, d, g = s["batch"], s["t"], s["h_kv"], s["ps"], s["d"], s["h_q"] // s["h_kv"]
    kv = _tile_values(s["kv4"][s["table"].clamp(min=0).long()], ps, d)  # [b][pages][h][2][ps][d]
    keys, values = (kv[:, :, :, i].transpose(1, 2).flatten(2, 3) for i in (0, 1))
    last = (s["lens"] - t)[:, None] + torch.arange(t, device="cuda")  # the newest token that position t sees
    visible = torch.arange(keys.shape[2], device="cuda") <= last[:, :, None]  # [b][t][n]
    visible = visible[:, None, :, None].expand(b, h, t, g, -1).flatten(2, 3)
    q = s["q"].unflatten(2, (h, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    o, lse = _attend(q, keys, values, visible)
    back = lambda x: x.unflatten(2, (t, g)).transpose(1, 2).flatten(2, 3)
    return back(o).contiguous(), back(lse).contiguous()


def _plain_logprobs(s):
    x = s["logits"].float()
    z = x * s["inv_temperature"]
    m = z.amax(dim=1, keepdim=True)
    p = torch.exp(z - m)
    total = p.sum(dim=1, keepdim=True)
    lse = (m + torch.log(total))[:, 0]
    p = p / total
    entropy = torch.log(total)[:, 0] - torch.where(p > 0, p * (z - m), 0.0).sum(dim=1)
    target = s["targets"].long()
    logprob = torch.where(target >= 0, torch.gather(z, 1, target.clamp(min=0)[:, None])[:, 0] - lse, 0.0)
    bits = x.view(torch.int32).long()  # whole numbers in the order of the logits, the lower index first among equals
    order = torch.where(bits < 0, -2147483648 - bits, bits) * 4294967296 - torch.arange(x.shape[1], device="cuda")
    ids = order.topk(s["top"], dim=1).indices
    return logprob, entropy, lse, ids.to(torch.int32), torch.gather(z, 1, ids) - lse[:, None]


_PLAIN = {"qk_norm_rope": _plain_qk, "kv_append_rope": _plain_append_rope, "kv4_append": _plain_kv4_append,
          "kv4_sparse": _plain_sparse, "kv4_dense": _plain_dense, "logprobs": _plain_logprobs}


# ------------------------------------------------------------------ the library's calls

def _own(s):
    import sparse_attention_decode_pages_gb300 as spd
    op = s["op"]
    if op == "logprobs":
        logprob, entropy, lse = s["out"]
        spd.token_logprobs(s["logits"], s["targets"], logprob, s["ws"], entropy=entropy, lse=lse, top_ids=s["top_ids"],
                           top_logprobs=s["top_logprobs"], inv_temperature=s["inv_temperature"])
        return logprob, entropy, lse, s["top_ids"], s["top_logprobs"]
    if op == "qk_norm_rope":
        spd.qk_norm_rope(s["q"], s["k"], s["positions"], s["rope"], s["q_out"], s["k_out"], q_weight=s["q_weight"],
                         k_weight=s["k_weight"], eps=EPS, interleaved=s["interleaved"])
        return s["q_out"], s["k_out"]
    dims = spd.dims_of(*s["dims"])
    if op == "kv_append_rope":
        spd.kv_append_rope(dims, s["t"], s["K"], s["V"], s["table"], s["lens"], s["q"], s["k"], s["v"], s["rope"], s["q_out"], s["summ"],
                           q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=s["interleaved"])
        return s["q_out"], s["K"], s["V"], s["summ"]
    if op == "kv4_append":
        spd.kv4_append(dims, s["t"], s["kv4"], s["table"], s["lens"], s["k"], s["v"], s["summ"])
        spd.kv4_read(dims, s["t"], s["kv4"], s["table"], s["lens"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"], s["summ"]
    if op == "kv4_sparse":
        spd.kv4_sparse_decode_attn(dims, s["q"], s["kv4"], s["table"], s["lens"], s["sel"], s["nsel"], s["pages"], s["o"], s["ws"], lse=s["lse"])
    else:
        spd.kv4_dense_verify_attn(dims, s["t"], s["q"], s["kv4"], s["table"], s["lens"], s["o"], s["ws"], lse=s["lse"])
    return s["o"], s["lse"]


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "logprobs":
        n = case["rows"] * case["n_vocab"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + case["rows"] * (16 + 8 * case["top"]), "flops": 6 * n}
    h_q, h_kv, d = case["h_q"], case["h_kv"], case["d"]
    if op == "qk_norm_rope":
        rows = case["rows"]
        return {"bytes": rows * (4 * (h_q + h_kv) * d + 4 * min(case["rot"], d) + 4), "flops": 8 * rows * (h_q + h_kv) * d}
    ps, t, lens = case["ps"], case.get("t", 1), _lengths(case)
    touched = [((n - 1) // ps - (n - t) // ps + 1, n - t - (n - t) // ps * ps) for n in lens]  # pages, older tokens in the first
    if op == "kv_append_rope":
        new = len(lens) * t
        moved = new * (4 * (h_q + 2 * h_kv) * d + 4 * case["rot"])
        return {"bytes": moved + sum(p * 4 * h_kv * d + old * 2 * h_kv * d for p, old in touched), "flops": new * 8 * (h_q + h_kv) * d}
    row4 = h_kv * d * 9 // 16  # bytes of one token's keys, or values, in 4 bits with their scales
    if op == "kv4_append":  # written, and read back as the values that it stands for
        new = len(lens) * t
        moved = new * (8 * h_kv * d + 4 * row4)
        return {"bytes": moved + sum(p * 4 * h_kv * d + old * row4 for p, old in touched), "flops": new * 16 * h_kv * d}
    if op == "kv4_sparse":
        tokens = sum(min(n, case["pages"] * ps) for n in lens)  # of each KV head
        rows = len(lens)
    else:
        tokens, rows = sum(lens), len(lens) * t
    return {"bytes": tokens * 2 * row4 + rows * h_q * (4 * d + 4), "flops": 4 * tokens * t * h_q * d}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_turn(x, weight, angles, rot, interleaved):
    """One tensor of head rows [n][heads][d]; angles [n][2][rot / 2], all in 64 bits: a complex product for each pair."""
    x = x.double()
    if weight is not None:
        x = x * weight.double() * (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).rsqrt()
    i = torch.arange(rot // 2, device=x.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    turn = torch.complex(angles[:, 0].double(), angles[:, 1].double())[:, None]
    pair = torch.complex(x[..., first], x[..., second]) * turn
    y = x.clone()
    y[..., first], y[..., second] = pair.real, pair.imag
    return y


def _exact_e4m3(v):
    """v >= 0 in 64 bits rounded to the nearest e4m3 value (ties to the even one), at most 448."""
    step = torch.exp2(torch.floor(torch.log2(v.clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(max=448.0)


def _exact_stored(x):
    """The values that x [..][d] is held as in 4 bits: the nearest of the sixteen codes' for its group's scale."""
    x = x.double().unflatten(-1, (-1, 16))
    s = _exact_e4m3(x.abs().amax(-1, keepdim=True) / 6)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    a = torch.where(s > 0, x.abs() / s, 0.0).clamp(max=6.0)
    upper = torch.searchsorted(grid, a).clamp(min=1, max=7)
    lower = upper - 1
    up, down = grid[upper] - a, a - grid[lower]
    c = torch.where((up < down) | ((up == down) & (upper % 2 == 0)), upper, lower)
    return (torch.copysign(grid[c], x) * s).flatten(-2)


def _exact_unpacked(tile, ps, d):
    """The 64-bit values [ps][d] of one tile of bytes, or [..][ps][d] of several."""
    codes, scales = tile[..., :ps * d // 2].int(), tile[..., ps * d // 2:].int()
    codes = torch.stack([codes % 16, codes // 16], -1).reshape(*tile.shape[:-1], ps, d // 16, 16)
    exponent, fraction = codes % 8 // 2, codes % 2
    value = torch.where(exponent > 0, (2 + fraction) * 2.0 ** (exponent - 2), fraction * 0.5).double()
    e, f = scales % 128 // 8, scales % 8
    scale = torch.where(e > 0, (8 + f) * torch.exp2((e - 10).double()), f * 2.0 ** -9)
    return (torch.where(codes >= 8, -value, value) * scale.reshape(*tile.shape[:-1], ps, d // 16, 1)).flatten(-2)


def _exact_attention(s):
    sparse, b, h = s["op"] == "kv4_sparse", s["batch"], s["h_kv"]
    ps, d, g, t = s["ps"], s["d"], s["h_q"] // s["h_kv"], s.get("t", 1)
    o = torch.empty((b, t, h, g, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((b, t, h, g), dtype=torch.float64, device="cuda")
    q = s["q"].reshape(b, t, h, g, d).double()
    for i, n in enumerate(s["lens"].tolist()):
        if sparse:
            k = int(s["nsel"][i, 0])
            logical = s["sel"][i, :, :k].long()
        else:
            logical = torch.arange(-(-n // ps), device="cuda")[None].expand(h, -1)
        tiles = s["kv4"][s["table"][i].long()[logical], torch.arange(h, device="cuda")[:, None]]
        keys, values = (_exact_unpacked(tiles[:, :, j], ps, d).flatten(1, 2) for j in (0, 1))
        at = (logical[:, :, None] * ps + torch.arange(ps, device="cuda")).flatten(1)
        seen = at[None] < (n - t + 1 + torch.arange(t, device="cuda"))[:, None, None]  # [t][h][tokens]
        z = torch.matmul(q[i].transpose(0, 1).reshape(h, t * g, d), keys.transpose(1, 2)).reshape(h, t, g, -1) * d ** -0.5
        z = torch.where(seen.transpose(0, 1)[:, :, None], z, -math.inf)
        total = torch.logsumexp(z, -1)
        lse[i] = total.transpose(0, 1)
        o[i] = torch.matmul(torch.exp(z - total[..., None]).flatten(1, 2), values).reshape(h, t, g, d).transpose(0, 1)
    return o.reshape(s["o"].shape), lse.reshape(s["lse"].shape)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "logprobs":
        x = s["logits"].double() * s["inv_temperature"]
        log_p = x - torch.logsumexp(x, 1, keepdim=True)
        picked = log_p.gather(1, s["targets"].long().clamp(min=0)[:, None])[:, 0]
        best = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True).indices[:, :case["top"]]
        entropy = -torch.xlogy(log_p.exp(), log_p.exp()).sum(1)
        return (torch.where(s["targets"] < 0, 0.0, picked), entropy, torch.logsumexp(x, 1), best.to(torch.int32), log_p.gather(1, best))
    if op == "qk_norm_rope":
        angles = s["rope"][s["positions"].long()]
        return tuple(_exact_turn(s[x], s[x + "_weight"], angles, case["rot"], case["interleaved"]) for x in ("q", "k"))
    if op in ("kv4_sparse", "kv4_dense"):
        return _exact_attention(s)
    t, ps = case["t"], case["ps"]
    summ = torch.zeros(s["summ"].shape, dtype=torch.float64, device="cuda")
    if op == "kv_append_rope":
        K, V, q = s["K"].double(), s["V"].double(), torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    else:
        new_k, new_v = _exact_stored(s["k"]), _exact_stored(s["v"])
    for i, n in enumerate(s["lens"].tolist()):
        at = torch.arange(n - t, n, device="cuda")
        page, slot = s["table"][i].long()[at // ps], at % ps
        first, pages = (n - t) // ps, -(-n // ps)
        rows = s["table"][i].long()[first:pages]
        if op == "kv_append_rope":
            angles = s["rope"][at]
            q[i] = _exact_turn(s["q"][i], s["q_weight"], angles, case["rot"], case["interleaved"])
            K[page, :, slot] = _exact_turn(s["k"][i], s["k_weight"], angles, case["rot"], case["interleaved"])
            V[page, :, slot] = s["v"][i].double()
            keys = K[rows].transpose(1, 2).flatten(0, 1)
        else:
            keys = _exact_unpacked(s["kv4"][rows, :, 0], ps, case["d"]).transpose(1, 2).flatten(0, 1)
            keys[n - t - first * ps:n - first * ps] = new_k[i]
        for j in range(pages - first):
            own_rows = keys[j * ps:min((j + 1) * ps, n - first * ps)]
            summ[i, :, first + j, 0], summ[i, :, first + j, 1] = own_rows.amin(0), own_rows.amax(0)
    return (q, K, V, summ) if op == "kv_append_rope" else (new_k, new_v, summ)
