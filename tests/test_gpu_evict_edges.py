"""The weights and the eviction where few calls go: wide page tables, paths with selections, shared pages; and what a sparse
decode gives over the shortened cache."""
import numpy as np
import pytest

from tests import tree_reference as ref
from tests.test_gpu_evict import check_weights
from tests.test_gpu_rope import dev, host, paged
from tests.test_gpu_tree import bf, check_node, context

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spd():
    import sparse_attention_decode_pages_gb300 as spd
    spd.spd_device_status(clear=True)
    return spd


def update(spd, rng, lens, T, H_q, H_kv, D, ps, tokens, with_path, pages):
    """One call against the 64-bit form, in a table for `tokens` tokens (or as wide as the longest sequence)."""
    import torch
    lens, pt, mp, n, K, V = paged(rng, lens, ps, H_kv, D)
    B, G = len(lens), H_q // H_kv
    if tokens // ps > mp:
        pt = np.concatenate([pt, np.full((B, tokens // ps - mp), -1, np.int32)], 1)
        mp = tokens // ps
    Kh = host(K)
    for b in range(B):
        if lens[b] % ps:
            K[int(pt[b, lens[b] // ps]), :, lens[b] % ps:] = float("nan")
    q = bf(rng.standard_normal((B, T, H_q, D)))
    count = np.minimum(lens, rng.integers(0, T + 1, B) if with_path else T).astype(np.int32)
    path = np.stack([np.concatenate([np.sort(rng.permutation(T)[: c]), np.full(T - c, -7)]) for c in count]).astype(np.int32)
    lse = rng.uniform(4, 9, (B, T, H_q)).astype(np.float32)
    args = dict(decay=0.75)
    if with_path or np.any(lens < T):
        path = path if with_path else np.where(np.arange(T) < count[:, None], np.arange(T), -7).astype(np.int32)
        args.update(path=dev(path), n_path=dev(count))
        with_path = True
    sel, nsel = np.full((B, H_kv, max(1, pages)), -3, np.int32), np.zeros((B, H_kv), np.int32)
    if pages:
        for b in range(B):
            P = -(-lens[b] // ps)
            for h in range(H_kv):
                nsel[b, h] = min(pages, P)
                sel[b, h, : nsel[b, h]] = np.sort(rng.permutation(P)[: nsel[b, h]])
        args.update(sel=dev(sel), nsel=dev(nsel))
    w_in = torch.rand((B, H_kv, mp * ps), device="cuda")
    out = torch.full_like(w_in, 5.0)
    spd.kv_weights_update(spd.dims_of(B, H_q, H_kv, D, ps, mp, n), T, q, dev(lse), K, dev(pt), dev(lens), out, w_in=w_in, **args)
    assert spd.spd_device_status(clear=True) == 0
    qh, scale = host(q), D ** -0.5
    for b in range(B):
        assert bool((out[b, :, lens[b]:] == 5.0).all())
        got, old = host(out[b, :, : lens[b]]), host(w_in[b, :, : lens[b]])
        rows = path[b, : count[b]] if with_path else np.arange(T)
        fresh = lens[b] - len(rows)
        keys = context(lens, pt, Kh, ps, b)
        for h in range(H_kv):
            visible = np.isin(np.arange(lens[b]) // ps, sel[b, h, : nsel[b, h]]) if pages else None
            total, spread = ref.weights(qh[b][rows].reshape(len(rows), H_kv, G, D)[:, h],
                                        lse[b][rows].reshape(len(rows), H_kv, G)[:, h].astype(np.float64), keys[:, h], scale, fresh, visible)
            check_weights(got[h], old[h], 0.75, fresh, lens[b], total, spread, len(rows) * G, (b, h))


WIDE = [  # lens, T, H_q, H_kv, D, ps, tokens of the table, path, pages
    ([0, 1, 17, 300, 4000], 1, 8, 2, 128, 16, 131072, False, 0),
    ([255, 256, 257, 5000, 700], 2, 6, 2, 64, 32, 65536, True, 0),
    ([60001] + 31 * [50, 700], 1, 4, 1, 64, 64, 1 << 18, False, 0),   # fewer CTAs a row than its table has runs
    ([0, 1, 17, 300, 4000], 7, 8, 2, 128, 16, 131072, True, 0),
    ([60001] + 31 * [50, 700], 10, 4, 1, 64, 64, 1 << 18, True, 0),
    ([0, 1, 17, 300, 4000], 1, 8, 2, 128, 16, 131072, False, 9),
    ([20000, 129, 0, 2000], 2, 6, 2, 64, 32, 1 << 18, True, 40),
    ([1600, 20, 7, 5000], 5, 8, 2, 128, 16, 0, True, 9),              # a path with a selection
    ([700, 64, 65], 64, 8, 1, 64, 64, 0, True, 3),
]


@pytest.mark.parametrize("lens,T,H_q,H_kv,D,ps,tokens,with_path,pages", WIDE)
def test_kv_weights_update_wide_tables_and_paths_with_selections(spd, lens, T, H_q, H_kv, D, ps, tokens, with_path, pages):
    update(spd, np.random.default_rng(T * 5 + pages), lens, T, H_q, H_kv, D, ps, tokens, with_path, pages)


@pytest.mark.parametrize("T,pages,tokens", [(2, 0, 0), (40, 0, 0), (3, 40, 0), (1, 0, 65536)])
@pytest.mark.parametrize("limit_ns", [1, 1500])
def test_kv_weights_update_writes_nothing_of_tokens_that_are_late(spd, T, pages, tokens, limit_ns):
    """Whatever the limit, a weight is the usual one or left as it was, with the timeout bit set."""
    import torch
    rng = np.random.default_rng(T)
    H_q, H_kv, D, ps = 8, 2, 128, 16
    lens, pt, mp, n, K, V = paged(rng, rng.integers(T, 6000, 40), ps, H_kv, D)
    B = len(lens)
    if tokens // ps > mp:
        pt = np.concatenate([pt, np.full((B, tokens // ps - mp), -1, np.int32)], 1)
        mp = tokens // ps
    q, lse = bf(rng.standard_normal((B, T, H_q, D))), dev(rng.uniform(4, 9, (B, T, H_q)).astype(np.float32))
    args = {}
    if pages:
        nsel = np.minimum(pages, -(-lens // ps))[:, None].repeat(H_kv, 1).astype(np.int32)
        args = dict(sel=dev(np.tile(np.arange(pages, dtype=np.int32), (B, H_kv, 1))), nsel=dev(nsel))
    w_in = torch.rand((B, H_kv, mp * ps), device="cuda")
    d_pt, d_lens = dev(pt), dev(lens)

    def update():
        w = torch.full_like(w_in, -1.0)
        spd.kv_weights_update(spd.dims_of(B, H_q, H_kv, D, ps, mp, n), T, q, lse, K, d_pt, d_lens, w, w_in=w_in, **args)
        return w, spd.spd_device_status(clear=True)

    want, status = update()
    assert status == 0
    usual = spd.spd_wait_limit_ns()
    try:
        spd.spd_set_wait_limit_ns(limit_ns)
        for _ in range(6):
            got, status = update()
            left = (got == -1.0) & (want != -1.0)
            assert torch.equal(got[~left], want[~left])
            assert status in (0, spd.DEV_TIMEOUT) and (status or not bool(left.any()))
    finally:
        spd.spd_set_wait_limit_ns(usual)
    assert torch.equal(update()[0], want)


@pytest.mark.parametrize("spare", [0, 4000])
def test_kv_evict_of_sequences_that_share_pages(spd, spare):
    """Three sequences begin with the same physical pages; each keeps its own choice of them, and they stay as they were."""
    import torch
    rng = np.random.default_rng(21 + spare)
    H, D, ps, budget, sink, recent = 2, 64, 16, 90, 5, 20
    lens = np.array([200, 163, 160, 80], np.int32)
    _, pt, mp, n, K, V = paged(rng, lens, ps, H, D)
    pt[1, :10], pt[2, :10] = pt[0, :10], pt[0, :10]         # 160 tokens of the first
    if spare:
        pt = np.concatenate([pt, np.full((4, spare), -1, np.int32)], 1)
        mp += spare
    new = np.minimum(lens, budget)
    dst, at = np.full_like(pt, -1), n
    for b in range(4):
        P = -(-new[b] // ps)
        dst[b, :P] = at + rng.permutation(P)
        at += P
    K, V = (torch.cat([x, torch.zeros((at - n, H, ps, D), dtype=torch.bfloat16, device="cuda")]) for x in (K, V))
    w = rng.random((4, H, mp * ps)).astype(np.float32)
    kept = torch.full((4, H, budget), -9, dtype=torch.int32, device="cuda")
    w_out, summ = torch.full((4, H, mp * ps), 5.0, device="cuda"), torch.full((4, H, mp, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    new_lens = torch.zeros(4, dtype=torch.int32, device="cuda")
    want = [host(x) for x in (K, V)]
    spd.kv_evict(spd.dims_of(4, H, H, D, ps, mp, at), budget, sink, recent, K, V, dev(pt), dev(lens), dev(w), dev(dst), kept, w_out, summ, new_lens)
    assert spd.spd_device_status(clear=True) == 0 and np.array_equal(new_lens.cpu().numpy(), new)
    want_summ = np.full((4, H, mp, 2, D), 7.0)
    for b in range(4):
        for h in range(H):
            stay = ref.kept(w[b, h], lens[b], budget, sink, recent)
            assert np.array_equal(kept[b, h, : len(stay)].cpu().numpy(), stay)
            assert np.array_equal(w_out[b, h, : len(stay)].cpu().numpy(), w[b, h, stay])
            j = np.arange(len(stay))
            for x in want:
                x[dst[b, j // ps], h, j % ps] = x[pt[b, stay // ps], h, stay % ps]
            for p in range(-(-len(stay) // ps)):
                rows = want[0][dst[b, p], h, : min(ps, len(stay) - p * ps)]
                want_summ[b, h, p] = rows.min(0), rows.max(0)
    assert np.array_equal(host(K), want[0]) and np.array_equal(host(V), want[1]) and np.array_equal(host(summ), want_summ)


def test_a_sparse_decode_over_the_shortened_cache(spd):
    """A tree's verification, append, weights and eviction, then page selection and sparse decode over what is left, each output
    against its 64-bit form on the inputs that it had."""
    import torch
    rng = np.random.default_rng(78)
    B, T, H_q, H_kv, D, ps, budget, k_max = 3, 12, 8, 2, 128, 16, 200, 6
    G, scale = H_q // H_kv, D ** -0.5
    base = np.array([250, 97, 400], np.int32)
    _, pt, mp, n, K, V = paged(rng, base + T, ps, H_kv, D)
    dst, P = np.full_like(pt, -1), -(-budget // ps)
    dst[:, :P] = n + np.arange(B * P).reshape(B, P)
    K, V = (torch.cat([x, torch.zeros((B * P, H_kv, ps, D), dtype=torch.bfloat16, device="cuda")]) for x in (K, V))
    dims = spd.dims_of(B, H_q, H_kv, D, ps, mp, n + B * P)
    parents = np.stack([ref.random_tree(rng, T, "random") for _ in range(B)])
    q, k, v, qd = (bf(rng.standard_normal(s)) for s in ((B, T, H_q, D), (B, T, H_kv, D), (B, T, H_kv, D), (B, H_q, D)))
    path, count = np.full((B, T), -1, np.int32), np.zeros(B, np.int32)
    sees = [ref.sees(p) for p in parents]
    for b in range(B):
        way = np.flatnonzero(sees[b][T - 1 - b])   # a node's ancestors and itself
        path[b, : len(way)], count[b] = way, len(way)
    z = lambda *shape, dtype=torch.int32: torch.zeros(shape, dtype=dtype, device="cuda")
    o, lse, od, lsed = z(B, T, H_q, D, dtype=torch.bfloat16), z(B, T, H_q, dtype=torch.float32), z(B, H_q, D, dtype=torch.bfloat16), z(B, H_q, dtype=torch.float32)
    summ, summ2 = (z(B, H_kv, mp, 2, D, dtype=torch.bfloat16) for _ in range(2))
    w, w2 = z(B, H_kv, mp * ps, dtype=torch.float32), z(B, H_kv, mp * ps, dtype=torch.float32)
    lens2, lens3, kept, sel, nsel = z(B), z(B), z(B, H_kv, budget), z(B, H_kv, k_max), z(B, H_kv)
    scores = z(B, H_kv, mp, dtype=torch.float32)
    pol = spd.Policy(0, k_max, 0, 0, 1, 0, 1, 1, 1, 1)
    ws = spd.workspace(max(spd.spd_tree_verify_workspace_size(dims, T), spd.spd_score_select_workspace_size(dims),
                           spd.spd_sparse_decode_workspace_size(dims, k_max)))
    d_pt, d_dst, d_base, d_par, d_path, d_count = (dev(x.astype(np.int32)) for x in (pt, dst, base, parents, path, count))
    Kh, Vh = host(K), host(V)
    spd.tree_verify_attn(dims, T, q, K, V, d_pt, d_base, k, v, d_par, o, ws, lse=lse)
    spd.kv_append_path(dims, T, K, V, d_pt, d_base, k, v, d_path, d_count, summ, lens2)
    spd.kv_weights_update(dims, T, q, lse, K, d_pt, lens2, w, path=d_path, n_path=d_count)
    spd.kv_evict(dims, budget, 4, 16, K, V, d_pt, lens2, w, d_dst, kept, w2, summ2, lens3)
    spd.pages_score_select(dims, qd, summ2, lens3, pol, sel, nsel, k_max, ws, scores=scores)
    spd.sparse_decode_attn(dims, qd, K, V, d_dst, lens3, sel, nsel, k_max, od, ws, lse=lsed)
    assert spd.spd_device_status(clear=True) == 0
    o, lse, od, lsed, q, k, v, qd, w, summ2, scores = (host(x) for x in (o, lse, od, lsed, q, k, v, qd, w, summ2, scores))
    kept, sel, nsel = (x.cpu().numpy() for x in (kept, sel, nsel))
    for b in range(B):
        keys, values = (np.concatenate([context(base, pt, c, ps, b), rows[b]]) for c, rows in ((Kh, k), (Vh, v)))
        for t in range(T):
            seen = np.concatenate([np.full(base[b], sees[b][t].any()), sees[b][t]])
            for hq in range(H_q):
                check_node(o[b, t, hq], lse[b, t, hq], q[b, t, hq], keys[:, hq // G], values[:, hq // G], scale, seen, (b, t, hq))
        way = path[b, : count[b]]
        keys, values = (np.concatenate([x[: base[b]], x[base[b] + way]]) for x in (keys, values))
        length = len(keys)
        assert int(lens2[b]) == length and int(lens3[b]) == min(length, budget)
        left = min(length, budget)
        for h in range(H_kv):
            total, spread = ref.weights(q[b, way].reshape(-1, H_kv, G, D)[:, h], lse[b, way].reshape(-1, H_kv, G)[:, h], keys[:, h], scale, base[b])
            check_weights(w[b, h], None, 1.0, base[b], length, total, spread, len(way) * G, (b, h))
            stay = ref.kept(w[b, h], length, budget, 4, 16)
            assert np.array_equal(kept[b, h, :left], stay)
            kk, vv = keys[stay, h], values[stay, h]
            pages = -(-left // ps)
            bounds = np.stack([np.stack([kk[p * ps: p * ps + ps].min(0), kk[p * ps: p * ps + ps].max(0)]) for p in range(pages)])
            assert np.array_equal(summ2[b, h, :pages], bounds)
            # an upper bound of q . k over a page, the group's largest: 2 D products and as many sums in fp32
            qs = qd[b, h * G: h * G + G]
            terms = np.maximum(qs[:, None] * bounds[None, :, 0], qs[:, None] * bounds[None, :, 1])  # [G][pages][D]
            score, room = terms.sum(-1).max(0), (np.abs(terms).sum(-1).max(0)) * 2 * D * 2.0 ** -24
            assert np.all(np.abs(scores[b, h, :pages] - score) <= room)
            m = min(k_max, pages)
            assert nsel[b, h] == m
            chosen = sel[b, h, :m]
            inner = [p for p in range(1, pages - 1)]
            best = sorted(inner, key=lambda p: (-scores[b, h, p], p))[: m - min(2, pages)]
            assert chosen.tolist() == sorted({0, pages - 1, *best})
            seen = np.isin(np.arange(left) // ps, chosen)
            for g in range(G):
                check_node(od[b, h * G + g], lsed[b, h * G + g], qs[g], kk, vv, scale, seen, (b, h, g))
