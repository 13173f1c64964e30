"""The cached tokens' attention weights and the eviction by them against their 64-bit forms on the GPU."""
import numpy as np
import pytest

from tests import tree_reference as ref
from tests.test_gpu_rope import dev, host, paged
from tests.test_gpu_tree import bf, context

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spd():
    import sparse_attention_decode_pages_gb300 as spd
    spd.spd_device_status(clear=True)
    return spd


# ---------------------------------------------------------------- weights

def check_weights(got, w_in, decay, fresh, length, total, spread, rows, what):
    """Each p is off by the logit's error (130 fp32 sums of products of `spread`, the exponent's roundings: 2^-22 of it) and
    ex2's 2^-22; the sum of `rows` of them and the old weight by (rows + 2) 2^-24 of itself."""
    want = np.zeros(length)
    if w_in is not None:
        want[:fresh] = decay * w_in[:fresh]
    want += total
    tol = spread * 140 * 2.0 ** -24 + total * 2.0 ** -21 + np.abs(want) * (rows + 2) * 2.0 ** -24 + total * rows * 2.0 ** -24
    err = np.abs(got[:length] - want)
    assert np.all(err <= tol), (what, float((err / np.maximum(tol, 1e-30)).max()))


WEIGHTS = [  # lens, T, H_q, H_kv, D, ps, path, with old weights, pages selected
    ([1, 16, 17, 600], 1, 8, 2, 128, 16, False, True, 0),
    ([40, 520, 1030], 7, 4, 1, 64, 32, True, True, 0),
    ([64, 65, 700], 64, 8, 1, 128, 64, True, False, 0),
    ([513, 12], 5, 6, 2, 64, 16, False, False, 0),
    ([100, 3, 1500], 3, 5, 5, 128, 16, True, True, 0),
    ([1600, 20, 7], 1, 8, 2, 128, 16, False, True, 9),
    ([1600, 500], 4, 3, 1, 64, 64, False, True, 5),
    ([200, 16, 900], 16, 8, 2, 64, 16, True, True, 0),
    ([129, 1300], 20, 14, 2, 128, 32, False, True, 0),
    ([700, 128, 64], 11, 3, 1, 128, 64, True, False, 0),
    ([4500, 0, 63], 63, 5, 1, 64, 16, True, True, 0),
]


@pytest.mark.parametrize("lens,T,H_q,H_kv,D,ps,with_path,old,pages", WEIGHTS)
def test_kv_weights_update(spd, lens, T, H_q, H_kv, D, ps, with_path, old, pages):
    """Against the 64-bit form, in place and not; what lies behind the lengths is left; empty slots hold NaN keys."""
    import torch
    rng = np.random.default_rng(T * 7 + D)
    lens, pt, mp, n, K, V = paged(rng, lens, ps, H_kv, D)
    B, G, N = len(lens), H_q // H_kv, mp * ps
    Kh = host(K)
    for b in range(B):
        if lens[b] % ps:
            K[int(pt[b, lens[b] // ps]), :, lens[b] % ps:] = float("nan")
    q = bf(rng.standard_normal((B, T, H_q, D)))
    scale = D ** -0.5
    count = np.minimum(lens, rng.integers(0, T + 1, B) if with_path else T).astype(np.int32)
    if with_path:
        count[-1] = min(T, lens[-1])
    path = np.stack([np.concatenate([np.sort(rng.permutation(T)[: c]), np.full(T - c, -7)]) for c in count]).astype(np.int32)
    lse = rng.uniform(4, 9, (B, T, H_q)).astype(np.float32)
    lse[rng.random(lse.shape) < 0.05] = -np.inf
    w_in = rng.uniform(0, 2, (B, H_kv, N)).astype(np.float32)
    w_in[..., ::5] = 0
    k_max = max(1, pages)
    sel, nsel = np.full((B, H_kv, k_max), -3, np.int32), np.zeros((B, H_kv), np.int32)
    for b in range(B):
        P = -(-lens[b] // ps)
        for h in range(H_kv):
            nsel[b, h] = min(pages, P) if h else min(max(0, pages - 1), P)
            sel[b, h, : nsel[b, h]] = np.sort(rng.permutation(P)[: nsel[b, h]])
    ok = [b for b in range(B) if with_path or lens[b] >= T]
    dims = spd.dims_of(B, H_q, H_kv, D, ps, mp, n)
    args = dict(decay=0.75)
    if with_path:
        args.update(path=dev(path), n_path=dev(count))
    if pages:
        args.update(sel=dev(sel), nsel=dev(nsel))
    results = []
    for in_place in (False, True):
        out = dev(w_in).clone() if in_place else torch.full((B, H_kv, N), 5.0, device="cuda")
        if in_place and not old:
            continue
        spd.kv_weights_update(dims, T, q, dev(lse), K, dev(pt), dev(lens), out, w_in=(out if in_place else dev(w_in)) if old else None, **args)
        assert spd.spd_device_status(clear=True) == (0 if len(ok) == B else spd.DEV_BAD_LEN)
        results.append(host(out))
        rest = w_in if in_place else np.full((B, H_kv, N), 5.0)
        for b in range(B):
            first = lens[b] if b in ok else 0
            assert np.array_equal(results[-1][b, :, first:], rest[b, :, first:])
    for b in ok:
        rows = path[b, : count[b]] if with_path else np.arange(T)
        fresh = lens[b] - len(rows)
        keys = context(lens, pt, Kh, ps, b)
        qh = host(q)[b][rows].reshape(len(rows), H_kv, G, D)
        ls = lse[b][rows].reshape(len(rows), H_kv, G).astype(np.float64)
        for h in range(H_kv):
            visible = np.isin(np.arange(lens[b]) // ps, sel[b, h, : nsel[b, h]]) if pages else None
            total, spread = ref.weights(qh[:, h], ls[:, h], keys[:, h], scale, fresh, visible)
            check_weights(results[0][b, h], w_in[b, h] if old else None, 0.75, fresh, lens[b], total, spread, len(rows) * G, (b, h))
            if old:
                assert np.array_equal(results[0][b, h, : lens[b]], results[1][b, h, : lens[b]])


def test_kv_weights_add_up_to_the_queries(spd):
    """With the attention's own lse every query row gives a weight of 1 in all: over a (sequence, KV head) the sums are the
    number of its rows, to 16 times the 2^-21 of a weight and the fp32 sums of a test."""
    import torch
    rng = np.random.default_rng(1)
    B, T, H_q, H_kv, D, ps = 3, 7, 8, 2, 128, 16
    lens, pt, mp, n, K, V = paged(rng, [300, 33, 1200], ps, H_kv, D)
    dims = spd.dims_of(B, H_q, H_kv, D, ps, mp, n)
    q = bf(rng.standard_normal((B, T, H_q, D)))
    o, lse = torch.empty_like(q), torch.empty((B, T, H_q), device="cuda")
    spd.dense_verify_attn(dims, T, q, K, V, dev(pt), dev(lens), o, spd.workspace(spd.spd_dense_verify_workspace_size(dims, T)), lse=lse)
    w = torch.zeros((B, H_kv, mp * ps), device="cuda")
    spd.kv_weights_update(dims, T, q, lse, K, dev(pt), dev(lens), w)
    assert np.abs(host(w).sum(-1) - T * H_q // H_kv).max() <= 28 * 1e-4


def test_kv_weights_update_bad_entries(spd):
    import torch
    rng = np.random.default_rng(6)
    B, T, H, D, ps = 6, 2, 2, 64, 16
    lens, pt, mp, n, K, V = paged(rng, [40] * B, ps, H, D)
    dims = spd.dims_of(B, H, H, D, ps, mp, n)
    q, lse = bf(rng.standard_normal((B, T, H, D))), dev(np.full((B, T, H), 5.0, np.float32))
    path, count = np.tile([0, 1], (B, 1)).astype(np.int32), np.full(B, 2, np.int32)
    good = torch.full((B, H, mp * ps), 3.0, device="cuda")
    spd.kv_weights_update(dims, T, q, lse, K, dev(pt), dev(lens), good, w_in=good, path=dev(path), n_path=dev(count))
    assert spd.spd_device_status(clear=True) == 0
    bad, table = lens.copy(), pt.copy()
    count[0], path[1, 1], bad[2], bad[3], table[4, 1] = 3, 2, mp * ps + 1, 1, n
    w = torch.full((B, H, mp * ps), 3.0, device="cuda")
    spd.kv_weights_update(dims, T, q, lse, K, dev(table), dev(bad), w, w_in=w, path=dev(path), n_path=dev(count))
    assert spd.spd_device_status(clear=True) == spd.DEV_BAD_TREE | spd.DEV_BAD_LEN | spd.DEV_BAD_PAGE
    assert bool((w[:4] == 3.0).all()) and torch.equal(w[5], good[5])
    good[4, :, 16:32] = 3.0
    assert torch.equal(w[4], good[4])
    sel, nsel = np.tile([0, 2], (B, H, 1)).astype(np.int32), np.full((B, H), 2, np.int32)
    want = torch.full((B, H, mp * ps), 3.0, device="cuda")
    spd.kv_weights_update(dims, T, q, lse, K, dev(pt), dev(lens), want, w_in=want, sel=dev(sel), nsel=dev(nsel))
    assert spd.spd_device_status(clear=True) == 0
    sel[0, 0], nsel[1, 0], nsel[2, 1] = [-1, 3], 3, -1
    w = torch.full((B, H, mp * ps), 3.0, device="cuda")
    spd.kv_weights_update(dims, T, q, lse, K, dev(pt), dev(lens), w, w_in=w, sel=dev(sel), nsel=dev(nsel))
    assert spd.spd_device_status(clear=True) == spd.DEV_BAD_SEL
    assert torch.equal(w[1], want[1]) and torch.equal(w[3:], want[3:]) and torch.equal(w[0, 1], want[0, 1])
    assert bool((w[2, 1, :38] == 3.0).all()) and bool((w[2, 1, 38:40] == 0.0).all()) and bool((w[0, 0, :38] == 3.0).all())


# ---------------------------------------------------------------- eviction

def weights_of(rng, kind, shape):
    w = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        w = np.round(w).astype(np.float32)          # many equal ones, many zeros
    elif kind == "same":
        w[:] = 0.25
    elif kind == "odd":
        w *= rng.choice([1, -1], shape).astype(np.float32)
        w[rng.random(shape) < 0.2] = np.nan
        w[rng.random(shape) < 0.1] = np.inf
        w[rng.random(shape) < 0.1] = -np.inf
        w[rng.random(shape) < 0.1] = -0.0
        w[rng.random(shape) < 0.1] = 0.0
    return w


EVICT = [  # lens, budget, sink, recent, H, D, ps, table's spare pages
    ([100, 33, 16, 0], 32, 4, 8, 2, 128, 16, 0),
    ([1000, 1, 999], 500, 0, 0, 3, 64, 32, 5),
    ([700, 65], 65, 65, 0, 1, 128, 64, 0),
    ([300, 301], 100, 1, 99, 2, 64, 16, 0),
    ([513], 1, 0, 0, 9, 64, 16, 3),
    ([2000, 17], 1999, 3, 17, 1, 128, 16, 0),
]


def evict(spd, rng, lens, budget, sink, recent, H, D, ps, spare, w_kind):
    """One call; checks all that it writes and that it writes nothing else."""
    import torch
    lens, pt, mp, n, K, V = paged(rng, lens, ps, H, D)
    B = len(lens)
    if spare:
        pt = np.concatenate([pt, np.full((B, spare), -1, np.int32)], 1)
        mp += spare
    new = np.minimum(lens, budget)
    dst = np.full_like(pt, -1)
    at = n
    for b in range(B):
        P = -(-new[b] // ps)
        dst[b, :P] = at + rng.permutation(P)
        at += P
    K, V = (torch.cat([x, bf(rng.standard_normal((at - n + 1, H, ps, D)))]) for x in (K, V))
    w = weights_of(rng, w_kind, (B, H, mp * ps))
    dims = spd.dims_of(B, H, H, D, ps, mp, at + 1)
    kept = torch.full((B, H, budget), -9, dtype=torch.int32, device="cuda")
    w_out = torch.full((B, H, mp * ps), 5.0, device="cuda")
    summ = torch.full((B, H, mp, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    new_lens = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    want = [host(x) for x in (K, V)]
    want_summ, want_w = np.full((B, H, mp, 2, D), 7.0), np.full((B, H, mp * ps), 5.0, np.float32)
    spd.kv_evict(dims, budget, sink, recent, K, V, dev(pt), dev(lens), dev(w), dev(dst), kept, w_out, summ, new_lens)
    assert spd.spd_device_status(clear=True) == 0
    assert np.array_equal(new_lens.cpu().numpy(), new)
    kept = kept.cpu().numpy()
    for b in range(B):
        for h in range(H):
            stay = ref.kept(w[b, h], lens[b], budget, sink, recent)
            assert np.array_equal(kept[b, h, : len(stay)], stay), (b, h)
            assert np.all(kept[b, h, len(stay):] == -9)
            j = np.arange(len(stay))
            for x in want:
                x[dst[b, j // ps], h, j % ps] = x[pt[b, stay // ps], h, stay % ps]
            want_w[b, h, : len(stay)] = w[b, h, stay]
            for p in range(-(-len(stay) // ps)):
                rows = want[0][dst[b, p], h, : min(ps, len(stay) - p * ps)]
                want_summ[b, h, p] = rows.min(0), rows.max(0)
    assert np.array_equal(host(K), want[0]) and np.array_equal(host(V), want[1])
    assert np.array_equal(w_out.cpu().numpy(), want_w, equal_nan=True) and np.array_equal(host(summ), want_summ)


@pytest.mark.parametrize("lens,budget,sink,recent,H,D,ps,spare", EVICT)
@pytest.mark.parametrize("kind", ["usual", "ties", "same", "odd"])
def test_kv_evict(spd, lens, budget, sink, recent, H, D, ps, spare, kind):
    evict(spd, np.random.default_rng(budget + D), lens, budget, sink, recent, H, D, ps, spare, kind)


@pytest.mark.parametrize("length,spare,budget", [(16384, 0, 5000), (16500, 0, 16400), (40000, 0, 3001), (131101, 0, 100), (900, 9000, 333), (140000, 1500, 70001)])
@pytest.mark.parametrize("kind", ["usual", "ties"])
def test_kv_evict_long_rows(spd, length, spare, budget, kind):
    """One CTA's tokens, a cluster's, and more than a cluster holds; short rows in a table for long ones."""
    evict(spd, np.random.default_rng(length), [length, 50], budget, 7, 50, 1, 64, 16, spare, kind)


def test_kv_evict_bad_entries(spd):
    import torch
    rng = np.random.default_rng(12)
    B, H, D, ps, budget = 4, 2, 64, 16, 24
    lens, pt, mp, n, K, V = paged(rng, [60, 50, 40, 90], ps, H, D, spare=10)
    free = np.setdiff1d(np.arange(n), pt[pt >= 0])
    dst = np.full_like(pt, -1)
    dst[:, :2] = free[:8].reshape(4, 2)
    w = dev(np.tile(np.arange(mp * ps, dtype=np.float32), (B, H, 1)))  # the newest tokens stay
    dims = spd.dims_of(B, H, H, D, ps, mp, n)

    def run(pt, dst, lens):
        out = [K.clone(), V.clone(), torch.full((B, H, budget), -9, dtype=torch.int32, device="cuda"), torch.full_like(w, 5.0),
               torch.full((B, H, mp, 2, D), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((B,), -9, dtype=torch.int32, device="cuda")]
        spd.kv_evict(dims, budget, 0, 0, out[0], out[1], dev(pt), dev(lens), w, dev(dst), out[2], out[3], out[4], out[5])
        return out

    good = run(pt, dst, lens)
    assert spd.spd_device_status(clear=True) == 0
    pt2, dst2, lens2 = pt.copy(), dst.copy(), lens.copy()
    pt2[0, 3] = n          # tokens 48 ... 59 of sequence 0: the last 12 of 36 ... 59
    dst2[1, 1] = -4
    lens2[2] = -5
    got = run(pt2, dst2, lens2)
    assert spd.spd_device_status(clear=True) == spd.DEV_BAD_PAGE | spd.DEV_BAD_LEN
    assert got[5].tolist() == [24, 24, 0, 24]
    good[0][dst[0, 0], :, 12:] = 0
    good[1][dst[0, 0], :, 12:] = 0
    for i, x in ((0, K), (1, V)):
        good[i][dst[0, 1], :, :8] = 0
        good[i][dst[1, 1]] = x[dst[1, 1]]
        good[i][dst[2, :2]] = x[dst[2, :2]]
        assert torch.equal(got[i], good[i])
    assert torch.equal(got[2][[0, 1, 3]], good[2][[0, 1, 3]]) and bool((got[2][2] == -9).all())
    assert torch.equal(got[4][3], good[4][3]) and bool((got[4][2] == 7.0).all()) and bool((got[4][1, :, 1] == 7.0).all())


def test_a_round_with_trees_and_eviction_as_it_is_used(spd):
    """Rotated projections, a tree's verification, acceptance, append and weights, then the eviction and a sparse decode over
    the shortened cache, captured as one graph, with nothing but the library's calls between: against the parts in 64 bits."""
    import torch
    rng = np.random.default_rng(77)
    B, T, H_q, H_kv, D, ps, n_vocab, budget, k_max = 3, 12, 8, 2, 128, 16, 500, 96, 4
    G = H_q // H_kv
    base = np.array([150, 97, 200], np.int32)
    _, pt, mp, n, K, V = paged(rng, base + T, ps, H_kv, D)
    dst = np.full_like(pt, -1)
    P = -(-budget // ps)
    dst[:, :P] = n + np.arange(B * P).reshape(B, P)
    K, V = (torch.cat([x, torch.zeros((B * P, H_kv, ps, D), dtype=torch.bfloat16, device="cuda")]) for x in (K, V))
    dims = spd.dims_of(B, H_q, H_kv, D, ps, mp, n + B * P)
    parents = np.stack([ref.random_tree(rng, T, "wide") for _ in range(B)]).astype(np.int32)
    depth = ref.sees(parents[0]).sum(1) - 1
    rows = bf(rng.standard_normal((B, T, (H_q + 2 * H_kv) * D)))
    q, k, v = (x.unflatten(2, (-1, D)) for x in torch.split(rows, [H_q * D, H_kv * D, H_kv * D], 2))
    ang = np.arange(256)[:, None] * 10000.0 ** (-np.arange(0, D, 2) / D)
    rope = dev(np.stack([np.cos(ang), np.sin(ang)], 1).astype(np.float32))
    positions = dev((base[:, None] + depth[None]).astype(np.int32))
    q_t = rng.exponential(size=(B, T, n_vocab)).astype(np.float32) ** 4
    q_t /= q_t.sum(-1, keepdims=True)
    draft = np.zeros((B, T), np.int32)
    for b in range(B):
        for x in range(1, T):
            draft[b, x] = np.argsort(-q_t[b, parents[b, x]])[(x - 1) % 3]
    u_acc, u_res = rng.random((B, T), np.float32) * np.float32(0.4), rng.random(B, np.float32)
    z = lambda *shape, dtype=torch.int32: torch.zeros(shape, dtype=dtype, device="cuda")
    qr, kr = z(B, T, H_q, D, dtype=torch.bfloat16), z(B, T, H_kv, D, dtype=torch.bfloat16)
    o, lse = z(B, T, H_q, D, dtype=torch.bfloat16), z(B, T, H_q, dtype=torch.float32)
    n_path, path, tokens, lens2, lens3 = z(B), z(B, T), z(B, T), z(B), z(B)
    summ, summ2 = (z(B, H_kv, mp, 2, D, dtype=torch.bfloat16) for _ in range(2))
    w0 = rng.uniform(0, 0.1, (B, H_kv, mp * ps)).astype(np.float32)
    w_in, w, w2 = dev(w0), z(B, H_kv, mp * ps, dtype=torch.float32), z(B, H_kv, mp * ps, dtype=torch.float32)
    kept, sel, nsel = z(B, H_kv, budget), z(B, H_kv, k_max), z(B, H_kv)
    qd, od = bf(rng.standard_normal((B, H_q, D))), z(B, H_q, D, dtype=torch.bfloat16)
    pol = spd.Policy(0, k_max, 0, 0, 1, 0, 1, 1, 1, 1)
    d = {x: dev(y) for x, y in dict(pt=pt, dst=dst, base=base, par=parents, q_t=q_t, draft=draft, ua=u_acc, ur=u_res).items()}
    ws = spd.workspace(max(spd.spd_tree_verify_workspace_size(dims, T), spd.spd_score_select_workspace_size(dims),
                           spd.spd_sparse_decode_workspace_size(dims, k_max)))
    K0, V0 = K.clone(), V.clone()

    def step():
        spd.qk_norm_rope(q, k, positions, rope, qr, kr)
        spd.tree_verify_attn(dims, T, qr, K, V, d["pt"], d["base"], kr, v, d["par"], o, ws, lse=lse)
        spd.spec_accept_tree(d["q_t"], d["draft"], d["par"], d["ua"], d["ur"], n_path, path, tokens)
        spd.kv_append_path(dims, T, K, V, d["pt"], d["base"], kr, v, path, n_path, summ, lens2)
        spd.kv_weights_update(dims, T, qr, lse, K, d["pt"], lens2, w, w_in=w_in, path=path, n_path=n_path)
        spd.kv_evict(dims, budget, 4, 16, K, V, d["pt"], lens2, w, d["dst"], kept, w2, summ2, lens3)
        spd.pages_score_select(dims, qd, summ2, lens3, pol, sel, nsel, k_max, ws)
        spd.sparse_decode_attn(dims, qd, K, V, d["dst"], lens3, sel, nsel, k_max, od, ws)

    outs = (o, lse, n_path, path, tokens, K, V, lens2, w, kept, w2, lens3, sel, nsel, od)
    step()
    torch.cuda.synchronize()
    first = [x.clone() for x in outs]
    for x in outs:
        x.zero_()
    K.copy_(K0)
    V.copy_(V0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    g.replay()
    torch.cuda.synchronize()
    assert spd.spd_device_status(clear=True) == 0
    for x, y in zip(outs, first):
        assert torch.equal(x, y)
    got_w = host(w)
    for b in range(B):
        c, p, t = ref.accept_tree(q_t[b], draft[b], parents[b], u_acc[b], u_res[b])
        assert int(n_path[b]) == c and np.array_equal(path[b].cpu(), p) and np.array_equal(tokens[b].cpu(), t)
        length = base[b] + c
        assert int(lens2[b]) == length and int(lens3[b]) == min(length, budget)
        keys = context(base + n_path.cpu().numpy(), pt, host(K), ps, b)
        assert np.array_equal(keys[base[b]:], host(kr)[b, p[:c]])
        for h in range(H_kv):
            # the accepted rows' weights, with the lse that the tree's verification gave: rows at their positions
            total, spread = ref.weights(host(qr)[b, p[:c]].reshape(c, H_kv, G, D)[:, h], host(lse)[b, p[:c]].reshape(c, H_kv, G)[:, h],
                                        keys[:, h], D ** -0.5, base[b])
            check_weights(got_w[b, h], w0[b, h], 1.0, base[b], length, total, spread, c * G, (b, h))
            assert np.array_equal(kept[b, h].cpu(), ref.kept(got_w[b, h], length, budget, 4, 16))
            stay = kept[b, h].cpu().numpy()
            j = np.arange(budget)
            assert np.array_equal(host(K)[dst[b, j // ps], h, j % ps], keys[stay, h])


def test_kv_evict_rows_beyond_shared_memory(spd):
    """A row that no cluster holds."""
    evict(spd, np.random.default_rng(4), [400001, 3000], 4096, 4, 500, 1, 64, 64, 0, "ties")


@pytest.mark.parametrize("longest", [700, 20011])
def test_kv_evict_many_rows(spd, longest):
    """More (sequence, KV head) rows than SMs: one CTA a row, and clusters of two."""
    rng = np.random.default_rng(longest)
    evict(spd, rng, [longest, *rng.integers(0, 400, 40)], 150, 2, 30, 4, 64, 32, 0, "usual")


def test_kv_weights_update_of_a_long_row(spd):
    """2^30 - 3 tokens of one page: the weights of the first, of some in the middle, and of the newest, which is fresh."""
    import torch
    ps, D, n = 64, 64, (1 << 30) - 3
    pages = 1 << 24
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    rng = np.random.default_rng(2)
    dims = spd.dims_of(1, 3, 1, D, ps, pages, 1)
    K = bf(rng.standard_normal((1, 1, ps, D)))
    pt = torch.zeros((1, pages), dtype=torch.int32, device="cuda")
    w = torch.ones((1, 1, pages * ps), device="cuda")
    q, lse = bf(rng.standard_normal((1, 1, 3, D))), dev(np.array([[[5.0, 6.0, 7.0]]], np.float32))
    spd.kv_weights_update(dims, 1, q, lse, K, pt, torch.tensor([n], dtype=torch.int32, device="cuda"), w, w_in=w, decay=0.5)
    assert spd.spd_device_status(clear=True) == 0
    total, spread = ref.weights(host(q)[0], lse.cpu().numpy()[0].astype(np.float64), host(K)[0, 0], D ** -0.5, ps)
    got = w[0, 0]
    for t0 in (0, 1 << 20, (1 << 29) + 64, (1 << 30) - 64):
        block = host(got[t0: t0 + ps])
        stop = min(ps, n - t0)
        fresh = n - 1 - t0
        check_weights(block, np.ones(ps), 0.5, fresh, stop, total[:stop], spread[:stop], 3, t0)
    assert got[n:].tolist() == [1.0] * 3


def test_caches_past_4_gib(spd):
    """Pages whose byte offset passes 32 bits: tree verification, append, weights and eviction between the cache's two ends."""
    import torch
    rng = np.random.default_rng(40)
    ps, H, D, T = 64, 8, 128, 5
    n = (5 << 30) // (H * ps * D * 2)
    lens, pt, mp, m, K, V = paged(rng, [150, 70], ps, H, D)
    far = np.where(pt >= 0, n - 1 - pt, -1).astype(np.int32)      # the same pages at the end of a large cache
    far[:, -1] = [n - 1 - m, n - 2 - m]                          # a spare page each, for what is appended
    big_K, big_V = (torch.zeros((n, H, ps, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for p in range(m):
        big_K[n - 1 - p], big_V[n - 1 - p] = K[p], V[p]
    q, k, v = (bf(rng.standard_normal((2, T, h, D))) for h in (2 * H, H, H))
    parents = dev(np.tile(np.array([-1, 0, 0, 1, 2], np.int32), (2, 1)))
    results = []
    for cache_K, cache_V, table, pages in ((K, V, pt, m), (big_K, big_V, far, n)):
        if pages == m:  # with the spare pages and those of the eviction behind the others
            extra = torch.zeros((6, H, ps, D), dtype=torch.bfloat16, device="cuda")
            cache_K, cache_V, pages = torch.cat([cache_K, extra]), torch.cat([cache_V, extra]), m + 6
            table = table.copy()
            table[:, -1] = [m, m + 1]
            dst = np.array([[m + 2, m + 3], [m + 4, m + 5]], np.int32)
        else:
            dst = np.array([[0, n // 2], [1, n // 2 + 1]], np.int32)
        dims = spd.dims_of(2, 2 * H, H, D, ps, table.shape[1], pages)
        dst_table = np.full_like(table, -1)
        dst_table[:, :2] = dst
        o, lse = torch.empty_like(q), torch.empty((2, T, 2 * H), device="cuda")
        d_pt, d_lens = dev(table), dev(lens)
        spd.tree_verify_attn(dims, T, q, cache_K, cache_V, d_pt, d_lens, k, v, parents, o, spd.workspace(spd.spd_tree_verify_workspace_size(dims, T)), lse=lse)
        path, count = dev(np.array([[0, 1, 3, -1, -1], [0, 2, -1, -1, -1]], np.int32)), dev(np.array([3, 2], np.int32))
        summ = torch.zeros((2, H, table.shape[1], 2, D), dtype=torch.bfloat16, device="cuda")
        new, new2 = (torch.zeros(2, dtype=torch.int32, device="cuda") for _ in range(2))
        spd.kv_append_path(dims, T, cache_K, cache_V, d_pt, d_lens, k, v, path, count, summ, new)
        w, w2 = (torch.zeros((2, H, table.shape[1] * ps), device="cuda") for _ in range(2))
        spd.kv_weights_update(dims, T, q, lse, cache_K, d_pt, new, w, path=path, n_path=count)
        kept = torch.full((2, H, 100), -1, dtype=torch.int32, device="cuda")
        spd.kv_evict(dims, 100, 4, 20, cache_K, cache_V, d_pt, new, w, dev(dst_table), kept, w2, summ, new2)
        assert spd.spd_device_status(clear=True) == 0
        results.append([o, lse, new, w, kept, w2, new2] + [x[dev(dst.reshape(-1).astype(np.int64))] for x in (cache_K, cache_V)])
    for x, y in zip(*results):
        assert torch.equal(x, y)


@pytest.mark.parametrize("length", [5000, 16000, 60001, 400003])
@pytest.mark.parametrize("values", [2, 3, 2048, 1 << 21])
def test_kv_evict_weights_that_differ_in_their_last_bits(spd, monkeypatch, length, values):
    """Keys with the same upper bits, more of them than go on alone, down to the last bit."""
    def close(rng, kind, shape):
        return (np.uint32(0x3F800000) + rng.integers(0, values, shape).astype(np.uint32)).view(np.float32) * np.float32(kind)
    monkeypatch.setitem(globals(), "weights_of", close)
    rng = np.random.default_rng(length + values)
    evict(spd, rng, [length, 700], length // 2, 3, 100, 1, 64, 64, 0, 1)
    evict(spd, rng, [length], length - 700, 0, 0, 1, 64, 64, 0, -1)


def test_kv_evict_weights_at_any_address(spd):
    """Weights that start at no multiple of 16 bytes."""
    import torch
    rng = np.random.default_rng(8)
    lens, budget, H, D, ps = [1001, 40, 333], 100, 2, 64, 16
    lens, pt, mp, n, K, V = paged(rng, lens, ps, H, D)
    B = len(lens)
    dst = np.full_like(pt, -1)
    dst[:, :7] = n + np.arange(B * 7).reshape(B, 7)
    K, V = (torch.cat([x, bf(rng.standard_normal((B * 7 + 1, H, ps, D)))]) for x in (K, V))
    w = rng.random((B, H, mp * ps)).astype(np.float32)
    dims = spd.dims_of(B, H, H, D, ps, mp, K.shape[0])
    for off in (1, 2, 3):
        at = torch.full((w.size + 4,), 9.0, device="cuda")[off: off + w.size].view(w.shape)
        at.copy_(dev(w))
        kept = torch.full((B, H, budget), -9, dtype=torch.int32, device="cuda")
        w_out = torch.full((w.size + 4,), 5.0, device="cuda")[off: off + w.size].view(w.shape)
        summ = torch.zeros((B, H, mp, 2, D), dtype=torch.bfloat16, device="cuda")
        new_lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        spd.kv_evict(dims, budget, 4, 10, K, V, dev(pt), dev(lens), at, dev(dst), kept, w_out, summ, new_lens)
        assert spd.spd_device_status(clear=True) == 0
        for b in range(B):
            for h in range(H):
                stay = ref.kept(w[b, h], lens[b], budget, 4, 10)
                assert np.array_equal(kept[b, h, : len(stay)].cpu().numpy(), stay)
                assert np.array_equal(w_out[b, h, : len(stay)].cpu().numpy(), w[b, h, stay])


@pytest.mark.parametrize("T,G", [(2, 3), (5, 8), (8, 1)])
def test_kv_weights_update_keys_and_rows_that_are_not_finite(spd, T, G):
    """Rows of lse = -inf add nothing, whatever their queries hold; a key of -inf logits gets nothing from any row, one of +inf
    logits infinity, a NaN key NaN, and no other token is touched by them."""
    import torch
    rng = np.random.default_rng(T)
    D, ps, length = 64, 16, 200
    lens, pt, mp, n, K, V = paged(rng, [length], ps, 1, D)
    q = np.abs(host(bf(rng.standard_normal((1, T, G, D)))))
    lse = rng.uniform(4, 9, (1, T, G)).astype(np.float32)
    for t, value in ((20, float("-inf")), (40, float("inf")), (41, float("nan"))):
        K[int(pt[0, t // ps]), 0, t % ps, 0] = value
    dead = [(0, 0), (T - 1, G - 1)]
    for (t, g), value in zip(dead, (np.nan, np.inf)):
        lse[0, t, g], q[0, t, g] = -np.inf, value
    keys = context(lens, pt, host(K), ps, 0)[:, 0]
    w_in = rng.uniform(0, 2, (1, 1, mp * ps)).astype(np.float32)
    out = torch.full((1, 1, mp * ps), 5.0, device="cuda")
    spd.kv_weights_update(spd.dims_of(1, G, 1, D, ps, mp, n), T, bf(q), dev(lse), K, dev(pt), dev(lens), out, w_in=dev(w_in), decay=0.5)
    assert spd.spd_device_status(clear=True) == 0
    got = host(out)[0, 0]
    assert got[20] == 0.5 * w_in[0, 0, 20] and np.isposinf(got[40]) and np.isnan(got[41])
    finite = keys.copy()
    finite[[20, 40, 41]] = 0
    q[0, [t for t, g in dead], [g for t, g in dead]] = 0
    total, spread = ref.weights(host(bf(q))[0], lse[0].astype(np.float64), finite, D ** -0.5, length - T)
    rest = np.delete(np.arange(length), [20, 40, 41])
    check_weights(got[rest], w_in[0, 0][rest], 0.5, length - T - 3, len(rest), total[rest], spread[rest], T * G, T)


@pytest.mark.parametrize("T,pages", [(2, 0), (40, 0), (3, 4)])
def test_kv_weights_update_with_waits_that_run_out(spd, T, pages):
    """A limit of 1 ns: the call ends, and the next one with the usual limit gives a clean one's bits."""
    import torch
    rng = np.random.default_rng(T)
    H_q, H_kv, D, ps = 8, 2, 128, 16
    lens, pt, mp, n, K, V = paged(rng, [3000, 200, 40], ps, H_kv, D)
    dims = spd.dims_of(3, H_q, H_kv, D, ps, mp, n)
    q, lse = bf(rng.standard_normal((3, T, H_q, D))), dev(rng.uniform(4, 9, (3, T, H_q)).astype(np.float32))
    args = {}
    if pages:
        args = dict(sel=dev(np.tile(np.array([0, 1, 2], np.int32), (3, H_kv, 1))), nsel=dev(np.full((3, H_kv), 3, np.int32)))

    def update():
        w = torch.zeros((3, H_kv, mp * ps), device="cuda")
        spd.kv_weights_update(dims, T, q, lse, K, dev(pt), dev(lens), w, **args)
        torch.cuda.synchronize()
        return w

    first = update()
    assert spd.spd_device_status(clear=True) == 0
    usual = spd.spd_wait_limit_ns()
    try:
        spd.spd_set_wait_limit_ns(1)
        for _ in range(3):
            update()
            assert spd.spd_device_status(clear=True) & ~spd.DEV_TIMEOUT == 0
    finally:
        spd.spd_set_wait_limit_ns(usual)
    assert torch.equal(update(), first) and spd.spd_device_status(clear=True) == 0


def test_kv_weights_update_of_a_long_row_many_queries(spd):
    """2^30 - 3 tokens of one page and 18 query rows."""
    import torch
    ps, D, T, n = 64, 64, 6, (1 << 30) - 3
    pages = 1 << 24
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    rng = np.random.default_rng(3)
    dims = spd.dims_of(1, 3, 1, D, ps, pages, 1)
    K = bf(rng.standard_normal((1, 1, ps, D)))
    pt = torch.zeros((1, pages), dtype=torch.int32, device="cuda")
    w = torch.ones((1, 1, pages * ps), device="cuda")
    q, lse = bf(rng.standard_normal((1, T, 3, D))), dev(rng.uniform(5, 8, (1, T, 3)).astype(np.float32))
    spd.kv_weights_update(dims, T, q, lse, K, pt, torch.tensor([n], dtype=torch.int32, device="cuda"), w, w_in=w, decay=0.5)
    assert spd.spd_device_status(clear=True) == 0
    got = w[0, 0]
    for t0 in (0, 1 << 20, (1 << 29) + 64, (1 << 30) - 64):
        block = host(got[t0: t0 + ps])
        stop, fresh = min(ps, n - t0), n - T - t0
        total, spread = ref.weights(host(q)[0], lse.cpu().numpy()[0].astype(np.float64), host(K)[0, 0], D ** -0.5, min(fresh, ps))
        check_weights(block, np.ones(ps), 0.5, fresh, stop, total[:stop], spread[:stop], 3 * T, t0)
    assert got[n:].tolist() == [1.0] * 3
