"""Tree verification, its acceptance and its append against their 64-bit forms on the GPU."""
import numpy as np
import pytest

from tests import ops_reference, tree_reference as ref
from tests.test_gpu_rope import dev, host, paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spd():
    import sparse_attention_decode_pages_gb300 as spd
    spd.spd_device_status(clear=True)
    return spd


def bf(x):
    import torch
    return dev(np.asarray(x, np.float32), torch.bfloat16)


def context(lens, pt, cache, ps, b):
    """Rows [len][H][D] of one sequence's cache (float64)."""
    at = np.arange(lens[b])
    return cache[pt[b, at // ps], :, at % ps]


# ---------------------------------------------------------------- attention

def check_node(o, lse, q, keys, values, scale, visible, what):
    """o: one rounding to bf16 (2^-8), weights rounded to bf16 (2^-8 of sum p |v|), products added up by the tensor
    cores, which cut below 2^-24 of a sum in each of n / 16 steps, and logits that are off by d: D fp32 sums of
    products that add up to at most `mag`, z itself rounded and raised by ex2 (2^-22), and the sum of n weights
    (2^-24 each): a weight's relative error, once in the numerator and once in the sum."""
    want, want_lse, pv, mag = ops_reference.attention(q, keys, values, scale, visible)
    n = int(visible.sum())
    d = mag * (len(q) + 4) * 2.0 ** -24 + 2.0 ** -21 + n * 2.0 ** -24 + (abs(want_lse) * 2.0 ** -22 if np.isfinite(want_lse) else 0.0)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * d + (n / 16 + 1) * 2.0 ** -23) * pv
    assert np.all(np.abs(o - want) <= tol), (what, float((np.abs(o - want) / np.maximum(tol, 1e-30)).max()))
    if np.isneginf(want_lse):
        assert np.isneginf(lse), what
    else:
        assert abs(lse - want_lse) <= d, (what, lse, want_lse)


def attend(spd, dims, T, q, K, V, pt, lens, k, v, parents, scale=None, ws=None, stream=None):
    import torch
    o = torch.full((dims.B, T, dims.H_q, dims.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((dims.B, T, dims.H_q), float("nan"), device="cuda")
    if ws is None:
        ws = torch.full((spd.spd_tree_verify_workspace_size(dims, T),), 0xAB, dtype=torch.uint8, device="cuda")
    spd.tree_verify_attn(dims, T, q, K, V, pt, lens, k, v, parents, o, ws, lse=lse, softmax_scale=scale, stream=stream)
    return o, lse


def poison(lens, pt, K, V, ps):
    """NaN and infinities in every slot that no token holds."""
    used = np.zeros((K.shape[0], ps), bool)
    for b, n in enumerate(lens):
        for t in range(n):
            used[pt[b, t // ps], t % ps] = True
    import torch
    free = dev(~used)[:, None, :, None].expand_as(K)
    for x, y in ((K, float("nan")), (V, float("inf"))):
        x.masked_fill_(free, y)
    V[..., ::2].masked_fill_(free[..., ::2], float("nan"))
    assert torch.isnan(K).any() or used.all()


def case(spd, rng, lens, T, H_q, H_kv, D, ps, trees, packed=True):
    import torch
    lens, pt, mp, n, K, V = paged(rng, lens, ps, H_kv, D)
    B = len(lens)
    poison(lens, pt, K, V, ps)
    if packed:
        rows = bf(rng.standard_normal((B, T, (H_q + 2 * H_kv) * D + 8)))
        q, k, v = (x.unflatten(2, (-1, D)) for x in torch.split(rows[..., :-8], [H_q * D, H_kv * D, H_kv * D], 2))
    else:
        q, k, v = (bf(rng.standard_normal((B, T, h, D))) for h in (H_q, H_kv, H_kv))
    parents = np.stack(trees)
    # rows of what is no node hold anything
    no = dev(~ref.sees(parents[0]).any(1)) if B == 1 else dev(np.stack([~ref.sees(p).any(1) for p in parents]))
    no = no.reshape(B, T)
    k[no] = float("nan")
    v[no] = float("inf")
    return spd.dims_of(B, H_q, H_kv, D, ps, mp, n), lens, pt, K, V, q, k, v, parents


def check_case(spd, dims, lens, pt, K, V, q, k, v, parents, scale=None, rows=None):
    B, T = parents.shape
    o, lse = attend(spd, dims, T, q, K, V, dev(pt), dev(lens), k, v, dev(parents.astype(np.int32)), scale)
    assert spd.spd_device_status(clear=True) == 0
    o, lse, qh, kh, vh, Kh, Vh = (host(x) for x in (o, lse, q, k, v, K, V))
    G = dims.H_q // dims.H_kv
    for b in range(B):
        s = ref.sees(parents[b])
        ck, cv = (context(lens, pt, x, dims.page_size, b) for x in (Kh, Vh))
        keys, values = np.concatenate([ck, kh[b]]), np.concatenate([cv, vh[b]])
        for t in range(T):
            if rows is not None and t not in rows:
                continue
            seen = np.concatenate([np.full(lens[b], s[t].any()), s[t]])
            for hq in range(dims.H_q):
                check_node(o[b, t, hq], lse[b, t, hq], qh[b, t, hq], keys[:, hq // G], values[:, hq // G],
                           dims.D ** -0.5 if scale is None else scale, seen, (b, t, hq))


ATTN = [  # lens, T, H_q, H_kv, D, ps, kind, packed
    ([1, 15, 16, 17, 100], 5, 8, 2, 128, 16, "random", True),
    ([0, 127, 128, 129], 1, 4, 4, 64, 32, "chain", False),
    ([255, 256, 257, 0], 8, 4, 1, 128, 64, "wide", True),
    ([513, 40], 33, 8, 2, 128, 16, "random", True),       # 132 rows: two tiles
    ([300, 700], 32, 8, 2, 64, 16, "chain", False),       # 128 rows
    ([200, 1000], 64, 8, 1, 128, 16, "random", True),     # 512 rows
    ([130], 64, 5, 1, 64, 32, "wide", True),              # 320 rows, groups that do not divide 128
    ([97, 31], 37, 7, 1, 128, 64, "random", False),       # 259 rows
    ([600], 64, 12, 4, 128, 32, "random", True),          # groups of 3
    ([2000], 2, 6, 1, 64, 16, "chain", True),
]


@pytest.mark.parametrize("lens,T,H_q,H_kv,D,ps,kind,packed", ATTN)
def test_tree_verify_attn(spd, lens, T, H_q, H_kv, D, ps, kind, packed):
    rng = np.random.default_rng(T * 31 + D + ps)
    trees = [ref.random_tree(rng, T, kind, T if b % 2 == 0 else max(1, T - 3)) for b in range(len(lens))]
    check_case(spd, *case(spd, rng, lens, T, H_q, H_kv, D, ps, trees, packed))


def test_tree_verify_attn_many_sequences(spd):
    """More (sequence, KV head) rows than SMs, of very different lengths, so that units end inside of others' shares."""
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 700, 50)
    lens[::9] = 0
    trees = [ref.random_tree(rng, 6, "random") for _ in lens]
    check_case(spd, *case(spd, rng, lens, 6, 8, 4, 64, 16, trees), rows={0, 3, 5})


def test_tree_verify_attn_of_a_chain_is_dense_verification(spd):
    """A chain on the cache against dense_verify_attn with the same tokens appended: each within its roundings (the
    outputs' 2^-8 and the weights' 2^-8 of values below 5) of the other."""
    import torch
    rng = np.random.default_rng(8)
    B, T, H_q, H_kv, D, ps = 3, 7, 8, 2, 128, 16
    base = np.array([500, 33, 16], np.int32)
    lens, pt, mp, n, K, V = paged(rng, base + T, ps, H_kv, D)
    dims = spd.dims_of(B, H_q, H_kv, D, ps, mp, n)
    q, k, v = (bf(rng.standard_normal((B, T, h, D))) for h in (H_q, H_kv, H_kv))
    o, lse = attend(spd, dims, T, q, K, V, dev(pt), dev(base), k, v, dev(np.tile(np.arange(-1, T - 1, dtype=np.int32), (B, 1))))
    summ = torch.zeros((B, H_kv, mp, 2, D), dtype=torch.bfloat16, device="cuda")
    spd.kv_append_refresh(dims, T, K, V, dev(pt), dev(lens), k, v, summ)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    spd.dense_verify_attn(dims, T, q, K, V, dev(pt), dev(lens), o2, spd.workspace(spd.spd_dense_verify_workspace_size(dims, T)), lse=lse2)
    assert np.abs(host(o) - host(o2)).max() <= 4 * 2.0 ** -8 * 5
    assert np.abs(host(lse) - host(lse2)).max() <= 1e-4
    assert spd.spd_device_status(clear=True) == 0


@pytest.mark.parametrize("D,T", [(128, 4), (64, 40)])
def test_tree_verify_attn_logits_that_grow(spd, D, T):
    """Maxima that move all along the sequence, by hundreds of powers of two in all, the node's own the largest or the
    smallest; and a negative scale."""
    rng = np.random.default_rng(D)
    trees = [ref.random_tree(rng, T, "random") for _ in range(2)]
    dims, lens, pt, K, V, q, k, v, parents = case(spd, rng, [900, 450], T, 4, 1, D, 16, trees, False)
    ramp = np.linspace(0, 6, 900)
    for b in range(2):
        for t in range(lens[b]):
            K[int(pt[b, t // 16]), :, t % 16] = bf(np.sign(host(q)[b, 0, :1]) * (ramp[t] if b == 0 else 6 - ramp[t]))
    check_case(spd, dims, lens, pt, K, V, q, k, v, parents, 0.5)
    check_case(spd, dims, lens, pt, K, V, q, k, v, parents, -0.25)
    check_case(spd, dims, lens, pt, K, V, q, k, v, parents, 0.0)


def test_tree_verify_attn_an_infinite_key(spd):
    """A key whose logit is -inf for every row weighs nothing; +inf and NaN logits make their rows NaN, and no others."""
    rng = np.random.default_rng(3)
    dims, lens, pt, K, V, q, k, v, parents = case(spd, rng, [300], 4, 2, 2, 64, 16, [ref.random_tree(rng, 4, "chain")], False)
    q[:, :, :, 0] = 1.0
    K[int(pt[0, 3]), 0, 5, 0] = float("-inf")   # token 53 of head 0
    K[int(pt[0, 7]), 1, 1, 0] = float("inf")    # token 113 of head 1
    o, lse = attend(spd, dims, 4, q, K, V, dev(pt), dev(lens), k, v, dev(parents.astype(np.int32)))
    o, lse, qh, kh, vh = (host(x) for x in (o, lse, q, k, v))
    keys = np.concatenate([context(lens, pt, host(K), 16, 0), kh[0]])[:, 0]
    values = np.concatenate([context(lens, pt, host(V), 16, 0), vh[0]])[:, 0]
    keys[53] = 0.0
    for t in range(4):
        seen = np.concatenate([np.ones(300, bool), ref.sees(parents[0])[t]])
        seen[53] = False
        check_node(o[0, t, 0], lse[0, t, 0], qh[0, t, 0], keys, values, 64 ** -0.5, seen, t)
    assert np.isnan(o[0, :, 1]).all() and np.all(np.isnan(lse[0, :, 1]) | np.isposinf(lse[0, :, 1]))


def test_tree_verify_attn_bad_entries(spd):
    """A parent that is not before its node, a page out of range, a length that the table has no room for: flagged, their
    rows or tokens left out, everything else as it should be."""
    rng = np.random.default_rng(17)
    T = 5
    trees = [np.array([-1, 0, 2, 1, 2]), np.array([-1, 0, 0, 1, 7]), np.array([-1, -3, 1, 0, 3]), np.array([-2] * 5), np.array([-1, 0, 1, 2, 3])]
    dims, lens, pt, K, V, q, k, v, parents = case(spd, rng, [60, 70, 80, 33, 50], T, 4, 2, 64, 16, trees, False)
    o, lse = attend(spd, dims, T, q, K, V, dev(pt), dev(lens), k, v, dev(parents.astype(np.int32)))
    assert spd.spd_device_status(clear=True) == spd.DEV_BAD_TREE
    good = (host(o), host(lse))
    for b in range(5):
        s = ref.sees(parents[b])
        for t in range(T):
            if not s[t].any():
                assert np.all(good[0][b, t] == 0) and np.all(np.isneginf(good[1][b, t])), (b, t)
            else:
                assert np.isfinite(good[0][b, t]).all()
    table, bad = pt.copy(), lens.copy()
    table[0, 1] = dims.num_phys_pages          # tokens 16 ... 31 of sequence 0
    table[2, 0] = -1
    bad[1] = dims.max_pages_per_seq * 16 + 1
    bad[4] = -1
    parents[0:3] = np.arange(-1, 4)
    o, lse = attend(spd, dims, T, q, K, V, dev(table), dev(bad), k, v, dev(parents.astype(np.int32)))
    assert spd.spd_device_status(clear=True) == spd.DEV_BAD_PAGE | spd.DEV_BAD_LEN
    o, lse = host(o), host(lse)
    for b in (1, 3, 4):
        assert np.all(o[b] == 0) and np.all(np.isneginf(lse[b]))
    kh, vh = np.nan_to_num(host(k), posinf=0.0), np.nan_to_num(host(v), posinf=0.0)
    for b, gone in ((0, range(16, 32)), (2, range(16))):
        keys, values = (np.concatenate([context(lens, pt, host(x), 16, b), y[b]]) for x, y in ((K, kh), (V, vh)))
        for t in range(T):
            seen = np.concatenate([np.ones(lens[b], bool), ref.sees(parents[b])[t]])
            seen[list(gone)] = False
            if np.isfinite(host(k)[b, : t + 1]).all():
                check_node(o[b, t, 1], lse[b, t, 1], host(q)[b, t, 1], keys[:, 0], values[:, 0], 64 ** -0.5, seen, (b, t))


def test_tree_verify_attn_on_a_stream_in_a_graph_and_in_one_workspace(spd):
    """Captured and replayed over changed inputs, on another stream than the tensors' own, through the workspace that other
    calls use, their tickets left as they were."""
    import torch
    rng = np.random.default_rng(23)
    T = 9
    dims, lens, pt, K, V, q, k, v, parents = case(spd, rng, [400, 90], T, 8, 2, 128, 16, [ref.random_tree(rng, T) for _ in range(2)], False)
    d_pt, d_lens, d_par = dev(pt), dev(lens), dev(parents.astype(np.int32))
    T2 = 4
    q2 = q[:, :T2].contiguous()
    ws = spd.workspace(max(spd.spd_tree_verify_workspace_size(dims, T), spd.spd_dense_verify_workspace_size(dims, T2, 3)))
    want = attend(spd, dims, T, q, K, V, d_pt, d_lens, k, v, d_par)
    want2 = torch.empty_like(q2)
    spd.dense_verify_attn(dims, T2, q2, K, V, d_pt, d_lens, want2, spd.workspace(ws.numel()), num_splits=3)
    for _ in range(2):
        for x, y in zip(attend(spd, dims, T, q, K, V, d_pt, d_lens, k, v, d_par, ws=ws), want):
            assert torch.equal(x, y)
        o2 = torch.empty_like(q2)
        spd.dense_verify_attn(dims, T2, q2, K, V, d_pt, d_lens, o2, ws, num_splits=3)
        assert torch.equal(o2, want2)
    side = torch.cuda.Stream()
    o, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        spd.tree_verify_attn(dims, T, q, K, V, d_pt, d_lens, k, v, d_par, o, ws, lse=lse)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    d_lens.sub_(dev(np.array([64, 5], np.int32)))
    q.mul_(0.5)
    g.replay()
    for x, y in zip((o, lse), attend(spd, dims, T, q, K, V, d_pt, d_lens, k, v, d_par)):
        assert torch.equal(x, y)
    assert spd.spd_device_status(clear=True) == 0


# ---------------------------------------------------------------- acceptance

def accept(spd, q, draft, parents, u_acc, u_res):
    import torch
    B, T, _ = q.shape
    out = torch.full((B,), -9, dtype=torch.int32, device="cuda"), *(torch.full((B, T), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    i32 = lambda x: dev(np.asarray(x).astype(np.int32))
    spd.spec_accept_tree(q if isinstance(q, torch.Tensor) else dev(q), i32(draft), i32(parents), dev(np.float32(u_acc)), dev(np.float32(u_res)), *out)
    return [x.cpu().numpy() for x in out]


def check_accept(spd, q, draft, parents, u_acc, u_res):
    got = accept(spd, q, draft, parents, u_acc, u_res)
    for b in range(len(q)):
        n, path, tokens = ref.accept_tree(q[b], draft[b], parents[b], u_acc[b], u_res[b])
        assert got[0][b] == n and np.array_equal(got[1][b], path) and np.array_equal(got[2][b], tokens), (b, got[0][b], n, got[1][b], path, got[2][b], tokens)
    return got


@pytest.mark.parametrize("n", [1, 2, 127, 1000, 4097, 30004])
@pytest.mark.parametrize("B,T,kind", [(1, 1, "chain"), (5, 8, "wide"), (7, 64, "random"), (40, 5, "chain")])
def test_spec_accept_tree(spd, n, B, T, kind):
    rng = np.random.default_rng(n + T)
    q = rng.exponential(size=(B, T, n)).astype(np.float32) ** 4
    q /= q.sum(-1, keepdims=True) * rng.choice([1.0, 0.5, 3.0], (B, T, 1))
    parents = np.stack([ref.random_tree(rng, T, kind, max(1, T - b % 3)) for b in range(B)])
    best = np.argsort(-q, -1)
    draft = np.zeros((B, T), np.int64)
    for b in range(B):
        for v in range(1, T):
            p = max(0, parents[b, v])
            draft[b, v] = best[b, p, rng.integers(0, min(n, 4))] if rng.random() < 0.9 else rng.integers(0, n)
    u_acc, u_res = rng.random((B, T), np.float32), rng.random(B, np.float32)
    u_acc[rng.random((B, T)) < 0.2] = 0.0
    u_acc[rng.random((B, T)) < 0.1] *= 2.0 ** -20   # numbers with more than 24 bits behind the point
    check_accept(spd, q, draft, parents, u_acc, u_res)
    assert spd.spd_device_status(clear=True) == 0


@pytest.mark.parametrize("kind,T", [("chain", 64), ("random", 64), ("wide", 40)])
def test_spec_accept_tree_long_walks(spd, kind, T):
    """Targets that hold 0.9 of a row on the tokens proposed: walks of many steps, to the last node of a chain."""
    rng = np.random.default_rng(T)
    B, n = 12, 5000
    parents = np.stack([ref.random_tree(rng, T, kind) for _ in range(B)])
    draft = rng.integers(0, n, (B, T))
    q = np.full((B, T, n), 0.1 / n, np.float32)
    for b in range(B):
        for v in range(1, T):
            q[b, parents[b, v], draft[b, v]] += np.float32(0.9 / (parents[b] == parents[b, v]).sum())
    u_acc, u_res = rng.random((B, T), np.float32), rng.random(B, np.float32)
    u_acc[::2] = 0.0  # the first child is always taken
    got = check_accept(spd, q, draft, parents, u_acc, u_res)
    if kind == "chain":
        assert np.all(got[0][::2] == T)
    assert spd.spd_device_status(clear=True) == 0


def test_spec_accept_tree_edges(spd):
    """Rows without weight, a row whose whole weight is tried, the same token twice, tokens outside the vocabulary, the last
    token's borders, values that are no probabilities, and sequences without a tree."""
    n, T = 300, 6
    q = np.zeros((9, T, n), np.float32)
    draft = np.tile(np.arange(T) + 10, (9, 1))
    parents = np.tile([-1, 0, 0, 0, 1, 2], (9, 1))
    u_acc, u_res = np.full((9, T), 0.5, np.float32), np.full(9, 0.999, np.float32)
    # 0: no weight anywhere
    q[1, 0, 11] = 0.25                                  # 1: all weight on the first child; its row has none
    q[2, 0, [11, 12, 13]] = [0.1, 0.1, 0.2]             # 2: every token tried and not taken, nothing left
    u_acc[2, 1:4] = [0.9, 0.9, 1.0]                     # (a number that is not below 1 is never taken)
    draft[3, 1:4] = 7                                   # 3: one token three times
    q[3, 0, 7], q[3, 0, 299] = 0.5, 0.5
    u_acc[3, 1:4] = [0.6, 0.0, 0.0]
    draft[4, 1:4] = [-1, n, 12]                         # 4: outside the vocabulary
    q[4, 0, 12], q[4, 2, 0] = 0.125, 1.0
    q[5, 0, [0, 128, 255, 299]] = [2.0, np.inf, -1.0, np.nan]  # 5: clamped to 1, 1, 0, 0
    u_res[5] = 0.5
    parents[6] = -2                                     # 6: no tree
    parents[7] = [-2, 0, 1, -2, -2, -2]                 # 7: a tree without its root
    q[7, :, 5] = 1.0
    q[8, 0, [0, 299]] = [2.0 ** -40, 1.0]               # 8: the smallest weight there is
    u_res[8] = 0.0
    u_acc[8] = 1.0
    got = check_accept(spd, q, draft, parents, u_acc, u_res)
    assert spd.spd_device_status(clear=True) == spd.DEV_BAD_TOKEN
    assert got[2][0, 0] == -1 and got[2][2, 0] == -1 and got[2][3, 0] == 299 and got[0][6] == got[0][7] == 0 and got[2][8, 0] == 0
    parents[8] = [-1, 0, 2, 3, -9, 0]                   # parents that are not before their nodes
    check_accept(spd, q, draft, parents, u_acc, u_res)
    assert spd.spd_device_status(clear=True) == spd.DEV_BAD_TOKEN | spd.DEV_BAD_TREE


def test_spec_accept_tree_follows_the_target(spd):
    """First tokens of 40,000 walks over one distribution: each token's share within 5 standard deviations of its
    probability, whatever the tree proposes."""
    import torch
    rng = np.random.default_rng(4)
    B, T, n = 40000, 4, 8
    p = np.float32([0.4, 0.25, 0.125, 0.1, 0.0625, 0.0375, 0.025, 0.0])
    draft = np.tile([0, 1, 0, 5], (B, 1))
    parents = np.tile([-1, 0, 0, 0], (B, 1))
    q = dev(p).expand(B, T, n).contiguous()
    tokens = accept(spd, q, draft, parents, rng.random((B, T), np.float32), rng.random(B, np.float32))[2][:, 0]
    share = np.bincount(tokens, minlength=n) / B
    assert np.all(np.abs(share - p) <= 5 * np.sqrt(p * (1 - p) / B)), share
    assert torch.cuda.is_available()


@pytest.mark.parametrize("B,n", [(1, 151936), (3, 151935), (70, 20001), (2, 1 << 21)])
def test_spec_accept_tree_large_vocabularies(spd, B, n):
    rng = np.random.default_rng(B)
    T = 5
    q = rng.exponential(size=(B, T, n)).astype(np.float32) ** 3 + np.float32(1e-9)
    q /= q.sum(-1, keepdims=True)
    parents = np.tile([-1, 0, 0, 1, 1], (B, 1))
    best = np.argsort(-q[:, :2], -1)[..., :2]
    draft = np.concatenate([np.zeros((B, 1), np.int64), best[:, 0], best[:, 1]], 1)
    q[:, 0, :] *= 0.5
    q[np.arange(B), 0, draft[:, 1]] += np.float32(0.5)
    check_accept(spd, q, draft, parents, rng.random((B, T), np.float32), rng.random(B, np.float32))
    assert spd.spd_device_status(clear=True) == 0


# ---------------------------------------------------------------- append

APPEND = [  # lens, T, ps, H, D
    ([0, 1, 15, 16, 17], 5, 16, 2, 128),
    ([31, 32, 40], 64, 32, 9, 64),
    ([63, 0, 100], 33, 64, 1, 128),
    ([7], 1, 16, 3, 64),
]


@pytest.mark.parametrize("lens,T,ps,H,D", APPEND)
@pytest.mark.parametrize("packed", [False, True])
def test_kv_append_path(spd, lens, T, ps, H, D, packed):
    """The whole cache and all summaries, bit for bit: what kv_append_refresh leaves for the path's rows."""
    import torch
    rng = np.random.default_rng(T + D)
    B = len(lens)
    base = np.asarray(lens, np.int32)
    _, pt, mp, n, K, V = paged(rng, base + T, ps, H, D)
    count = rng.integers(0, T + 1, B).astype(np.int32)
    count[0] = min(T, 3)
    count[-1] = T
    path = np.full((B, T), -5, np.int32)
    for b in range(B):
        path[b, : count[b]] = rng.permutation(T)[: count[b]]
    if packed:
        rows = bf(rng.standard_normal((B, T, 2 * H * D + 16)))
        k, v = rows[..., : H * D].unflatten(2, (H, D)), rows[..., H * D: 2 * H * D].unflatten(2, (H, D))
    else:
        k, v = (bf(rng.standard_normal((B, T, H, D))) for _ in range(2))
    dims = spd.dims_of(B, H, H, D, ps, mp, n)
    summ = torch.full((B, H, mp, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    want_K, want_V, want_summ = K.clone(), V.clone(), summ.clone()
    for b in range(B):  # each sequence by itself
        if count[b] == 0:
            continue
        one = spd.dims_of(1, H, H, D, ps, mp, n)
        at = dev(path[b, : count[b]].astype(np.int64))
        part = want_summ[b: b + 1].clone()
        spd.kv_append_refresh(one, int(count[b]), want_K, want_V, dev(pt[b: b + 1]), dev(base[b: b + 1] + count[b: b + 1]),
                              k[b, at][None].contiguous(), v[b, at][None].contiguous(), part)
        want_summ[b] = part[0]
    new = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    spd.kv_append_path(dims, T, K, V, dev(pt), dev(base), k, v, dev(path), dev(count), summ, new)
    assert spd.spd_device_status(clear=True) == 0
    assert torch.equal(K, want_K) and torch.equal(V, want_V) and torch.equal(summ, want_summ)
    assert np.array_equal(new.cpu().numpy(), base + count)


def test_kv_append_path_skips_what_it_cannot_place(spd):
    import torch
    rng = np.random.default_rng(2)
    B, T, ps, H, D = 7, 4, 16, 2, 64
    base = np.array([3, 3, 3, 0, -1, 14, 10], np.int32)
    _, pt, mp, n, K, V = paged(rng, np.full(B, 20), ps, H, D)
    count = np.array([5, 2, -1, 2, 1, 4, 0], np.int32)
    path = np.tile(np.arange(T, dtype=np.int32), (B, 1))
    path[1, 1] = 4
    base[3] = mp * ps - 1
    pt[5, 1] = n  # the second page of sequence 5
    k, v = (bf(rng.standard_normal((B, T, H, D))) for _ in range(2))
    summ = torch.full((B, H, mp, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    before = K.clone(), V.clone()
    new = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    spd.kv_append_path(spd.dims_of(B, H, H, D, ps, mp, n), T, K, V, dev(pt), dev(base), k, v, dev(path), dev(count), summ, new)
    assert spd.spd_device_status(clear=True) == spd.DEV_BAD_TREE | spd.DEV_BAD_LEN | spd.DEV_BAD_PAGE
    assert new.tolist() == [3, 3, 3, mp * ps - 1, -1, 18, 10]
    for x, y, rows in ((K, before[0], k), (V, before[1], v)):
        y[int(pt[5, 0]), :, 14:16] = rows[5, :2].transpose(0, 1)
        assert torch.equal(x, y)
    assert bool((summ[[0, 1, 2, 3, 4, 6]] == 7.0).all()) and bool((summ[5, :, 1:] == 7.0).all()) and not bool((summ[5, :, 0] == 7.0).any())


def test_tree_verify_attn_values_that_are_not_finite(spd):
    """An infinite or NaN value of a node reaches the rows that see it, and no others; no-node rows reach none."""
    rng = np.random.default_rng(31)
    T, D = 6, 64
    parents = np.array([-1, 0, 0, 1, 2, -2])
    dims, lens, pt, K, V, q, k, v, parents = case(spd, rng, [140], T, 8, 2, D, 16, [parents], True)
    clean = v.clone()
    v[0, 1, 0, 5], v[0, 2, 0, 5], v[0, 2, 1, 63], v[0, 4, 0, 7] = float("inf"), float("-inf"), float("nan"), float("nan")
    clean[0, 1, 0, 5] = clean[0, 2, 0, 5] = clean[0, 2, 1, 63] = clean[0, 4, 0, 7] = 0.0
    args = (dev(pt), dev(lens), k)
    o, lse = (host(x) for x in attend(spd, dims, T, q, K, V, *args, v, dev(parents.astype(np.int32))))
    o2, lse2 = (host(x) for x in attend(spd, dims, T, q, K, V, *args, clean, dev(parents.astype(np.int32))))
    assert np.array_equal(lse, lse2)
    for hq in range(4):                       # head 0
        for t in (1, 3):
            o2[0, t, hq, 5] = np.inf
        for t in (2, 4):
            o2[0, t, hq, 5] = -np.inf
        o2[0, 4, hq, 7] = np.nan
        o2[0, [2, 4], 4 + hq, 63] = np.nan    # head 1
    assert np.array_equal(o, o2, equal_nan=True)
    assert spd.spd_device_status(clear=True) == 0


@pytest.mark.parametrize("lens,T,H_q,H_kv,D", [([700, 300], 9, 8, 2, 128), ([700, 300], 64, 4, 1, 128), ([2000, 0], 50, 8, 1, 64)])
def test_tree_verify_attn_with_waits_that_run_out(spd, lens, T, H_q, H_kv, D):
    """A limit that no copy meets: the calls return with the timeout bit (or, should every copy be early, clean), all
    of their waits over, and later calls with the usual limit are those of before."""
    import torch
    rng = np.random.default_rng(T)
    dims, lens, pt, K, V, q, k, v, parents = case(spd, rng, lens, T, H_q, H_kv, D, 16, [ref.random_tree(rng, T, nodes=T - b) for b in range(2)])
    args = (dims, T, q, K, V, dev(pt), dev(lens), k, v, dev(parents.astype(np.int32)))
    first = attend(spd, *args)
    assert spd.spd_device_status(clear=True) == 0
    usual = spd.spd_wait_limit_ns()
    try:
        spd.spd_set_wait_limit_ns(1)
        for _ in range(2):
            attend(spd, *args)
            torch.cuda.synchronize()
            assert spd.spd_device_status(clear=True) & ~spd.DEV_TIMEOUT == 0
    finally:
        spd.spd_set_wait_limit_ns(usual)
    for got, want in zip(attend(spd, *args), first):
        assert torch.equal(got, want)
    assert spd.spd_device_status(clear=True) == 0


@pytest.mark.parametrize("seed", range(16))
def test_tree_verify_attn_of_any_shape(spd, seed):
    """Heads, nodes, pages, lengths and trees drawn together, several sequences to none."""
    rng = np.random.default_rng(1000 + seed)
    H_kv = int(rng.integers(1, 5))
    G, T, D, ps = int(rng.integers(1, 9)), int(rng.integers(1, 65)), int(rng.choice([64, 128])), int(rng.choice([16, 32, 64]))
    B = int(rng.integers(1, 7))
    lens = rng.integers(0, int(rng.choice([20, 300, 900])), B)
    trees = [ref.random_tree(rng, T, str(rng.choice(["chain", "wide", "random"])), int(rng.integers(0, T + 1))) for _ in range(B)]
    check_case(spd, *case(spd, rng, lens, T, G * H_kv, H_kv, D, ps, trees, bool(rng.integers(2))), rows=set(rng.integers(0, T, 6).tolist()))


def test_tree_verify_attn_on_two_streams_at_once(spd):
    """Calls that overlap, each with a workspace of its own: the bits of calls by themselves."""
    import torch
    rng = np.random.default_rng(12)
    calls = []
    for T, D in ((30, 128), (7, 64)):
        dims, lens, pt, K, V, q, k, v, parents = case(spd, rng, rng.integers(500, 4000, 30), T, 8, 2, D, 16, [ref.random_tree(rng, T) for _ in range(30)])
        calls.append((dims, T, q, K, V, dev(pt), dev(lens), k, v, dev(parents.astype(np.int32))))
    want = [attend(spd, *c) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    out = []
    for _ in range(4):
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                out.append(attend(spd, *c))
    torch.cuda.synchronize()
    for i, got in enumerate(out):
        for x, y in zip(got, want[i % 2]):
            assert torch.equal(x, y)
    assert spd.spd_device_status(clear=True) == 0


def test_tree_verify_attn_the_longest_sequence(spd):
    """2^30 - 5 tokens, all but the last page one and the same: the last token, whose weight is e^40 times the others', decides;
    what lies behind it is NaN."""
    import torch
    ps, D, n = 16, 64, (1 << 30) - 5
    pages = 1 << 26
    dims = spd.dims_of(1, 2, 1, D, ps, pages, 2)
    K, V = torch.zeros((2, 1, ps, D), dtype=torch.bfloat16, device="cuda"), torch.ones((2, 1, ps, D), dtype=torch.bfloat16, device="cuda")
    last = (n - 1) % ps
    K[1, 0, last], V[1, 0, last] = 5.0, 5.0
    K[1, 0, last + 1:], V[1, 0, last + 1:] = float("nan"), float("inf")
    pt = torch.zeros((1, pages), dtype=torch.int32, device="cuda")
    pt[0, -1] = 1
    q = torch.ones((1, 2, 2, D), dtype=torch.bfloat16, device="cuda")   # logits 40 (scale 1 / 8) and 0
    k, v = torch.zeros((1, 2, 1, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 2, 1, D), dtype=torch.bfloat16, device="cuda")
    o, lse = attend(spd, dims, 2, q, K, V, pt, torch.tensor([n], dtype=torch.int32, device="cuda"), k, v, dev(np.array([[-1, 0]], np.int32)))
    assert spd.spd_device_status(clear=True) == 0
    # the others' share of the weight is 2^30 e^-40 = 4.6e-9
    assert np.abs(host(o) - 5.0).max() <= 5 * 2.0 ** -8 and np.abs(host(lse) - 40.0).max() <= 40 * 2.0 ** -20
