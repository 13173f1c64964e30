"""qk_norm_rope and kv_append_rope against the 64-bit form and against each other, on the GPU."""
import numpy as np
import pytest

from tests import ops_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spd():
    import sparse_attention_decode_pages_gb300 as spd
    spd.spd_device_status(clear=True)
    return spd


def dev(x, dtype=None):
    import torch
    t = torch.as_tensor(np.ascontiguousarray(x))
    return t.to(device="cuda", dtype=dtype or t.dtype)


def projection(rng, rows, H_q, H_kv, D, packed):
    """bf16 q, k, v rows [rows][heads][D]: slices of one buffer with some channels to spare, or buffers of their own."""
    import torch
    if packed:
        x = dev(rng.standard_normal((rows, (H_q + 2 * H_kv) * D + 24)).astype(np.float32), torch.bfloat16)
        parts = torch.split(x[:, : (H_q + 2 * H_kv) * D], [H_q * D, H_kv * D, H_kv * D], 1)
        return [p.unflatten(1, (-1, D)) for p in parts]
    return [dev(rng.standard_normal((rows, h, D)).astype(np.float32), torch.bfloat16) for h in (H_q, H_kv, H_kv)]


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def check_turned(got, x, weight, table, positions, eps, interleaved, what):
    """One rounding to bf16 (half a step, 2^-8 of the value).  Before it: the sum of 128 squares in chains of
    at most 12 additions, rsqrt (2 ulp), and 5 products and sums, each 2^-24 of what it is made of: under
    2^-19 of the magnitudes that meet in an output."""
    y, mag = ref.norm_rope(host(x), None if weight is None else host(weight), table, positions, eps, interleaved)
    err = np.abs(host(got) - y)
    tol = 2.0 ** -8 * np.abs(y) + 2.0 ** -19 * mag
    assert np.all(err <= tol), (what, float((err / np.maximum(tol, 1e-30)).max()))


CASES = [  # rows, H_q, H_kv, D, rot, interleaved, norm, packed
    (1, 32, 8, 128, 128, False, "both", True),
    (5, 4, 2, 64, 64, True, "both", False),
    (7, 7, 1, 128, 48, False, "both", True),
    (33, 3, 3, 64, 8, True, "q", True),
    (64, 8, 1, 128, 64, True, "k", False),
    (19, 5, 5, 128, 0, False, "both", False),
    (257, 16, 8, 64, 24, False, "none", True),
]


@pytest.mark.parametrize("rows,H_q,H_kv,D,rot,inter,norm,packed", CASES)
def test_qk_norm_rope_matches_the_64_bit_form(spd, rows, H_q, H_kv, D, rot, inter, norm, packed):
    import torch
    rng = np.random.default_rng(rows * 7 + D)
    q, k, _ = projection(rng, rows, H_q, H_kv, D, packed)
    n_pos = 5000
    table = ref.rope_table(n_pos, rot)
    positions = rng.integers(0, n_pos, rows)
    positions[0] = n_pos - 1
    wq = dev(1 + 0.3 * rng.standard_normal(D), torch.bfloat16) if norm in ("both", "q") else None
    wk = dev(1 + 0.3 * rng.standard_normal(D), torch.bfloat16) if norm in ("both", "k") else None
    qo = torch.full((rows, H_q, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    ko = torch.full((rows, H_kv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    rope = dev(table) if rot else None
    spd.qk_norm_rope(q, k, dev(positions.astype(np.int32)), rope, qo, ko, q_weight=wq, k_weight=wk, interleaved=inter)
    torch.cuda.synchronize()
    assert spd.spd_device_status(clear=True) == 0
    check_turned(qo, q, wq, table, positions, 1e-6, inter, "q")
    check_turned(ko, k, wk, table, positions, 1e-6, inter, "k")


def test_qk_norm_rope_one_side_in_place_and_zero_rows(spd):
    import torch
    rng = np.random.default_rng(3)
    q, k, _ = projection(rng, 9, 4, 2, 128, False)
    table = dev(ref.rope_table(64, 128))
    pos = dev(np.arange(9, dtype=np.int32))
    both_q, both_k = torch.empty_like(q), torch.empty_like(k)
    spd.qk_norm_rope(q, k, pos, table, both_q, both_k)
    only = torch.empty_like(k)
    spd.qk_norm_rope(None, k, pos, table, None, only)
    assert torch.equal(only, both_k)
    spd.qk_norm_rope(q, None, pos, table, q, None)  # in place
    assert torch.equal(q, both_q)
    z = torch.zeros((3, 4, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(z)
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    spd.qk_norm_rope(z, None, pos[:3].contiguous(), table, out, None, q_weight=w)
    assert torch.count_nonzero(out) == 0
    spd.qk_norm_rope(z[:0], None, pos[:0], table, out[:0], None)


def test_qk_norm_rope_position_outside_the_table(spd):
    import torch
    rng = np.random.default_rng(4)
    q, k, _ = projection(rng, 4, 4, 2, 64, False)
    pos = dev(np.array([3, -1, 64, 63], np.int32))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    table = ref.rope_table(64, 64)
    spd.qk_norm_rope(q, k, pos, dev(table), qo, ko)
    torch.cuda.synchronize()
    assert spd.spd_device_status(clear=True) == spd.DEV_BAD_POS
    assert torch.count_nonzero(qo[1:3]) == 0 and torch.count_nonzero(ko[1:3]) == 0
    check_turned(qo[[0, 3]], q[[0, 3]], None, table, [3, 63], 0, False, "q")


def paged(rng, lens, ps, H_kv, D, spare=2):
    """A random page table over the sequences' pages and some spare ones, and bf16 K, V of normal numbers."""
    import torch
    lens = np.asarray(lens, np.int32)
    pages = -(-lens // ps)
    mp = int(max(1, pages.max())) + 1
    n = int(pages.sum()) + spare
    pt = np.full((len(lens), mp), -1, np.int32)
    perm = rng.permutation(n)
    at = 0
    for b, p in enumerate(pages):
        pt[b, :p] = perm[at: at + p]
        at += p
    K = dev(rng.standard_normal((n, H_kv, ps, D)).astype(np.float32), torch.bfloat16)
    V = dev(rng.standard_normal((n, H_kv, ps, D)).astype(np.float32), torch.bfloat16)
    return lens, pt, mp, n, K, V


def test_kv_append_rope_to_the_longest_sequence(spd):
    """The newest two of 2^31 - 1 tokens, in the last page of a table of 2^27."""
    import torch
    D, ps, mp = 64, 16, 1 << 27
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    rng = np.random.default_rng(9)
    dims = spd.dims_of(1, 1, 1, D, ps, mp, 2)
    pt, lens = torch.ones((1, mp), dtype=torch.int32, device="cuda"), torch.tensor([(1 << 31) - 1], dtype=torch.int32, device="cuda")
    pt[0, -1] = 0
    summ = torch.empty((1, 1, mp, 2, D), dtype=torch.bfloat16, device="cuda")
    summ[0, 0, -2:] = 7.0
    K, V = (dev(rng.standard_normal((2, 1, ps, D)).astype(np.float32), torch.bfloat16) for _ in range(2))
    want_K, want_V = K.clone(), V.clone()
    k, v = (dev(rng.standard_normal((1, 2, 1, D)).astype(np.float32), torch.bfloat16) for _ in range(2))
    spd.kv_append_rope(dims, 2, K, V, pt, lens, None, k, v, None, None, summ)
    torch.cuda.synchronize()
    assert spd.spd_device_status(clear=True) == 0
    want_K[0, 0, 13:15], want_V[0, 0, 13:15] = k[0, :, 0], v[0, :, 0]
    assert torch.equal(K, want_K) and torch.equal(V, want_V)
    held = want_K[0, 0, :15]
    assert torch.equal(summ[0, 0, -1], torch.stack([held.amin(0), held.amax(0)])) and torch.all(summ[0, 0, -2] == 7.0)


APPEND = [  # lens, T, ps, H_q, H_kv, D, rot, interleaved, norm
    ([1, 17, 16, 130], 1, 16, 8, 2, 128, 128, False, True),
    ([40, 33, 64], 33, 32, 7, 1, 64, 32, True, True),
    ([100, 65, 71, 130], 65, 64, 3, 3, 128, 40, False, False),
    ([500], 7, 16, 32, 8, 64, 0, False, True),
    ([16, 2049], 16, 16, 18, 9, 128, 128, True, True),
]


@pytest.mark.parametrize("lens,T,ps,H_q,H_kv,D,rot,inter,norm", APPEND)
@pytest.mark.parametrize("packed", [True, False])
def test_kv_append_rope_is_the_two_calls(spd, lens, T, ps, H_q, H_kv, D, rot, inter, norm, packed):
    """Bit for bit: q_out, K, V and the summaries of qk_norm_rope followed by kv_append_refresh; and the keys
    against the 64-bit form."""
    import torch
    rng = np.random.default_rng(T * 11 + D)
    lens, pt, mp, n, K, V = paged(rng, lens, ps, H_kv, D)
    B = len(lens)
    q, k, v = projection(rng, B * T, H_q, H_kv, D, packed)
    wq = dev(1 + 0.3 * rng.standard_normal(D), torch.bfloat16) if norm else None
    wk = dev(1 + 0.3 * rng.standard_normal(D), torch.bfloat16) if norm else None
    table = ref.rope_table(2100, rot)
    rope = dev(table) if rot else None
    dims = spd.dims_of(B, H_q, H_kv, D, ps, mp, n)
    d_pt, d_lens = dev(pt), dev(lens)
    K2, V2 = K.clone(), V.clone()
    summ = torch.full((B, H_kv, mp, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    summ2 = summ.clone()
    qo, qo2 = (torch.full((B, T, H_q, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    shape4 = [x.unflatten(0, (B, T)) for x in (q, k, v)]
    spd.kv_append_rope(dims, T, K, V, d_pt, d_lens, *shape4, rope, qo, summ, q_weight=wq, k_weight=wk, interleaved=inter)
    pos = (lens[:, None] - T + np.arange(T)).reshape(-1)
    k2 = torch.empty((B * T, H_kv, D), dtype=torch.bfloat16, device="cuda")
    spd.qk_norm_rope(q, k, dev(pos.astype(np.int32)), rope, qo2, k2, q_weight=wq, k_weight=wk, interleaved=inter)
    spd.kv_append_refresh(dims, T, K2, V2, d_pt, d_lens, k2, v.contiguous(), summ2)
    torch.cuda.synchronize()
    assert spd.spd_device_status(clear=True) == 0
    for a, b, what in ((qo, qo2, "q"), (K, K2, "K"), (V, V2, "V"), (summ, summ2, "summaries")):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)), what
    check_turned(k2, k, wk, table, pos, 1e-6, inter, "k")
    # keys and values only: the same cache without queries
    K3, V3, summ3 = K2.clone(), V2.clone(), torch.full_like(summ, 7.0)
    spd.kv_append_rope(dims, T, K3, V3, d_pt, d_lens, None, k, v, rope, None, summ3, k_weight=wk, interleaved=inter)
    assert torch.equal(K3, K2) and torch.equal(V3, V2) and torch.equal(summ3.view(torch.int16), summ2.view(torch.int16))


@pytest.mark.parametrize("rot", [64, 0])
def test_kv_append_rope_skips_what_it_cannot_place(spd, rot):
    """A sequence that is too short, one too long, one past the table, a page id outside the cache: the others
    are as without them, what is skipped is left as it was, and its queries are zeros (but for the bad page's)."""
    import torch
    rng = np.random.default_rng(8)
    T, ps, H_q, H_kv, D = 3, 16, 4, 2, 64
    lens, pt, mp, n, K, V = paged(rng, [20, 30, 40, 35, 50], ps, H_kv, D)
    B = len(lens)
    bad = lens.copy()
    bad[0], bad[1] = 2, mp * ps + 1
    pt_bad = pt.copy()
    pt_bad[3, 32 // ps] = n  # the page of sequence 3's three new tokens
    q, k, v = projection(rng, B * T, H_q, H_kv, D, True)
    table = dev(ref.rope_table(49, rot)) if rot else None
    dims = spd.dims_of(B, H_q, H_kv, D, ps, mp, n)
    K0, V0 = K.clone(), V.clone()
    summ = torch.full((B, H_kv, mp, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    qo = torch.full((B, T, H_q, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    spd.kv_append_rope(dims, T, K, V, dev(pt_bad), dev(bad), q, k, v, table, qo, summ)
    torch.cuda.synchronize()
    want = spd.DEV_BAD_LEN | spd.DEV_BAD_PAGE | (spd.DEV_BAD_POS if rot else 0)
    assert spd.spd_device_status(clear=True) == want
    skipped = [0, 1, 4] if rot else [0, 1]  # length 50 is past a table of 49 positions
    for b in range(B):
        rows = pt[b, : -(-int(lens[b]) // ps)].tolist()
        same = torch.equal(K[rows], K0[rows]) and torch.equal(V[rows], V0[rows])
        assert same == (b in skipped or b == 3), b
        zero = torch.count_nonzero(qo[b]) == 0
        assert bool(zero) == (b in skipped), b
        assert not torch.isnan(qo[b].float()).any()
        assert bool((summ[b] == 7.0).all()) == (b in skipped or b == 3), b


def test_kv_append_rope_under_a_graph_and_on_a_stream(spd):
    import torch
    rng = np.random.default_rng(12)
    T, ps, H_q, H_kv, D = 2, 16, 8, 2, 128
    lens, pt, mp, n, K, V = paged(rng, [20, 33], ps, H_kv, D)
    q, k, v = projection(rng, 4, H_q, H_kv, D, True)
    table = dev(ref.rope_table(64, D))
    dims = spd.dims_of(2, H_q, H_kv, D, ps, mp, n)
    d_pt, d_lens = dev(pt), dev(lens)
    outs = []
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    for how in ("plain", "stream", "graph"):
        Kc, Vc = K.clone(), V.clone()
        summ = torch.zeros((2, H_kv, mp, 2, D), dtype=torch.bfloat16, device="cuda")
        qo = torch.zeros((2, T, H_q, D), dtype=torch.bfloat16, device="cuda")
        args = (dims, T, Kc, Vc, d_pt, d_lens, q, k, v, table, qo, summ)
        torch.cuda.synchronize()
        if how == "plain":
            spd.kv_append_rope(*args)
        elif how == "stream":
            spd.kv_append_rope(*args, stream=side)
        else:
            with torch.cuda.graph(graph):
                spd.kv_append_rope(*args)
            graph.replay()
        torch.cuda.synchronize()
        outs.append((qo, Kc, Vc, summ))
    for other in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], other))
