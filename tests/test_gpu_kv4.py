"""The 4-bit paged cache on the GPU: its numbers bit for bit, its attention against the 64-bit form over them."""
import numpy as np
import pytest

from tests import ops_reference as ref
from tests.test_gpu_rope import dev, host, paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spd():
    import sparse_attention_decode_pages_gb300 as spd
    spd.spd_device_status(clear=True)
    return spd


def rows_bf16(rng, *shape, spread=False):
    """bf16 values as float64: normal, or over many powers of two with zeros, ties and tiny groups among them."""
    x = rng.standard_normal(shape)
    if spread:
        x = x * 2.0 ** rng.integers(-14, 12, (*shape[:-1], 1))
        flat = x.reshape(-1, 16)
        flat[::7] = 0.0
        flat[1::7] = np.round(flat[1::7] * 4) / 4  # many exact ties
        flat[2::11] *= 2.0 ** -12                   # scales below the smallest e4m3 number
        flat[3::11, 0] = 5000.0                     # scales past the largest
    return ref.bf16(x)


def to_dev(x):
    import torch
    return dev(x.astype(np.float32), torch.bfloat16)


def append_reference(kv4, pt, lens, T, k, v, ps, k_exp, v_exp):
    """kv4 (numpy bytes) with the T newest tokens written; the summaries' bf16 values of the touched pages."""
    kv4 = kv4.copy()
    H, D = k.shape[2], k.shape[3]
    summ = {}
    for b, n in enumerate(lens):
        if n < T:
            continue
        for p in range((n - T) // ps, -(-n // ps)):
            for h in range(H):
                tile = kv4[pt[b, p], h]
                for half, (rows, e) in enumerate(((k, k_exp), (v, v_exp))):
                    codes, scale = (x.copy() for x in ref.kv4_unpack(tile[half], ps, D))
                    for pos in range(max(p * ps, n - T), min((p + 1) * ps, n)):
                        codes[pos % ps], scale[pos % ps] = ref.kv4_quantise(rows[b, pos - (n - T), h], e)
                    tile[half] = ref.kv4_pack(codes, scale)
                    if half == 0:
                        val = ref.kv4_values(codes, scale, e)[: min(ps, n - p * ps)]
                        summ[b, h, p] = (val.min(0), val.max(0))
    return kv4, summ


APPEND = [  # lens, T, ps, H, D, k_exp, v_exp
    ([1, 17, 16, 130], 1, 16, 2, 128, 0, 0),
    ([40, 33, 64], 33, 32, 1, 64, 3, -5),
    ([100, 65, 71, 130], 65, 64, 3, 128, -2, 4),
    ([500], 7, 16, 9, 64, 0, -1),
]


@pytest.mark.parametrize("lens,T,ps,H,D,k_exp,v_exp", APPEND)
@pytest.mark.parametrize("spread", [False, True])
def test_kv4_append_and_read_are_exact(spd, lens, T, ps, H, D, k_exp, v_exp, spread):
    """Every byte of the cache (old slots and spare pages too), the summaries, and the values read back."""
    import torch
    rng = np.random.default_rng(T * 13 + D + spread)
    lens, pt, mp, n, _, _ = paged(rng, lens, ps, H, D)
    B = len(lens)
    kv4 = rng.integers(0, 256, (n, H, 2, ps * D * 9 // 16)).astype(np.uint8)
    # older tokens: scales without NaN
    kv4[..., ps * D // 2:] &= 0x7F
    kv4[..., ps * D // 2:][kv4[..., ps * D // 2:] == 0x7F] = 0x30
    k, v = (rows_bf16(rng, B, T, H, D, spread=spread) for _ in range(2))
    want, want_summ = append_reference(kv4, pt, lens, T, k, v, ps, k_exp, v_exp)
    dims = spd.dims_of(B, H, H, D, ps, mp, n)
    cache, summ = dev(kv4), torch.full((B, H, mp, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    spd.kv4_append(dims, T, cache, dev(pt), dev(lens), to_dev(k), to_dev(v), summ, k_exp=k_exp, v_exp=v_exp)
    ko, vo = (torch.full((B, T, H, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    spd.kv4_read(dims, T, cache, dev(pt), dev(lens), ko, vo, k_exp=k_exp, v_exp=v_exp)
    torch.cuda.synchronize()
    assert spd.spd_device_status(clear=True) == 0
    assert np.array_equal(cache.cpu().numpy(), want)
    got = host(summ)
    expect = np.full(got.shape, 7.0)
    for (b, h, p), (lo, hi) in want_summ.items():
        expect[b, h, p, 0], expect[b, h, p, 1] = lo, hi
    assert np.array_equal(got, expect)
    for out, rows, e in ((ko, k, k_exp), (vo, v, v_exp)):
        assert np.array_equal(host(out), ref.kv4_values(*ref.kv4_quantise(rows, e), e))


@pytest.mark.parametrize("k_exp,v_exp", [(0, 7), (-64, 64)])
def test_kv4_codes_of_every_quotient(spd, k_exp, v_exp):
    """Every scale against every bf16 magnitude from 2^-5 scales to the largest code, both signs, and zeros of both."""
    import torch
    ps, H, D = 64, 1, 128
    scales = ref.e4m3_values()[1:]
    mags = np.outer(np.arange(128, 256), 2.0 ** np.arange(-12, -4)).reshape(-1)  # [2^-5, 16) times a power of two
    groups = []
    for s in scales:
        x = mags * 2.0 ** np.floor(np.log2(s))
        x = np.concatenate([x[x < 6 * s], [0.0, -0.0]])
        x = np.concatenate([x, -x])
        x = np.append(x, np.zeros(-len(x) % 15)).reshape(-1, 15)
        groups.append(np.concatenate([np.full((len(x), 1), 6 * s), x], 1))  # 6 s: the group's scale is s
    g = np.concatenate(groups)
    g = np.concatenate([g, np.zeros((-len(g) % (D // 16), 16))])
    T = len(g) * 16 // D
    lens, pt, mp, n, _, _ = paged(np.random.default_rng(1), [T], ps, H, D)
    k, v = (g.reshape(1, T, H, D) * 2.0 ** e for e in (k_exp, v_exp))
    assert np.array_equal(k, ref.bf16(k)) and np.array_equal(v, ref.bf16(v))
    want, _ = append_reference(np.zeros((n, H, 2, ps * D * 9 // 16), np.uint8), pt, lens, T, k, v, ps, k_exp, v_exp)
    dims = spd.dims_of(1, H, H, D, ps, mp, n)
    cache, summ = spd.kv4_cache(dims), torch.zeros((1, H, mp, 2, D), dtype=torch.bfloat16, device="cuda")
    spd.kv4_append(dims, T, cache, dev(pt), dev(lens), to_dev(k), to_dev(v), summ, k_exp=k_exp, v_exp=v_exp)
    assert spd.spd_device_status(clear=True) == 0
    assert np.array_equal(cache.cpu().numpy(), want)


def test_kv4_append_of_infinities_and_nan(spd):
    import torch
    rng = np.random.default_rng(5)
    ps, H, D = 16, 2, 64
    lens, pt, mp, n, _, _ = paged(rng, [16], ps, H, D)
    k = rows_bf16(rng, 1, 16, H, D)
    k[0, 0, 0, 3], k[0, 1, 0, 20], k[0, 2, 1, :16], k[0, 3, 1, 5] = np.inf, -np.inf, np.nan, np.nan
    v = k[:, ::-1].copy()
    dims = spd.dims_of(1, H, H, D, ps, mp, n)
    cache, summ = spd.kv4_cache(dims), torch.zeros((1, H, mp, 2, D), dtype=torch.bfloat16, device="cuda")
    ko, vo = (torch.empty((1, 16, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    spd.kv4_append(dims, 16, cache, dev(pt), dev(lens), to_dev(k), to_dev(v), summ)
    spd.kv4_read(dims, 16, cache, dev(pt), dev(lens), ko, vo)
    for out, rows in ((ko, k), (vo, v)):
        assert np.array_equal(host(out), ref.kv4_values(*ref.kv4_quantise(rows, 0), 0))
    assert host(ko)[0, 0, 0, 3] == 6 * 448 and host(ko)[0, 1, 0, 20] == -6 * 448
    assert np.all(host(ko)[0, 2, 1, :16] == 0) and host(ko)[0, 3, 1, 5] == 0


def test_kv4_append_skips_what_it_cannot_place(spd):
    import torch
    rng = np.random.default_rng(6)
    T, ps, H, D = 3, 16, 2, 64
    lens, pt, mp, n, _, _ = paged(rng, [20, 30, 40, 35], ps, H, D)
    bad, pt_bad = lens.copy(), pt.copy()
    bad[0], bad[1] = 2, mp * ps + 1
    pt_bad[3, 2] = -5
    kv4 = rng.integers(0, 120, (n, H, 2, ps * D * 9 // 16)).astype(np.uint8)
    k, v = (rows_bf16(rng, 4, T, H, D) for _ in range(2))
    dims = spd.dims_of(4, H, H, D, ps, mp, n)
    cache, summ = dev(kv4), torch.full((4, H, mp, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    spd.kv4_append(dims, T, cache, dev(pt_bad), dev(bad), to_dev(k), to_dev(v), summ)
    assert spd.spd_device_status(clear=True) == spd.DEV_BAD_LEN | spd.DEV_BAD_PAGE
    ko, vo = (torch.full((4, T, H, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    spd.kv4_read(dims, T, cache, dev(pt_bad), dev(bad), ko, vo)
    assert spd.spd_device_status(clear=True) == spd.DEV_BAD_LEN | spd.DEV_BAD_PAGE
    got = cache.cpu().numpy()
    for b in range(4):
        rows = pt[b, : -(-int(lens[b]) // ps)]
        assert np.array_equal(got[rows], kv4[rows]) == (b != 2), b
        assert bool(torch.count_nonzero(ko[b]) == 0) == (b != 2) and bool(torch.count_nonzero(vo[b]) == 0) == (b != 2)
        assert bool((summ[b] == 7.0).all()) == (b != 2), b


# ---------------------------------------------------------------- attention

def make_cache(rng, lens, ps, H, D, k_exp=0, v_exp=0, poison=True):
    """A page table and a cache of quantised normal rows; slots behind the lengths hold any bytes (NaN scales too)."""
    lens, pt, mp, n, _, _ = paged(rng, lens, ps, H, D)
    kv4 = rng.integers(0, 256, (n, H, 2, ps * D * 9 // 16)).astype(np.uint8)
    if poison:
        kv4[..., ps * D // 2:] = 0x7F
    vals = []
    for b, ln in enumerate(lens):
        rows = [rows_bf16(rng, ln, H, D) * 2.0 ** e for e in (k_exp, v_exp)]
        out = []
        for half, (x, e) in enumerate(zip(rows, (k_exp, v_exp))):
            codes, scale = ref.kv4_quantise(x, e)
            out.append(ref.kv4_values(codes, scale, e))
            for p in range(-(-ln // ps)):
                lo, hi = p * ps, min((p + 1) * ps, ln)
                for h in range(H):
                    c, s = (y.copy() for y in ref.kv4_unpack(kv4[pt[b, p], h, half], ps, D))
                    c[: hi - lo], s[: hi - lo] = codes[lo:hi, h], scale[lo:hi, h]
                    kv4[pt[b, p], h, half] = ref.kv4_pack(c, s)
        vals.append(out)
    return lens, pt, mp, n, kv4, vals


def check_row(o, lse, q, keys, values, scale, visible, what):
    """o: one rounding to bf16 (2^-8), weights rounded to fp16 (2^-11 of sum p |v|; below 2^-32 of the largest
    they are dropped), and logits that are off by d: D fp32 sums of products that add up to at most `mag`, the
    query's channels kept to 2^-25 of the largest, and z itself rounded and raised by ex2 (2^-22): a weight's
    relative error, once in the numerator and once in the sum."""
    want, want_lse, pv, mag = ref.attention(q, keys, values, scale, visible)
    d = mag * (len(q) + 4) * 2.0 ** -24 + 2.0 ** -21 + (abs(want_lse) * 2.0 ** -22 if np.isfinite(want_lse) else 0.0)
    drop = len(keys) * 2.0 ** -32 * np.abs(values).max(0, initial=0.0)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * d) * pv + drop
    assert np.all(np.abs(o - want) <= tol), (what, float((np.abs(o - want) / np.maximum(tol, 1e-30)).max()))
    if np.isneginf(want_lse):
        assert np.isneginf(lse), what
    else:
        assert abs(lse - want_lse) <= d, (what, lse, want_lse)


DENSE = [  # lens, T, H_q, H_kv, D, ps, splits
    ([1, 16, 17, 100], 1, 8, 2, 128, 16, 0),
    ([7, 64, 200], 7, 4, 1, 128, 16, 3),
    ([33, 40, 129], 5, 6, 2, 64, 32, 0),
    ([64, 63, 150], 8, 16, 2, 128, 64, 2),
    ([300], 2, 7, 1, 64, 16, 5),
    ([2000], 1, 3, 3, 128, 32, 0),
    ([70, 31], 16, 4, 2, 64, 16, 0),
    ([90, 65], 13, 1, 1, 128, 64, 1),
    ([140, 12], 12, 8, 2, 64, 32, 0),
]


@pytest.mark.parametrize("lens,T,H_q,H_kv,D,ps,splits", DENSE)
def test_kv4_dense_verify(spd, lens, T, H_q, H_kv, D, ps, splits):
    import torch
    rng = np.random.default_rng(len(lens) * 100 + T + D)
    k_exp, v_exp = (2, -3) if T % 2 else (0, 0)
    lens, pt, mp, n, kv4, vals = make_cache(rng, lens, ps, H_kv, D, k_exp, v_exp)
    B, G = len(lens), H_q // H_kv
    q = rows_bf16(rng, B, T, H_q, D) * 2.0 ** rng.integers(-3, 2, (B, T, H_q, 1))
    dims = spd.dims_of(B, H_q, H_kv, D, ps, mp, n)
    ws = spd.workspace(spd.spd_kv4_dense_verify_workspace_size(dims, T, splits))
    o = torch.full((B, T, H_q, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, T, H_q), float("nan"), device="cuda")
    scale = 0.11
    args = (dims, T, to_dev(q), dev(kv4), dev(pt), dev(lens), o, ws)
    for _ in range(2):  # the workspace is left as it was found
        spd.kv4_dense_verify_attn(*args, lse=lse, num_splits=splits, softmax_scale=scale, k_exp=k_exp, v_exp=v_exp)
    torch.cuda.synchronize()
    assert spd.spd_device_status(clear=True) == 0
    og, lg = host(o), host(lse)
    for b in range(B):
        for t in range(T):
            seen = np.arange(lens[b]) <= lens[b] - T + t
            for hq in range(H_q):
                check_row(og[b, t, hq], lg[b, t, hq], q[b, t, hq], vals[b][0][:, hq // G], vals[b][1][:, hq // G], scale,
                          seen, (b, t, hq))
    again = torch.empty_like(o)
    spd.kv4_dense_verify_attn(*args[:6], again, ws, num_splits=splits, softmax_scale=scale, k_exp=k_exp, v_exp=v_exp)
    assert torch.equal(again, o)  # and without lse


SPARSE = [  # lens, H_q, H_kv, D, ps, k_max, splits
    ([1, 16, 17, 100, 250], 8, 2, 128, 16, 5, 0),
    ([600, 33, 129], 6, 2, 64, 32, 9, 3),
    ([640, 63], 16, 2, 128, 64, 4, 2),
    ([900], 7, 1, 64, 16, 40, 7),
    ([500, 20], 3, 3, 128, 16, 31, 1),
]


@pytest.mark.parametrize("lens,H_q,H_kv,D,ps,k_max,splits", SPARSE)
def test_kv4_sparse_decode(spd, lens, H_q, H_kv, D, ps, k_max, splits):
    """Random selections in any order, a row with none, and one whose last page is not among its pages."""
    import torch
    rng = np.random.default_rng(k_max + D)
    lens, pt, mp, n, kv4, vals = make_cache(rng, lens, ps, H_kv, D)
    B, G = len(lens), H_q // H_kv
    sel = np.full((B, H_kv, k_max), 1 << 20, np.int32)
    nsel = np.zeros((B, H_kv), np.int32)
    for b in range(B):
        P = -(-int(lens[b]) // ps)
        for h in range(H_kv):
            nsel[b, h] = 0 if (b == 0 and h == 1) else rng.integers(1, min(P, k_max) + 1)
            sel[b, h, : nsel[b, h]] = rng.permutation(P)[: nsel[b, h]]
    q = rows_bf16(rng, B, H_q, D)
    dims = spd.dims_of(B, H_q, H_kv, D, ps, mp, n)
    ws = spd.workspace(spd.spd_kv4_sparse_decode_workspace_size(dims, k_max, splits))
    o = torch.full((B, H_q, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H_q), float("nan"), device="cuda")
    for _ in range(2):
        spd.kv4_sparse_decode_attn(dims, to_dev(q), dev(kv4), dev(pt), dev(lens), dev(sel), dev(nsel), k_max, o, ws,
                                   lse=lse, num_splits=splits)
    torch.cuda.synchronize()
    assert spd.spd_device_status(clear=True) == 0
    og, lg = host(o), host(lse)
    for b in range(B):
        for hq in range(H_q):
            h = hq // G
            pages = set(sel[b, h, : nsel[b, h]].tolist())
            seen = np.array([j // ps in pages for j in range(lens[b])])
            check_row(og[b, hq], lg[b, hq], q[b, hq], vals[b][0][:, h], vals[b][1][:, h], D ** -0.5, seen, (b, hq))


LONG = [  # len, T, H_q, H_kv, D, ps, splits
    (9001, 1, 4, 1, 128, 16, 1),
    (9001, 2, 8, 2, 64, 64, 2),
    (5003, 7, 4, 1, 128, 16, 1),
    (5003, 7, 4, 1, 64, 32, 2),
    (4500, 9, 7, 1, 128, 64, 1),
]


@pytest.mark.parametrize("length,T,H_q,H_kv,D,ps,splits", LONG)
def test_kv4_long_sequences(spd, length, T, H_q, H_kv, D, ps, splits):
    """Many turns of every ring and of the page lookups, in few splits; and, for one position, the same tokens
    as a selection of every page."""
    import torch
    rng = np.random.default_rng(length + T)
    lens, pt, mp, n, kv4, vals = make_cache(rng, [length, 40], ps, H_kv, D)
    G = H_q // H_kv
    q = rows_bf16(rng, 2, T, H_q, D)
    dims = spd.dims_of(2, H_q, H_kv, D, ps, mp, n)
    ws = spd.workspace(spd.spd_kv4_dense_verify_workspace_size(dims, T, splits))
    o = torch.full((2, T, H_q, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, T, H_q), float("nan"), device="cuda")
    spd.kv4_dense_verify_attn(dims, T, to_dev(q), dev(kv4), dev(pt), dev(lens), o, ws, lse=lse, num_splits=splits)
    assert spd.spd_device_status(clear=True) == 0
    for b in range(2):
        for t in range(T):
            seen = np.arange(lens[b]) <= lens[b] - T + t
            for hq in range(H_q):
                check_row(host(o)[b, t, hq], host(lse)[b, t, hq], q[b, t, hq], vals[b][0][:, hq // G], vals[b][1][:, hq // G],
                          D ** -0.5, seen, (b, t, hq))
    if T == 1:
        k_max = mp
        sel = np.zeros((2, H_kv, k_max), np.int32)
        nsel = np.zeros((2, H_kv), np.int32)
        for b in range(2):
            P = -(-int(lens[b]) // ps)
            for h in range(H_kv):
                sel[b, h, :P], nsel[b, h] = rng.permutation(P), P
        ws = spd.workspace(spd.spd_kv4_sparse_decode_workspace_size(dims, k_max, splits))
        spd.kv4_sparse_decode_attn(dims, to_dev(q), dev(kv4), dev(pt), dev(lens), dev(sel), dev(nsel), k_max, o, ws, lse=lse,
                                   num_splits=splits)
        assert spd.spd_device_status(clear=True) == 0
        for b in range(2):
            for hq in range(H_q):
                check_row(host(o)[b, 0, hq], host(lse)[b, 0, hq], q[b, 0, hq], vals[b][0][:, hq // G], vals[b][1][:, hq // G],
                          D ** -0.5, np.ones(lens[b], bool), (b, hq))


def test_kv4_the_longest_sequence(spd):
    """2^31 - 1 tokens, every page of them the same physical page of zero keys and of ones (33/32 as held) as values: the
    two newest tokens appended, with their summary, read back, and attended to by one query row."""
    import torch
    D, ps, mp, length = 64, 16, 1 << 27, (1 << 31) - 1
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    dims = spd.dims_of(1, 1, 1, D, ps, mp, 2)
    pt, lens = torch.ones((1, mp), dtype=torch.int32, device="cuda"), torch.tensor([length], dtype=torch.int32, device="cuda")
    pt[0, -1] = 0
    summ = torch.empty((1, 1, mp, 2, D), dtype=torch.bfloat16, device="cuda")
    summ[0, 0, -2:] = 7.0
    zeros, ones = (torch.full((1, 16, 1, D), x, dtype=torch.bfloat16, device="cuda") for x in (0.0, 1.0))
    cache = spd.kv4_cache(dims)
    small = spd.dims_of(2, 1, 1, D, ps, 1, 2)
    spd.kv4_append(small, 16, cache, torch.tensor([[0], [1]], dtype=torch.int32, device="cuda"),
                   torch.tensor([16, 16], dtype=torch.int32, device="cuda"), zeros.repeat(2, 1, 1, 1), ones.repeat(2, 1, 1, 1),
                   torch.empty((2, 1, 1, 2, D), dtype=torch.bfloat16, device="cuda"))
    before = cache.clone()
    rng = np.random.default_rng(8)
    k, v = (to_dev(ref.bf16(rng.standard_normal((1, 2, 1, D)))) for _ in range(2))
    spd.kv4_append(dims, 2, cache, pt, lens, k, v, summ)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    spd.kv4_read(dims, 2, cache, pt, lens, ko, vo)
    want = ref.kv4_values(*ref.kv4_quantise(host(k), 0), 0)
    assert np.array_equal(host(ko), want) and np.array_equal(host(vo), ref.kv4_values(*ref.kv4_quantise(host(v), 0), 0))
    assert np.array_equal(host(summ[0, 0, -1]), np.stack([np.minimum(want[0, :, 0].min(0), 0), np.maximum(want[0, :, 0].max(0), 0)]))
    assert torch.all(summ[0, 0, -2] == 7.0) and torch.equal(cache[1], before[1])
    cache.copy_(before)
    q = to_dev(rows_bf16(rng, 1, 1, 1, D))
    o, lse = torch.full_like(q, float("nan")), torch.full((1, 1, 1), float("nan"), device="cuda")
    spd.kv4_dense_verify_attn(dims, 1, q, cache, pt, lens, o, spd.workspace(spd.spd_kv4_dense_verify_workspace_size(dims, 1)), lse=lse)
    assert spd.spd_device_status(clear=True) == 0
    assert np.all(host(o) == ref.kv4_values(*ref.kv4_quantise(np.ones(16), 0), 0)[0])
    assert np.all(np.abs(host(lse) - np.log(float(length))) <= 32 * 2.0 ** -22)


@pytest.mark.parametrize("T,H_q", [(1, 4), (4, 8), (7, 4), (8, 8)])
@pytest.mark.parametrize("D", [64, 128])
def test_kv4_empty_and_short_sequences(spd, T, H_q, D):
    """Idle slots of a padded batch: no tokens at all, and fewer tokens than positions (rows that see nothing give
    zeros and -inf), beside ordinary sequences."""
    import torch
    rng = np.random.default_rng(T + D)
    lens, pt, mp, n, kv4, vals = make_cache(rng, [0, 3, 50, 0, 129], 16, 1, D)
    q = rows_bf16(rng, 5, T, H_q, D)
    dims = spd.dims_of(5, H_q, 1, D, 16, mp, n)
    ws = spd.workspace(spd.spd_kv4_dense_verify_workspace_size(dims, T, 0))
    o = torch.full((5, T, H_q, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, T, H_q), float("nan"), device="cuda")
    spd.kv4_dense_verify_attn(dims, T, to_dev(q), dev(kv4), dev(pt), dev(lens), o, ws, lse=lse)
    assert spd.spd_device_status(clear=True) == 0
    for b in range(5):
        for t in range(T):
            seen = np.arange(lens[b]) <= lens[b] - T + t
            for hq in range(H_q):
                check_row(host(o)[b, t, hq], host(lse)[b, t, hq], q[b, t, hq], vals[b][0][:, 0], vals[b][1][:, 0], D ** -0.5,
                          seen, (b, t, hq))
    assert torch.count_nonzero(o[0]) == 0 and torch.count_nonzero(o[3]) == 0


@pytest.mark.parametrize("T", [1, 3, 8])
@pytest.mark.parametrize("D", [64, 128])
def test_kv4_logits_that_grow_along_the_sequence(spd, T, D):
    """The largest logit moves up by tens of nats, again and again: every rescaling of what was summed before.
    Some rows fall instead, and some heads see the growth from the other side."""
    import torch
    rng = np.random.default_rng(T * D)
    H_q, length, ps = 4, 1500, 32
    lens, pt, mp, n, _, _ = paged(rng, [length], ps, 1, D)
    u = np.where(rng.random(D) < 0.5, 1.0, -1.0)
    k = ref.bf16(np.linspace(0.5, 6.0, length)[:, None, None] * u + 0.1 * rng.standard_normal((length, 1, D)))
    v = rows_bf16(rng, length, 1, D)
    dims = spd.dims_of(1, H_q, 1, D, ps, mp, n)
    cache, summ = spd.kv4_cache(dims), torch.zeros((1, 1, mp, 2, D), dtype=torch.bfloat16, device="cuda")
    spd.kv4_append(dims, length, cache, dev(pt), dev(lens), to_dev(k[None]), to_dev(v[None]), summ)
    kd, vd = ref.kv4_values(*ref.kv4_quantise(k, 0), 0)[:, 0], ref.kv4_values(*ref.kv4_quantise(v, 0), 0)[:, 0]
    q = ref.bf16(np.array([3.0, -2.0, 0.7, 8.0])[None, None, :, None] * u + 0.2 * rng.standard_normal((1, T, H_q, D)))
    for splits in (1, 3):
        ws = spd.workspace(spd.spd_kv4_dense_verify_workspace_size(dims, T, splits))
        o, lse = torch.empty((1, T, H_q, D), dtype=torch.bfloat16, device="cuda"), torch.empty((1, T, H_q), device="cuda")
        spd.kv4_dense_verify_attn(dims, T, to_dev(q), cache, dev(pt), dev(lens), o, ws, lse=lse, num_splits=splits)
        assert spd.spd_device_status(clear=True) == 0
        for t in range(T):
            for hq in range(H_q):
                check_row(host(o)[0, t, hq], host(lse)[0, t, hq], q[0, t, hq], kd, vd, D ** -0.5,
                          np.arange(length) <= length - T + t, (splits, t, hq))


@pytest.mark.parametrize("T,H_q", [(5, 7), (8, 8), (9, 7)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("splits", [1, 3])
def test_kv4_logits_that_grow_under_many_query_rows(spd, T, H_q, D, splits):
    """33 to 64 query rows of a KV head whose largest logit moves up again and again, rows that fall among them: what was
    summed before is rescaled at many steps, in units that start with and without a visible token."""
    import torch
    rng = np.random.default_rng(T * D + splits)
    length, ps = 1500, 16
    lens, pt, mp, n, _, _ = paged(rng, [length, T - 2], ps, 1, D)
    u = np.where(rng.random(D) < 0.5, 1.0, -1.0)
    k = ref.bf16(np.linspace(0.5, 6.0, length)[:, None, None] * u + 0.1 * rng.standard_normal((length, 1, D)))
    v = rows_bf16(rng, length, 1, D)
    dims = spd.dims_of(2, H_q, 1, D, ps, mp, n)
    one = spd.dims_of(1, H_q, 1, D, ps, mp, n)
    cache, summ = spd.kv4_cache(dims), torch.zeros((1, 1, mp, 2, D), dtype=torch.bfloat16, device="cuda")
    for b in range(2):
        m = int(lens[b])
        spd.kv4_append(one, m, cache, dev(pt[b: b + 1]), dev(lens[b: b + 1]), to_dev(k[None, :m]), to_dev(v[None, :m]), summ)
    kd, vd = ref.kv4_values(*ref.kv4_quantise(k, 0), 0)[:, 0], ref.kv4_values(*ref.kv4_quantise(v, 0), 0)[:, 0]
    size = np.resize(np.array([3.0, -2.0, 0.7, 8.0, 1.5]), H_q)
    q = ref.bf16(size[None, None, :, None] * u + 0.2 * rng.standard_normal((2, T, H_q, D)))
    ws = spd.workspace(spd.spd_kv4_dense_verify_workspace_size(dims, T, splits))
    got = []
    for _ in range(2):
        o = torch.full((2, T, H_q, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((2, T, H_q), float("nan"), device="cuda")
        spd.kv4_dense_verify_attn(dims, T, to_dev(q), cache, dev(pt), dev(lens), o, ws, lse=lse, num_splits=splits)
        got.append((o, lse))
    assert spd.spd_device_status(clear=True) == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    og, lg = host(o), host(lse)
    for b in range(2):
        m = int(lens[b])
        for t in range(T):
            for hq in range(H_q):
                check_row(og[b, t, hq], lg[b, t, hq], q[b, t, hq], kd[:m], vd[:m], D ** -0.5, np.arange(m) <= m - T + t,
                          (b, t, hq))


def test_kv4_attention_extremes(spd):
    """Large and tiny queries, logits that grow along the sequence (the reference maximum moves again and again)
    and one token that outweighs the rest."""
    import torch
    rng = np.random.default_rng(21)
    H_q, H_kv, D, ps = 4, 1, 128, 16
    lens, pt, mp, n, kv4, vals = make_cache(rng, [400], ps, H_kv, D)
    q = rows_bf16(rng, 1, 1, H_q, D)
    q[0, 0, 0] *= 2.0 ** 40
    q[0, 0, 1] *= 2.0 ** -60
    q[0, 0, 2] = 0.0
    q[0, 0, 3, 1:] = 0.0
    dims = spd.dims_of(1, H_q, H_kv, D, ps, mp, n)
    for scale in (2.0 ** -42, 0.3):
        qq = q.copy()
        if scale == 0.3:
            qq[0, 0, 0] = ref.bf16(vals[0][0][399, 0] * 4)  # the last key: far above the others
        ws = spd.workspace(spd.spd_kv4_dense_verify_workspace_size(dims, 1, 0))
        o = torch.empty((1, 1, H_q, D), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((1, 1, H_q), device="cuda")
        spd.kv4_dense_verify_attn(dims, 1, to_dev(qq), dev(kv4), dev(pt), dev(lens), o, ws, lse=lse, softmax_scale=scale)
        for hq in range(H_q):
            check_row(host(o)[0, 0, hq], host(lse)[0, 0, hq], qq[0, 0, hq], vals[0][0][:, 0], vals[0][1][:, 0], scale,
                      np.ones(400, bool), (scale, hq))


def test_kv4_attention_bad_entries(spd):
    """Entries that point outside the sequence or the cache are skipped, lengths the table cannot hold give empty
    rows, and the other rows are as without them."""
    import torch
    rng = np.random.default_rng(31)
    H_q, H_kv, D, ps, k_max = 4, 2, 64, 16, 4
    lens, pt, mp, n, kv4, vals = make_cache(rng, [70, 60, 50, 64], ps, H_kv, D)
    sel = np.tile(np.arange(k_max, dtype=np.int32), (4, H_kv, 1))
    nsel = np.full((4, H_kv), k_max, np.int32)
    q = to_dev(rows_bf16(rng, 4, H_q, D))
    dims = spd.dims_of(4, H_q, H_kv, D, ps, mp, n)
    ws = spd.workspace(max(spd.spd_kv4_sparse_decode_workspace_size(dims, k_max), spd.spd_kv4_dense_verify_workspace_size(dims, 1)))

    def run(pt, lens, sel, nsel):
        o = torch.full((4, H_q, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        spd.kv4_sparse_decode_attn(dims, q, dev(kv4), dev(pt), dev(lens), dev(sel), dev(nsel), k_max, o, ws)
        od = torch.full((4, 1, H_q, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        spd.kv4_dense_verify_attn(dims, 1, q.unsqueeze(1).contiguous(), dev(kv4), dev(pt), dev(lens), od, ws)
        return o, od[:, 0], spd.spd_device_status(clear=True)

    good, good_d, status = run(pt, lens, sel, nsel)
    assert status == 0
    sel2, nsel2, pt2, lens2 = sel.copy(), nsel.copy(), pt.copy(), lens.copy()
    sel2[0, 0, 1], sel2[0, 1, 2] = -3, 1 << 20
    nsel2[1, 0], nsel2[1, 1] = -1, k_max + 5
    pt2[2, 1] = n + 7
    lens2[3] = mp * ps + 1
    o, od, status = run(pt2, lens2, sel2, nsel2)
    assert status == spd.DEV_BAD_SEL | spd.DEV_BAD_PAGE | spd.DEV_BAD_LEN
    assert not torch.isnan(o.float()).any() and not torch.isnan(od.float()).any()
    assert torch.count_nonzero(o[3]) == 0 and torch.count_nonzero(od[3]) == 0
    assert torch.count_nonzero(o[1, : H_q // H_kv]) == 0
    assert torch.equal(o[1, H_q // H_kv:], good[1, H_q // H_kv:])
    assert torch.equal(od[:2], good_d[:2])
    # the skipped page of sequence 2: as a selection without it
    sel3 = sel.copy()
    sel3[2, :, 1:3] = sel[2, :, 2:4]
    nsel3 = nsel.copy()
    nsel3[2] = 3
    less, _, _ = run(pt, lens, sel3, nsel3)
    assert np.abs(host(o)[2] - host(less)[2]).max() <= 2 ** -7 * np.abs(host(less)[2]).max()


def test_kv4_step_as_it_is_used(spd):
    """Projection rows -> qk_norm_rope -> kv4_append -> pages_score_select -> kv4_sparse_decode_attn, the same
    captured as a graph, and the verification of two positions over the same cache."""
    import torch
    rng = np.random.default_rng(41)
    B, H_q, H_kv, D, ps, k_max = 3, 8, 2, 64, 16, 4
    lens, pt, mp, n, kv4, vals = make_cache(rng, [100, 130, 75], ps, H_kv, D)
    dims = spd.dims_of(B, H_q, H_kv, D, ps, mp, n)
    cache = dev(kv4)
    # summaries of the whole cache first: every token appended again, in one call per sequence length
    summ = torch.zeros((B, H_kv, mp, 2, D), dtype=torch.bfloat16, device="cuda")
    for b in range(B):
        one = spd.dims_of(1, H_q, H_kv, D, ps, mp, n)
        ln = int(lens[b])
        kk, vv = (to_dev(vals[b][i][None]) for i in (0, 1))
        spd.kv4_append(one, ln, cache, dev(pt[b: b + 1]), dev(lens[b: b + 1]), kk, vv, summ[b: b + 1])
    before = cache.cpu().numpy()
    for b in range(B):  # values that are representable are stored as they are
        for p in range(-(-int(lens[b]) // ps)):
            m = min(ps, int(lens[b]) - p * ps)
            for h in range(H_kv):
                for half in (0, 1):
                    c, s = ref.kv4_unpack(before[pt[b, p], h, half], ps, D)
                    assert np.array_equal(ref.kv4_values(c, s, 0)[:m], vals[b][half][p * ps: p * ps + m, h])
    x = to_dev(rows_bf16(rng, B, H_q + 2 * H_kv, D))
    q_in, k_in, v_in = torch.split(x, [H_q, H_kv, H_kv], 1)
    w = to_dev(1 + 0.1 * rng.standard_normal(D))
    table = dev(ref.rope_table(256, D))
    pos = dev((lens - 1).astype(np.int32))
    q, k = torch.empty((B, H_q, D), dtype=torch.bfloat16, device="cuda"), torch.empty((B, H_kv, D), dtype=torch.bfloat16, device="cuda")
    v = v_in.contiguous()
    sel = torch.zeros((B, H_kv, k_max), dtype=torch.int32, device="cuda")
    nsel = torch.zeros((B, H_kv), dtype=torch.int32, device="cuda")
    pol = spd.Policy(0, k_max, 0, 0, 1, 0, 1, 1, 1, 1)
    ws = spd.workspace(max(spd.spd_score_select_workspace_size(dims), spd.spd_kv4_sparse_decode_workspace_size(dims, k_max),
                           spd.spd_kv4_dense_verify_workspace_size(dims, 2)))
    o = torch.empty((B, H_q, D), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((B, H_q), device="cuda")
    d_pt, d_lens = dev(pt), dev(lens)

    def step():
        spd.qk_norm_rope(q_in, k_in, pos, table, q, k, q_weight=w, k_weight=w)
        spd.kv4_append(dims, 1, cache, d_pt, d_lens, k, v, summ)
        spd.pages_score_select(dims, q, summ, d_lens, pol, sel, nsel, k_max, ws)
        spd.kv4_sparse_decode_attn(dims, q, cache, d_pt, d_lens, sel, nsel, k_max, o, ws, lse=lse)

    step()
    torch.cuda.synchronize()
    assert spd.spd_device_status(clear=True) == 0
    first = [t.clone() for t in (q, k, cache, summ, sel, nsel, o, lse)]
    for b in range(B):
        for i, rows in enumerate((k, v)):
            vals[b][i][-1] = ref.kv4_values(*ref.kv4_quantise(host(rows)[b], 0), 0)
        for h in range(H_kv):  # the selection by the score's definition over the values as held
            P = -(-int(lens[b]) // ps)
            lo = np.array([vals[b][0][p * ps: min((p + 1) * ps, lens[b]), h].min(0) for p in range(P)])
            hi = np.array([vals[b][0][p * ps: min((p + 1) * ps, lens[b]), h].max(0) for p in range(P)])
            qs = host(q)[b, h * 4: h * 4 + 4]
            score = np.maximum(qs[:, None] * lo, qs[:, None] * hi).sum(-1).max(0)
            chosen = sel[b, h].tolist()
            assert chosen == sorted(set(chosen)) and 0 in chosen and P - 1 in chosen
            worst = min(score[p] for p in chosen if p not in (0, P - 1))
            rest = [score[p] for p in range(P) if p not in chosen]
            assert max(rest) <= worst * (1 + 1e-5)
            seen = np.array([j // ps in chosen for j in range(lens[b])])
            for hq in range(h * 4, h * 4 + 4):
                check_row(host(o)[b, hq], host(lse)[b, hq], host(q)[b, hq], vals[b][0][:, h], vals[b][1][:, h], D ** -0.5,
                          seen, (b, hq))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (q, k, o, lse):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (q, k, cache, summ, sel, nsel, o, lse)))
    q2 = rows_bf16(rng, B, 2, H_q, D)
    o2 = torch.empty((B, 2, H_q, D), dtype=torch.bfloat16, device="cuda")
    lse2 = torch.empty((B, 2, H_q), device="cuda")
    spd.kv4_dense_verify_attn(dims, 2, to_dev(q2), cache, d_pt, d_lens, o2, ws, lse=lse2)
    for b in range(B):
        for t in range(2):
            for hq in range(H_q):
                check_row(host(o2)[b, t, hq], host(lse2)[b, t, hq], q2[b, t, hq], vals[b][0][:, hq // 4], vals[b][1][:, hq // 4],
                          D ** -0.5, np.arange(lens[b]) <= lens[b] - 2 + t, (b, t, hq))


def test_kv4_cache_past_4_gib(spd):
    """Pages whose byte offset in the cache passes 32 bits."""
    import torch
    rng = np.random.default_rng(51)
    H, D, ps = 8, 128, 64
    tile = ps * D * 9 // 8
    n = (5 << 30) // (H * tile)
    lens, pt, mp, m, kv4, vals = make_cache(rng, [150], ps, H, D)
    cache = torch.zeros((n, H, 2, tile // 2), dtype=torch.uint8, device="cuda")
    far = np.array([n - 1, 3, n - 5])
    for p in range(3):
        cache[int(far[p])] = dev(kv4[pt[0, p]])
    pt2 = pt.copy()
    pt2[0, :3] = far
    dims = spd.dims_of(1, H, H, D, ps, mp, n)
    q = rows_bf16(rng, 1, 1, H, D)
    o, lse = torch.empty((1, 1, H, D), dtype=torch.bfloat16, device="cuda"), torch.empty((1, 1, H), device="cuda")
    ws = spd.workspace(spd.spd_kv4_dense_verify_workspace_size(dims, 1))
    spd.kv4_dense_verify_attn(dims, 1, to_dev(q), cache, dev(pt2), dev(lens), o, ws, lse=lse)
    for h in range(H):
        check_row(host(o)[0, 0, h], host(lse)[0, 0, h], q[0, 0, h], vals[0][0][:, h], vals[0][1][:, h], D ** -0.5,
                  np.ones(150, bool), h)
    q9 = rows_bf16(rng, 1, 9, H, D)  # the kernel for more query rows
    o9, lse9 = torch.empty((1, 9, H, D), dtype=torch.bfloat16, device="cuda"), torch.empty((1, 9, H), device="cuda")
    ws9 = spd.workspace(spd.spd_kv4_dense_verify_workspace_size(dims, 9))
    spd.kv4_dense_verify_attn(dims, 9, to_dev(q9), cache, dev(pt2), dev(lens), o9, ws9, lse=lse9)
    for t in range(9):
        check_row(host(o9)[0, t, 3], host(lse9)[0, t, 3], q9[0, t, 3], vals[0][0][:, 3], vals[0][1][:, 3], D ** -0.5,
                  np.arange(150) <= 150 - 9 + t, t)
    k, v = (rows_bf16(rng, 1, 2, H, D) for _ in range(2))
    summ = torch.zeros((1, H, mp, 2, D), dtype=torch.bfloat16, device="cuda")
    ko, vo = (torch.empty((1, 2, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    spd.kv4_append(dims, 2, cache, dev(pt2), dev(lens), to_dev(k), to_dev(v), summ)
    spd.kv4_read(dims, 2, cache, dev(pt2), dev(lens), ko, vo)
    assert np.array_equal(host(ko), ref.kv4_values(*ref.kv4_quantise(k, 0), 0))
    assert np.array_equal(host(vo), ref.kv4_values(*ref.kv4_quantise(v, 0), 0))
    assert spd.spd_device_status(clear=True) == 0


def test_one_workspace_for_calls_of_different_sizes(spd):
    """Split calls of few and of many rows and scored rows through one buffer, in turn: the bits of buffers of their own."""
    import torch
    rng = np.random.default_rng(77)
    calls = []
    for lens, T, H_q, H_kv, splits in (([200, 90, 310], 3, 16, 8, 3), ([400], 1, 2, 1, 4), ([250, 130], 1, 32, 16, 2)):
        lens, pt, mp, n, kv4, _ = make_cache(rng, lens, 16, H_kv, 64)
        dims, B = spd.dims_of(len(lens), H_q, H_kv, 64, 16, mp, n), len(lens)
        q, args = to_dev(rows_bf16(rng, B, T, H_q, 64)), (dev(kv4), dev(pt), dev(lens))

        def attend(ws, dims=dims, T=T, q=q, args=args, splits=splits):
            o = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
            lse = torch.full(q.shape[:-1], float("nan"), device="cuda")
            spd.kv4_dense_verify_attn(dims, T, q, *args, o, ws, lse=lse, num_splits=splits)
            return o, lse

        calls.append((spd.spd_kv4_dense_verify_workspace_size(dims, T, splits), attend))
    for rows in (3, 70):
        x, t = dev(rng.standard_normal((rows, 20001)).astype(np.float32)), dev(rng.integers(0, 20001, rows).astype(np.int32))

        def score(ws, rows=rows, x=x, t=t):
            out = [torch.full((rows,), float("nan"), device="cuda") for _ in range(3)]
            ids, top = torch.full((rows, 5), -9, dtype=torch.int32, device="cuda"), torch.zeros((rows, 5), device="cuda")
            spd.token_logprobs(x, t, out[0], ws, entropy=out[1], lse=out[2], top_ids=ids, top_logprobs=top)
            return (*out, ids, top)

        calls.append((spd.spd_token_logprobs_workspace_size(rows, 20001, 5), score))
    want = [f(spd.workspace(size)) for size, f in calls]
    ws = spd.workspace(max(size for size, _ in calls))
    for i in (0, 1, 0, 3, 2, 4, 1, 3, 0, 2, 3, 4, 0):
        for got, ref_ in zip(calls[i][1](ws), want[i]):
            assert torch.equal(got, ref_), i
    assert spd.spd_device_status(clear=True) == 0


def test_one_workspace_for_every_call(spd):
    """Scoring, attention over both caches (in few splits, in many, joined in groups) and scored rows, of several sizes, in
    any order through one buffer that a step has used before: the bits of buffers of their own."""
    import torch
    rng = np.random.default_rng(99)
    calls, steps = [], []
    for lens, T, H_q, H_kv, D, ps, k_max in (([16384, 9000], 7, 32, 8, 128, 16, 64), ([16400], 1, 64, 8, 128, 16, 1024),
                                             ([700, 40, 0, 333, 512], 2, 8, 4, 64, 32, 8), ([90] * 70, 3, 4, 4, 64, 16, 4)):
        lens, pt, mp, n, K, V = paged(rng, lens, ps, H_kv, D)
        B = len(lens)
        dims, d_pt, d_lens = spd.dims_of(B, H_q, H_kv, D, ps, mp, n), dev(pt), dev(lens)
        kv4 = rng.integers(0, 256, (n, H_kv, 2, ps * D * 9 // 16)).astype(np.uint8)
        kv4[..., ps * D // 2:] = rng.integers(0x30, 0x3C, kv4[..., ps * D // 2:].shape)
        kv4 = dev(kv4)
        lo = rng.standard_normal((B, H_kv, mp, 1, D))
        summ = to_dev(ref.bf16(np.concatenate([lo, lo + 1], 3)))
        q = to_dev(rows_bf16(rng, B, T, H_q, D))
        q1 = q[:, 0].contiguous()
        pol = spd.Policy(0, k_max, 0, 0, 1, 0, 1, 1, 1, 1)
        sel = torch.zeros((B, H_kv, k_max), dtype=torch.int32, device="cuda")
        nsel = torch.zeros((B, H_kv), dtype=torch.int32, device="cuda")

        def select(ws, q1=q1, dims=dims, summ=summ, d_lens=d_lens, pol=pol, sel=sel, nsel=nsel, k_max=k_max):
            a, b = torch.full_like(sel, -1), torch.full_like(nsel, -1)
            spd.pages_score_select(dims, q1, summ, d_lens, pol, a, b, k_max, ws)
            a[torch.arange(k_max, device="cuda") >= b[..., None]] = 0
            return a, b

        first = select(spd.workspace(spd.spd_score_select_workspace_size(dims)))
        sel.copy_(first[0])
        nsel.copy_(first[1])

        def attend(f, *args, like=None):
            def run(ws):
                o = torch.full_like(like, float("nan"))
                lse = torch.full(like.shape[:-1], float("nan"), device="cuda")
                f(*args, o, ws, lse=lse)
                return o, lse
            return run

        steps.append((spd.spd_sparse_decode_step_workspace_size(dims, k_max),
                      lambda ws, a=(dims, K, V, d_pt, d_lens, None, None, q1, summ, pol, sel.clone(), nsel.clone(), k_max):
                      spd.sparse_decode_step(*a, torch.empty_like(a[7]), ws)))
        calls += [
            (spd.spd_score_select_workspace_size(dims), select),
            (spd.spd_sparse_decode_workspace_size(dims, k_max),
             attend(spd.sparse_decode_attn, dims, q1, K, V, d_pt, d_lens, sel, nsel, k_max, like=q1)),
            (spd.spd_dense_verify_workspace_size(dims, T), attend(spd.dense_verify_attn, dims, T, q, K, V, d_pt, d_lens, like=q)),
            (spd.spd_kv4_sparse_decode_workspace_size(dims, k_max),
             attend(spd.kv4_sparse_decode_attn, dims, q1, kv4, d_pt, d_lens, sel, nsel, k_max, like=q1)),
            (spd.spd_kv4_dense_verify_workspace_size(dims, T),
             attend(spd.kv4_dense_verify_attn, dims, T, q, kv4, d_pt, d_lens, like=q)),
        ]
    for rows, n in ((70, 20001), (3, 151936)):
        x, t = dev(rng.standard_normal((rows, n)).astype(np.float32)), dev(rng.integers(0, n, rows).astype(np.int32))

        def score(ws, rows=rows, x=x, t=t):
            out = [torch.full((rows,), float("nan"), device="cuda") for _ in range(3)]
            ids, top = torch.full((rows, 5), -9, dtype=torch.int32, device="cuda"), torch.zeros((rows, 5), device="cuda")
            spd.token_logprobs(x, t, out[0], ws, entropy=out[1], lse=out[2], top_ids=ids, top_logprobs=top)
            return (*out, ids, top)

        calls.append((spd.spd_token_logprobs_workspace_size(rows, n, 5), score))
    want = [f(spd.workspace(size)) for size, f in calls]
    ws = spd.workspace(max(size for size, _ in calls + steps))
    steps[2][1](ws)
    order = np.concatenate([np.arange(len(calls)), *(rng.permutation(len(calls)) for _ in range(8))])
    wrong = []
    for before, i in zip([-1, *order], order):
        wrong += [(int(before), int(i)) for got, own in zip(calls[i][1](ws), want[i]) if not torch.equal(got, own)]
    assert not wrong, wrong
    assert spd.spd_device_status(clear=True) == 0


@pytest.mark.parametrize("T,H_q,D,splits", [(1, 8, 128, 2), (1, 8, 64, 1), (6, 16, 128, 2), (7, 8, 64, 1)])
def test_kv4_attention_with_waits_that_run_out(spd, T, H_q, D, splits):
    """A limit that no copy meets: the calls return with the timeout bit (or, should every copy be early, clean), all
    of their waits over, and later calls with the usual limit are those of before."""
    import torch
    rng = np.random.default_rng(T + D)
    lens, pt, mp, n, kv4, _ = make_cache(rng, [700, 300], 16, 2, D)
    dims = spd.dims_of(2, H_q, 2, D, 16, mp, n)
    q, cache, d_pt, d_lens = to_dev(rows_bf16(rng, 2, T, H_q, D)), dev(kv4), dev(pt), dev(lens)
    size = spd.spd_kv4_dense_verify_workspace_size(dims, T, splits)

    def run():
        o = torch.full((2, T, H_q, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((2, T, H_q), float("nan"), device="cuda")
        spd.kv4_dense_verify_attn(dims, T, q, cache, d_pt, d_lens, o, spd.workspace(size), lse=lse, num_splits=splits)
        torch.cuda.synchronize()
        return o, lse

    first = run()
    assert spd.spd_device_status(clear=True) == 0
    usual = spd.spd_wait_limit_ns()
    try:
        spd.spd_set_wait_limit_ns(1)
        for _ in range(3):
            run()
            assert spd.spd_device_status(clear=True) & ~spd.DEV_TIMEOUT == 0
    finally:
        spd.spd_set_wait_limit_ns(usual)
    for got, want in zip(run(), first):
        assert torch.equal(got, want)
    assert spd.spd_device_status(clear=True) == 0


@pytest.mark.parametrize("lens,T,H_q,H_kv,D,splits", [
    ([6000], 8, 8, 1, 128, 40), ([5000, 900, 0], 6, 8, 1, 64, 33), ([4100, 8200], 1, 8, 1, 128, 100), ([6500, 70], 2, 8, 2, 64, 136),
])
def test_kv4_splits_joined_in_groups(spd, lens, T, H_q, H_kv, D, splits):
    """So many partials that they are joined in two steps: against one unit a row, and twice through one workspace."""
    import torch
    rng = np.random.default_rng(splits)
    lens, pt, mp, n, kv4, vals = make_cache(rng, lens, 16, H_kv, D)
    B = len(lens)
    dims = spd.dims_of(B, H_q, H_kv, D, 16, mp, n)
    items = mp
    units = -(-items // -(-items // splits))  # of a row, as the call cuts it
    assert units * T * (H_q // H_kv) * D * 4 > 256 << 10
    q, cache, d_pt, d_lens = rows_bf16(rng, B, T, H_q, D), dev(kv4), dev(pt), dev(lens)
    ws = spd.workspace(spd.spd_kv4_dense_verify_workspace_size(dims, T, splits))
    got = []
    for s in (splits, splits, 1):
        o = torch.full((B, T, H_q, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((B, T, H_q), float("nan"), device="cuda")
        spd.kv4_dense_verify_attn(dims, T, to_dev(q), cache, d_pt, d_lens, o, ws, lse=lse, num_splits=s)
        got.append((host(o), host(lse)))
    assert spd.spd_device_status(clear=True) == 0
    assert all(np.array_equal(x, y) for x, y in zip(got[0], got[1]))
    G = H_q // H_kv
    for b in range(B):
        for t in range(T):
            seen = np.arange(lens[b]) <= lens[b] - T + t
            for hq in (0, H_q - 1):
                for og, lg in (got[0], got[2]):
                    check_row(og[b, t, hq], lg[b, t, hq], q[b, t, hq], vals[b][0][:, hq // G], vals[b][1][:, hq // G], D ** -0.5, seen, (b, t, hq))
