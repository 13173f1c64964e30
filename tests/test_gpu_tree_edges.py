"""Tree verification and acceptance where few calls go: numbers of one and more, short wait limits, many sequences, many parts,
long sums."""
import numpy as np
import pytest

from tests import tree_reference as ref
from tests.test_gpu_rope import dev, host
from tests.test_gpu_tree import attend, case, check_accept, check_case, check_node

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spd():
    import sparse_attention_decode_pages_gb300 as spd
    spd.spd_device_status(clear=True)
    return spd


@pytest.mark.parametrize("u", [1.0, 8.0, 2.0 ** 21, 2.0 ** 22, 1.5 * 2.0 ** 22, 2.0 ** 23, 3e38])
def test_spec_accept_tree_numbers_of_one_and_more(spd, u):
    """A number of 1 or more takes no child and draws the last token of positive weight, also where its product with the
    row's sum passes 64 bits (2^22 times four weights of 2^40 is 2^64)."""
    T, n = 3, 7
    q = np.zeros((3, T, n), np.float32)
    q[0, :, :4] = 1.0
    q[1, :, :5] = 1.0
    q[2, :, 2] = 0.75
    draft, parents = np.tile([0, 2, 1], (3, 1)), np.tile([-1, 0, 0], (3, 1))
    got = check_accept(spd, q, draft, parents, np.full((3, T), u, np.float32), np.full(3, u, np.float32))
    assert got[0].tolist() == [1, 1, 1] and got[2][:, 0].tolist() == [3, 4, -1]
    assert spd.spd_device_status(clear=True) == 0


@pytest.mark.parametrize("u", [4.0, 8.0, 24.0])
def test_spec_accept_tree_numbers_of_one_and_more_long_rows(spd, u):
    """Row sums of 2^61, the largest there are."""
    n = 1 << 21
    q = np.ones((1, 2, n), np.float32)
    q[0, 1] = 0.0
    got = check_accept(spd, q, np.array([[0, 5]]), np.array([[-1, 0]]), np.full((1, 2), u, np.float32), np.float32([u]))
    assert got[0][0] == 1 and got[2][0, 0] == n - 1


def walks(B, T, n):
    """Arguments of spec_accept_tree with walks of several steps, made on the GPU."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(n)
    q = torch.rand((B, T, n), generator=gen, device="cuda") ** 8
    draft = torch.randint(0, n, (B, T), generator=gen, device="cuda")
    parents = torch.clamp(torch.arange(T, device="cuda") - 1, min=-1) // 2
    parents[0] = -1
    parents = parents.repeat(B, 1)
    for x in range(1, T):  # a token proposed weighs more than all others together
        q[torch.arange(B), parents[:, x], draft[:, x]] = 0.3 * n
    q /= q.sum(2, keepdim=True)
    u_acc, u_res = (torch.rand(shape, generator=gen, device="cuda") for shape in ((B, T), (B,)))
    return q, draft.to(torch.int32), parents.to(torch.int32).contiguous(), u_acc, u_res


def accepted(spd, *args):
    import torch
    B, T = args[1].shape
    out = [torch.full(shape, -9, dtype=torch.int32, device="cuda") for shape in ((B,), (B, T), (B, T))]
    spd.spec_accept_tree(*args, *out)
    return out


@pytest.mark.parametrize("B,T,n", [(64, 15, 151936), (3, 8, 151936), (400, 5, 32000), (20, 6, 4099)])
def test_spec_accept_tree_with_waits_that_run_out(spd, B, T, n):
    """A limit that no copy meets: the calls return with the timeout bit (or, should every copy be early, clean), and later calls
    with the usual limit are those of before."""
    import torch
    args = walks(B, T, n)
    want = accepted(spd, *args)
    assert spd.spd_device_status(clear=True) == 0 and int(want[0].max()) > 2  # (five nodes in pairs are three deep)
    usual = spd.spd_wait_limit_ns()
    try:
        spd.spd_set_wait_limit_ns(1)
        for _ in range(2):
            accepted(spd, *args)
            assert spd.spd_device_status(clear=True) & ~spd.DEV_TIMEOUT == 0
    finally:
        spd.spd_set_wait_limit_ns(usual)
    for got, x in zip(accepted(spd, *args), want):
        assert torch.equal(got, x)
    assert spd.spd_device_status(clear=True) == 0


@pytest.mark.parametrize("B,T,n", [(64, 15, 151936), (3, 8, 151936), (400, 5, 32000)])
@pytest.mark.parametrize("limit_ns", [1, 3000])
def test_spec_accept_tree_writes_nothing_of_a_sequence_whose_copies_are_late(spd, B, T, n, limit_ns):
    """Whatever the limit, a sequence's outputs are those of the usual one, or left as they were with the timeout bit set."""
    args = walks(B, T, n)
    want = [x.cpu().numpy() for x in accepted(spd, *args)]
    assert spd.spd_device_status(clear=True) == 0
    usual = spd.spd_wait_limit_ns()
    try:
        spd.spd_set_wait_limit_ns(limit_ns)
        for _ in range(6):
            got = [x.cpu().numpy() for x in accepted(spd, *args)]
            status = spd.spd_device_status(clear=True)
            late = got[0] == -9
            assert np.all(got[1][late] == -9) and np.all(got[2][late] == -9)
            for x, y in zip(got, want):
                assert np.array_equal(x[~late], y[~late])
            assert status == (spd.DEV_TIMEOUT if late.any() else 0), (status, late.sum())
    finally:
        spd.spd_set_wait_limit_ns(usual)


def test_tree_verify_attn_a_limit_shorter_than_a_part(spd):
    """A limit is one of a single wait: a part of 65,536 tokens takes many times the limit, no copy in it does."""
    import torch
    B, T, H_q, H_kv, D, ps, n = 19, 32, 64, 8, 128, 16, 65536
    dims = spd.dims_of(B, H_q, H_kv, D, ps, n // ps, n // ps)
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *shape: torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    K, V = r(n // ps, H_kv, ps, D), r(n // ps, H_kv, ps, D)
    pt = torch.arange(n // ps, dtype=torch.int32, device="cuda").repeat(B, 1)  # all sequences over the same pages
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    parents = dev(np.tile(ref.random_tree(np.random.default_rng(0), T).astype(np.int32), (B, 1)))
    args = (dims, T, r(B, T, H_q, D), K, V, pt, lens, r(B, T, H_kv, D), r(B, T, H_kv, D), parents)
    ws = spd.workspace(spd.spd_tree_verify_workspace_size(dims, T))
    want = attend(spd, *args, ws=ws)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    attend(spd, *args, ws=ws)
    end.record()
    assert spd.spd_device_status(clear=True) == 0
    limit_ns = 200_000
    assert begin.elapsed_time(end) * 1e6 > 2 * limit_ns  # (one part a CTA)
    usual = spd.spd_wait_limit_ns()
    try:
        spd.spd_set_wait_limit_ns(limit_ns)
        for _ in range(3):
            got = attend(spd, *args, ws=ws)
            assert spd.spd_device_status(clear=True) == 0
            for x, y in zip(got, want):
                assert torch.equal(x, y)
    finally:
        spd.spd_set_wait_limit_ns(usual)


@pytest.mark.parametrize("lens,T,H_q,H_kv,D", [([700, 300], 9, 8, 2, 128), ([700, 300], 64, 4, 1, 128), ([2000, 0], 50, 8, 1, 64),
                                               ([9000], 5, 4, 1, 64), (list(range(0, 4000, 50)), 20, 8, 2, 128), (list(range(0, 4000, 50)), 50, 8, 2, 64)])
@pytest.mark.parametrize("limit_ns", [1, 1500])
def test_tree_verify_attn_writes_nothing_of_parts_that_are_late(spd, lens, T, H_q, H_kv, D, limit_ns):
    """Whatever the limit, each output is the usual one's or left as it was (with the timeout bit set), also where partials are
    joined and the workspace holds those of another call."""
    import torch
    rng = np.random.default_rng(T)
    dims, lens, pt, K, V, q, k, v, parents = case(spd, rng, lens, T, H_q, H_kv, D, 16, [ref.random_tree(rng, T) for _ in lens])
    args = (dims, T, q, K, V, dev(pt), dev(lens), k, v, dev(parents.astype(np.int32)))
    ws = spd.workspace(spd.spd_tree_verify_workspace_size(dims, T))
    want = attend(spd, *args, ws=ws)
    other = (dims, T, torch.randn_like(q.contiguous()), *args[3:])
    assert spd.spd_device_status(clear=True) == 0
    usual = spd.spd_wait_limit_ns()
    for _ in range(8):
        attend(spd, *other, ws=ws)
        torch.cuda.synchronize()
        try:
            spd.spd_set_wait_limit_ns(limit_ns)
            got = attend(spd, *args, ws=ws)  # (outputs that begin as NaN)
            status = spd.spd_device_status(clear=True)
        finally:
            spd.spd_set_wait_limit_ns(usual)
        missing = [torch.isnan(x) for x in got]
        for x, y, m in zip(got, want, missing):
            assert torch.equal(x[~m], y[~m])
        assert status in (0, spd.DEV_TIMEOUT) and (status or not any(bool(m.any()) for m in missing))
    for x, y in zip(attend(spd, *args, ws=ws), want):
        assert torch.equal(x, y)
    assert spd.spd_device_status(clear=True) == 0


@pytest.mark.parametrize("B", [385, 800])
def test_tree_verify_attn_more_sequences_than_a_cta_has_threads(spd, B):
    """Short sequences of unequal lengths, several empty: a thread's run of them where shares are cut."""
    rng = np.random.default_rng(B)
    lens = np.where(rng.random(B) < 0.2, 0, rng.integers(0, 200, B))
    lens[[0, -1]] = 0, 1500
    T = 3
    trees = [ref.random_tree(rng, T, "random", int(rng.integers(0, T + 1))) for _ in range(B)]
    check_case(spd, *case(spd, rng, lens, T, 2, 1, 64, 16, trees))


def test_tree_verify_attn_a_bad_length_among_many_sequences(spd):
    """The rows of a sequence that the page table has no room for are of no node, all others' bits are those without it."""
    import torch
    rng = np.random.default_rng(5)
    B, T = 500, 4
    lens = rng.integers(0, 150, B)
    trees = [ref.random_tree(rng, T) for _ in range(B)]
    dims, lens, pt, K, V, q, k, v, parents = case(spd, rng, lens, T, 4, 2, 64, 16, trees)
    args = (dims, T, q, K, V, dev(pt))
    rest = (k, v, dev(parents.astype(np.int32)))
    room = pt.shape[1] * 16
    clean = lens.copy()
    clean[[7, 250, 499]] = 0
    bad = clean.copy()
    bad[[7, 250, 499]] = room + 1, -1, 2 ** 31 - 1
    want = attend(spd, *args, dev(clean), *rest)
    assert spd.spd_device_status(clear=True) == 0
    o, lse = attend(spd, *args, dev(bad), *rest)
    assert spd.spd_device_status(clear=True) == spd.DEV_BAD_LEN
    assert bool((o[[7, 250, 499]] == 0).all()) and bool(torch.isneginf(lse[[7, 250, 499]]).all())
    good = np.setdiff1d(np.arange(B), [7, 250, 499])
    assert torch.equal(o[good], want[0][good]) and torch.equal(lse[good], want[1][good])


@pytest.mark.parametrize("lens,T,H_q,H_kv,D,ps,rows", [
    ([23545], 51, 8, 2, 128, 16, {0, 17, 50}),      # two units in 76 parts each
    ([18001], 3, 2, 1, 64, 32, None),               # one in 142
    ([40003, 300, 0], 33, 4, 1, 128, 64, {0, 31, 32}),
])
def test_tree_verify_attn_units_in_many_parts(spd, lens, T, H_q, H_kv, D, ps, rows):
    """Tens of partials of a row, joined by several threads each."""
    rng = np.random.default_rng(T)
    trees = [ref.random_tree(rng, T) for _ in lens]
    check_case(spd, *case(spd, rng, lens, T, H_q, H_kv, D, ps, trees), rows=rows)


@pytest.mark.parametrize("lg_tokens,low,T,G,D", [(17, 1e-4, 32, 8, 64), (20, 7e-4, 32, 8, 64), (22, 1e-4, 32, 8, 64), (21, 1e-4, 29, 8, 128),
                                                 (20, 1e-4, 4, 4, 128), (22, 1e-4, 5, 3, 64)])
def test_tree_verify_attn_long_sums_of_one_sign(spd, lg_tokens, low, T, G, D):
    """Equal logits over 2^17 and more tokens that one CTA goes over: channel c's mean is 1 + m / 64 * 2^-7 for an m that grows with c,
    so a result is 1 + 2^-7 where the mean, less what the tensor cores cut (`low` of it at most), is above 1 + 2^-8, and 1 where it
    is below.  (Sums that lose their small parts give 1 everywhere.)"""
    import torch
    B, ps, n = 152, 64, 1 << lg_tokens
    dims = spd.dims_of(B, G, 1, D, ps, n // ps, 1)
    K = torch.zeros((1, 1, ps, D), dtype=torch.bfloat16, device="cuda")
    m = np.arange(D) * 64 // D
    V = (1.0 + (torch.arange(ps, device="cuda")[:, None] < dev(m)) * 2.0 ** -7).to(torch.bfloat16)[None, None].contiguous()
    pt = torch.zeros((B, n // ps), dtype=torch.int32, device="cuda")
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = torch.ones((B, T, G, D), dtype=torch.bfloat16, device="cuda")
    k, v = torch.full((B, T, 1, D), -100.0, dtype=torch.bfloat16, device="cuda"), torch.zeros((B, T, 1, D), dtype=torch.bfloat16, device="cuda")
    parents = dev(np.tile(np.arange(-1, T - 1, dtype=np.int32), (B, 1)))
    o, lse = attend(spd, dims, T, q, K, V, pt, lens, k, v, parents)
    assert spd.spd_device_status(clear=True) == 0
    mean = 1.0 + m / 64 * 2.0 ** -7
    o = host(o)
    assert np.all(np.isin(o, [1.0, 1.0 + 2.0 ** -7]))
    assert np.all(o[..., mean * (1 - low) > 1.0 + 2.0 ** -8] == 1.0 + 2.0 ** -7)
    assert np.all(o[..., mean < 1.0 + 2.0 ** -8] == 1.0)
    # n weights of 1 add up exactly below 2^24; log2 is off by an ulp (2^-19 at most), its product with ln 2 is rounded
    assert np.abs(host(lse) - lg_tokens * np.log(2.0)).max() <= lg_tokens * 2.0 ** -22


@pytest.mark.parametrize("T,G,D,B", [(32, 8, 64, 152), (4, 2, 128, 152), (32, 8, 128, 100), (7, 2, 64, 90)])
def test_tree_verify_attn_long_sums_of_weights_below_one(spd, T, G, D, B):
    """2^22 - 5 tokens, one of 64 of them with a larger logit: weights of 0.7 add up as they should, from one reference to a
    later one (the last token's logit is 15 above all others)."""
    import torch
    ps, n = 64, (1 << 22) - 5
    pages = -(-n // ps)
    dims = spd.dims_of(B, G, 1, D, ps, pages, 2)
    K, V = torch.zeros((2, 1, ps, D), dtype=torch.bfloat16, device="cuda"), torch.ones((2, 1, ps, D), dtype=torch.bfloat16, device="cuda")
    K[:, 0, 0] = 0.35 / D ** 0.5
    K[1, 0, (n - 1) % ps] = 15.0 / D ** 0.5
    pt = torch.zeros((B, pages), dtype=torch.int32, device="cuda")
    pt[:, -1] = 1
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = torch.ones((B, T, G, D), dtype=torch.bfloat16, device="cuda")
    k, v = torch.full((B, T, 1, D), -100.0, dtype=torch.bfloat16, device="cuda"), torch.zeros((B, T, 1, D), dtype=torch.bfloat16, device="cuda")
    o, lse = attend(spd, dims, T, q, K, V, pt, lens, k, v, dev(np.tile(np.arange(-1, T - 1, dtype=np.int32), (B, 1))))
    assert spd.spd_device_status(clear=True) == 0
    z = host(K)[:, 0].sum(-1) * D ** -0.5
    count = np.array([(pages - 1), 1])[:, None] * np.ones(ps)
    count[1, (n - 1) % ps + 1:] = 0
    want = np.log((count * np.exp(z)).sum())
    # logits: D exact products; the exponent's and ex2's 2^-22 and 2^-24 * 15 each; sums of 36 in a tile, 512 tiles, 64 of these
    # sums and two streams, each off by 2^-24 at most; log2 and its product
    assert np.abs(host(lse) - want).max() <= (36 + 512 + 64 + 2) * 2.0 ** -24 + 16 * 2.0 ** -22 + 22 * 2.0 ** -22
    # values of 1: the weights' rounding (2^-9 of each), the tensor cores' cut (1e-4) and the result's rounding
    assert np.abs(host(o) - 1.0).max() <= 2.0 ** -9 + 1e-4 + 2.0 ** -8


@pytest.mark.parametrize("T,G,D,B", [(32, 8, 64, 110), (5, 4, 128, 110)])
def test_tree_verify_attn_long_sequences_of_any_values(spd, T, G, D, B):
    """200,001 tokens for each of many sequences (all over the same pages), logits that rise and fall along them, shares that cut
    most of the sequences."""
    import torch
    rng = np.random.default_rng(T)
    ps, n = 64, 200001
    pages = -(-n // ps)
    dims = spd.dims_of(B, G, 1, D, ps, pages, pages)
    gen = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *shape: torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    K, V = r(pages, 1, ps, D), r(pages, 1, ps, D)
    K *= (1.5 + torch.sin(torch.arange(pages, device="cuda") / 300.0))[:, None, None, None].to(torch.bfloat16)
    V[pages // 3: pages // 2] += 1.0
    table = rng.permutation(pages).astype(np.int32)
    parents = ref.random_tree(rng, T)
    q, k, v = r(B, T, G, D), r(B, T, 1, D), r(B, T, 1, D)
    o, lse = attend(spd, dims, T, q, K, V, dev(np.tile(table, (B, 1))), torch.full((B,), n, dtype=torch.int32, device="cuda"), k, v,
                    dev(np.tile(parents.astype(np.int32), (B, 1))))
    assert spd.spd_device_status(clear=True) == 0
    ck, cv = (host(x)[table, 0].reshape(-1, D)[:n] for x in (K, V))
    sees = ref.sees(parents)
    for b in (0, 1, B // 2, B - 1):
        keys, values = (np.concatenate([c, host(x[b, :, 0])]) for c, x in ((ck, k), (cv, v)))
        for t, hq in ((0, 0), (T - 1, G - 1)):
            seen = np.concatenate([np.ones(n, bool), sees[t]])
            check_node(host(o[b, t, hq]), float(lse[b, t, hq]), host(q[b, t, hq]), keys, values, D ** -0.5, seen, (b, t, hq))
