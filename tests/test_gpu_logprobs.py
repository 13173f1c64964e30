"""token_logprobs against the 64-bit form on the GPU."""
import numpy as np
import pytest

from tests import ops_reference as ref
from tests.test_gpu_rope import dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spd():
    import sparse_attention_decode_pages_gb300 as spd
    spd.spd_device_status(clear=True)
    return spd


def call(spd, logits, targets, top_k, inv_t=1.0):
    """logits: a device tensor [rows][n] (any row stride); numpy results."""
    import torch
    rows, n = logits.shape
    out = [torch.full((rows,), float("nan"), device="cuda") for _ in range(3)]
    ids = torch.full((rows, top_k), -9, dtype=torch.int32, device="cuda") if top_k else None
    tops = torch.full((rows, top_k), float("nan"), device="cuda") if top_k else None
    ws = spd.workspace(spd.spd_token_logprobs_workspace_size(rows, n, top_k))
    for _ in range(2):  # the workspace is left as it was found
        spd.token_logprobs(logits, dev(targets.astype(np.int32)), out[0], ws, entropy=out[1], lse=out[2], top_ids=ids,
                           top_logprobs=tops, inv_temperature=inv_t)
    torch.cuda.synchronize()
    return [host(t) for t in out] + ([ids.cpu().numpy(), host(tops)] if top_k else [None, None])


def check(got, x, targets, inv_t, top_k):
    """fp32 throughout: z = x * inv_t is off by 2^-24 |z|, exp by 2^-21 more of itself; sums of n positive terms in
    chains of at most 600 additions by 600 * 2^-24 of themselves; log and the last sums by 2^-23 of what they hold.
    The entropy is log S - T / S with T a sum of terms of one sign up to the largest: its relative error is a sum's."""
    lp, ent, lse, ids, tops = ref.logprobs(x, targets, inv_t, top_k)
    with np.errstate(invalid="ignore"):
        zmax = np.array([np.abs(r[np.isfinite(r)] * inv_t).max(initial=0.0) for r in x])
    base = 600 * 2.0 ** -24 + 2.0 ** -20 + 8 * zmax * 2.0 ** -24

    def near(a, b, tol, what):
        special = ~np.isfinite(b)
        assert np.array_equal(a[special], b[special], equal_nan=True), (what, a[special], b[special])
        err = np.abs(a - b)[~special]
        tol = np.broadcast_to(tol, b.shape)[~special]
        assert np.all(err <= tol), (what, float((err / tol).max()))

    near(got[2], lse, base, "lse")
    near(got[0], lp, 2 * base, "logprob")
    near(got[1], ent, base * (4 + 4 * np.where(np.isfinite(ent), np.abs(ent), 0)), "entropy")
    if top_k:
        assert np.array_equal(got[3], ids), np.argwhere(got[3] != ids)[:5]
        near(got[4], tops, 2 * base[:, None], "top")


@pytest.mark.parametrize("n", [1, 2, 31, 500, 4097, 20003])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("top_k", [0, 1, 5, 32])
def test_sizes_and_types(spd, n, dtype, top_k):
    import torch
    rng = np.random.default_rng(n + top_k)
    rows = 5
    x = dev((rng.standard_normal((rows, n)) * 3).astype(np.float32), torch.bfloat16 if dtype == "bf16" else torch.float32)
    t = rng.integers(-1, n, rows)
    check(call(spd, x, t, top_k, 0.7), host(x), t, float(np.float32(0.7)), top_k)
    assert spd.spd_device_status(clear=True) == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("offset,stride", [(0, 1003), (1, 1001), (3, 1010), (7, 1024)])
def test_strided_and_unaligned_rows(spd, dtype, offset, stride):
    """Rows of 1001 logits that start anywhere; what lies between them is NaN."""
    import torch
    rng = np.random.default_rng(offset)
    buf = np.full(offset + 9 * stride + 1001, np.nan, np.float32)
    for r in range(9):
        buf[offset + r * stride: offset + r * stride + 1001] = rng.standard_normal(1001) * 4
    d = dev(buf, torch.bfloat16 if dtype == "bf16" else torch.float32)
    x = d[offset:].as_strided((9, 1001), (stride, 1), d.storage_offset() + offset)
    t = rng.integers(0, 1001, 9)
    check(call(spd, x, t, 7), host(x), t, 1.0, 7)


def test_ties_go_to_the_lower_token(spd):
    import torch
    rng = np.random.default_rng(2)
    x = np.round(rng.standard_normal((6, 3000)) * 2).astype(np.float32)
    x[1] = 0.0
    x[1, ::2] = -0.0  # equal to 0
    x[2] = 5.0
    x[3, 100:] = -np.inf
    t = np.zeros(6, int)
    for dt in (torch.float32, torch.bfloat16):
        check(call(spd, dev(x, dt), t, 32), x.astype(np.float64), t, 1.0, 32)


def test_orders_that_defeat_a_running_bound(spd):
    """Ascending and descending rows, all large values in one place, and few values above a masked row."""
    n = 9001
    x = np.zeros((5, n), np.float32)
    x[0] = np.linspace(-5, 5, n)
    x[1] = np.linspace(5, -5, n)
    x[2, 4000:4040] = 3 + np.arange(40)
    x[3] = -np.inf
    x[3, [17, 8999, 4]] = [1.0, 2.0, 1.0]
    x[4] = np.tile(np.linspace(-4, 4, 13), n // 13 + 1)[:n]
    t = np.array([n - 1, 0, 4039, 17, 12])
    check(call(spd, dev(x), t, 32), x.astype(np.float64), t, 1.0, 32)
    check(call(spd, dev(x), t, 9, 3.0), x.astype(np.float64), t, 3.0, 9)


def test_masked_infinite_and_nan_logits(spd):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((7, 600)) * 3).astype(np.float32)
    x[0] = -np.inf                     # nothing is left
    x[1, :599] = -np.inf               # one token is left
    x[2, 5] = np.nan
    x[3, 7] = -np.inf                  # the target itself is masked
    x[4] = np.finfo(np.float32).min    # a mask of the type's lowest value everywhere
    x[5, ::2] = np.finfo(np.float32).min
    x[6, 0] = 3e38
    t = np.array([3, 599, 9, 7, 2, 1, 0])
    check(call(spd, dev(x), t, 4), x.astype(np.float64), t, 1.0, 4)
    got = call(spd, dev(x), np.full(7, -1), 0)
    assert np.all(got[0] == 0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [601, 1001, 50257])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("inv_t", [0.5, 1.0, 2.0])
def test_one_token_left_under_a_finite_mask(spd, dtype, n, offset, inv_t):
    """Masks of the type's lowest value and of -1e38 that leave a row's first, last or any token, in rows whose ends lie
    outside their whole vectors.  A masked token's weight is exactly 0, so the tolerances are those of the few
    that are left: z to 2^-24 of 9 at most, exp and the sums by 2^-20."""
    import torch
    t_dtype = torch.bfloat16 if dtype == "bf16" else torch.float32
    lowest = torch.finfo(t_dtype).min
    left = [{n - 1: 2.5}, {0: -3.0}, {0: 1.0, n - 1: 4.0}, {n // 2: 0.5}, {n - 1: 2.0, n - 2: 2.0, 1: 3.0}, {n - 1: 0.0}]
    buf = torch.full((offset + len(left) * n,), lowest, dtype=t_dtype, device="cuda")
    x = buf[offset:].view(len(left), n)
    x[4:] = -1e38
    for r, tokens in enumerate(left):
        for token, logit in tokens.items():
            x[r, token] = logit
    t = np.array([max(tokens) for tokens in left])
    got = call(spd, x, t, 0, inv_t)
    lp, ent, lse, _, _ = ref.logprobs(host(x), t, inv_t, 0)
    for a, b in zip(got, (lp, ent, lse)):
        assert np.all(np.abs(a - b) <= 2.0 ** -20 * (1 + 8 * np.abs(b)) + 9 * 2.0 ** -22), (a, b)
    assert spd.spd_device_status(clear=True) == 0


@pytest.mark.parametrize("n", [600, 601, 20003])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_an_infinite_logit(spd, n, dtype):
    """+inf in a vector, as a row's single first or last token, beside a second one, and with all else masked."""
    import torch
    rng = np.random.default_rng(n)
    x = (rng.standard_normal((6, n)) * 3).astype(np.float32)
    x[0, 5], x[1, 0], x[2, n - 1], x[3, [7, n // 2]] = np.inf, np.inf, np.inf, np.inf
    x[4], x[4, n - 1] = -np.inf, np.inf
    d = dev(x, torch.bfloat16 if dtype == "bf16" else torch.float32)
    t = np.array([5, 3, n - 1, 0, n - 1, 2])
    with np.errstate(invalid="ignore"):
        check(call(spd, d, t, 6), host(d), t, 1.0, 6)
    got = call(spd, d, t, 6)
    assert np.isnan(np.stack(got[:3])[:, :5]).all() and not np.isnan(np.stack(got[:3])[:, 5]).any()
    assert np.array_equal(got[3][:5, 0], [5, 0, n - 1, 7, n - 1]) and got[3][3, 1] == n // 2 and np.all(got[3][4, 1:] == -1)


def test_targets_outside_the_vocabulary(spd):
    rng = np.random.default_rng(4)
    x = rng.standard_normal((4, 50)).astype(np.float32)
    t = np.array([-1, 50, -7, 3])
    got = call(spd, dev(x), t, 0)
    assert spd.spd_device_status(clear=True) == spd.DEV_BAD_TOKEN
    want = ref.logprobs(x.astype(np.float64), np.array([-1, -1, -1, 3]), 1.0, 0)
    assert np.all(got[0][:3] == 0) and abs(got[0][3] - want[0][3]) < 1e-5


@pytest.mark.parametrize("rows,n", [(1, 151936), (3, 32000), (700, 2000), (450, 5000)])
def test_many_and_few_rows(spd, rows, n):
    import torch
    rng = np.random.default_rng(rows)
    x = dev((rng.standard_normal((rows, n)) * 3).astype(np.float32), torch.bfloat16 if rows % 2 else torch.float32)
    t = rng.integers(-1, n, rows)
    some = sorted(set(rng.integers(0, rows, 6).tolist()) | {0, rows - 1})
    got = [g[some] for g in call(spd, x, t, 20, 1.1)]
    check(got, host(x)[some], t[some], float(np.float32(1.1)), 20)


def test_a_round_as_it_is_used(spd):
    """spec_accept's tokens scored against the target's logits, on a stream of its own and as a graph."""
    import torch
    rng = np.random.default_rng(6)
    B, k, n = 5, 3, 777
    logits = dev((rng.standard_normal((B, k + 1, n)) * 2).astype(np.float32))
    probs = torch.softmax(logits, -1).contiguous()
    draft_p = torch.softmax(logits[:, :k] + 0.3 * torch.randn((B, k, n), device="cuda"), -1).contiguous()
    draft = torch.multinomial(draft_p.view(-1, n), 1).view(B, k).to(torch.int32)
    u_acc, u_res = torch.rand((B, k), device="cuda"), torch.rand(B, device="cuda")
    n_acc = torch.zeros(B, dtype=torch.int32, device="cuda")
    tokens = torch.zeros((B, k + 1), dtype=torch.int32, device="cuda")
    lp = torch.empty((B, k + 1), device="cuda")
    lse = torch.empty((B, k + 1), device="cuda")
    ws = spd.workspace(spd.spd_token_logprobs_workspace_size(B * (k + 1), n, 0))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def step(**kw):
        spd.spec_accept(draft_p, probs, draft, u_acc, u_res, n_acc, tokens, **kw)
        spd.token_logprobs(logits, tokens, lp, ws, lse=lse, **kw)

    step(stream=side)
    torch.cuda.synchronize()
    first, toks = lp.clone(), tokens.cpu().numpy()
    want = ref.logprobs(host(logits).reshape(-1, n), toks.reshape(-1), 1.0, 0)
    assert np.abs(host(lp).reshape(-1) - want[0]).max() < 1e-4 and np.all(host(lp)[toks < 0] == 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lp.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(lp, first)
    assert spd.spd_device_status(clear=True) == 0
