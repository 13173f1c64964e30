"""Tree verification and acceptance where few calls go: numbers of one and more, short wait limits, many sequences, many parts,
long sums."""
import numpy as np
import pytest

from tests import tree_reference as ref
from tests.test_gpu_rope import dev, host
from tests.test_gpu_tree import attend, case, check_accept, check_case

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
