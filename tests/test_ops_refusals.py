"""What the rotation, the 4-bit cache and the token log probabilities refuse, without a GPU."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4


@pytest.fixture(scope="module")
def spd():
    from sparse_attention_decode_pages_gb300 import _build
    _build.build()
    import sparse_attention_decode_pages_gb300 as spd
    return spd


P = ctypes.c_void_p
A, ODD = 0x10000, 0x10002  # addresses that are never read: every call below is refused before a launch


def rope(spd, **over):
    f = dict(table=A, n_pos=64, rot_dim=64, interleaved=0, eps=1e-6, q_weight=None, k_weight=None)
    f.update(over)
    return spd.Rope(*f.values())


def qk(spd, r, rows=4, H_q=4, H_kv=2, D=64, q=A, qs=256, k=A, ks=128, pos=A, qo=A, ko=A):
    return spd.lib().qk_norm_rope(rows, H_q, H_kv, D, ctypes.byref(r) if r else None, q, qs, k, ks, pos, qo, ko, None)


def test_qk_norm_rope_refusals(spd):
    assert qk(spd, None) == INVALID
    assert qk(spd, rope(spd), D=96) == UNSUPPORTED
    for rot in (-8, 4, 72):
        assert qk(spd, rope(spd, rot_dim=rot)) == UNSUPPORTED
    for eps in (-1.0, float("nan"), float("inf")):
        assert qk(spd, rope(spd, eps=eps)) == INVALID
    assert qk(spd, rope(spd, table=None)) == INVALID
    assert qk(spd, rope(spd, table=ODD)) == INVALID
    assert qk(spd, rope(spd, n_pos=0)) == INVALID
    assert qk(spd, rope(spd, q_weight=ODD)) == INVALID
    assert qk(spd, rope(spd), qs=255) == INVALID       # below the row
    assert qk(spd, rope(spd), ks=132) == INVALID       # rows off 16 bytes
    assert qk(spd, rope(spd), H_q=0) == INVALID
    assert qk(spd, rope(spd), q=ODD) == INVALID
    assert qk(spd, rope(spd), qo=None) == INVALID
    assert qk(spd, rope(spd), pos=None) == INVALID
    assert qk(spd, rope(spd), rows=-1) == INVALID
    assert qk(spd, rope(spd), rows=1 << 31) == UNSUPPORTED
    assert qk(spd, rope(spd), rows=0) == OK
    assert qk(spd, rope(spd), q=None, k=None) == OK


def test_kv_append_rope_refusals(spd):
    d = spd.dims_of(2, 4, 2, 64, 16, 8, 16)

    def call(dims=d, T=1, r=rope(spd), K=A, q=A, qs=256, k=A, v=A, vs=128, qo=A, summ=A):
        return spd.lib().kv_append_rope(ctypes.byref(dims), T, ctypes.byref(r), K, A, A, A, q, qs, k, 128, v, vs, qo,
                                        summ, None)

    assert call(T=0) == INVALID and call(T=4097) == INVALID
    assert call(dims=spd.dims_of(2, 4, 2, 96, 16, 8, 16)) == UNSUPPORTED
    assert call(r=rope(spd, rot_dim=12)) == UNSUPPORTED
    assert call(K=None) == INVALID and call(k=None) == INVALID and call(v=None) == INVALID and call(summ=None) == INVALID
    assert call(K=ODD) == INVALID and call(v=ODD) == INVALID
    assert call(q=None) == INVALID and call(qo=None) == INVALID   # q and q_out go together
    assert call(vs=64) == INVALID and call(vs=132) == INVALID
    assert call(dims=spd.dims_of(0, 4, 2, 64, 16, 8, 16)) == OK


def test_kv4_refusals(spd):
    L = spd.lib()
    d = spd.dims_of(2, 4, 2, 64, 16, 8, 16)
    z = spd.dims_of(0, 4, 2, 64, 16, 8, 16)
    B = ctypes.byref
    for f in (lambda dims, T, c, ke, ve, k: L.kv4_append(B(dims), T, c, ke, ve, A, A, k, A, A, None),
              lambda dims, T, c, ke, ve, k: L.kv4_read(B(dims), T, c, ke, ve, A, A, k, A, None)):
        assert f(d, 0, A, 0, 0, A) == INVALID and f(d, 4097, A, 0, 0, A) == INVALID
        assert f(d, 1, A, 65, 0, A) == INVALID and f(d, 1, A, 0, -65, A) == INVALID
        assert f(d, 1, None, 0, 0, A) == INVALID and f(d, 1, ODD, 0, 0, A) == INVALID
        assert f(d, 1, A, 0, 0, None) == INVALID and f(d, 1, A, 0, 0, ODD) == INVALID
        assert f(spd.dims_of(2, 4, 2, 64, 24, 8, 16), 1, A, 0, 0, A) == UNSUPPORTED
        assert f(z, 1, A, 0, 0, A) == OK

    def sparse(dims=d, q=A, c=A, ke=0, sel=A, k_max=4, splits=0, scale=0.1, o=A):
        return L.kv4_sparse_decode_attn(B(dims), q, c, ke, 0, A, A, sel, A, k_max, splits, scale, o, None, A, 1 << 20, None)

    def dense(dims=d, T=1, q=A, c=A, ve=0, splits=0, scale=0.1):
        return L.kv4_dense_verify_attn(B(dims), T, q, c, 0, ve, A, A, splits, scale, A, None, A, 1 << 20, None)

    assert sparse(k_max=0) == INVALID and sparse(sel=None) == INVALID and sparse(q=None) == INVALID
    assert sparse(c=ODD) == INVALID and sparse(o=ODD) == INVALID and sparse(ke=99) == INVALID
    assert sparse(scale=float("nan")) == INVALID and sparse(splits=-1) == INVALID
    assert sparse(scale=1e30, ke=64) == INVALID
    assert sparse(dims=z) == OK and dense(dims=z) == OK
    assert dense(T=0) == UNSUPPORTED and dense(T=33) == UNSUPPORTED
    assert dense(q=ODD) == INVALID and dense(ve=-99) == INVALID and dense(scale=float("inf")) == INVALID
    assert L.spd_kv4_sparse_decode_workspace_size(B(d), 0, 0) == 0
    assert L.spd_kv4_dense_verify_workspace_size(B(d), 33, 0) == 0


@pytest.mark.parametrize("B,H_kv", [(1, 1), (2, 8), (2048, 8), (5000, 8)])
def test_scores_lie_behind_every_calls_tickets(spd, B, H_kv):
    """A queue of 16 bytes and the tickets of 16,384 rows, or of the call's own where they are more."""
    d = spd.dims_of(B, H_kv, H_kv, 64, 16, 9, 16)
    size = spd.lib().spd_score_select_workspace_size(ctypes.byref(d))
    assert size - B * H_kv * 9 * 4 >= 16 + 4 * max(16384, B * H_kv)


def test_token_logprobs_refusals(spd):
    def call(rows=2, n=50, x=A, bf=0, stride=50, t=A, inv=1.0, lp=A, k=0, ids=None, tops=None):
        return spd.lib().token_logprobs(rows, n, x, bf, stride, t, inv, lp, None, None, k, ids, tops, A, 1 << 20, None)

    assert call(rows=-1) == INVALID and call(rows=1 << 31) == INVALID
    assert call(n=0) == UNSUPPORTED and call(n=(1 << 21) + 1, stride=1 << 22) == UNSUPPORTED
    assert call(k=33) == UNSUPPORTED and call(k=-1) == UNSUPPORTED
    assert call(stride=49) == INVALID
    for inv in (0.0, -1.0, float("nan"), float("inf")):
        assert call(inv=inv) == INVALID
    assert call(x=None) == INVALID and call(t=None) == INVALID
    assert call(k=3) == INVALID and call(k=3, ids=A) == INVALID
    assert call(x=A + 2) == INVALID and call(x=A + 1, bf=1) == INVALID
    assert call(rows=0) == OK
    assert spd.lib().spd_token_logprobs_workspace_size(1, 0, 0) == 0


def test_token_logprobs_refuses_a_temperature_past_its_exponents(spd):
    """Differences of logits are scaled by inv_temperature * log2(e): where that is infinite, 0 times it is NaN."""
    for inv in (2.4e38, 3e38, 3.4028e38):
        assert spd.lib().token_logprobs(2, 50, A, 0, 50, A, inv, A, None, None, 0, None, None, A, 1 << 20, None) == INVALID


def test_the_binding_checks_its_tensors(spd):
    """Host tensors are refused before anything is called (types, sizes and strides need a device tensor)."""
    import torch
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(spd.SpdError):
        spd.qk_norm_rope(x, None, None, None, x, None)
    with pytest.raises(spd.SpdError):
        spd.qk_norm_rope(None, None, None, None, None, None)
    with pytest.raises(spd.SpdError):
        spd.token_logprobs(torch.zeros((2, 50)), torch.zeros(2, dtype=torch.int32), torch.zeros(2), torch.zeros(16, dtype=torch.uint8))
    assert spd._row_stride(torch.zeros((3, 2, 12, 64))[:, :, 2:6], 64, "q") == 12 * 64
    assert spd._row_stride(torch.zeros((1, 1, 4, 64)), 64, "q") == 256
    for bad in (torch.zeros((2, 4, 128))[:, :, ::2], torch.zeros((2, 8, 64))[:, ::2], torch.zeros((3, 4, 4, 64))[:, :2]):
        with pytest.raises(spd.SpdError):
            spd._row_stride(bad, 64, "q")


def test_the_reference_format_is_the_one_described():
    """The 64-bit form that the GPU tests hold the cache to: worked by hand."""
    import numpy as np
    from tests import ops_reference as ref
    assert ref.e4m3_values()[-1] == 448 and ref.e4m3_values()[1] == 2.0 ** -9
    x = np.array([0.25, -0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.26, 5.1, -3.49, 0, 4.99, 2.51, 0.74])
    codes, scale = ref.kv4_quantise(x, 0)
    assert scale.tolist() == [0x38]  # 1.0
    assert codes.tolist() == [0, 8, 2, 2, 4, 4, 6, 6, 7, 1, 7, 13, 0, 6, 5, 1]
    tile = ref.kv4_pack(np.tile(codes, (2, 1)), np.tile(scale, (2, 1)))
    assert tile.tolist()[:2] == [0x80, 0x22] and tile.tolist()[-2:] == [0x38, 0x38]
    c, s = ref.kv4_unpack(tile, 2, 16)
    assert np.array_equal(c[1], codes) and np.array_equal(ref.kv4_values(c, s, 3)[0], ref.kv4_values(codes, scale, 0) * 8)
