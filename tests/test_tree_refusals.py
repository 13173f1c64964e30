"""What the tree calls and the eviction refuse, without a GPU, and their 64-bit forms by hand."""
import ctypes

import numpy as np
import pytest

from tests import tree_reference as ref

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
A, ODD = 0x10000, 0x10002  # addresses that are never read: every call below is refused before a launch
C = 0x20000


@pytest.fixture(scope="module")
def spd():
    from sparse_attention_decode_pages_gb300 import _build
    _build.build()
    import sparse_attention_decode_pages_gb300 as spd
    return spd


def both(spd):
    return spd.dims_of(2, 4, 2, 64, 16, 8, 16), spd.dims_of(0, 4, 2, 64, 16, 8, 16)


def test_tree_verify_attn_refusals(spd):
    d, z = both(spd)

    def call(dims=d, T=4, q=A, qs=256, K=A, V=A, pt=A, lens=A, k=A, ks=128, v=A, vs=128, par=A, scale=0.1, o=A, ws=A):
        return spd.lib().tree_verify_attn(ctypes.byref(dims), T, q, qs, K, V, pt, lens, k, ks, v, vs, par, scale, o, None,
                                          ws, 1 << 30, None)

    assert call(T=0) == UNSUPPORTED and call(T=65) == UNSUPPORTED
    assert call(dims=spd.dims_of(2, 4, 2, 96, 16, 8, 16)) == UNSUPPORTED
    assert call(dims=spd.dims_of(2, 4, 2, 64, 24, 8, 16)) == UNSUPPORTED
    assert call(dims=spd.dims_of(2, 36, 4, 64, 16, 8, 16)) == UNSUPPORTED
    assert call(dims=spd.dims_of(8193, 4, 2, 64, 16, 8, 16)) == UNSUPPORTED      # B * H_kv > 16384
    assert call(dims=spd.dims_of(1, 4, 2, 64, 64, (1 << 24) + 1, 16)) == UNSUPPORTED  # positions past 2^30
    for name in ("q", "K", "V", "pt", "lens", "k", "v", "par", "o"):
        assert call(**{name: None}) == INVALID, name
    for name in ("q", "K", "V", "k", "v", "o"):
        assert call(**{name: ODD}) == INVALID, name
    assert call(qs=255) == INVALID and call(qs=264 - 4) == INVALID and call(ks=120) == INVALID and call(vs=132) == INVALID
    for s in (float("nan"), float("inf"), 3e38):
        assert call(scale=s) == INVALID
    assert call(dims=z) == OK
    assert spd.lib().spd_tree_verify_workspace_size(ctypes.byref(d), 0) == 0
    assert spd.lib().spd_tree_verify_workspace_size(ctypes.byref(d), 65) == 0


def test_spec_accept_tree_refusals(spd):
    def call(B=2, T=4, n=50, q=A, draft=A, par=A, ua=A, ur=A, np_=A, path=A, tok=A):
        return spd.lib().spec_accept_tree(B, T, n, q, draft, par, ua, ur, np_, path, tok, None)

    assert call(B=-1) == INVALID and call(B=1 << 27) == UNSUPPORTED
    assert call(T=0) == UNSUPPORTED and call(T=65) == UNSUPPORTED
    assert call(n=0) == UNSUPPORTED and call(n=(1 << 21) + 1) == UNSUPPORTED
    for name in ("q", "draft", "par", "ua", "ur", "np_", "path", "tok"):
        assert call(**{name: None}) == INVALID, name
    assert call(q=ODD) == INVALID
    assert call(B=0) == OK


def test_kv_append_path_refusals(spd):
    d, z = both(spd)

    def call(dims=d, T=4, K=A, V=A, pt=A, lens=A, k=A, ks=128, v=A, vs=128, path=A, n=A, summ=A, new=C):
        return spd.lib().kv_append_path(ctypes.byref(dims), T, K, V, pt, lens, k, ks, v, vs, path, n, summ, new, None)

    assert call(T=0) == UNSUPPORTED and call(T=65) == UNSUPPORTED
    assert call(dims=spd.dims_of(2, 4, 2, 80, 16, 8, 16)) == UNSUPPORTED
    for name in ("K", "V", "pt", "lens", "k", "v", "path", "n", "summ", "new"):
        assert call(**{name: None}) == INVALID, name
    for name in ("K", "V", "k", "v", "summ"):
        assert call(**{name: ODD}) == INVALID, name
    assert call(ks=64) == INVALID and call(vs=129) == INVALID
    assert call(new=A) == INVALID   # the lengths themselves
    assert call(dims=z) == OK


def test_kv_weights_update_refusals(spd):
    d, z = both(spd)

    def call(dims=d, T=4, q=A, lse=A, K=A, pt=A, lens=A, path=None, n=None, sel=None, nsel=None, k_max=0, decay=1.0,
             scale=0.1, w_in=A, w_out=A):
        return spd.lib().kv_weights_update(ctypes.byref(dims), T, q, lse, K, pt, lens, path, n, sel, nsel, k_max, decay, scale,
                                           w_in, w_out, None)

    assert call(T=0) == UNSUPPORTED and call(T=65) == UNSUPPORTED
    assert call(dims=spd.dims_of(2, 4, 2, 64, 24, 8, 16)) == UNSUPPORTED
    assert call(dims=spd.dims_of(1, 4, 2, 64, 64, (1 << 24) + 1, 16)) == UNSUPPORTED
    for name in ("q", "lse", "K", "pt", "lens", "w_out"):
        assert call(**{name: None}) == INVALID, name
    assert call(q=ODD) == INVALID and call(K=ODD) == INVALID
    assert call(path=A) == INVALID and call(n=A) == INVALID
    assert call(sel=A, k_max=4) == INVALID and call(nsel=A) == INVALID and call(sel=A, nsel=A) == INVALID
    for x in (float("nan"), float("inf")):
        assert call(decay=x) == INVALID and call(scale=x) == INVALID
    assert call(dims=z) == OK


def test_kv_evict_refusals(spd):
    d, z = both(spd)

    def call(dims=d, budget=32, sink=4, recent=8, K=A, V=A, pt=A, lens=A, w=A, dst=C, kept=A, w_out=C, summ=A, new=C):
        return spd.lib().kv_evict(ctypes.byref(dims), budget, sink, recent, K, V, pt, lens, w, dst, kept, w_out, summ, new, None)

    assert call(budget=0) == INVALID and call(sink=-1) == INVALID and call(recent=-1) == INVALID
    assert call(budget=11) == INVALID and call(sink=(1 << 31) - 1, recent=(1 << 31) - 1) == INVALID
    assert call(dims=spd.dims_of(2, 4, 2, 64, 8, 8, 16)) == UNSUPPORTED
    assert call(dims=spd.dims_of(1, 4, 2, 64, 64, (1 << 24) + 1, 16)) == UNSUPPORTED
    for name in ("K", "V", "pt", "lens", "w", "dst", "kept", "w_out", "summ", "new"):
        assert call(**{name: None}) == INVALID, name
    for name in ("K", "V", "summ"):
        assert call(**{name: ODD}) == INVALID, name
    assert call(dst=A) == INVALID and call(w_out=A) == INVALID and call(new=A) == INVALID
    assert call(dims=z) == OK


def test_the_binding_refuses_host_tensors(spd):
    import torch
    d, _ = both(spd)
    f, i = torch.zeros((2, 4, 50)), torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(spd.SpdError):
        spd.spec_accept_tree(f, i, i, f[..., 0], f[:, 0, 0], i[:, 0], i, i)
    x = torch.zeros((2, 4, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(spd.SpdError):
        spd.kv_append_path(d, 4, x, x, i, i, x, x, i, i, x, i)


def test_the_64_bit_forms_by_hand():
    s = ref.sees([-1, 0, 0, 1, -2, 4, 9, -1, 7])
    assert [np.flatnonzero(r).tolist() for r in s] == [[0], [0, 1], [0, 2], [0, 1, 3], [], [], [], [7], [7, 8]]
    q = np.zeros((4, 5), np.float32)
    q[0] = [0.5, 0.25, 0.25, 0, 0]
    q[2] = [0, 0, 0, 0.5, 0.5]
    u = np.float32([0, 0.5, 0.25, 0])
    # node 1 proposes token 0 (weight 1/2 of 1): u = 0.5 fails; node 2 token 1 (1/4 of 1/2): 0.25 passes; then node 3
    # proposes token 2, which has no weight behind node 2, and the draw from (3, 4) at 0.5 gives 4
    assert [x.tolist() if hasattr(x, "tolist") else x for x in ref.accept_tree(q, [9, 0, 1, 2], [-1, 0, 0, 2], u, 0.5)] == \
        [2, [0, 2, -1, -1], [1, 4, -1, -1]]
    # with the first child's token tried and lost, the draw is from what is left
    assert ref.accept_tree(q, [9, 0, 0, 0], [-1, 0, 0, 0], np.float32([0, 0.75, 0, 0]), 0.0)[2].tolist() == [1, -1, -1, -1]
    w = np.array([0.0, 3.0, np.nan, 3.0, -1.0, 2.0, 7.0])
    assert ref.kept(w, 7, 4, 1, 1).tolist() == [0, 1, 3, 6] and ref.kept(w, 7, 6, 1, 1).tolist() == [0, 1, 3, 4, 5, 6]
    assert ref.kept(w, 3, 4, 1, 1).tolist() == [0, 1, 2]
