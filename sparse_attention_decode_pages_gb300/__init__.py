"""Sparse paged decode attention for GB300: a thin Python binding over ``libspd.so``.

The functions here carry the names of the C ABI (``include/spd.h``) and only
marshal arguments: every step runs in the library's CUDA kernels.  PyTorch
supplies device memory and the current stream.  There is no fallback: if the
library is missing or a call fails, a ``SpdError`` is raised.

Tensors: bf16 data may be ``torch.bfloat16`` or ``torch.uint16`` (same bits);
index data is ``torch.int32``; everything contiguous and on the current device.
Workspaces are zero-initialised byte tensors (see ``workspace``); each call
leaves its counters at zero, so a workspace can be reused on one stream.
"""
from __future__ import annotations

import ctypes
import math
import os

__all__ = [
    "SpdError", "Dims", "Policy", "RoundDesc", "Round", "lib", "dims_of", "policy_of", "workspace",
    "pages_summarize", "kv_append_refresh", "pages_score_select", "pages_append_score_select",
    "sparse_decode_attn", "sparse_decode_attn_noalloc", "sparse_decode_step", "dense_verify_attn",
    "lse_merge", "spec_accept", "spd_device_status", "spd_score_select_workspace_size",
    "spd_sparse_decode_workspace_size", "spd_dense_verify_workspace_size",
    "spd_sparse_decode_step_workspace_size", "spd_set_wait_limit_ns", "spd_wait_limit_ns",
    "DEV_BAD_PAGE", "DEV_BAD_SEL", "DEV_TIMEOUT", "DEV_BAD_LEN", "DEV_BAD_TOKEN", "DEV_BAD_POS",
    "Rope", "qk_norm_rope", "kv_append_rope", "kv4_cache", "kv4_append", "kv4_read",
    "kv4_sparse_decode_attn", "kv4_dense_verify_attn", "token_logprobs",
    "spd_kv4_sparse_decode_workspace_size", "spd_kv4_dense_verify_workspace_size",
    "spd_token_logprobs_workspace_size", "DEV_BAD_TREE", "tree_verify_attn", "spec_accept_tree",
    "kv_append_path", "kv_weights_update", "kv_evict", "spd_tree_verify_workspace_size",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspd.so")

# device status bits (SPD_DEV_* in include/spd.h)
DEV_BAD_PAGE, DEV_BAD_SEL, DEV_TIMEOUT, DEV_BAD_LEN, DEV_BAD_TOKEN = 0x1, 0x2, 0x4, 0x8, 0x10
DEV_BAD_POS, DEV_BAD_TREE = 0x20, 0x40
_STATUS = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "CUDA", 4: "WORKSPACE"}
_MODES = {"fixed": 0, "linear": 1, "fraction": 2, "top_p": 3}


class SpdError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"spd {_STATUS.get(status, status)}: {message}")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H_q", ctypes.c_int32), ("H_kv", ctypes.c_int32),
                ("D", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32), ("num_phys_pages", ctypes.c_int64)]


class Policy(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("fixed_pages", ctypes.c_int32),
                ("min_tokens", ctypes.c_int64), ("slope_num", ctypes.c_int64),
                ("slope_den", ctypes.c_int64), ("intercept", ctypes.c_int64),
                ("frac_num", ctypes.c_int64), ("frac_den", ctypes.c_int64),
                ("sink_pages", ctypes.c_int32), ("local_pages", ctypes.c_int32),
                ("top_p", ctypes.c_float), ("score_scale", ctypes.c_float)]


class Rope(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("n_pos", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p)]


class RoundDesc(ctypes.Structure):
    _fields_ = [("dims", Dims), ("k", ctypes.c_int32),
                ("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("summ", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("q_draft", ctypes.c_void_p), ("k_draft", ctypes.c_void_p), ("v_draft", ctypes.c_void_p),
                ("q_verify", ctypes.c_void_p), ("k_verify", ctypes.c_void_p), ("v_verify", ctypes.c_void_p),
                ("policy", Policy), ("k_max", ctypes.c_int32),
                ("sel", ctypes.c_void_p), ("nsel", ctypes.c_void_p),
                ("o_draft", ctypes.c_void_p), ("lse_draft", ctypes.c_void_p),
                ("o_verify", ctypes.c_void_p), ("lse_verify", ctypes.c_void_p),
                ("n_vocab", ctypes.c_int32),
                ("p_draft", ctypes.c_void_p), ("q_target", ctypes.c_void_p),
                ("draft_tokens", ctypes.c_void_p), ("u_acc", ctypes.c_void_p), ("u_res", ctypes.c_void_p),
                ("n_accepted", ctypes.c_void_p), ("tokens", ctypes.c_void_p),
                ("ws_select", ctypes.c_void_p), ("ws_select_bytes", ctypes.c_size_t),
                ("ws_sparse", ctypes.c_void_p), ("ws_sparse_bytes", ctypes.c_size_t),
                ("ws_verify", ctypes.c_void_p), ("ws_verify_bytes", ctypes.c_size_t),
                ("sparse_splits", ctypes.c_int32), ("verify_splits", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float)]


_lib = None


def lib():
    """Load libspd.so (fails loudly when it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise SpdError(3, f"{LIB_PATH} is missing: build it with "
                              "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        DP, PP = ctypes.POINTER(Dims), ctypes.POINTER(Policy)
        L.spd_version.restype = i32
        L.spd_last_error.restype = ctypes.c_char_p
        L.spd_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), i32]
        L.spd_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
        L.spd_wait_limit_ns.restype = ctypes.c_uint64
        L.spd_score_select_workspace_size.argtypes = [DP]
        L.spd_score_select_workspace_size.restype = sz
        L.spd_sparse_decode_workspace_size.argtypes = [DP, i32, i32]
        L.spd_sparse_decode_workspace_size.restype = sz
        L.spd_dense_verify_workspace_size.argtypes = [DP, i32, i32]
        L.spd_dense_verify_workspace_size.restype = sz
        L.pages_summarize.argtypes = [DP, P, P, P, P, i32, P, P]
        L.pages_score_select.argtypes = [DP, P, P, P, PP, P, P, i32, P, P, sz, P]
        L.sparse_decode_attn.argtypes = [DP, P, P, P, P, P, P, P, i32, i32, ctypes.c_float,
                                         P, P, P, sz, P]
        L.dense_verify_attn.argtypes = [DP, i32, P, P, P, P, P, i32, ctypes.c_float, P, P, P, sz, P]
        L.sparse_decode_attn_noalloc.argtypes = [DP, P, P, P, P, P, P, P, i32, i32, ctypes.c_float,
                                                 P, P, P]
        L.lse_merge.argtypes = [i32, i32, i32, P, P, P, P, P]
        L.kv_append_refresh.argtypes = [DP, i32, P, P, P, P, P, P, P, P]
        L.spec_accept.argtypes = [i32, i32, i32, P, P, P, P, P, P, P, P]
        L.pages_append_score_select.argtypes = [DP, P, P, P, P, P, P, P, P, PP, P, P, i32, P, P, sz, P]
        L.spd_sparse_decode_step_workspace_size.argtypes = [DP, i32]
        L.spd_sparse_decode_step_workspace_size.restype = sz
        L.sparse_decode_step.argtypes = [DP, P, P, P, P, P, P, P, P, PP, P, P, i32, ctypes.c_float, P, P,
                                         P, sz, P]
        RP, i64, f32, u8 = ctypes.POINTER(Rope), ctypes.c_int64, ctypes.c_float, P
        L.qk_norm_rope.argtypes = [i64, i32, i32, i32, RP, P, i64, P, i64, P, P, P, P]
        L.kv_append_rope.argtypes = [DP, i32, RP, P, P, P, P, P, i64, P, i64, P, i64, P, P, P]
        L.kv4_append.argtypes = [DP, i32, u8, i32, i32, P, P, P, P, P, P]
        L.kv4_read.argtypes = [DP, i32, u8, i32, i32, P, P, P, P, P]
        L.spd_kv4_sparse_decode_workspace_size.argtypes = [DP, i32, i32]
        L.spd_kv4_sparse_decode_workspace_size.restype = sz
        L.spd_kv4_dense_verify_workspace_size.argtypes = [DP, i32, i32]
        L.spd_kv4_dense_verify_workspace_size.restype = sz
        L.kv4_sparse_decode_attn.argtypes = [DP, P, u8, i32, i32, P, P, P, P, i32, i32, f32, P, P, P, sz, P]
        L.kv4_dense_verify_attn.argtypes = [DP, i32, P, u8, i32, i32, P, P, i32, f32, P, P, P, sz, P]
        L.spd_token_logprobs_workspace_size.argtypes = [i64, i32, i32]
        L.spd_token_logprobs_workspace_size.restype = sz
        L.token_logprobs.argtypes = [i64, i32, P, i32, i64, P, f32, P, P, P, i32, P, P, P, sz, P]
        L.spd_tree_verify_workspace_size.argtypes = [DP, i32]
        L.spd_tree_verify_workspace_size.restype = sz
        L.tree_verify_attn.argtypes = [DP, i32, P, i64, P, P, P, P, P, i64, P, i64, P, f32, P, P, P, sz, P]
        L.spec_accept_tree.argtypes = [i32, i32, i32, P, P, P, P, P, P, P, P, P]
        L.kv_append_path.argtypes = [DP, i32, P, P, P, P, P, i64, P, i64, P, P, P, P, P]
        L.kv_weights_update.argtypes = [DP, i32, P, P, P, P, P, P, P, P, P, i32, f32, f32, P, P, P]
        L.kv_evict.argtypes = [DP, i32, i32, i32, P, P, P, P, P, P, P, P, P, P, P]
        L.spd_round_create.argtypes = [ctypes.POINTER(RoundDesc), ctypes.POINTER(ctypes.c_void_p)]
        L.spd_round_launch.argtypes = [P, i32, P]
        L.spd_round_destroy.argtypes = [P]
        L.spd_round_destroy.restype = None
        for f in ("spd_device_status", "spd_set_wait_limit_ns", "pages_summarize", "pages_score_select",
                  "sparse_decode_attn", "dense_verify_attn", "lse_merge",
                  "sparse_decode_attn_noalloc", "kv_append_refresh", "spec_accept",
                  "pages_append_score_select", "sparse_decode_step", "qk_norm_rope", "kv_append_rope",
                  "kv4_append", "kv4_read", "kv4_sparse_decode_attn", "kv4_dense_verify_attn",
                  "token_logprobs", "tree_verify_attn", "spec_accept_tree", "kv_append_path",
                  "kv_weights_update", "kv_evict", "spd_round_create", "spd_round_launch"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(status: int):
    if status != 0:
        raise SpdError(status, lib().spd_last_error().decode(errors="replace"))


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise SpdError(1, "tensor is not on a CUDA device")
    if not t.is_contiguous():
        raise SpdError(1, "tensor is not contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def dims_of(B, H_q, H_kv, D, page_size, max_pages_per_seq, num_phys_pages) -> Dims:
    return Dims(B, H_q, H_kv, D, page_size, max_pages_per_seq, num_phys_pages)


def policy_of(p) -> Policy:
    """A ``Policy`` from any object with the fields of ``workloads.BudgetPolicy``."""
    return Policy(_MODES[p.mode] if isinstance(p.mode, str) else int(p.mode), p.fixed_pages,
                  p.min_tokens, p.slope_num, p.slope_den, p.intercept, p.frac_num, p.frac_den,
                  p.sink_pages, p.local_pages, float(getattr(p, "top_p", 0.0)),
                  float(getattr(p, "score_scale", 0.0)))


def _size(v: int, what: str) -> int:
    if v == 0:
        raise SpdError(1, f"{what}: " + lib().spd_last_error().decode(errors="replace"))
    return v


def spd_score_select_workspace_size(dims: Dims) -> int:
    """Bytes of workspace pages_score_select needs for these dims."""
    return _size(lib().spd_score_select_workspace_size(ctypes.byref(dims)), "score_select workspace")


def spd_sparse_decode_workspace_size(dims: Dims, k_max: int, num_splits: int = 0) -> int:
    """Bytes of workspace sparse_decode_attn needs (num_splits 0: the automatic split count)."""
    return _size(lib().spd_sparse_decode_workspace_size(ctypes.byref(dims), k_max, num_splits),
                 "sparse_decode workspace")


def spd_dense_verify_workspace_size(dims: Dims, T: int, num_splits: int = 0) -> int:
    """Bytes of workspace dense_verify_attn needs for T positions."""
    return _size(lib().spd_dense_verify_workspace_size(ctypes.byref(dims), T, num_splits),
                 "dense_verify workspace")


def workspace(nbytes: int, device=None):
    """A zeroed byte tensor usable as a workspace (allocated by PyTorch, not the library)."""
    import torch
    return torch.zeros(max(1, int(nbytes)), dtype=torch.uint8, device=device or "cuda")


def spd_device_status(clear: bool = False) -> int:
    """The device status word (DEV_* bits raised by kernels since the last clear); waits for the device."""
    v = ctypes.c_uint32(0)
    _check(lib().spd_device_status(ctypes.byref(v), 1 if clear else 0))
    return v.value


def spd_set_wait_limit_ns(ns: int):
    """Limit (ns) of every bounded wait in kernels launched from now on (2 s by default)."""
    _check(lib().spd_set_wait_limit_ns(int(ns)))


def spd_wait_limit_ns() -> int:
    """The current limit of the kernels' bounded waits, in nanoseconds."""
    return int(lib().spd_wait_limit_ns())


def pages_summarize(dims: Dims, K, page_table, seq_lens, summ, only_pages=None, stream=None):
    """Per-page key min / max summaries into summ (all pages, or the listed b * max_pages + p slots)."""
    n_only = 0 if only_pages is None else only_pages.numel()
    _check(lib().pages_summarize(ctypes.byref(dims), _ptr(K), _ptr(page_table), _ptr(seq_lens),
                                 _ptr(only_pages), n_only, _ptr(summ), _stream(stream)))


def kv_append_refresh(dims: Dims, T: int, K, V, page_table, seq_lens, k_new, v_new, summ,
                      stream=None):
    """Write the T newest tokens into the paged cache and rebuild the summaries of their pages."""
    _check(lib().kv_append_refresh(ctypes.byref(dims), T, _ptr(K), _ptr(V), _ptr(page_table),
                                   _ptr(seq_lens), _ptr(k_new), _ptr(v_new), _ptr(summ),
                                   _stream(stream)))


def spec_accept(p_draft, q_target, draft, u_acc, u_res, n_accepted, tokens, stream=None):
    """p_draft [B][k][n], q_target [B][k+1][n] (fp32), draft int32 [B][k], u_acc [B][k], u_res [B]."""
    B, k, n = p_draft.shape
    _check(lib().spec_accept(B, k, n, _ptr(p_draft), _ptr(q_target), _ptr(draft), _ptr(u_acc),
                             _ptr(u_res), _ptr(n_accepted), _ptr(tokens), _stream(stream)))


def pages_append_score_select(dims: Dims, K, V, page_table, seq_lens, k_new, v_new, q, summ, policy,
                              sel, nsel, k_max: int, ws, scores=None, stream=None):
    """kv_append_refresh (T = 1) fused into pages_score_select's pass over the summaries."""
    pol = policy if isinstance(policy, Policy) else policy_of(policy)
    _check(lib().pages_append_score_select(ctypes.byref(dims), _ptr(K), _ptr(V), _ptr(page_table),
                                           _ptr(seq_lens), _ptr(k_new), _ptr(v_new), _ptr(q), _ptr(summ),
                                           ctypes.byref(pol), _ptr(sel), _ptr(nsel), k_max, _ptr(scores),
                                           _ptr(ws), ws.numel(), _stream(stream)))


def spd_sparse_decode_step_workspace_size(dims: Dims, k_max: int) -> int:
    """Bytes of workspace sparse_decode_step needs."""
    return _size(lib().spd_sparse_decode_step_workspace_size(ctypes.byref(dims), k_max), "decode step workspace")


def sparse_decode_step(dims: Dims, K, V, page_table, seq_lens, k_new, v_new, q, summ, policy, sel, nsel,
                       k_max: int, o, ws, lse=None, softmax_scale: float | None = None, stream=None):
    """Append (k_new / v_new may be None) + score + select + sparse attention in one call."""
    pol = policy if isinstance(policy, Policy) else policy_of(policy)
    scale = 1.0 / math.sqrt(dims.D) if softmax_scale is None else softmax_scale
    _check(lib().sparse_decode_step(ctypes.byref(dims), _ptr(K), _ptr(V), _ptr(page_table), _ptr(seq_lens),
                                    _ptr(k_new), _ptr(v_new), _ptr(q), _ptr(summ), ctypes.byref(pol), _ptr(sel),
                                    _ptr(nsel), k_max, scale, _ptr(o), _ptr(lse), _ptr(ws), ws.numel(),
                                    _stream(stream)))


def pages_score_select(dims: Dims, q, summ, seq_lens, policy, sel, nsel, k_max: int, ws,
                       scores=None, stream=None):
    """Page upper-bound scores and the budgeted selection (ascending page ids) per (sequence, KV head)."""
    pol = policy if isinstance(policy, Policy) else policy_of(policy)
    _check(lib().pages_score_select(ctypes.byref(dims), _ptr(q), _ptr(summ), _ptr(seq_lens),
                                    ctypes.byref(pol), _ptr(sel), _ptr(nsel), k_max,
                                    _ptr(scores), _ptr(ws), ws.numel(), _stream(stream)))


def sparse_decode_attn(dims: Dims, q, K, V, page_table, seq_lens, sel, nsel, k_max: int, o, ws,
                       lse=None, num_splits: int = 0, softmax_scale: float | None = None,
                       stream=None):
    """Attention of the decode query over the selected pages (split-K, merged)."""
    scale = 1.0 / math.sqrt(dims.D) if softmax_scale is None else softmax_scale
    _check(lib().sparse_decode_attn(ctypes.byref(dims), _ptr(q), _ptr(K), _ptr(V), _ptr(page_table),
                                    _ptr(seq_lens), _ptr(sel), _ptr(nsel), k_max, num_splits,
                                    scale, _ptr(o), _ptr(lse), _ptr(ws), ws.numel(),
                                    _stream(stream)))


def sparse_decode_attn_noalloc(dims: Dims, q, K, V, page_table, seq_lens, sel, nsel, k_max: int, o,
                               lse=None, num_splits: int = 0, softmax_scale: float | None = None,
                               stream=None):
    """sparse_decode_attn without a workspace: its scratch is a fixed array inside the library."""
    scale = 1.0 / math.sqrt(dims.D) if softmax_scale is None else softmax_scale
    _check(lib().sparse_decode_attn_noalloc(ctypes.byref(dims), _ptr(q), _ptr(K), _ptr(V),
                                            _ptr(page_table), _ptr(seq_lens), _ptr(sel), _ptr(nsel),
                                            k_max, num_splits, scale, _ptr(o), _ptr(lse),
                                            _stream(stream)))


def dense_verify_attn(dims: Dims, T: int, q, K, V, page_table, seq_lens, o, ws, lse=None,
                      num_splits: int = 0, softmax_scale: float | None = None, stream=None):
    """Causal attention of the T newest positions over the whole cache."""
    scale = 1.0 / math.sqrt(dims.D) if softmax_scale is None else softmax_scale
    _check(lib().dense_verify_attn(ctypes.byref(dims), T, _ptr(q), _ptr(K), _ptr(V),
                                   _ptr(page_table), _ptr(seq_lens), num_splits, scale, _ptr(o),
                                   _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))


def lse_merge(part_o, part_lse, o, lse=None, stream=None):
    """Merge split partials (part_o [S][rows][D], part_lse [S][rows]) by the log-sum-exp rule."""
    S, rows, D = part_o.shape
    _check(lib().lse_merge(S, rows, D, _ptr(part_o), _ptr(part_lse), _ptr(o), _ptr(lse),
                           _stream(stream)))


_B16 = _I32 = _F32 = _U8 = _LOGITS = ()  # accepted types, set with torch's first use
_raw_stream = _device = None


def _here(stream):
    """The current device and the raw stream to launch on (the given one has to be of that device)."""
    if _device is None:
        _first_use()
    dev = _device()
    if stream is None:
        return dev, _raw_stream(dev)
    if stream.device.index != dev:
        raise SpdError(1, "the stream is not of the current CUDA device")
    return dev, stream.cuda_stream


def _first_use():
    global _raw_stream, _device, _B16, _I32, _F32, _U8, _LOGITS
    import torch
    _B16, _I32, _F32, _U8 = (torch.bfloat16, torch.uint16), (torch.int32,), (torch.float32,), (torch.uint8,)
    _LOGITS = (torch.float32, torch.bfloat16)
    if not torch.cuda.is_available():
        raise SpdError(3, "no CUDA device")
    torch.cuda.init()
    # the current device, and its stream's handle without a Stream object around it, as plain
    # numbers (1 us less a call)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _arg(t, dtypes, what: str, dev: int, numel: int | None = None, rows: bool = False):
    """The address of a tensor of device `dev`, its type and size checked (None passes).

    rows: a [..., heads, D] view whose heads and channels are contiguous and whose leading
    dimensions are one stride apart (a slice of a fused projection; see _row_stride)."""
    if t is None:
        return None
    if (t.dtype in dtypes and t.get_device() == dev and (numel is None or t.numel() == numel)
            and (rows or t.is_contiguous())):
        return t.data_ptr()
    if t.get_device() != dev:
        raise SpdError(1, f"{what} is not on the current CUDA device")
    if t.dtype not in dtypes:
        raise SpdError(1, f"{what} is {t.dtype}, not {' or '.join(map(str, dtypes))}")
    if numel is not None and t.numel() != numel:
        raise SpdError(1, f"{what} has {t.numel()} elements, not {numel}")
    raise SpdError(1, f"{what} is not contiguous")


def _row_stride(t, D: int, what: str) -> int:
    """Elements between the rows [heads][D] of a [..., heads, D] view (see _arg)."""
    shape, stride = t.shape, t.stride()
    dims = len(shape)
    if dims < 3 or shape[-1] != D:
        raise SpdError(1, f"{what} must be [..., heads, {D}], not {list(shape)}")
    if stride[-1] != 1 or (stride[-2] != D and shape[-2] > 1):
        raise SpdError(1, f"{what}: the heads and channels of a row must be contiguous")
    if dims == 3:
        return stride[0] if shape[0] > 1 else shape[1] * D
    if dims == 4 and shape[0] > 1 and (shape[1] == 1 or stride[0] == stride[1] * shape[1]):
        return stride[0] if shape[1] == 1 else stride[1]
    step, n = None, 1
    for size, s in zip(reversed(shape[:-2]), reversed(stride[:-2])):
        if size == 1:
            continue
        if step is None:
            step = s
        elif s != step * n:
            raise SpdError(1, f"{what}: the rows must be one stride apart")
        n *= size
    return step if step is not None else shape[-2] * D


def _rope_of(rope, q_weight, k_weight, eps: float, interleaved: bool, D: int, dev: int) -> Rope:
    n_pos, rot, table = 0, 0, None
    if rope is not None:
        shape = rope.shape
        if len(shape) != 3 or shape[1] != 2:
            raise SpdError(1, f"rope must be [n_pos, 2, rot_dim / 2], not {list(shape)}")
        n_pos, rot, table = shape[0], 2 * shape[2], _arg(rope, _F32, "rope", dev)
    return Rope(table, n_pos, rot, 1 if interleaved else 0, eps,
                None if q_weight is None else _arg(q_weight, _B16, "q_weight", dev, D),
                None if k_weight is None else _arg(k_weight, _B16, "k_weight", dev, D))


def qk_norm_rope(q, k, positions, rope, q_out, k_out, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, stream=None):
    """Norm and rotation of query rows q [..., H_q, D] and key rows k [..., H_kv, D] (either may be
    None) at positions [...]; rope fp32 [n_pos, 2, rot_dim / 2] (None: norm only)."""
    one = q if q is not None else k
    if one is None:
        raise SpdError(1, "q and k are both None")
    dev, st = _here(stream)
    D = one.shape[-1]
    rows = one.numel() // max(1, one.shape[-2] * D)
    r = _rope_of(rope, q_weight, k_weight, eps, interleaved, D, dev)
    hq = qs = hk = ks = 0
    qp = qo = kp = ko = None
    if q is not None:
        hq, qs = q.shape[-2], _row_stride(q, D, "q")
        qp = _arg(q, _B16, "q", dev, rows * hq * D, True)
        qo = _arg(q_out, _B16, "q_out", dev, rows * hq * D)
    if k is not None:
        hk, ks = k.shape[-2], _row_stride(k, D, "k")
        kp = _arg(k, _B16, "k", dev, rows * hk * D, True)
        ko = _arg(k_out, _B16, "k_out", dev, rows * hk * D)
    pos = _arg(positions, _I32, "positions", dev, rows) if r.rot_dim else None
    _check(lib().qk_norm_rope(rows, hq, hk, D, ctypes.byref(r), qp, qs, kp, ks, pos, qo, ko, st))


def kv_append_rope(dims: Dims, T: int, K, V, page_table, seq_lens, q, k, v, rope, q_out, summ, q_weight=None,
                   k_weight=None, eps: float = 1e-6, interleaved: bool = False, stream=None):
    """Norm and rotate the T newest tokens' keys into the paged cache (values as they are), rebuild
    their pages' summaries, and write the rotated queries to q_out; q and q_out may be None."""
    dev, st = _here(stream)
    B, D, H, pages = dims.B, dims.D, dims.H_kv, dims.max_pages_per_seq
    n, cache = B * T, dims.num_phys_pages * H * dims.page_size * D
    r = _rope_of(rope, q_weight, k_weight, eps, interleaved, D, dev)
    _check(lib().kv_append_rope(
        ctypes.byref(dims), T, ctypes.byref(r), _arg(K, _B16, "K", dev, cache), _arg(V, _B16, "V", dev, cache),
        _arg(page_table, _I32, "page_table", dev, B * pages), _arg(seq_lens, _I32, "seq_lens", dev, B),
        _arg(q, _B16, "q", dev, n * dims.H_q * D, True), 0 if q is None else _row_stride(q, D, "q"),
        _arg(k, _B16, "k", dev, n * H * D, True), _row_stride(k, D, "k"),
        _arg(v, _B16, "v", dev, n * H * D, True), _row_stride(v, D, "v"),
        _arg(q_out, _B16, "q_out", dev, n * dims.H_q * D), _arg(summ, _B16, "summ", dev, B * H * pages * 2 * D), st))


def kv4_cache(dims: Dims, device=None):
    """An empty 4-bit cache for these dims: uint8 [num_phys_pages][H_kv][2][page_size * D * 9 / 16]."""
    import torch
    return torch.zeros((dims.num_phys_pages, dims.H_kv, 2, dims.page_size * dims.D * 9 // 16),
                       dtype=torch.uint8, device=device or "cuda")


def _kv4(dims: Dims, kv4, dev: int):
    return _arg(kv4, _U8, "kv4", dev, dims.num_phys_pages * dims.H_kv * dims.page_size * dims.D * 9 // 8)


def kv4_append(dims: Dims, T: int, kv4, page_table, seq_lens, k_new, v_new, summ, k_exp: int = 0,
               v_exp: int = 0, stream=None):
    """Quantise the T newest tokens into the 4-bit cache and rebuild the summaries of their pages."""
    dev, st = _here(stream)
    B, pages = dims.B, dims.max_pages_per_seq
    row = dims.H_kv * dims.D
    _check(lib().kv4_append(
        ctypes.byref(dims), T, _kv4(dims, kv4, dev), k_exp, v_exp,
        _arg(page_table, _I32, "page_table", dev, B * pages), _arg(seq_lens, _I32, "seq_lens", dev, B),
        _arg(k_new, _B16, "k_new", dev, B * T * row), _arg(v_new, _B16, "v_new", dev, B * T * row),
        _arg(summ, _B16, "summ", dev, B * pages * 2 * row), st))


def kv4_read(dims: Dims, T: int, kv4, page_table, seq_lens, k_out, v_out, k_exp: int = 0, v_exp: int = 0,
             stream=None):
    """The T newest tokens of every sequence as the bf16 values that the 4-bit cache holds."""
    dev, st = _here(stream)
    B, n = dims.B, dims.B * T * dims.H_kv * dims.D
    _check(lib().kv4_read(
        ctypes.byref(dims), T, _kv4(dims, kv4, dev), k_exp, v_exp,
        _arg(page_table, _I32, "page_table", dev, B * dims.max_pages_per_seq),
        _arg(seq_lens, _I32, "seq_lens", dev, B), _arg(k_out, _B16, "k_out", dev, n),
        _arg(v_out, _B16, "v_out", dev, n), st))


def spd_kv4_sparse_decode_workspace_size(dims: Dims, k_max: int, num_splits: int = 0) -> int:
    """Bytes of workspace kv4_sparse_decode_attn needs."""
    return _size(lib().spd_kv4_sparse_decode_workspace_size(ctypes.byref(dims), k_max, num_splits),
                 "kv4_sparse_decode workspace")


def spd_kv4_dense_verify_workspace_size(dims: Dims, T: int, num_splits: int = 0) -> int:
    """Bytes of workspace kv4_dense_verify_attn needs for T positions."""
    return _size(lib().spd_kv4_dense_verify_workspace_size(ctypes.byref(dims), T, num_splits),
                 "kv4_dense_verify workspace")


def kv4_sparse_decode_attn(dims: Dims, q, kv4, page_table, seq_lens, sel, nsel, k_max: int, o, ws, lse=None,
                           num_splits: int = 0, softmax_scale: float | None = None, k_exp: int = 0,
                           v_exp: int = 0, stream=None):
    """sparse_decode_attn over the 4-bit cache."""
    dev, st = _here(stream)
    scale = 1.0 / math.sqrt(dims.D) if softmax_scale is None else softmax_scale
    B, D, H, rows = dims.B, dims.D, dims.H_kv, dims.B * dims.H_q
    _check(lib().kv4_sparse_decode_attn(
        ctypes.byref(dims), _arg(q, _B16, "q", dev, rows * D), _kv4(dims, kv4, dev), k_exp, v_exp,
        _arg(page_table, _I32, "page_table", dev, B * dims.max_pages_per_seq),
        _arg(seq_lens, _I32, "seq_lens", dev, B), _arg(sel, _I32, "sel", dev, B * H * k_max),
        _arg(nsel, _I32, "nsel", dev, B * H), k_max, num_splits, scale, _arg(o, _B16, "o", dev, rows * D),
        _arg(lse, _F32, "lse", dev, rows), _arg(ws, _U8, "ws", dev), ws.numel(), st))


def kv4_dense_verify_attn(dims: Dims, T: int, q, kv4, page_table, seq_lens, o, ws, lse=None,
                          num_splits: int = 0, softmax_scale: float | None = None, k_exp: int = 0,
                          v_exp: int = 0, stream=None):
    """dense_verify_attn over the 4-bit cache."""
    dev, st = _here(stream)
    scale = 1.0 / math.sqrt(dims.D) if softmax_scale is None else softmax_scale
    B, D, rows = dims.B, dims.D, dims.B * T * dims.H_q
    _check(lib().kv4_dense_verify_attn(
        ctypes.byref(dims), T, _arg(q, _B16, "q", dev, rows * D), _kv4(dims, kv4, dev), k_exp, v_exp,
        _arg(page_table, _I32, "page_table", dev, B * dims.max_pages_per_seq),
        _arg(seq_lens, _I32, "seq_lens", dev, B), num_splits, scale, _arg(o, _B16, "o", dev, rows * D),
        _arg(lse, _F32, "lse", dev, rows), _arg(ws, _U8, "ws", dev), ws.numel(), st))


def spd_token_logprobs_workspace_size(rows: int, n_vocab: int, top_k: int = 0) -> int:
    """Bytes of workspace token_logprobs needs."""
    return _size(lib().spd_token_logprobs_workspace_size(rows, n_vocab, top_k), "token_logprobs workspace")


def token_logprobs(logits, targets, logprobs, ws, entropy=None, lse=None, top_ids=None, top_logprobs=None,
                   inv_temperature: float = 1.0, stream=None):
    """Log probabilities of targets [...] under logits [..., n_vocab] (fp32 or bf16; rows may be one
    stride apart), with the optional entropy and lse [...] and the alternatives [..., top_k]."""
    dev, st = _here(stream)
    n = logits.shape[-1]
    rows = logits.numel() // max(1, n)
    step = n
    if logits.dim() == 2 and logits.stride(1) == 1:
        step = logits.stride(0) if rows > 1 else n
    elif logits.dim() > 1:  # as rows of one "head" of n channels
        step = _row_stride(logits.unsqueeze(-2), n, "logits")
    elif n > 1 and logits.stride(0) != 1:
        raise SpdError(1, "logits: a row must be contiguous")
    top_k = 0 if top_ids is None else top_ids.shape[-1]
    _check(lib().token_logprobs(
        rows, n, _arg(logits, _LOGITS, "logits", dev, None, True), 1 if logits.dtype is _LOGITS[1] else 0, step,
        _arg(targets, _I32, "targets", dev, rows), inv_temperature, _arg(logprobs, _F32, "logprobs", dev, rows),
        _arg(entropy, _F32, "entropy", dev, rows), _arg(lse, _F32, "lse", dev, rows), top_k,
        _arg(top_ids, _I32, "top_ids", dev, rows * top_k),
        _arg(top_logprobs, _F32, "top_logprobs", dev, rows * top_k), _arg(ws, _U8, "ws", dev), ws.numel(), st))


def spd_tree_verify_workspace_size(dims: Dims, T: int) -> int:
    """Bytes of workspace tree_verify_attn needs for trees of T nodes."""
    return _size(lib().spd_tree_verify_workspace_size(ctypes.byref(dims), T), "tree_verify workspace")


def tree_verify_attn(dims: Dims, T: int, q, K, V, page_table, seq_lens, k_tree, v_tree, parents, o, ws, lse=None,
                     softmax_scale: float | None = None, stream=None):
    """Attention of every node of a tree of drafted tokens over the cache, its ancestors and itself.

    q [B, T, H_q, D], k_tree and v_tree [B, T, H_kv, D] may be views of one projection; parents int32 [B, T];
    seq_lens counts the cache without the tree."""
    dev, st = _here(stream)
    scale = 1.0 / math.sqrt(dims.D) if softmax_scale is None else softmax_scale
    B, D, H, n = dims.B, dims.D, dims.H_kv, dims.B * T
    cache = dims.num_phys_pages * H * dims.page_size * D
    _check(lib().tree_verify_attn(
        ctypes.byref(dims), T, _arg(q, _B16, "q", dev, n * dims.H_q * D, True), _row_stride(q, D, "q"),
        _arg(K, _B16, "K", dev, cache), _arg(V, _B16, "V", dev, cache),
        _arg(page_table, _I32, "page_table", dev, B * dims.max_pages_per_seq),
        _arg(seq_lens, _I32, "seq_lens", dev, B), _arg(k_tree, _B16, "k_tree", dev, n * H * D, True),
        _row_stride(k_tree, D, "k_tree"), _arg(v_tree, _B16, "v_tree", dev, n * H * D, True),
        _row_stride(v_tree, D, "v_tree"), _arg(parents, _I32, "parents", dev, n), scale,
        _arg(o, _B16, "o", dev, n * dims.H_q * D), _arg(lse, _F32, "lse", dev, n * dims.H_q),
        _arg(ws, _U8, "ws", dev), ws.numel(), st))


def spec_accept_tree(q_target, draft, parents, u_acc, u_res, n_path, path, tokens, stream=None):
    """The accepted path through a tree: q_target fp32 [B, T, n], draft and parents int32 [B, T], u_acc [B, T],
    u_res [B]; writes n_path [B], path and tokens [B, T]."""
    dev, st = _here(stream)
    if q_target.dim() != 3:
        raise SpdError(1, f"q_target must be [B, T, n_vocab], not {list(q_target.shape)}")
    B, T, n = q_target.shape
    _check(lib().spec_accept_tree(
        B, T, n, _arg(q_target, _F32, "q_target", dev), _arg(draft, _I32, "draft", dev, B * T),
        _arg(parents, _I32, "parents", dev, B * T), _arg(u_acc, _F32, "u_acc", dev, B * T),
        _arg(u_res, _F32, "u_res", dev, B), _arg(n_path, _I32, "n_path", dev, B), _arg(path, _I32, "path", dev, B * T),
        _arg(tokens, _I32, "tokens", dev, B * T), st))


def kv_append_path(dims: Dims, T: int, K, V, page_table, seq_lens, k_tree, v_tree, path, n_path, summ, new_lens,
                   stream=None):
    """Append the accepted nodes' keys and values (rows path[b, :n_path[b]] of k_tree, v_tree [B, T, H_kv, D]) to
    the cache, rebuild their pages' summaries, and write the new lengths."""
    dev, st = _here(stream)
    B, D, H, pages = dims.B, dims.D, dims.H_kv, dims.max_pages_per_seq
    n, cache = B * T * H * D, dims.num_phys_pages * H * dims.page_size * D
    _check(lib().kv_append_path(
        ctypes.byref(dims), T, _arg(K, _B16, "K", dev, cache), _arg(V, _B16, "V", dev, cache),
        _arg(page_table, _I32, "page_table", dev, B * pages), _arg(seq_lens, _I32, "seq_lens", dev, B),
        _arg(k_tree, _B16, "k_tree", dev, n, True), _row_stride(k_tree, D, "k_tree"),
        _arg(v_tree, _B16, "v_tree", dev, n, True), _row_stride(v_tree, D, "v_tree"),
        _arg(path, _I32, "path", dev, B * T), _arg(n_path, _I32, "n_path", dev, B),
        _arg(summ, _B16, "summ", dev, B * H * pages * 2 * D), _arg(new_lens, _I32, "new_lens", dev, B), st))


def kv_weights_update(dims: Dims, T: int, q, lse, K, page_table, seq_lens, w_out, w_in=None, path=None, n_path=None,
                      sel=None, nsel=None, decay: float = 1.0, softmax_scale: float | None = None, stream=None):
    """Add the newest queries' attention weights to those of the cached tokens, w [B, H_kv, max_pages * page_size]
    (w_in may be w_out, or None for weights that start at 0)."""
    dev, st = _here(stream)
    scale = 1.0 / math.sqrt(dims.D) if softmax_scale is None else softmax_scale
    B, D, H, pages, rows = dims.B, dims.D, dims.H_kv, dims.max_pages_per_seq, dims.B * T * dims.H_q
    n_w = B * H * pages * dims.page_size
    k_max = 0 if sel is None else sel.shape[-1]
    _check(lib().kv_weights_update(
        ctypes.byref(dims), T, _arg(q, _B16, "q", dev, rows * D), _arg(lse, _F32, "lse", dev, rows),
        _arg(K, _B16, "K", dev, dims.num_phys_pages * H * dims.page_size * D),
        _arg(page_table, _I32, "page_table", dev, B * pages), _arg(seq_lens, _I32, "seq_lens", dev, B),
        _arg(path, _I32, "path", dev, B * T), _arg(n_path, _I32, "n_path", dev, B),
        _arg(sel, _I32, "sel", dev, B * H * k_max), _arg(nsel, _I32, "nsel", dev, B * H), k_max, decay, scale,
        _arg(w_in, _F32, "w_in", dev, n_w), _arg(w_out, _F32, "w_out", dev, n_w), st))


def kv_evict(dims: Dims, budget: int, n_sink: int, n_recent: int, K, V, page_table, seq_lens, weights, dst_table,
             kept, weights_out, summ, new_lens, stream=None):
    """Copy the `budget` tokens of each KV head that stay (the first n_sink, the newest n_recent, and those of the
    largest weights) to the pages of dst_table; kept int32 [B, H_kv, budget] gets their old positions."""
    dev, st = _here(stream)
    B, D, H, pages = dims.B, dims.D, dims.H_kv, dims.max_pages_per_seq
    n_w, cache = B * H * pages * dims.page_size, dims.num_phys_pages * H * dims.page_size * D
    _check(lib().kv_evict(
        ctypes.byref(dims), budget, n_sink, n_recent, _arg(K, _B16, "K", dev, cache), _arg(V, _B16, "V", dev, cache),
        _arg(page_table, _I32, "page_table", dev, B * pages), _arg(seq_lens, _I32, "seq_lens", dev, B),
        _arg(weights, _F32, "weights", dev, n_w), _arg(dst_table, _I32, "dst_table", dev, B * pages),
        _arg(kept, _I32, "kept", dev, B * H * budget), _arg(weights_out, _F32, "weights_out", dev, n_w),
        _arg(summ, _B16, "summ", dev, B * H * pages * 2 * D), _arg(new_lens, _I32, "new_lens", dev, B), st))


class Round:
    """spd_round: one S3R round (k sparse draft steps, verification, sampling) as two
    CUDA graphs built by the library.  Takes device tensors laid out as include/spd.h
    states; keeps them referenced while the round lives.  ``sampling`` is None or a dict
    with p_draft, q_target, draft_tokens, u_acc, u_res, n_accepted, tokens."""

    def __init__(self, dims: Dims, k: int, K, V, summ, page_table, seq_lens, q_draft, k_draft,
                 v_draft, q_verify, k_verify, v_verify, policy, k_max: int, sel, nsel, o_draft,
                 o_verify, ws_select, ws_sparse, ws_verify, lse_draft=None, lse_verify=None,
                 sampling=None, sparse_splits: int = 0, verify_splits: int = 0,
                 softmax_scale: float | None = None):
        pol = policy if isinstance(policy, Policy) else policy_of(policy)
        scale = 1.0 / math.sqrt(dims.D) if softmax_scale is None else softmax_scale
        smp = sampling or {}
        self._keep = [K, V, summ, page_table, seq_lens, q_draft, k_draft, v_draft, q_verify,
                      k_verify, v_verify, sel, nsel, o_draft, o_verify, ws_select, ws_sparse,
                      ws_verify, lse_draft, lse_verify, *smp.values()]
        n_vocab = int(smp["q_target"].shape[-1]) if smp else 0
        g = lambda name: _ptr(smp.get(name))
        d = RoundDesc(dims, k, _ptr(K), _ptr(V), _ptr(summ), _ptr(page_table), _ptr(seq_lens),
                      _ptr(q_draft), _ptr(k_draft), _ptr(v_draft), _ptr(q_verify), _ptr(k_verify),
                      _ptr(v_verify), pol, k_max, _ptr(sel), _ptr(nsel), _ptr(o_draft),
                      _ptr(lse_draft), _ptr(o_verify), _ptr(lse_verify), n_vocab,
                      g("p_draft"), g("q_target"), g("draft_tokens"), g("u_acc"), g("u_res"),
                      g("n_accepted"), g("tokens"),
                      _ptr(ws_select), ws_select.numel(), _ptr(ws_sparse), ws_sparse.numel(),
                      _ptr(ws_verify), ws_verify.numel(), sparse_splits, verify_splits, scale)
        h = ctypes.c_void_p()
        _check(lib().spd_round_create(ctypes.byref(d), ctypes.byref(h)))
        self._h = h

    def launch(self, part: int = 2, stream=None):
        """Replay part 0 (draft steps), 1 (verification + sampling) or 2 (both)."""
        _check(lib().spd_round_launch(self._h, part, _stream(stream)))

    def close(self):
        if getattr(self, "_h", None):
            lib().spd_round_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
