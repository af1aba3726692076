"""ctypes binding of libfa_gb300.so (include/fa.h): argument marshalling only.

The functions named like the C entry points (``fa_fwd``, ``fa_bwd``, ...) pass raw
device pointers straight through.  ``forward`` / ``backward`` are conveniences that
take torch CUDA tensors, allocate the outputs and the workspace with torch and call
the same entry points on torch's current stream.  Every step of the computation runs
in the library's kernels; there is no CPU path.  Loading fails loudly when the
library is missing or cannot be built.
"""
from __future__ import annotations

import ctypes
import operator
import os
import threading

from . import build as _build

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_WORKSPACE = 3
FA_ERR_CUDA = 4
FA_ERR_TIMEOUT = 5
FA_ERR_DEVICE_CHECK = 6

FA_FLAG_VALIDATE_CU = 1
FA_FLAG_NO_SPLIT = 2
FA_FLAG_DETERMINISTIC = 4
FA_DTYPE_BF16 = 0
FA_DTYPE_E4M3 = 1
FA_DTYPE_F16 = 2

EXPORTS = ("fa_fwd", "fa_bwd", "fa_fwd_workspace_size", "fa_bwd_workspace_size", "fa_read_device_status",
           "fa_status_string", "fa_profile_enable", "fa_profile_read", "fa_version", "fa_fwd_noalloc",
           "fa_qk_norm_rope", "fa_qk_norm_rope_bwd", "fa_qk_norm_rope_bwd_workspace_size", "fa_page_plan",
           "fa_qk_norm_rope_append8")

FA_ROPE_MAX_AXES = 4
FA_ROPE_MAX_PAIRS = 128

FA_NOALLOC_SCRATCH_BYTES = 64 << 20


class FaParams(ctypes.Structure):
    """Mirror of ``fa_params``."""
    _fields_ = [
        ("B", ctypes.c_int), ("s_q", ctypes.c_int), ("s_kv", ctypes.c_int),
        ("h_q", ctypes.c_int), ("h_kv", ctypes.c_int), ("d", ctypes.c_int),
        ("softmax_scale", ctypes.c_float), ("causal", ctypes.c_int),
        ("window_left", ctypes.c_int), ("window_right", ctypes.c_int),
        ("sinks", ctypes.c_void_p), ("cu_seqlens_q", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p),
        ("max_seqlen_q", ctypes.c_int), ("max_seqlen_k", ctypes.c_int), ("flags", ctypes.c_uint),
        ("seqused_k", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("page_size", ctypes.c_int),
        ("max_blocks_per_seq", ctypes.c_int), ("num_pages", ctypes.c_int),
        ("dtype", ctypes.c_int), ("q_descale", ctypes.c_void_p), ("k_descale", ctypes.c_void_p),
        ("v_descale", ctypes.c_void_p), ("seqused_q", ctypes.c_void_p),
        ("wait_limit_ns", ctypes.c_ulonglong), ("cache_dtype", ctypes.c_int), ("scale_block", ctypes.c_int),
        ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
    ]


class FaRopeParams(ctypes.Structure):
    """Mirror of ``fa_rope_params``."""
    _fields_ = [
        ("T", ctypes.c_int), ("h_q", ctypes.c_int), ("h_kv", ctypes.c_int), ("d", ctypes.c_int),
        ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("seq_len", ctypes.c_int), ("max_pos", ctypes.c_int),
        ("eps", ctypes.c_float), ("dtype", ctypes.c_int), ("weight_f32", ctypes.c_int),
        ("q_stride", ctypes.c_longlong), ("k_stride", ctypes.c_longlong), ("v_stride", ctypes.c_longlong),
        ("dq_stride", ctypes.c_longlong), ("dk_stride", ctypes.c_longlong),
        ("positions", ctypes.c_void_p), ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p),
        ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("slots", ctypes.c_void_p),
        ("num_slots", ctypes.c_longlong), ("status", ctypes.c_void_p), ("zero_skipped", ctypes.c_int),
        ("wait_limit_ns", ctypes.c_ulonglong), ("axes", ctypes.c_int), ("no_norm", ctypes.c_int),
        ("pair_axis", ctypes.c_ubyte * FA_ROPE_MAX_PAIRS),
    ]


class FaCache8Params(ctypes.Structure):
    """Mirror of ``fa_cache8_params``."""
    _fields_ = [("B", ctypes.c_int), ("page_size", ctypes.c_int), ("max_blocks_per_seq", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("scale_block", ctypes.c_int), ("cu_seqlens_q", ctypes.c_void_p), ("seqused_k", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p)]


class FaPagePlanParams(ctypes.Structure):
    """Mirror of ``fa_page_plan_params``."""
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("page_size", ctypes.c_int),
                ("max_blocks_per_seq", ctypes.c_int), ("num_pages", ctypes.c_int), ("n_free", ctypes.c_int)]


class FaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {fa_status_string(code)} (status {code})")


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Loads (building first if stale) the CUDA library; raises if that is impossible.

    With FA_TRACE=1 in the environment the trace build (libfa_gb300_trace.so, whose
    kernels record per-role event traces into the workspace; see trace.py) is loaded
    instead of the product library."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        trace = os.environ.get("FA_TRACE", "") == "1"
        path = _build.TRACE_LIB if trace else _build.LIB
        if build_if_missing:
            _build.build(trace=trace)
        if not os.path.exists(path):
            raise RuntimeError(f"CUDA library {path} is missing; run exact_attention_bwd_gb300/build.py")
        lib = ctypes.CDLL(path)
        P = ctypes.POINTER(FaParams)
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        lib.fa_fwd.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.fa_fwd.restype = ctypes.c_int
        lib.fa_bwd.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.fa_bwd.restype = ctypes.c_int
        lib.fa_fwd_workspace_size.argtypes = [P]
        lib.fa_fwd_workspace_size.restype = sz
        lib.fa_bwd_workspace_size.argtypes = [P]
        lib.fa_bwd_workspace_size.restype = sz
        lib.fa_read_device_status.argtypes = [vp, vp]
        lib.fa_read_device_status.restype = ctypes.c_int
        lib.fa_status_string.argtypes = [ctypes.c_int]
        lib.fa_status_string.restype = ctypes.c_char_p
        lib.fa_profile_enable.argtypes = [ctypes.c_int]
        lib.fa_profile_enable.restype = ctypes.c_int
        lib.fa_profile_read.argtypes = [ctypes.c_char_p, ctypes.POINTER(ctypes.c_float)]
        lib.fa_profile_read.restype = ctypes.c_int
        lib.fa_fwd_noalloc.argtypes = [P, vp, vp, vp, vp, vp, vp]
        lib.fa_fwd_noalloc.restype = ctypes.c_int
        R, L = ctypes.POINTER(FaRopeParams), ctypes.POINTER(FaPagePlanParams)
        lib.fa_qk_norm_rope.argtypes = [R] + [vp] * 8
        lib.fa_qk_norm_rope.restype = ctypes.c_int
        lib.fa_qk_norm_rope_bwd.argtypes = [R] + [vp] * 9 + [sz, vp]
        lib.fa_qk_norm_rope_bwd.restype = ctypes.c_int
        lib.fa_qk_norm_rope_bwd_workspace_size.argtypes = [R]
        lib.fa_qk_norm_rope_bwd_workspace_size.restype = sz
        lib.fa_qk_norm_rope_append8.argtypes = [R, ctypes.POINTER(FaCache8Params)] + [vp] * 9
        lib.fa_qk_norm_rope_append8.restype = ctypes.c_int
        lib.fa_page_plan.argtypes = [L] + [vp] * 12
        lib.fa_page_plan.restype = ctypes.c_int
        lib.fa_version.argtypes = []
        lib.fa_version.restype = ctypes.c_char_p
        _lib = lib
        return lib


# ----------------------------------------------------------------------------------------------
# raw entry points (same names as the C ABI)
# ----------------------------------------------------------------------------------------------

def fa_fwd(params: FaParams, q, k, v, o, lse, workspace, workspace_bytes, stream) -> int:
    return load().fa_fwd(ctypes.byref(params), q, k, v, o, lse, workspace, workspace_bytes, stream)


def fa_fwd_noalloc(params: FaParams, q, k, v, o, lse, stream) -> int:
    """fa_fwd on the library's built-in scratch array: for callers that cannot allocate."""
    return load().fa_fwd_noalloc(ctypes.byref(params), q, k, v, o, lse, stream)


def fa_bwd(params: FaParams, q, k, v, o, lse, dout, dq, dk, dv, dsinks, workspace, workspace_bytes,
           stream) -> int:
    return load().fa_bwd(ctypes.byref(params), q, k, v, o, lse, dout, dq, dk, dv, dsinks, workspace,
                         workspace_bytes, stream)


def fa_fwd_workspace_size(params: FaParams) -> int:
    return int(load().fa_fwd_workspace_size(ctypes.byref(params)))


def fa_bwd_workspace_size(params: FaParams) -> int:
    return int(load().fa_bwd_workspace_size(ctypes.byref(params)))


def fa_qk_norm_rope(params: FaRopeParams, q, k, v, q_out, k_out, k_cache, v_cache, stream) -> int:
    return load().fa_qk_norm_rope(ctypes.byref(params), q, k, v, q_out, k_out, k_cache, v_cache, stream)


def fa_qk_norm_rope_bwd_workspace_size(params: FaRopeParams) -> int:
    return int(load().fa_qk_norm_rope_bwd_workspace_size(ctypes.byref(params)))


def fa_qk_norm_rope_bwd(params: FaRopeParams, q, k, dq_out, dk_out, dq, dk, dq_weight, dk_weight, workspace, workspace_bytes,
                        stream) -> int:
    return load().fa_qk_norm_rope_bwd(ctypes.byref(params), q, k, dq_out, dk_out, dq, dk, dq_weight, dk_weight, workspace,
                                      workspace_bytes, stream)


def fa_qk_norm_rope_append8(params: FaRopeParams, cache: FaCache8Params, q, k, v, q_out, k_cache, v_cache, k_scale, v_scale,
                            stream) -> int:
    return load().fa_qk_norm_rope_append8(ctypes.byref(params), ctypes.byref(cache), q, k, v, q_out, k_cache, v_cache, k_scale,
                                          v_scale, stream)


def fa_page_plan(params: FaPagePlanParams, cached, fresh, free_pages, free_head, block_table, cu_seqlens_q, seqused_k,
                 positions, slots, free_head_out, status, stream) -> int:
    return load().fa_page_plan(ctypes.byref(params), cached, fresh, free_pages, free_head, block_table, cu_seqlens_q,
                               seqused_k, positions, slots, free_head_out, status, stream)


def fa_read_device_status(workspace, stream) -> int:
    return load().fa_read_device_status(workspace, stream)


def fa_status_string(code: int) -> str:
    return load().fa_status_string(code).decode()


def fa_profile_enable(on: bool) -> int:
    return load().fa_profile_enable(1 if on else 0)


def fa_profile_read(kernel: str):
    ms = ctypes.c_float(0.0)
    rc = load().fa_profile_read(kernel.encode(), ctypes.byref(ms))
    return rc, float(ms.value)


def fa_version() -> str:
    return load().fa_version().decode()


# ----------------------------------------------------------------------------------------------
# torch conveniences: allocation and stream plumbing only
# ----------------------------------------------------------------------------------------------

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def make_params(q, k, *, causal=False, window=(-1, -1), softmax_scale=None, sinks=None, cu_q=None,
                cu_k=None, flags=0, seqused_k=None, block_table=None, s_kv=None, dtype=None, q_descale=None,
                k_descale=None, v_descale=None, seqused_q=None, wait_limit_ns=0, max_seqlen_q=0) -> FaParams:
    """fa_params from tensor shapes: [B,S,H,D] dense or [T,H,D] packed (with cu_q / cu_k).

    With a block_table ([B, max_blocks_per_seq] int32), k is a page pool
    [num_pages, page_size, h_kv, d] and s_kv (the logical cache length) must be given; q is
    dense, or packed with cu_q (then seqused_k must be given, and cu_k not).
    seqused_q / seqused_k: int32 [B] queries / keys used per sequence, or None."""
    if block_table is not None:
        if cu_q is not None:
            (s_q, h_q, d), B = q.shape, cu_q.numel() - 1
        else:
            B, s_q, h_q, d = q.shape
        num_pages, page_size, h_kv, _ = k.shape
        if s_kv is None:
            raise ValueError("a paged cache needs the logical cache length s_kv")
    elif cu_q is None:
        B, s_q, h_q, d = q.shape
        _, s_kv, h_kv, _ = k.shape
    else:
        T_q, h_q, d = q.shape
        T_k, h_kv, _ = k.shape
        B, s_q, s_kv = cu_q.numel() - 1, T_q, T_k
    p = FaParams()
    p.B, p.s_q, p.s_kv, p.h_q, p.h_kv, p.d = B, s_q, s_kv, h_q, h_kv, d
    p.softmax_scale = float(softmax_scale) if softmax_scale else 0.0
    p.causal = 1 if causal else 0
    p.window_left, p.window_right = int(window[0]), int(window[1])
    p.sinks = None if sinks is None else sinks.data_ptr()
    p.cu_seqlens_q = None if cu_q is None else cu_q.data_ptr()
    p.cu_seqlens_k = None if cu_k is None else cu_k.data_ptr()
    p.max_seqlen_q, p.max_seqlen_k = int(max_seqlen_q), 0
    p.flags = flags
    p.seqused_k = None if seqused_k is None else seqused_k.data_ptr()
    p.seqused_q = None if seqused_q is None else seqused_q.data_ptr()
    p.dtype = FA_DTYPE_BF16 if dtype is None else int(dtype)
    p.q_descale = None if q_descale is None else q_descale.data_ptr()
    p.k_descale = None if k_descale is None else k_descale.data_ptr()
    p.v_descale = None if v_descale is None else v_descale.data_ptr()
    p.wait_limit_ns = int(wait_limit_ns)
    if block_table is not None:
        p.block_table = block_table.data_ptr()
        p.page_size, p.num_pages = int(page_size), int(num_pages)
        p.max_blocks_per_seq = int(block_table.shape[1])
    return p


_type_codes = {}


def _type_code(t):
    """FA_DTYPE_* code of a torch dtype, or None when the library does not take it."""
    if not _type_codes:
        import torch
        _type_codes.update({torch.bfloat16: FA_DTYPE_BF16, torch.float16: FA_DTYPE_F16, torch.uint8: FA_DTYPE_E4M3})
    return _type_codes.get(t)


def _stream():
    """torch's current stream of the current device, as the C ABI takes it."""
    import torch
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _check_tensors(q, named):
    """Every tensor handed to the library: on q's CUDA device (the C ABI takes plain device
    pointers; a host pointer there would be dereferenced by the kernels), contiguous (the
    layouts are dense [B, S, H, D], [T, H, D] or the stated vectors), with the given element
    type and element count or shape.  named: (name, tensor or None, dtype, shape or count)."""
    import torch
    if q.device.type != "cuda":
        raise ValueError(f"q must be a CUDA tensor; it is on {q.device}")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    for name, t, dtype, want in named:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if t.device != q.device:
            raise ValueError(f"{name} is on {t.device}; every tensor must be on q's device {q.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}; it is {t.dtype}")
        if isinstance(want, int):
            if t.numel() != want:
                raise ValueError(f"{name} must have {want} elements; it has {t.numel()}")
        elif want is not None and tuple(t.shape) != tuple(want):
            raise ValueError(f"{name} must have shape {tuple(want)}; it has {tuple(t.shape)}")


def _vector_args(p, sinks, cu_q, cu_k, seqused_q, seqused_k):
    """The optional per-head / per-sequence vectors of a call, for _check_tensors."""
    import torch
    i32, f32 = torch.int32, torch.float32
    return [("sinks", sinks, f32, p.h_q), ("cu_q", cu_q, i32, p.B + 1), ("cu_k", cu_k, i32, p.B + 1),
            ("seqused_q", seqused_q, i32, p.B), ("seqused_k", seqused_k, i32, p.B)]


def _kv_shape(p, k, cu_q, block_table):
    """The shape k must have: [B, s_kv, h_kv, d] dense, [T_k, h_kv, d] packed, or a page pool
    [num_pages, page_size, h_kv, d]; B and d are q's (so no kernel reads past k's end)."""
    if block_table is not None:
        return (p.num_pages, p.page_size, p.h_kv, p.d)
    if cu_q is not None:
        return (p.s_kv, p.h_kv, p.d)
    return (p.B, p.s_kv, p.h_kv, p.d)


def forward(q, k, v, *, causal=False, window=(-1, -1), softmax_scale=None, sinks=None, cu_q=None, cu_k=None,
            flags=0, out=None, lse=None, workspace=None, seqused_k=None, block_table=None, s_kv=None,
            descale=None, seqused_q=None, wait_limit_ns=0, max_seqlen_q=0, cache_scale=None):
    """Runs fa_fwd on torch CUDA tensors; returns (o, lse, workspace).

    Packed queries over a paged cache: q [T, h_q, d] with cu_q, seqused_k, block_table and s_kv
    (no cu_k); max_seqlen_q is the most new tokens of a sequence, if the caller knows it.  Rows that no
    sequence covers are not written, in given tensors or in those made here.  cache_scale = (k_scale,
    v_scale), fp32 [num_pages, page_size / scale_block, h_kv], with k and v uint8 (e4m3 bytes) is the
    same over a cache in 8 bits, as qk_norm_rope_append8 fills it; q is bfloat16 or float16.

    q, k, v are all bfloat16, all float16, or all uint8 = e4m3 bytes (FA_DTYPE_E4M3);
    descale = (q, k, v) fp32 [B * h_kv] factors or None (all 1).  The output has the
    inputs' type (bf16 for e4m3 inputs)."""
    import torch
    if block_table is not None and cu_q is not None and cu_k is None:
        if descale is not None:
            raise TypeError("descale factors apply to e4m3 (uint8) inputs only")
        return _forward_paged(q, k, v, causal, window, softmax_scale, sinks, cu_q, flags, out, lse, workspace, seqused_k,
                              block_table, s_kv, seqused_q, wait_limit_ns, max_seqlen_q, cache_scale)
    if cache_scale is not None:
        raise ValueError("cache_scale goes with packed queries over a paged cache (cu_q, seqused_k and block_table, no cu_k)")
    fp8 = q.dtype == torch.uint8
    if _type_code(q.dtype) is None or k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must all be bfloat16, all float16 or all uint8 (e4m3 bytes); "
                        f"got {q.dtype}, {k.dtype}, {v.dtype}")
    if descale is not None and not fp8:
        raise TypeError("descale factors apply to e4m3 (uint8) inputs only")
    dq_, dk_, dv_ = descale if descale is not None else (None, None, None)
    p = make_params(q, k, causal=causal, window=window, softmax_scale=softmax_scale, sinks=sinks, cu_q=cu_q,
                    cu_k=cu_k, flags=flags, seqused_k=seqused_k, block_table=block_table, s_kv=s_kv,
                    dtype=_type_code(q.dtype), q_descale=dq_, k_descale=dk_, v_descale=dv_,
                    seqused_q=seqused_q, wait_limit_ns=wait_limit_ns)
    lse_shape = (p.B, p.h_q, p.s_q) if cu_q is None else (p.h_q, p.s_q)
    _check_tensors(q, [("k", k, None, _kv_shape(p, k, cu_q, block_table)), ("v", v, None, k.shape),
                       ("out", out, torch.bfloat16 if fp8 else q.dtype, q.shape), ("lse", lse, torch.float32, lse_shape),
                       ("workspace", workspace, torch.uint8, None),
                       ("block_table", block_table, torch.int32, None if block_table is None else
                        (p.B, p.max_blocks_per_seq)),
                       ("q_descale", dq_, torch.float32, p.B * p.h_kv), ("k_descale", dk_, torch.float32, p.B * p.h_kv),
                       ("v_descale", dv_, torch.float32, p.B * p.h_kv)]
                   + _vector_args(p, sinks, cu_q, cu_k, seqused_q, seqused_k))
    nbytes = fa_fwd_workspace_size(p)
    if nbytes == 0:
        raise FaError(FA_ERR_UNSUPPORTED, "fa_fwd_workspace_size")
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16 if fp8 else q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty(lse_shape, dtype=torch.float32, device=q.device)
    rc = fa_fwd(p, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), _stream())
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd")
    return out, lse, workspace


def backward(q, k, v, o, lse, dout, *, causal=False, window=(-1, -1), softmax_scale=None, sinks=None,
             cu_q=None, cu_k=None, flags=0, workspace=None, grads=None, seqused_q=None, seqused_k=None,
             wait_limit_ns=0):
    """Runs fa_bwd on torch CUDA tensors; returns (dq, dk, dv, dsinks, workspace).

    q, k, v, o, dout (and dq, dk, dv when given) are all bfloat16 or all float16."""
    import torch
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"the backward takes bfloat16 or float16 tensors; q is {q.dtype}")
    named = [("k", k), ("v", v), ("o", o), ("dout", dout)]
    if grads is not None:
        named += [("dq", grads[0]), ("dk", grads[1]), ("dv", grads[2])]
    for name, t in named:
        if t.dtype != q.dtype:
            raise TypeError(f"the backward's tensors must share q's type {q.dtype}; {name} is {t.dtype}")
    p = make_params(q, k, causal=causal, window=window, softmax_scale=softmax_scale, sinks=sinks, cu_q=cu_q,
                    cu_k=cu_k, flags=flags, seqused_q=seqused_q, seqused_k=seqused_k, dtype=_type_code(q.dtype),
                    wait_limit_ns=wait_limit_ns)
    lse_shape = (p.B, p.h_q, p.s_q) if cu_q is None else (p.h_q, p.s_q)
    g = (None, None, None, None) if grads is None else tuple(grads)
    _check_tensors(q, [("k", k, None, _kv_shape(p, k, cu_q, None)), ("v", v, None, k.shape), ("o", o, None, q.shape),
                       ("lse", lse, torch.float32, lse_shape), ("dout", dout, None, q.shape),
                       ("dq", g[0], None, q.shape), ("dk", g[1], None, k.shape), ("dv", g[2], None, k.shape),
                       ("dsinks", g[3], torch.float32, p.h_q), ("workspace", workspace, torch.uint8, None)]
                   + _vector_args(p, sinks, cu_q, cu_k, seqused_q, seqused_k))
    if lse is None:
        raise ValueError("the backward needs the forward's lse")
    nbytes = fa_bwd_workspace_size(p)
    if nbytes == 0:
        raise FaError(FA_ERR_UNSUPPORTED, "fa_bwd_workspace_size")
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    if grads is None:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dsinks = None if sinks is None else torch.empty_like(sinks)
    else:
        dq, dk, dv, dsinks = grads
    rc = fa_bwd(p, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                _ptr(dsinks), _ptr(workspace), workspace.numel(), _stream())
    if rc != FA_OK:
        raise FaError(rc, "fa_bwd")
    return dq, dk, dv, dsinks, workspace


def _on_device(t, call, *args, **kw):
    """call(*args, **kw) with t's device current (the library launches on the current device)."""
    import torch
    with torch.cuda.device(t.device):
        return call(*args, **kw)


def _device_index(t):
    """The index of t's CUDA device."""
    try:
        i = t.get_device()
    except AttributeError:
        raise TypeError(f"a torch tensor is wanted, not {type(t).__name__}") from None
    if i < 0:
        raise ValueError(f"the tensors must be CUDA tensors; one is on {t.device}")
    return i


def _check(dev, *named):
    """Each (name, tensor or None, dtype, size): a contiguous tensor of that type on device `dev`, of the
    shape `size`, or where that is a number, of so many elements.  The calls of a serving step are short,
    so this is written for speed: one expression a tensor, the wording only where it fails."""
    for name, t, dtype, size in named:
        if t is None or (t.dtype is dtype and t.get_device() == dev and (t.numel() if type(size) is int else t.shape) == size
                         and t.is_contiguous()):
            continue
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}; every tensor must be on device {dev}")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}; it is {t.dtype}")
        if type(size) is int:
            if t.numel() != size:
                raise ValueError(f"{name} must have {size} elements; it has {t.numel()}")
        elif t.shape != size:
            raise ValueError(f"{name} must have the shape {tuple(size)}; it has {tuple(t.shape)}")
        raise ValueError(f"{name} must be contiguous")


def _forward_paged(q, k, v, causal, window, softmax_scale, sinks, cu_q, flags, out, lse, workspace, seqused_k, block_table, s_kv,
                   seqused_q, wait_limit_ns, max_seqlen_q, cache_scale):
    """forward() for packed queries over a paged cache."""
    import torch
    dev = _device_index(q)
    if dev != torch._C._cuda_getDevice():
        return _on_device(q, _forward_paged, q, k, v, causal, window, softmax_scale, sinks, cu_q, flags, out, lse, workspace,
                          seqused_k, block_table, s_kv, seqused_q, wait_limit_ns, max_seqlen_q, cache_scale)
    kind = q.dtype
    code = _type_code(kind)
    if code is None:
        raise TypeError(f"q, k, v must all be bfloat16 or all float16; q is {kind}")
    if q.dim() != 3 or k.dim() != 4 or block_table.dim() != 2:
        raise ValueError("q must be [T, h_q, d], k and v [num_pages, page_size, h_kv, d], block_table [B, max_blocks_per_seq]")
    if s_kv is None or seqused_k is None:
        raise ValueError("packed queries over a paged cache need seqused_k and the longest cache's length s_kv")
    T, h_q, d = q.shape
    num_pages, page_size, h_kv, dk = k.shape
    B, blocks = block_table.shape
    if dk != d or v.shape != k.shape:
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} must have one shape and q's head dimension {d}")
    i32, f32 = torch.int32, torch.float32
    stored = kind
    if cache_scale is not None:
        if code == FA_DTYPE_E4M3:
            raise TypeError("over a cache in 8 bits q is bfloat16 or float16")
        stored, (k_scale, v_scale) = torch.uint8, cache_scale
        block = _cache8(dev, k, v, k_scale, v_scale, h_kv, d)[2]
    _check(dev, ("q", q, kind, T * h_q * d), ("k", k, stored, k.numel()), ("v", v, stored, v.numel()), ("cu_q", cu_q, i32, B + 1),
           ("seqused_k", seqused_k, i32, B), ("block_table", block_table, i32, B * blocks), ("sinks", sinks, f32, h_q),
           ("seqused_q", seqused_q, i32, B))
    if out is not None or lse is not None or workspace is not None:
        _check(dev, ("out", out, kind, q.shape), ("lse", lse, f32, (h_q, T)),
               ("workspace", workspace, torch.uint8, 0 if workspace is None else workspace.numel()))
    lib = load()
    p = FaParams(B, T, s_kv, h_q, h_kv, d, softmax_scale or 0.0, 1 if causal else 0, window[0], window[1],
                 None if sinks is None else sinks.data_ptr(), cu_q.data_ptr(), None, max_seqlen_q, 0, flags, seqused_k.data_ptr(),
                 block_table.data_ptr(), page_size, blocks, num_pages, code, None, None, None,
                 None if seqused_q is None else seqused_q.data_ptr(), wait_limit_ns)
    if cache_scale is not None:
        p.cache_dtype, p.scale_block, p.k_scale, p.v_scale = FA_DTYPE_E4M3, block, k_scale.data_ptr(), v_scale.data_ptr()
    ref = ctypes.byref(p)
    nbytes = lib.fa_fwd_workspace_size(ref)
    if nbytes == 0:
        raise FaError(FA_ERR_UNSUPPORTED, "fa_fwd_workspace_size")
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(h_q, T, dtype=f32, device=q.device)
    rc = lib.fa_fwd(ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                    workspace.numel(), torch._C._cuda_getCurrentRawStream(dev))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd")
    return out, lse, workspace


def _rows(name, t):
    """(tokens, heads, d, elements from token to token) of [T, h, d] or [B, S, h, d] rows, whose
    heads are contiguous and whose tokens lie at one stride (a slice of a fused projection)."""
    shape, st = t.shape, t.stride()
    if len(st) == 3:
        T, h, d = shape
        if T > 1 and st[2] == 1 and (h == 1 or st[1] == d):
            return T, h, d, st[0]
    elif len(st) != 4:
        raise ValueError(f"{name} must be [T, h, d] or [B, S, h, d]")
    h, d = shape[-2:]
    if t.numel() and (st[-1] != 1 or (h > 1 and st[-2] != d)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    T, step = shape[-3], st[-3]
    if len(shape) == 4:
        if shape[0] > 1 and T > 1 and st[0] != T * step:
            raise ValueError(f"{name}: the tokens must lie at one stride")
        if T == 1:
            step = st[0]
        T *= shape[0]
    return T, h, d, step if T > 1 else h * d


def _like(name, t, kind, dev):
    """t has q's type and device."""
    if t.dtype is not kind or t.get_device() != dev:
        raise TypeError(f"{name} must have the type and device of q")


def _set_axes(p, positions, pair_axis, norm):
    """The parameters' axes (positions [axes, T], the axis of each pair) and whether there is a norm."""
    p.no_norm = 0 if norm else 1
    if pair_axis is None:
        return
    p.axes = axes = positions.shape[0]
    if not 1 <= axes <= FA_ROPE_MAX_AXES:
        raise ValueError(f"positions must have 1 to {FA_ROPE_MAX_AXES} axes; they have {axes}")
    if len(pair_axis) != p.rot_dim // 2:
        raise ValueError(f"pair_axis must have {p.rot_dim // 2} entries, one for each pair; it has {len(pair_axis)}")
    try:
        # (bytes() of an array would be its memory, not its entries)
        pairs = bytes(pair_axis if isinstance(pair_axis, (tuple, list)) else list(map(operator.index, pair_axis)))
    except (TypeError, ValueError):
        pairs = b"\xff"
    if pairs.translate(None, b"\0\1\2\3"[:axes]):  # (what is left when the axes are taken out)
        raise ValueError(f"pair_axis must hold axes (0 to {axes - 1})")
    ctypes.memmove(p.pair_axis, pairs, len(pairs))


def _rope_params(dev, q, k, q_weight, k_weight, cos, sin, positions, seq_len, eps, interleaved, status, pair_axis, norm):
    import torch
    T, h_q, d, q_stride = _rows("q", q)
    kind = q.dtype
    _like("k", k, kind, dev)
    Tk, h_kv, dk, k_stride = _rows("k", k)
    code = _type_code(kind)
    if code is None or code == FA_DTYPE_E4M3:
        raise TypeError(f"q and k must be bfloat16 or float16; q is {kind}")
    if Tk != T or dk != d or k.dim() != q.dim() or k.shape[0] != q.shape[0]:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} must have the same tokens and head dimension")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    if pair_axis is not None and (positions is None or positions.dim() < 2):
        raise ValueError("pair_axis goes with positions [axes, T]")
    if not norm and (q_weight is not None or k_weight is not None):
        raise ValueError("without the norm there are no weights")
    max_pos = half = 0
    if cos is not None:
        max_pos, half = cos.shape
    wt = q_weight if q_weight is not None else k_weight
    wtype = kind if wt is None else wt.dtype
    if wtype is not kind and wtype is not torch.float32:
        raise TypeError(f"the weights must be {kind} or float32; they are {wtype}")
    _check(dev, ("cos", cos, torch.float32, (max_pos, half)), ("sin", sin, torch.float32, (max_pos, half)),
           ("q_weight", q_weight, wtype, d), ("k_weight", k_weight, wtype, d),
           ("positions", positions, torch.int32, T if pair_axis is None or positions is None else positions.shape[0] * T),
           ("status", status, torch.int32, 1))
    if seq_len is None:
        seq_len = max(1, q.shape[1] if q.dim() == 4 else T)
    p = FaRopeParams(T, h_q, h_kv, d, 2 * half, 1 if interleaved else 0, seq_len, max_pos, eps, code, 1 if wtype is not kind else 0,
                     q_stride, k_stride, h_kv * d, h_q * d, h_kv * d, None if positions is None else positions.data_ptr(),
                     None if cos is None else cos.data_ptr(), None if sin is None else sin.data_ptr(),
                     None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(),
                     None, 0, None if status is None else status.data_ptr())
    if not norm or pair_axis is not None:
        _set_axes(p, positions, pair_axis, norm)
    return p


def qk_norm_rope(q, k, q_weight, k_weight, cos, sin, *, positions=None, seq_len=None, eps=1e-6, interleaved=False,
                 v=None, k_cache=None, v_cache=None, slots=None, out=None, status=None, wait_limit_ns=0, pair_axis=None,
                 norm=True):
    """Runs fa_qk_norm_rope on torch CUDA tensors; returns (q_out, k_out).

    q [T, h_q, d] and k [T, h_kv, d] (or [B, S, h, d]) may be slices of a fused projection;
    q_weight, k_weight [d] (or None: ones) have their type or are fp32; cos, sin are fp32
    [max_pos, rot_dim / 2] (or None: no rotation); positions int32 [T], by default the token's
    place in its sequence of seq_len (S, or T).  positions int32 [axes, T] with pair_axis (a sequence:
    for each pair of the rotated part its axis) turn each pair by its own axis's position; norm=False leaves the norm
    out (no weights).  With v, k_cache, v_cache ([num_pages, page_size,
    h_kv, d]) and slots (int32 [T]) keys and values go to the paged cache, and k_out is None
    unless out = (q_out, k_out) gives one.  A padding token (position -1, or one outside the tables) is
    skipped: its rows are zero in the tensors made here, and left as they were in given ones and in the
    cache.  status: int32 [1] or None (bad positions and slots, and a wait past wait_limit_ns, are then not
    reported)."""
    import torch
    dev = _device_index(q)
    if dev != torch._C._cuda_getDevice():
        return _on_device(q, qk_norm_rope, q, k, q_weight, k_weight, cos, sin, positions=positions, seq_len=seq_len, eps=eps,
                          interleaved=interleaved, v=v, k_cache=k_cache, v_cache=v_cache, slots=slots, out=out, status=status,
                          wait_limit_ns=wait_limit_ns, pair_axis=pair_axis, norm=norm)
    p = _rope_params(dev, q, k, q_weight, k_weight, cos, sin, positions, seq_len, eps, interleaved, status, pair_axis, norm)
    p.wait_limit_ns = wait_limit_ns
    kind = q.dtype
    append = v is not None or k_cache is not None or v_cache is not None or slots is not None
    if append:
        if v is None or k_cache is None or v_cache is None or slots is None:
            raise ValueError("an append takes v, k_cache, v_cache and slots together")
        if v.shape != k.shape:
            raise ValueError(f"v must have k's shape {tuple(k.shape)}; it has {tuple(v.shape)}")
        _like("v", v, kind, dev)
        p.v_stride = _rows("v", v)[3]
        if k_cache.dim() != 4 or v_cache.shape != k_cache.shape or k_cache.shape[2:] != k.shape[-2:]:
            raise ValueError(f"k_cache {tuple(k_cache.shape)} and v_cache {tuple(v_cache.shape)} must be [num_pages, page_size, "
                             f"{p.h_kv}, {p.d}]")
        n = k_cache.numel()
        _check(dev, ("k_cache", k_cache, kind, n), ("v_cache", v_cache, kind, n), ("slots", slots, torch.int32, p.T))
        p.slots, p.num_slots = slots.data_ptr(), n // (p.h_kv * p.d)
    if out is None:
        p.zero_skipped = 1
        q_out = torch.empty(q.shape, dtype=kind, device=q.device)
        k_out = None if append else torch.empty(k.shape, dtype=kind, device=q.device)
    else:
        q_out, k_out = out
        _check(dev, ("q_out", q_out, kind, q.shape), ("k_out", k_out, kind, k.shape))
        if q_out is None:
            q_out = torch.zeros(q.shape, dtype=kind, device=q.device)
        if k_out is None and not append:
            k_out = torch.zeros(k.shape, dtype=kind, device=q.device)
    rc = load().fa_qk_norm_rope(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr() if append else None, q_out.data_ptr(),
                                None if k_out is None else k_out.data_ptr(), k_cache.data_ptr() if append else None,
                                v_cache.data_ptr() if append else None, torch._C._cuda_getCurrentRawStream(dev))
    if rc != FA_OK:
        raise FaError(rc, "fa_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_backward(q, k, dq_out, dk_out, q_weight, k_weight, cos, sin, *, positions=None, seq_len=None, eps=1e-6,
                          interleaved=False, grads=None, workspace=None, status=None, wait_limit_ns=0, pair_axis=None,
                          norm=True):
    """Runs fa_qk_norm_rope_bwd on torch CUDA tensors; returns (dq, dk, dq_weight, dk_weight).

    q, k and the arguments behind dk_out are those of qk_norm_rope; dq_out, dk_out (contiguous)
    are the gradients of its outputs.  grads: (dq, dk, dq_weight, dk_weight) to write, dq and dk at
    any token stride (slices of a fused projection's gradient); the weights' are fp32 [d].  A padding
    token (position -1, or one outside the tables) has a zero gradient in the tensors made here; in given
    ones its rows are left as they were.  With norm=False q and k are not read (None will do), and the
    weights' gradients are None."""
    import torch
    if not norm:
        q, k = dq_out, dk_out  # (their shapes)
    dev = _device_index(q)
    if dev != torch._C._cuda_getDevice():
        return _on_device(q, qk_norm_rope_backward, q, k, dq_out, dk_out, q_weight, k_weight, cos, sin, positions=positions,
                          seq_len=seq_len, eps=eps, interleaved=interleaved, grads=grads, workspace=workspace, status=status,
                          wait_limit_ns=wait_limit_ns, pair_axis=pair_axis, norm=norm)
    p = _rope_params(dev, q, k, q_weight, k_weight, cos, sin, positions, seq_len, eps, interleaved, status, pair_axis, norm)
    p.wait_limit_ns = wait_limit_ns
    kind = q.dtype
    _check(dev, ("dq_out", dq_out, kind, q.numel()), ("dk_out", dk_out, kind, k.numel()))
    if dq_out.shape != q.shape or dk_out.shape != k.shape:
        raise ValueError(f"dq_out and dk_out must have the shapes {tuple(q.shape)} and {tuple(k.shape)}")
    if grads is None:
        empty, at = torch.empty, q.device
        dq, dk = empty(q.shape, dtype=kind, device=at), empty(k.shape, dtype=kind, device=at)
        dwq = dwk = None
        if norm:
            dwq, dwk = empty(p.d, dtype=torch.float32, device=at), empty(p.d, dtype=torch.float32, device=at)
        p.zero_skipped = 1
    else:
        dq, dk, dwq, dwk = grads
        if dq.shape != q.shape or dk.shape != k.shape:
            raise ValueError(f"dq and dk must have the shapes {tuple(q.shape)} and {tuple(k.shape)}")
        _like("dq", dq, kind, dev)
        _like("dk", dk, kind, dev)
        p.dq_stride, p.dk_stride = _rows("dq", dq)[3], _rows("dk", dk)[3]
        if (dwq is None or dwk is None) == bool(norm):
            raise ValueError("the weights' gradients are wanted with the norm, and not without it")
        _check(dev, ("dq_weight", dwq, torch.float32, p.d), ("dk_weight", dwk, torch.float32, p.d))
    lib, ref = load(), ctypes.byref(p)
    nbytes = lib.fa_qk_norm_rope_bwd_workspace_size(ref)
    if nbytes == 0:
        raise FaError(FA_ERR_UNSUPPORTED, "fa_qk_norm_rope_bwd_workspace_size")
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    else:
        _check(dev, ("workspace", workspace, torch.uint8, workspace.numel()))
    rc = lib.fa_qk_norm_rope_bwd(ref, q.data_ptr(), k.data_ptr(), dq_out.data_ptr(), dk_out.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                 None if dwq is None else dwq.data_ptr(), None if dwk is None else dwk.data_ptr(),
                                 workspace.data_ptr(), workspace.numel(),
                                 torch._C._cuda_getCurrentRawStream(dev))
    if rc != FA_OK:
        raise FaError(rc, "fa_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


def _cache8(dev, k_cache, v_cache, k_scale, v_scale, h_kv, d):
    """(num_pages, page_size, scale_block) of an 8-bit cache, whose tensors are checked."""
    import torch
    if k_cache.dim() != 4 or k_scale.dim() != 3:
        raise ValueError(f"k_cache and v_cache must be [num_pages, page_size, {h_kv}, {d}], k_scale and v_scale [num_pages, "
                         f"page_size / scale_block, {h_kv}]")
    num_pages, page_size = k_cache.shape[:2]
    blocks = k_scale.shape[1]
    if blocks < 1 or page_size % blocks:
        raise ValueError(f"k_scale has {blocks} blocks for pages of {page_size} rows")
    pool, scales = (num_pages, page_size, h_kv, d), (num_pages, blocks, h_kv)
    _check(dev, ("k_cache", k_cache, torch.uint8, pool), ("v_cache", v_cache, torch.uint8, pool),
           ("k_scale", k_scale, torch.float32, scales), ("v_scale", v_scale, torch.float32, scales))
    return num_pages, page_size, page_size // blocks


def qk_norm_rope_append8(q, k, v, q_weight, k_weight, cos, sin, *, k_cache, v_cache, k_scale, v_scale, cu_q, seqused_k,
                         block_table, positions, eps=1e-6, interleaved=False, pair_axis=None, norm=True, out=None, status=None,
                         wait_limit_ns=0):
    """Runs fa_qk_norm_rope_append8 on torch CUDA tensors; returns q_out [T, h_q, d].

    q, k and v (slices of a fused projection will do), weights, tables, positions (int32 [T] or
    [axes, T], with pair_axis), norm and status are those of qk_norm_rope.  k_cache, v_cache: uint8 (e4m3
    bytes) [num_pages, page_size, h_kv, d]; k_scale, v_scale: fp32 [num_pages, page_size / scale_block, h_kv],
    which gives the block; cu_q [B + 1], seqused_k [B] (the new tokens included) and block_table
    [B, max_blocks_per_seq] are what page_plan makes and forward takes.  out: q_out to write (rows of
    skipped tokens are left as they were there, and zero in the one made here)."""
    import torch
    dev = _device_index(q)
    if dev != torch._C._cuda_getDevice():
        return _on_device(q, qk_norm_rope_append8, q, k, v, q_weight, k_weight, cos, sin, k_cache=k_cache, v_cache=v_cache,
                          k_scale=k_scale, v_scale=v_scale, cu_q=cu_q, seqused_k=seqused_k, block_table=block_table,
                          positions=positions, eps=eps, interleaved=interleaved, pair_axis=pair_axis, norm=norm, out=out,
                          status=status, wait_limit_ns=wait_limit_ns)
    if positions is None:
        raise ValueError("an append needs the tokens' positions")
    p = _rope_params(dev, q, k, q_weight, k_weight, cos, sin, positions, None, eps, interleaved, status, pair_axis, norm)
    p.wait_limit_ns = wait_limit_ns
    kind = q.dtype
    if v.shape != k.shape:
        raise ValueError(f"v must have k's shape {tuple(k.shape)}; it has {tuple(v.shape)}")
    _like("v", v, kind, dev)
    p.v_stride = _rows("v", v)[3]
    num_pages, page_size, block = _cache8(dev, k_cache, v_cache, k_scale, v_scale, p.h_kv, p.d)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks_per_seq]")
    B, blocks = block_table.shape
    _check(dev, ("cu_q", cu_q, torch.int32, B + 1), ("seqused_k", seqused_k, torch.int32, B),
           ("block_table", block_table, torch.int32, B * blocks), ("out", out, kind, q.shape))
    if out is None:
        p.zero_skipped = 1
        out = torch.empty(q.shape, dtype=kind, device=q.device)
    c = FaCache8Params(B, page_size, blocks, num_pages, block, cu_q.data_ptr(), seqused_k.data_ptr(), block_table.data_ptr())
    rc = load().fa_qk_norm_rope_append8(ctypes.byref(p), ctypes.byref(c), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                        k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                        torch._C._cuda_getCurrentRawStream(dev))
    if rc != FA_OK:
        raise FaError(rc, "fa_qk_norm_rope_append8")
    return out


def page_plan(cached, fresh, block_table, free_pages, *, page_size, num_pages, tokens, free_head=None, out=None, status=None):
    """Runs fa_page_plan on int32 torch CUDA tensors; returns (cu_seqlens_q, seqused_k, positions,
    slots, free_head_out) and writes the new pages' entries into block_table [B, max_blocks].

    cached, fresh: [B] tokens in the cache and new ones; free_pages: pages to take from, from
    index free_head ([1], None: 0) on; tokens: rows of the packed batch (positions and slots are
    -1 behind the last new token).  out: the five results' tensors to write, status: [1] or None."""
    import torch
    dev = _device_index(cached)
    if dev != torch._C._cuda_getDevice():
        return _on_device(cached, page_plan, cached, fresh, block_table, free_pages, page_size=page_size, num_pages=num_pages,
                          tokens=tokens, free_head=free_head, out=out, status=status)
    B, i32 = cached.numel(), torch.int32
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks_per_seq]")
    blocks, n_free = block_table.shape[1], free_pages.numel()
    _check(dev, ("cached", cached, i32, B), ("fresh", fresh, i32, B), ("block_table", block_table, i32, B * blocks),
           ("free_pages", free_pages, i32, n_free), ("free_head", free_head, i32, 1), ("status", status, i32, 1))
    if out is None:
        # (five allocations take less host time than one and five views of it: 9.4 against 12.3 us)
        empty, at = torch.empty, cached.device
        out = [empty(n, dtype=i32, device=at) for n in (B + 1, B, tokens, tokens, 1)]
    else:
        _check(dev, *((name, t, i32, size) for name, t, size in zip(("cu_seqlens_q", "seqused_k", "positions", "slots", "free_head_out"),
                                                                    out, ((B + 1,), (B,), (tokens,), (tokens,), 1))))
    cu, used, positions, slots, head_out = out
    p = FaPagePlanParams(B, tokens, page_size, blocks, num_pages, n_free)
    rc = load().fa_page_plan(ctypes.byref(p), cached.data_ptr(), fresh.data_ptr(), free_pages.data_ptr(),
                             None if free_head is None else free_head.data_ptr(), block_table.data_ptr(), cu.data_ptr(),
                             used.data_ptr(), positions.data_ptr(), slots.data_ptr(), head_out.data_ptr(),
                             None if status is None else status.data_ptr(), torch._C._cuda_getCurrentRawStream(dev))
    if rc != FA_OK:
        raise FaError(rc, "fa_page_plan")
    return cu, used, positions, slots, head_out


def device_status(workspace) -> int:
    return fa_read_device_status(_ptr(workspace), _stream())
