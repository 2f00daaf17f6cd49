"""B200-native DeepSeek Sparse Attention (DSA) hot path.

The compute lives in ``libdsa.so`` (CUDA for sm_100a, C ABI in
``include/dsa.h``); this module only marshals torch tensors into that ABI.
Every function has the name of its C entry point and takes device tensors
plus the stream it should run on (default: torch's current stream).  There is
no CPU path: if the library is missing, importing the binding fails.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "DSAError", "lib_path", "load", "dsa_version", "dsa_status_string",
    "dsa_indexer_logits", "dsa_topk", "dsa_sparse_mla_fwd", "dsa_forward",
    "dsa_forward_workspace_size", "dsa_get_device_error", "dsa_forward_noalloc",
    "dsa_forward_host", "dsa_forward_host_workspace_size", "dsa_indexer_kl",
    "dsa_indexer_kl_workspace_size", "dsa_masked_mha_fwd", "dsa_masked_mha_workspace_size",
    "dsa_debug_fault_injection", "dsa_indexer_backward", "dsa_forward_fused",
    "dsa_forward_fused_workspace_size", "dsa_paged_mla_decode",
    "dsa_paged_mla_decode_workspace_size", "dsa_paged_attn_mass", "dsa_cache_evict",
    "dsa_window_mha_fwd", "EXPORTED",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libdsa.so")
_lib = None

# Every symbol include/dsa.h declares.
EXPORTED = (
    "dsa_indexer_logits", "dsa_topk", "dsa_sparse_mla_fwd", "dsa_forward",
    "dsa_forward_workspace_size", "dsa_status_string", "dsa_get_device_error", "dsa_version",
    "dsa_forward_noalloc", "dsa_forward_host", "dsa_forward_host_workspace_size",
    "dsa_indexer_kl", "dsa_indexer_kl_workspace_size", "dsa_masked_mha_fwd",
    "dsa_masked_mha_workspace_size", "dsa_debug_fault_injection", "dsa_indexer_backward",
    "dsa_forward_fused", "dsa_forward_fused_workspace_size", "dsa_paged_mla_decode",
    "dsa_paged_mla_decode_workspace_size", "dsa_paged_attn_mass", "dsa_cache_evict",
    "dsa_window_mha_fwd",
)

STATUS = {
    0: "DSA_OK", 1: "DSA_ERR_INVALID_ARG", 2: "DSA_ERR_UNSUPPORTED", 3: "DSA_ERR_ALIGNMENT",
    4: "DSA_ERR_WORKSPACE", 5: "DSA_ERR_CUDA", 6: "DSA_ERR_TIMEOUT", 7: "DSA_ERR_BOUNDS",
}


class DSAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {STATUS.get(self.status, self.status)} "
                         f"({dsa_status_string(self.status)})")


def lib_path() -> str:
    return _LIB_PATH


def load():
    """Loads libdsa.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: build it with "
                          "`python -m sparse_attention_08_b200._build`")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    lib.dsa_indexer_logits.argtypes = [P, P, P, P, P, P, P, I, I, I, I64, I64, I, I, P, I64, P]
    lib.dsa_topk.argtypes = [P, I64, P, P, I, I, I, I64, I, P, P, P]
    lib.dsa_sparse_mla_fwd.argtypes = [P, P, P, P, P, I, I, I, I64, I64, I, I, I, I, F, P, P, P]
    lib.dsa_forward.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I64, I64, I, I, I, I, I, I, F,
                                P, P, P, P, ctypes.c_size_t, P]
    lib.dsa_forward_fused.argtypes = lib.dsa_forward.argtypes
    lib.dsa_forward_fused_workspace_size.argtypes = [I64, I64, I, I, I, I]
    lib.dsa_forward_fused_workspace_size.restype = ctypes.c_size_t
    lib.dsa_forward_noalloc.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I64, I64, I, I, I, I,
                                        I, I, F, P, P, P, P]
    lib.dsa_forward_host.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I64, I64, I, I, I, I, I,
                                     I, F, P, P, I, P, ctypes.c_size_t, P, I]
    lib.dsa_indexer_kl.argtypes = [P, P, P, P, P, I64, P, P, I, I, I, I64, I64, I, I, I, F, P, P,
                                   P, P, ctypes.c_size_t, P]
    lib.dsa_indexer_kl.restype = I
    lib.dsa_indexer_kl_workspace_size.argtypes = [I64, I, I]
    lib.dsa_indexer_kl_workspace_size.restype = ctypes.c_size_t
    lib.dsa_masked_mha_fwd.argtypes = [P, P, P, P, P, P, I, I, I, I64, I64, I, I, I, I, F, P, P, P,
                                       ctypes.c_size_t, P]
    lib.dsa_masked_mha_fwd.restype = I
    lib.dsa_masked_mha_workspace_size.argtypes = [I64, I]
    lib.dsa_masked_mha_workspace_size.restype = ctypes.c_size_t
    lib.dsa_forward_host_workspace_size.argtypes = [I64, I, I, I, I, I, I, I, I]
    lib.dsa_forward_host_workspace_size.restype = ctypes.c_size_t
    for name in ("dsa_indexer_logits", "dsa_topk", "dsa_sparse_mla_fwd", "dsa_forward",
                 "dsa_forward_noalloc", "dsa_forward_host", "dsa_forward_fused"):
        getattr(lib, name).restype = I
    lib.dsa_forward_workspace_size.argtypes = [I64, I, I]
    lib.dsa_forward_workspace_size.restype = ctypes.c_size_t
    lib.dsa_status_string.argtypes = [I]
    lib.dsa_status_string.restype = ctypes.c_char_p
    lib.dsa_get_device_error.argtypes = [P]
    lib.dsa_get_device_error.restype = I
    lib.dsa_indexer_backward.argtypes = [P, P, P, P, P, P, I64, P, P, I, I, I, I64, I64, I, I, P,
                                         P, P, P]
    lib.dsa_indexer_backward.restype = I
    lib.dsa_paged_mla_decode.argtypes = [P, P, I64, I, I64, P, I64, I, P, I, I, I, I, I, I, I, F,
                                         P, P, P, ctypes.c_size_t, P]
    lib.dsa_paged_mla_decode.restype = I
    lib.dsa_paged_mla_decode_workspace_size.argtypes = [I, I, I]
    lib.dsa_paged_mla_decode_workspace_size.restype = ctypes.c_size_t
    lib.dsa_paged_attn_mass.argtypes = [P, P, I64, I, I64, P, I64, I, P, I, I, I, I, I, I, F, P, P,
                                        P, I64, P]
    lib.dsa_paged_attn_mass.restype = I
    lib.dsa_cache_evict.argtypes = [P, I64, I, I64, P, I64, I, P, I, I, P, I64, I, I, I, P, I64, I,
                                    P, P, P, I64, P]
    lib.dsa_cache_evict.restype = I
    lib.dsa_window_mha_fwd.argtypes = [P, P, P, P, P, I, I, I, I64, I64, I, I, I, I, I, F, P, P, P]
    lib.dsa_window_mha_fwd.restype = I
    lib.dsa_debug_fault_injection.argtypes = [ctypes.c_uint64, I]
    lib.dsa_debug_fault_injection.restype = None
    lib.dsa_version.argtypes = []
    lib.dsa_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def dsa_debug_fault_injection(wait_limit_ns: int = 0, drop_first_key_load: bool = False):
    """Test hook: the wait limit of later launches (0 = the default 2 s) and a
    one-shot request that the next launch of dsa_indexer_logits (or of the paged
    decode and totals, or of the windowed prompt attention) leave out keys that it
    waits for, so a bounded wait runs out (DSA_ERR_TIMEOUT)."""
    load().dsa_debug_fault_injection(int(wait_limit_ns), 1 if drop_first_key_load else 0)


def dsa_version() -> str:
    return load().dsa_version().decode()


def dsa_status_string(status: int) -> str:
    return load().dsa_status_string(int(status)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(rc: int, where: str):
    if rc != 0:
        raise DSAError(rc, where)


def _need(t, dtype, name, ndim=None):
    import torch
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")
    del torch


def dsa_indexer_logits(q_fp8, q_scale, w, k_fp8, k_scale, cu_seqlens_q, cu_seqlens_k, B,
                       max_len_q, max_len_k, logits, ld_logits=None, stream=None):
    """Indexer scores into logits (f32, row stride ld_logits).  q_fp8 / k_fp8
    are uint8 (or float8_e4m3fn) tensors [T_q, H_I, d_I] / [T_k, d_I]."""
    import torch
    q8 = q_fp8.view(torch.uint8) if q_fp8.dtype == torch.float8_e4m3fn else q_fp8
    k8 = k_fp8.view(torch.uint8) if k_fp8.dtype == torch.float8_e4m3fn else k_fp8
    _need(q8, torch.uint8, "q_fp8", 3)
    _need(k8, torch.uint8, "k_fp8", 2)
    _need(q_scale, torch.float32, "q_scale")
    _need(w, torch.float32, "w")
    _need(k_scale, torch.float32, "k_scale")
    _need(cu_seqlens_q, torch.int32, "cu_seqlens_q")
    _need(cu_seqlens_k, torch.int32, "cu_seqlens_k")
    if ld_logits is None:
        ld_logits = logits.stride(0)
    T_q, H_I, d_I = q8.shape
    rc = load().dsa_indexer_logits(_ptr(q8), _ptr(q_scale), _ptr(w), _ptr(k8), _ptr(k_scale),
                                   _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), int(B), int(max_len_q),
                                   int(max_len_k), int(T_q), int(k8.shape[0]), int(H_I), int(d_I),
                                   _ptr(logits), int(ld_logits), _stream(stream))
    _check(rc, "dsa_indexer_logits")


def dsa_indexer_backward(q_fp8, q_scale, w, k_fp8, k_scale, g, cu_seqlens_q, cu_seqlens_k, B,
                         max_len_q, max_len_k, dq, dw, dk, ld_g=None, stream=None):
    """The indexer's backward: dq [T_q, 64, 128], dw [T_q, 64], dk [T_k, 128]
    (f32) from the upstream score gradient g (f32, row stride ld_g)."""
    import torch
    q8 = q_fp8.view(torch.uint8) if q_fp8.dtype == torch.float8_e4m3fn else q_fp8
    k8 = k_fp8.view(torch.uint8) if k_fp8.dtype == torch.float8_e4m3fn else k_fp8
    _need(q8, torch.uint8, "q_fp8", 3)
    _need(k8, torch.uint8, "k_fp8", 2)
    for t, n in ((q_scale, "q_scale"), (w, "w"), (k_scale, "k_scale"), (dw, "dw")):
        _need(t, torch.float32, n)
    _need(dq, torch.float32, "dq", 3)
    _need(dk, torch.float32, "dk", 2)
    _need(cu_seqlens_q, torch.int32, "cu_seqlens_q")
    _need(cu_seqlens_k, torch.int32, "cu_seqlens_k")
    if g.dtype != torch.float32 or not g.is_cuda or g.stride(1) != 1:
        raise ValueError("g must be a CUDA float32 tensor with contiguous rows")
    if ld_g is None:
        ld_g = g.stride(0)
    T_q, H_I, d_I = q8.shape
    rc = load().dsa_indexer_backward(_ptr(q8), _ptr(q_scale), _ptr(w), _ptr(k8), _ptr(k_scale),
                                     _ptr(g), int(ld_g), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                                     int(B), int(max_len_q), int(max_len_k), int(T_q),
                                     int(k8.shape[0]), int(H_I), int(d_I), _ptr(dq), _ptr(dw),
                                     _ptr(dk), _stream(stream))
    _check(rc, "dsa_indexer_backward")


def dsa_topk(logits, cu_seqlens_q, cu_seqlens_k, B, max_len_q, max_len_k, k, idx_out,
             val_out=None, ld_logits=None, total_q=None, stream=None):
    import torch
    _need(idx_out, torch.int32, "idx_out", 2)
    _need(val_out, torch.float32, "val_out", 2)
    if logits.dtype != torch.float32 or not logits.is_cuda:
        raise ValueError("logits must be a CUDA float32 tensor")
    if ld_logits is None:
        ld_logits = logits.stride(0)
    if total_q is None:
        total_q = idx_out.shape[0]
    rc = load().dsa_topk(_ptr(logits), int(ld_logits), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                         int(B), int(max_len_q), int(max_len_k), int(total_q), int(k),
                         _ptr(idx_out), _ptr(val_out), _stream(stream))
    _check(rc, "dsa_topk")


def dsa_sparse_mla_fwd(q, kv, idx, cu_seqlens_q, cu_seqlens_k, B, max_len_q, max_len_k,
                       sm_scale, out, lse=None, stream=None):
    import torch
    _need(q, torch.bfloat16, "q", 3)
    _need(kv, torch.bfloat16, "kv", 2)
    _need(idx, torch.int32, "idx", 2)
    _need(out, torch.bfloat16, "out", 3)
    _need(lse, torch.float32, "lse", 2)
    T_q, H, d_qk = q.shape
    rc = load().dsa_sparse_mla_fwd(_ptr(q), _ptr(kv), _ptr(idx), _ptr(cu_seqlens_q),
                                   _ptr(cu_seqlens_k), int(B), int(max_len_q), int(max_len_k),
                                   int(T_q), int(kv.shape[0]), int(H), int(d_qk),
                                   int(out.shape[2]), int(idx.shape[1]), float(sm_scale),
                                   _ptr(out), _ptr(lse), _stream(stream))
    _check(rc, "dsa_sparse_mla_fwd")


def dsa_forward_workspace_size(total_q, max_len_k, k) -> int:
    return int(load().dsa_forward_workspace_size(int(total_q), int(max_len_k), int(k)))


def dsa_forward(q_fp8, q_scale, w, k_fp8, k_scale, q, kv, cu_seqlens_q, cu_seqlens_k, B,
                max_len_q, max_len_k, k, sm_scale, out, lse, workspace, idx_out=None,
                stream=None):
    import torch
    q8 = q_fp8.view(torch.uint8) if q_fp8.dtype == torch.float8_e4m3fn else q_fp8
    k8 = k_fp8.view(torch.uint8) if k_fp8.dtype == torch.float8_e4m3fn else k_fp8
    _need(q8, torch.uint8, "q_fp8", 3)
    _need(k8, torch.uint8, "k_fp8", 2)
    _need(q, torch.bfloat16, "q", 3)
    _need(kv, torch.bfloat16, "kv", 2)
    _need(out, torch.bfloat16, "out", 3)
    _need(lse, torch.float32, "lse", 2)
    _need(idx_out, torch.int32, "idx_out", 2)
    T_q, H_I, d_I = q8.shape
    _, H, d_qk = q.shape
    rc = load().dsa_forward(_ptr(q8), _ptr(q_scale), _ptr(w), _ptr(k8), _ptr(k_scale), _ptr(q),
                            _ptr(kv), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), int(B),
                            int(max_len_q), int(max_len_k), int(T_q), int(k8.shape[0]), int(H_I),
                            int(d_I), int(H), int(d_qk), int(out.shape[2]), int(k),
                            float(sm_scale), _ptr(out), _ptr(lse), _ptr(idx_out),
                            _ptr(workspace), int(workspace.numel() * workspace.element_size()),
                            _stream(stream))
    _check(rc, "dsa_forward")


def dsa_forward_fused_workspace_size(total_q, total_k, B, max_len_k, k, d_I) -> int:
    return int(load().dsa_forward_fused_workspace_size(int(total_q), int(total_k), int(B),
                                                       int(max_len_k), int(k), int(d_I)))


def dsa_forward_fused(q_fp8, q_scale, w, k_fp8, k_scale, q, kv, cu_seqlens_q, cu_seqlens_k, B,
                      max_len_q, max_len_k, k, sm_scale, out, lse, workspace, idx_out=None,
                      stream=None):
    """dsa_forward with the indexer and top-k fused into two passes over the
    keys (the score matrix stays out of HBM); same results, bit for bit.  The
    workspace holds dsa_forward_fused_workspace_size bytes."""
    import torch
    q8 = q_fp8.view(torch.uint8) if q_fp8.dtype == torch.float8_e4m3fn else q_fp8
    k8 = k_fp8.view(torch.uint8) if k_fp8.dtype == torch.float8_e4m3fn else k_fp8
    _need(q8, torch.uint8, "q_fp8", 3)
    _need(k8, torch.uint8, "k_fp8", 2)
    _need(q, torch.bfloat16, "q", 3)
    _need(kv, torch.bfloat16, "kv", 2)
    _need(out, torch.bfloat16, "out", 3)
    _need(lse, torch.float32, "lse", 2)
    _need(idx_out, torch.int32, "idx_out", 2)
    T_q, H_I, d_I = q8.shape
    _, H, d_qk = q.shape
    rc = load().dsa_forward_fused(
        _ptr(q8), _ptr(q_scale), _ptr(w), _ptr(k8), _ptr(k_scale), _ptr(q), _ptr(kv),
        _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), int(B), int(max_len_q), int(max_len_k), int(T_q),
        int(k8.shape[0]), int(H_I), int(d_I), int(H), int(d_qk), int(out.shape[2]), int(k),
        float(sm_scale), _ptr(out), _ptr(lse), _ptr(idx_out), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), _stream(stream))
    _check(rc, "dsa_forward_fused")


def dsa_forward_noalloc(q_fp8, q_scale, w, k_fp8, k_scale, q, kv, cu_seqlens_q, cu_seqlens_k, B,
                        max_len_q, max_len_k, k, sm_scale, out, lse, idx_out=None, stream=None):
    """dsa_forward without a workspace, for callers that cannot allocate device
    memory: the scratch lives in a fixed 48 MiB device array inside the
    library (see include/dsa.h).  Raises DSAError(DSA_ERR_WORKSPACE) when the
    problem's scratch exceeds it."""
    import torch
    q8 = q_fp8.view(torch.uint8) if q_fp8.dtype == torch.float8_e4m3fn else q_fp8
    k8 = k_fp8.view(torch.uint8) if k_fp8.dtype == torch.float8_e4m3fn else k_fp8
    _need(q8, torch.uint8, "q_fp8", 3)
    _need(k8, torch.uint8, "k_fp8", 2)
    _need(q, torch.bfloat16, "q", 3)
    _need(kv, torch.bfloat16, "kv", 2)
    _need(out, torch.bfloat16, "out", 3)
    _need(lse, torch.float32, "lse", 2)
    _need(idx_out, torch.int32, "idx_out", 2)
    T_q, H_I, d_I = q8.shape
    _, H, d_qk = q.shape
    rc = load().dsa_forward_noalloc(_ptr(q8), _ptr(q_scale), _ptr(w), _ptr(k8), _ptr(k_scale),
                                    _ptr(q), _ptr(kv), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                                    int(B), int(max_len_q), int(max_len_k), int(T_q),
                                    int(k8.shape[0]), int(H_I), int(d_I), int(H), int(d_qk),
                                    int(out.shape[2]), int(k), float(sm_scale), _ptr(out),
                                    _ptr(lse), _ptr(idx_out), _stream(stream))
    _check(rc, "dsa_forward_noalloc")


def _need_host(t, dtype, name, ndim=None):
    if t is None:
        return
    if t.is_cuda:
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")


def dsa_forward_host_workspace_size(total_k, max_len_k, B, H_I, d_I, H, k, chunk_q,
                                    n_streams) -> int:
    return int(load().dsa_forward_host_workspace_size(int(total_k), int(max_len_k), int(B),
                                                      int(H_I), int(d_I), int(H), int(k),
                                                      int(chunk_q), int(n_streams)))


def dsa_forward_host(q_fp8, q_scale, w, k_fp8, k_scale, q, kv, cu_seqlens_q, cu_seqlens_k, B,
                     max_len_q, max_len_k, k, sm_scale, out, lse, chunk_q, workspace, streams):
    """dsa_forward over host tensors (pin them for the copies to overlap):
    the library uploads the key side once and the query rows in chunks of
    chunk_q rows spread over `streams` (torch.cuda.Stream objects), and returns
    with `out` / `lse` (host tensors) filled.  `workspace` is a uint8 CUDA
    tensor of dsa_forward_host_workspace_size(...) bytes."""
    import torch
    q8 = q_fp8.view(torch.uint8) if q_fp8.dtype == torch.float8_e4m3fn else q_fp8
    k8 = k_fp8.view(torch.uint8) if k_fp8.dtype == torch.float8_e4m3fn else k_fp8
    for t, dt, name, nd in ((q8, torch.uint8, "q_fp8", 3), (k8, torch.uint8, "k_fp8", 2),
                            (q_scale, torch.float32, "q_scale", 2), (w, torch.float32, "w", 2),
                            (k_scale, torch.float32, "k_scale", 1),
                            (q, torch.bfloat16, "q", 3), (kv, torch.bfloat16, "kv", 2),
                            (cu_seqlens_q, torch.int32, "cu_seqlens_q", 1),
                            (cu_seqlens_k, torch.int32, "cu_seqlens_k", 1),
                            (out, torch.bfloat16, "out", 3), (lse, torch.float32, "lse", 2)):
        _need_host(t, dt, name, nd)
    _need(workspace, torch.uint8, "workspace", 1)
    T_q, H_I, d_I = q8.shape
    _, H, d_qk = q.shape
    arr = (ctypes.c_void_p * len(streams))(*[s.cuda_stream for s in streams])
    rc = load().dsa_forward_host(_ptr(q8), _ptr(q_scale), _ptr(w), _ptr(k8), _ptr(k_scale),
                                 _ptr(q), _ptr(kv), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                                 int(B), int(max_len_q), int(max_len_k), int(T_q),
                                 int(k8.shape[0]), int(H_I), int(d_I), int(H), int(d_qk),
                                 int(out.shape[2]), int(k), float(sm_scale), _ptr(out),
                                 _ptr(lse), int(chunk_q), _ptr(workspace),
                                 int(workspace.numel()), arr, len(streams))
    _check(rc, "dsa_forward_host")


def dsa_indexer_kl_workspace_size(total_q, H, k) -> int:
    return int(load().dsa_indexer_kl_workspace_size(int(total_q), int(H), int(k)))


def dsa_indexer_kl(q, kv, idx, lse, logits, cu_seqlens_q, cu_seqlens_k, B, max_len_q, max_len_k,
                   k, sm_scale, kl_out, grad_out=None, target_out=None, workspace=None,
                   ld_logits=None, stream=None):
    """The indexer's KL training signal over each query's selection (see
    include/dsa.h): kl_out [T_q], and optionally the gradient with respect to
    the selected indexer scores and the head-averaged attention target, both
    [T_q, k] in index-row order.  `workspace` (uint8 CUDA tensor) is allocated
    here when not given."""
    import torch
    _need(q, torch.bfloat16, "q", 3)
    _need(kv, torch.bfloat16, "kv", 2)
    _need(idx, torch.int32, "idx", 2)
    _need(lse, torch.float32, "lse", 2)
    _need(kl_out, torch.float32, "kl_out", 1)
    _need(grad_out, torch.float32, "grad_out", 2)
    _need(target_out, torch.float32, "target_out", 2)
    T_q, H, d_qk = q.shape
    nbytes = dsa_indexer_kl_workspace_size(T_q, H, k)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    ld = logits.stride(0) if ld_logits is None else ld_logits
    rc = load().dsa_indexer_kl(_ptr(q), _ptr(kv), _ptr(idx), _ptr(lse), _ptr(logits), int(ld),
                               _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), int(B), int(max_len_q),
                               int(max_len_k), int(T_q), int(kv.shape[0]), int(H), int(d_qk),
                               int(k), float(sm_scale), _ptr(kl_out), _ptr(grad_out),
                               _ptr(target_out), _ptr(workspace), int(workspace.numel()),
                               _stream(stream))
    _check(rc, "dsa_indexer_kl")


def dsa_masked_mha_workspace_size(total_q, max_len_k) -> int:
    return int(load().dsa_masked_mha_workspace_size(int(total_q), int(max_len_k)))


def dsa_masked_mha_fwd(q, k, v, idx, cu_seqlens_q, cu_seqlens_k, B, max_len_q, max_len_k,
                       topk, sm_scale, out, lse=None, workspace=None, stream=None):
    """The masked MHA mode (see include/dsa.h): dense per-head attention of
    q [T_q, H, 192] over k [T_k, H, 192], v [T_k, H, 128], restricted to each
    query's selected set idx [T_q, topk]; writes out [T_q, H, 128] (bf16) and
    lse [T_q, H] (fp32, optional).  `workspace` (uint8 CUDA tensor) is
    allocated here when not given."""
    import torch
    _need(q, torch.bfloat16, "q", 3)
    _need(k, torch.bfloat16, "k", 3)
    _need(v, torch.bfloat16, "v", 3)
    _need(idx, torch.int32, "idx", 2)
    _need(out, torch.bfloat16, "out", 3)
    _need(lse, torch.float32, "lse", 2)
    T_q, H, d_qk = q.shape
    nbytes = dsa_masked_mha_workspace_size(T_q, max_len_k)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    rc = load().dsa_masked_mha_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(cu_seqlens_q),
                                   _ptr(cu_seqlens_k), int(B), int(max_len_q), int(max_len_k),
                                   int(T_q), int(k.shape[0]), int(H), int(d_qk), int(v.shape[2]),
                                   int(topk), float(sm_scale), _ptr(out), _ptr(lse),
                                   _ptr(workspace), int(workspace.numel()), _stream(stream))
    _check(rc, "dsa_masked_mha_fwd")


class _On:
    """The device (its number) and stream a call runs on: the given stream (a torch stream or
    a raw handle), or the device's current one.  Entered around the launch; on
    the current device and stream, the common case, that does nothing."""

    __slots__ = ("handle", "_ctx")

    def __init__(self, device, stream):
        import torch
        on = getattr(stream, "device", None)
        if on is not None and on.index != device:
            raise ValueError(f"stream is on {on}, the tensors on cuda:{device}")
        self._ctx = ()
        if device != torch.cuda.current_device():
            self._ctx = (torch.cuda.device(device),)
        if stream is None:
            # (the handle alone: building a Stream object takes 2 us)
            self.handle = torch._C._cuda_getCurrentRawStream(device)
        else:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            self.handle = stream.cuda_stream
            # a workspace allocated inside belongs to this stream
            self._ctx += (torch.cuda.stream(stream),)

    def __enter__(self):
        for c in self._ctx:
            c.__enter__()
        return self.handle

    def __exit__(self, *exc):
        for c in reversed(self._ctx):
            c.__exit__(*exc)


def _ten(t, dtype, shape, dev, name):
    """Checks a contiguous CUDA tensor of a shape on device number dev (None
    passes) and returns its address."""
    if t is None:
        return None
    if (t.dtype is dtype and t.shape == shape and t.get_device() == dev and dev >= 0
            and t.is_contiguous()):
        return t.data_ptr()
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be on cuda:{max(dev, 0)}, got {t.device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _rows(t, dtype, B, least, dev, name):
    """Checks a CUDA matrix [B, >= least] whose rows are contiguous (None
    passes); returns its address and row stride."""
    if t is None:
        return None, 0
    if t.dtype != dtype or t.get_device() != dev or dev < 0 or t.dim() != 2 or t.shape[0] != B:
        raise ValueError(f"{name} must be a {dtype} matrix of {B} rows on cuda:{max(dev, 0)}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    n = t.shape[1]
    if n < least:
        raise ValueError(f"{name} must have at least {least} columns, got {n}")
    ld, step = t.stride()
    if n > 1 and step != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), (ld if B > 1 else n)


def _dims(t, n, name):
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dims, got {t.dim()}")
    return t.shape


def _cache(kv_cache, block_table, seq_lens):
    """Checks the tensors of a paged cache; returns its arguments in the C ABI's
    order, the number of sequences last, and the device's number."""
    import torch
    n_pages, page, width = _dims(kv_cache, 3, "kv_cache")
    if kv_cache.dtype != torch.bfloat16 or width != 576 or not kv_cache.is_cuda:
        raise ValueError("kv_cache must be a CUDA torch.bfloat16 tensor [n_pages, page_size, 576]")
    dev = kv_cache.get_device()
    stride, row, col = kv_cache.stride()
    if n_pages == 1:
        stride = page * 576
    if col != 1 or (page > 1 and row != 576):
        raise ValueError("kv_cache rows must lie one after the other within a page")
    (B,) = _dims(seq_lens, 1, "seq_lens")
    lens = _ten(seq_lens, torch.int32, (B,), dev, "seq_lens")
    table, ld = _rows(block_table, torch.int32, B, 1, dev, "block_table")
    return (kv_cache.data_ptr(), n_pages, page, stride, table, ld, block_table.shape[1], lens,
            B), dev


def dsa_window_mha_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k, B, max_len_q, max_len_k, window,
                       sinks, sm_scale, out, lse=None, stream=None):
    """Per-head attention of q [T_q, H, 192] over k [T_k, H, 192], v
    [T_k, H, 128], each query over its last `window` keys (0: all) and the
    sequence's first `sinks` (see include/dsa.h); writes out [T_q, H, 128]
    (bf16) and lse [T_q, H] (fp32, optional)."""
    import torch
    bf16, i32 = torch.bfloat16, torch.int32
    B = int(B)
    T_q, H, d_qk = _dims(q, 3, "q")
    T_k, d_v = _dims(k, 3, "k")[0], _dims(v, 3, "v")[2]
    dev = q.get_device()
    pq = _ten(q, bf16, (T_q, H, d_qk), dev, "q")
    pk = _ten(k, bf16, (T_k, H, d_qk), dev, "k")
    pv = _ten(v, bf16, (T_k, H, d_v), dev, "v")
    po = _ten(out, bf16, (T_q, H, d_v), dev, "out")
    pl = _ten(lse, torch.float32, (T_q, H), dev, "lse")
    cq = _ten(cu_seqlens_q, i32, (B + 1,), dev, "cu_seqlens_q")
    ck = _ten(cu_seqlens_k, i32, (B + 1,), dev, "cu_seqlens_k")
    with _On(dev, stream) as st:
        rc = load().dsa_window_mha_fwd(pq, pk, pv, cq, ck, B, int(max_len_q), int(max_len_k), T_q,
                                       T_k, H, d_qk, d_v, int(window), int(sinks),
                                       float(sm_scale), po, pl, st)
    _check(rc, "dsa_window_mha_fwd")


def dsa_paged_mla_decode_workspace_size(B, H, max_len_k) -> int:
    return int(load().dsa_paged_mla_decode_workspace_size(int(B), int(H), int(max_len_k)))


def dsa_paged_mla_decode(q, kv_cache, block_table, seq_lens, max_len_k, sm_scale, out, lse=None,
                         window=0, sinks=0, workspace=None, stream=None):
    """Attention of one new token per sequence, q [B, H, 576], over a paged
    latent cache (see include/dsa.h): kv_cache [n_pages, page_size, 576] (pages
    may be strided), block_table [B, pages], seq_lens [B].  Writes out
    [B, H, 512] (bf16) and lse [B, H] (fp32, optional).  window > 0 limits a
    token to its last `window` entries and the first `sinks`.  `workspace`
    (uint8 CUDA tensor) is allocated here, on the call's stream, when not
    given."""
    import torch
    max_len_k = int(max_len_k)
    cache, dev = _cache(kv_cache, block_table, seq_lens)
    B = cache[-1]
    _, H, d_qk = _dims(q, 3, "q")
    d_v = _dims(out, 3, "out")[2]
    pq = _ten(q, torch.bfloat16, (B, H, d_qk), dev, "q")
    po = _ten(out, torch.bfloat16, (B, H, d_v), dev, "out")
    pl = _ten(lse, torch.float32, (B, H), dev, "lse")
    pw = None if workspace is None else _ten(workspace, torch.uint8, (workspace.numel(),), dev,
                                             "workspace")
    lib = load()
    with _On(dev, stream) as st:
        if pw is None:
            nbytes = lib.dsa_paged_mla_decode_workspace_size(B, H, max_len_k)
            workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
            pw = workspace.data_ptr()
        rc = lib.dsa_paged_mla_decode(pq, *cache, max_len_k, H, d_qk, d_v, int(window),
                                      int(sinks), float(sm_scale), po, pl, pw, workspace.numel(),
                                      st)
    _check(rc, "dsa_paged_mla_decode")


def dsa_paged_attn_mass(q, kv_cache, block_table, seq_lens, lse, max_len_k, sm_scale, mass_out,
                        mass_in=None, window=0, sinks=0, stream=None):
    """Adds to mass_in [B, >= max_len_k] (None: zeros) the attention weight each
    cached entry got from the newest token, summed over the heads, into mass_out
    (which may be mass_in); lse as dsa_paged_mla_decode wrote it for the same
    arguments (see include/dsa.h)."""
    import torch
    f32 = torch.float32
    max_len_k = int(max_len_k)
    cache, dev = _cache(kv_cache, block_table, seq_lens)
    B = cache[-1]
    _, H, d_qk = _dims(q, 3, "q")
    pq = _ten(q, torch.bfloat16, (B, H, d_qk), dev, "q")
    pl = _ten(lse, f32, (B, H), dev, "lse")
    po, ld = _rows(mass_out, f32, B, max_len_k, dev, "mass_out")
    pi, ld_in = _rows(mass_in, f32, B, max_len_k, dev, "mass_in")
    if pi is not None and ld_in != ld and B > 1:
        raise ValueError("mass_in and mass_out must have the same row stride")
    with _On(dev, stream) as st:
        rc = load().dsa_paged_attn_mass(pq, *cache, max_len_k, H, d_qk, int(window), int(sinks),
                                        float(sm_scale), pl, pi, po, ld, st)
    _check(rc, "dsa_paged_attn_mass")


def dsa_cache_evict(kv_cache, block_table, seq_lens, mass, max_len_k, budget, sinks, recent,
                    new_block_table, new_lens, idx_out, new_mass=None, stream=None):
    """Cuts each sequence of a paged cache down to `budget` entries by mass
    [B, >= max_len_k]: the first `sinks`, the last `recent` and the heaviest
    between are copied to the pages of new_block_table; writes new_lens [B],
    idx_out [B, budget] (old positions, -1 padded) and new_mass
    [B, >= budget] (optional).  See include/dsa.h."""
    import torch
    i32, f32 = torch.int32, torch.float32
    max_len_k, budget = int(max_len_k), int(budget)
    cache, dev = _cache(kv_cache, block_table, seq_lens)
    B = cache[-1]
    pm, ld = _rows(mass, f32, B, max_len_k, dev, "mass")
    pt, ld_t = _rows(new_block_table, i32, B, 1, dev, "new_block_table")
    pn = _ten(new_lens, i32, (B,), dev, "new_lens")
    pi = _ten(idx_out, i32, (B, budget), dev, "idx_out")
    po, ld_o = _rows(new_mass, f32, B, budget, dev, "new_mass")
    with _On(dev, stream) as st:
        rc = load().dsa_cache_evict(*cache, max_len_k, pm, ld, budget, int(sinks), int(recent), pt,
                                    ld_t, new_block_table.shape[1], pn, pi, po, ld_o, st)
    _check(rc, "dsa_cache_evict")


def dsa_get_device_error(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device error
    status: 0 = DSA_OK, 6 = DSA_ERR_TIMEOUT, 7 = DSA_ERR_BOUNDS."""
    return int(load().dsa_get_device_error(_stream(stream)))
