"""GB300-native Lookahead-Sparse-Attention c4 indexer.

Thin Python binding of ``libfm_index.so`` (C ABI in ``include/fm_index.h``):
the functions below carry the C names and only marshal torch tensors into
pointers, sizes and the current CUDA stream.  Every step of the indexer runs
in the library's sm_103a kernels; there is no Python or CPU fallback, and
importing a function whose library is missing raises.

PyTorch provides device memory and streams only.
"""
from __future__ import annotations

import ctypes
import os
import struct

__all__ = [
    "FmError", "lib", "fm_version", "fm_last_error", "fm_device_status", "fm_check_device_status", "fm_memindex_score_mask",
    "fm_topk_workspace", "fm_topk_select", "fm_native_topk_paged_workspace", "fm_native_topk_paged",
    "fm_index_prefill_workspace", "fm_index_prefill_topk", "fm_native_topk_paged_noalloc", "fm_page_recall",
    "fm_native_topk_paged_ex", "fm_memindex_fp8_workspace", "fm_memindex_score_mask_fp8",
    "fm_index_prefill_scores", "fm_retriever_workspace", "fm_retriever_score_mask", "fm_query_chain_workspace",
    "fm_query_chain", "fm_query_chain_layers_workspace", "fm_query_chain_layers", "fm_qk_norm_rope",
    "fm_csa_attn_workspace", "fm_csa_attn", "fm_csa_attn_tree", "fm_prompt_attn", "fm_kv_append_fp8",
    "fm_kv_attn_fp8_workspace", "fm_kv_attn_fp8", "LIB_PATH",
]

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfm_index.so")

FM_OK, FM_ERR_INVALID_ARG, FM_ERR_UNSUPPORTED, FM_ERR_CUDA = 0, 1, 2, 3
FM_ERR_DEVICE_BOUNDS, FM_ERR_WORKSPACE, FM_ERR_DEVICE_TIMEOUT = 4, 5, 6
FM_DEVERR_PAGE_RANGE, FM_DEVERR_TIMEOUT, FM_DEVERR_DUP_PAGE = 0x1, 0x2, 0x4
FM_DTYPE_BF16, FM_DTYPE_FP8_E4M3 = 1, 2  # key element types of a paged pool
FM_NOALLOC_SCRATCH_BYTES = 16 << 20  # the no-allocation paged top-k's built-in scratch (fm_index.h)

_VP, _I64, _I32, _F, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


class FmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"fm status {status}: {message}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libfm_index.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        L.fm_version.restype = ctypes.c_int
        L.fm_last_error.restype = ctypes.c_char_p
        L.fm_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), _I32, _VP]
        L.fm_check_device_status.argtypes = [_VP]
        L.fm_check_device_status.restype = ctypes.c_int
        L.fm_memindex_score_mask.argtypes = [_VP, _VP, _VP, _I64, _I64, _I32, _I32, _I64, _I32, _I32, _F, _VP,
                                             _VP, _VP, _VP]
        for name in ("fm_topk_workspace",):
            if hasattr(L, name):
                getattr(L, name).argtypes = [_I32, _I64]
                getattr(L, name).restype = _SZ
        if hasattr(L, "fm_topk_select"):
            L.fm_topk_select.argtypes = [_VP, _I64, _VP, _I32, _I64, _I32, _VP, _VP, _VP, _SZ, _VP]
        if hasattr(L, "fm_native_topk_paged_workspace"):
            L.fm_native_topk_paged_workspace.argtypes = [_I32, _I32]
            L.fm_native_topk_paged_workspace.restype = _SZ
            L.fm_native_topk_paged.argtypes = [_VP, _VP, _VP, _I32, _VP, _I64, _VP, _VP, _VP, _I32, _I32, _I32,
                                               _I32, _I32, _VP, _VP, _VP, _SZ, _VP]
        if hasattr(L, "fm_native_topk_paged_ex"):
            L.fm_native_topk_paged_ex.argtypes = [_VP, _VP, _VP, _I32, _VP, _I64, _VP, _VP, _VP, _I32, _I32, _I32,
                                                  _I32, _I32, _VP, _I64, _I32, _I32, _VP, _VP, _VP, _SZ, _VP]
        if hasattr(L, "fm_native_topk_paged_noalloc"):
            L.fm_native_topk_paged_noalloc.argtypes = [_VP, _VP, _VP, _VP, _I64, _VP, _VP, _VP, _I32, _I32, _I32,
                                                       _I32, _I32, _VP, _VP, _VP]
            L.fm_native_topk_paged_noalloc.restype = ctypes.c_int
        if hasattr(L, "fm_index_prefill_workspace"):
            L.fm_index_prefill_workspace.argtypes = [_I32, _I64]
            L.fm_index_prefill_workspace.restype = _SZ
            L.fm_index_prefill_topk.argtypes = [_VP, _VP, _VP, _VP, _I32, _I64, _I32, _I32, _I32, _I32, _VP, _VP,
                                                _VP, _SZ, _VP]
        if hasattr(L, "fm_index_prefill_scores"):
            L.fm_index_prefill_scores.argtypes = [_VP, _VP, _VP, _VP, _I32, _I64, _I32, _I32, _I32, _VP, _VP]
            L.fm_index_prefill_scores.restype = ctypes.c_int
        if hasattr(L, "fm_memindex_score_mask_fp8"):
            L.fm_memindex_fp8_workspace.argtypes = [_I32, _I32]
            L.fm_memindex_fp8_workspace.restype = _SZ
            L.fm_memindex_score_mask_fp8.argtypes = [_VP, _VP, _VP, _VP, _I64, _I64, _I64, _I64, _I32, _I32, _I64,
                                                     _I32, _I32, _F, _VP, _VP, _VP, _VP, _SZ, _VP]
        if hasattr(L, "fm_retriever_score_mask"):
            L.fm_retriever_workspace.argtypes = [_I32, _I32, _I32]
            L.fm_retriever_workspace.restype = _SZ
            L.fm_retriever_score_mask.argtypes = [_VP, _VP, _VP, _I64, _I64, _I32, _I32, _I64, _I32, _I32, _I32, _F,
                                                  _VP, _VP, _VP, _VP, _SZ, _VP]
        if hasattr(L, "fm_query_chain"):
            L.fm_query_chain_workspace.argtypes = [_I32, _I32, _I32]
            L.fm_query_chain_workspace.restype = _SZ
            _D = ctypes.c_double
            L.fm_query_chain.argtypes = [_VP, _VP, _VP, _VP, _VP, _VP, _I32, _I32, _I32, _I32, _I32, _I32, _D, _D, _D,
                                         _D, _D, _F, _VP, _VP, _VP, _VP, _SZ, _VP]
        if hasattr(L, "fm_query_chain_layers"):
            _D = ctypes.c_double
            L.fm_query_chain_layers_workspace.argtypes = [_I32, _I32, _I32, _I32]
            L.fm_query_chain_layers_workspace.restype = _SZ
            L.fm_query_chain_layers.argtypes = [_I32, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _I32, _I32, _I32, _I32,
                                                _I32, _D, _D, _D, _D, _D, _F, _VP, _VP, _VP, _VP, _SZ, _VP]
            L.fm_query_chain_layers.restype = ctypes.c_int
        if hasattr(L, "fm_qk_norm_rope"):
            _D = ctypes.c_double
            L.fm_qk_norm_rope.argtypes = [_VP, _I32, _I32, _I32, _D, _D, _D, _D, _D, _F, _VP, _I64, _I32, _VP, _VP, _VP,
                                          _I64, _I32, _VP, _VP, _VP, _I64, _I64, _VP, _VP]
            L.fm_qk_norm_rope.restype = L.fm_qk_norm_rope_packed.restype = ctypes.c_int
            L.fm_qk_norm_rope_packed.argtypes = [ctypes.c_char_p]
        if hasattr(L, "fm_csa_attn"):
            L.fm_csa_attn_workspace.argtypes = [_I32, _I32]
            L.fm_csa_attn_workspace.restype = _SZ
            head = [_VP, _I32, _I32, _I32, _VP, _I64, _I64, _VP, _I32, _I32, _VP, _VP, _I64, _I32, _VP, _I64, _I64, _VP,
                    _I32, _VP, _F]
            tail = [_VP, _VP, _VP, _SZ, _VP]
            L.fm_csa_attn.argtypes = head + tail
            L.fm_csa_attn_tree.argtypes = head + [_VP, _I32, _VP] + tail
            L.fm_csa_attn_packed.argtypes = [ctypes.c_char_p]
            L.fm_csa_attn.restype = L.fm_csa_attn_tree.restype = L.fm_csa_attn_packed.restype = ctypes.c_int
        if hasattr(L, "fm_kv_attn_fp8"):
            L.fm_kv_attn_fp8_workspace.argtypes = [_I32, _I32, _I32, _I32]
            L.fm_kv_attn_fp8_workspace.restype = _SZ
            for name in ("fm_prompt_attn", "fm_kv_append_fp8", "fm_kv_attn_fp8"):
                getattr(L, name).argtypes = [ctypes.c_char_p]
                getattr(L, name).restype = ctypes.c_int
        if hasattr(L, "fm_page_recall"):
            L.fm_page_recall.argtypes = [_VP, _I32, _I64, _I64, _I64, _I32, _VP, _VP, _VP, _VP]
        for name in ("fm_memindex_score_mask", "fm_topk_select", "fm_native_topk_paged", "fm_index_prefill_topk",
                     "fm_device_status", "fm_page_recall", "fm_native_topk_paged_ex", "fm_memindex_score_mask_fp8"):
            if hasattr(L, name):
                getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(status: int) -> None:
    if status != FM_OK:
        raise FmError(status, fm_last_error())


def _stream(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def fm_version() -> int:
    return lib().fm_version()


def fm_last_error() -> str:
    return lib().fm_last_error().decode()


def fm_device_status(reset: bool = True, stream=None) -> int:
    v = ctypes.c_uint32(0)
    _check(lib().fm_device_status(ctypes.byref(v), int(reset), _stream(stream)))
    return v.value


def fm_check_device_status(stream=None) -> None:
    """Raise FmError (FM_ERR_DEVICE_BOUNDS or FM_ERR_DEVICE_TIMEOUT) when a
    kernel flagged the device status word since its last reset; clears it."""
    _check(lib().fm_check_device_status(_stream(stream)))


def fm_memindex_score_mask(q, w, keys, mask_out, maxsig_out=None, logits_out=None, threshold: float = 0.5,
                           stream=None) -> None:
    """q [B,L,64,128] bf16, w [B,L,64] fp32, keys [B,L,S,128] bf16 (any b/l
    strides, rows dense), mask_out [B, ceil(S/32)] int32/uint32,
    maxsig_out [B,S] fp32 or None, logits_out [B,L,S] fp32 or None."""
    B, L, n_h, d = q.shape
    S = keys.shape[2]
    if keys.stride(3) != 1 or keys.stride(2) != d:
        raise ValueError("keys rows must be dense [.., S, d]")
    _check(lib().fm_memindex_score_mask(_ptr(q), _ptr(w), _ptr(keys), keys.stride(0), keys.stride(1), B, L, S, n_h,
                                        d, float(threshold), _ptr(mask_out), _ptr(maxsig_out), _ptr(logits_out),
                                        _stream(stream)))


def fm_memindex_fp8_workspace(B: int, L: int) -> int:
    return lib().fm_memindex_fp8_workspace(B, L)


def fm_memindex_score_mask_fp8(q, w, k8, k_scale, mask_out, maxsig_out=None, logits_out=None, threshold: float = 0.5,
                               workspace=None, stream=None) -> None:
    """q [B,L,64,128] bf16, w [B,L,64] fp32, k8 [B,L,S,128] uint8 E4M3 codes
    (any b/l strides, rows dense), k_scale [B,L,S] fp32 (any b/l strides,
    unit s stride), mask_out [B, ceil(S/32)], maxsig_out [B,S] or None,
    logits_out [B,L,S] or None, workspace >= fm_memindex_fp8_workspace(B, L)."""
    B, L, n_h, d = q.shape
    S = k8.shape[2]
    if k8.stride(3) != 1 or k8.stride(2) != d or k_scale.stride(2) != 1:
        raise ValueError("k8 rows must be dense [.., S, d] and k_scale rows dense [.., S]")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fm_memindex_score_mask_fp8(_ptr(q), _ptr(w), _ptr(k8), _ptr(k_scale), k8.stride(0), k8.stride(1),
                                            k_scale.stride(0), k_scale.stride(1), B, L, S, n_h, d, float(threshold),
                                            _ptr(mask_out), _ptr(maxsig_out), _ptr(logits_out), _ptr(workspace),
                                            ws_bytes, _stream(stream)))


# The retriever's rotary hyperparameters ("FlashMemory-DeepSeek-V4" README, "Hyperparameters").
RETRIEVER_ROPE = dict(rope_base=160000.0, rope_factor=16.0, rope_orig_len=65536.0, rope_beta_fast=32.0,
                      rope_beta_slow=1.0)


def fm_query_chain_workspace(T: int, r: int, n_h: int) -> int:
    return lib().fm_query_chain_workspace(T, r, n_h)


def fm_query_chain(hidden, wq_a, q_norm, wq_b, w_proj, pos, q_out, w_out, q_out_f32=None, eps: float = 1e-6,
                   workspace=None, stream=None, **rope) -> None:
    """hidden [T,dim] bf16, wq_a [r,dim], q_norm [r], wq_b [n_h*128, r], w_proj [n_h,dim] bf16,
    pos [T] int64 -> q_out [T,n_h,128] bf16, w_out [T,n_h] fp32 (q_out_f32 optional)."""
    cfg = dict(RETRIEVER_ROPE, **rope)
    T, dim = hidden.shape
    r = wq_a.shape[0]
    n_h = w_proj.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fm_query_chain(_ptr(hidden), _ptr(wq_a), _ptr(q_norm), _ptr(wq_b), _ptr(w_proj), _ptr(pos), T, dim,
                                r, n_h, 128, 64, cfg["rope_base"], cfg["rope_factor"], cfg["rope_orig_len"],
                                cfg["rope_beta_fast"], cfg["rope_beta_slow"], float(eps), _ptr(q_out),
                                _ptr(q_out_f32), _ptr(w_out), _ptr(workspace), ws_bytes, _stream(stream)))


def fm_query_chain_layers_workspace(L: int, T: int, r: int, n_h: int) -> int:
    return lib().fm_query_chain_layers_workspace(L, T, r, n_h)


def fm_query_chain_layers(hidden, wq_a, q_norm, wq_b, w_proj, pos, q_out, w_out, q_out_f32=None, eps: float = 1e-6,
                          workspace=None, stream=None, **rope) -> None:
    """hidden, wq_a, q_norm, wq_b, w_proj: sequences of L device tensors (one
    per layer, shapes as fm_query_chain); pos [T] int64 -> q_out [T,L,n_h,128]
    bf16, w_out [T,L,n_h] fp32 (q_out_f32 optional)."""
    cfg = dict(RETRIEVER_ROPE, **rope)
    L = len(hidden)
    T, dim = hidden[0].shape
    r = wq_a[0].shape[0]
    n_h = w_proj[0].shape[0]
    arr = lambda ts: (ctypes.c_void_p * L)(*[t.data_ptr() for t in ts])
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fm_query_chain_layers(L, arr(hidden), arr(wq_a), arr(q_norm), arr(wq_b), arr(w_proj), _ptr(pos), T,
                                       dim, r, n_h, 128, 64, cfg["rope_base"], cfg["rope_factor"],
                                       cfg["rope_orig_len"], cfg["rope_beta_fast"], cfg["rope_beta_slow"], float(eps),
                                       _ptr(q_out), _ptr(q_out_f32), _ptr(w_out), _ptr(workspace), ws_bytes,
                                       _stream(stream)))


ENSEMBLE_MAX, ENSEMBLE_MEAN = 0, 1


def fm_retriever_workspace(B: int, L: int, n_h: int = 128) -> int:
    return lib().fm_retriever_workspace(B, L, n_h)


def fm_retriever_score_mask(q, w, compressed_k, mask_out, ens_out=None, logits_out=None, ensemble: int = ENSEMBLE_MAX,
                            threshold: float = 0.5, workspace=None, stream=None) -> None:
    """q [B,L,n_h,128] bf16 (n_h 64 or 128), w [B,L,n_h] fp32, compressed_k
    [B,L,S,132] uint8 packed rows (any b/l strides, rows dense), mask_out
    [B, ceil(S/32)], ens_out [B,S] or None, logits_out [B,L,S] or None,
    ensemble ENSEMBLE_MAX or ENSEMBLE_MEAN, workspace >=
    fm_retriever_workspace(B, L, n_h)."""
    B, L, n_h, d = q.shape
    S = compressed_k.shape[2]
    if compressed_k.stride(3) != 1 or compressed_k.stride(2) != d + 4:
        raise ValueError("compressed_k rows must be dense [.., S, 132]")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fm_retriever_score_mask(_ptr(q), _ptr(w), _ptr(compressed_k), compressed_k.stride(0),
                                         compressed_k.stride(1), B, L, S, n_h, d, int(ensemble), float(threshold),
                                         _ptr(mask_out), _ptr(ens_out), _ptr(logits_out), _ptr(workspace), ws_bytes,
                                         _stream(stream)))


def fm_topk_workspace(rows: int, n: int) -> int:
    return lib().fm_topk_workspace(rows, n)


def fm_topk_select(scores, k: int, idx_out, score_out=None, n_valid=None, n=None, workspace=None,
                   stream=None) -> None:
    """scores [rows, ld] fp32 (row stride ld, unit column stride); n_valid [rows]
    int32 or None; idx_out [rows, k] int32; score_out [rows, k] fp32 or None."""
    rows, ld = scores.shape[0], scores.stride(0)
    n = scores.shape[1] if n is None else n
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fm_topk_select(_ptr(scores), ld, _ptr(n_valid), rows, n, k, _ptr(idx_out), _ptr(score_out),
                                _ptr(workspace), ws_bytes, _stream(stream)))


def fm_native_topk_paged_workspace(Q: int, R: int) -> int:
    return lib().fm_native_topk_paged_workspace(Q, R)


def _key_dtype(k_pool) -> int:
    """The pool's key type from its tensor dtype: uint8 holds E4M3 codes;
    int16 / bfloat16 hold bf16 keys."""
    import torch
    if k_pool.dtype == torch.uint8:
        return FM_DTYPE_FP8_E4M3
    if k_pool.dtype in (torch.int16, torch.bfloat16):
        return FM_DTYPE_BF16
    raise ValueError(f"k_pool dtype {k_pool.dtype}: uint8 (E4M3 codes) or int16/bfloat16 (bf16 keys)")


def fm_native_topk_paged(q, w, k_pool, k_scale, page_phys, page_logical, k: int, idx_out, score_out=None,
                         n_res=None, workspace=None, stream=None) -> None:
    """q [Q,64,128] bf16, w [Q,64] fp32, k_pool [P,64,128]: uint8 E4M3 codes
    with k_scale [P,64] fp32, or int16/bfloat16 bf16 keys with k_scale None;
    page_phys/page_logical [Q,R] int32, n_res [Q] int32 or None, idx_out
    [Q,k] int32, score_out [Q,k] fp32 or None."""
    Q, n_h, d = q.shape
    R = page_phys.shape[1]
    P = k_pool.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fm_native_topk_paged(_ptr(q), _ptr(w), _ptr(k_pool), _key_dtype(k_pool), _ptr(k_scale), P,
                                      _ptr(page_phys),
                                      _ptr(page_logical), _ptr(n_res), Q, R, n_h, d, k, _ptr(idx_out),
                                      _ptr(score_out), _ptr(workspace), ws_bytes, _stream(stream)))


def fm_native_topk_paged_ex(q, w, k_pool, k_scale, page_phys, page_logical, k: int, idx_out, score_out=None,
                            n_res=None, res_mask=None, mask_group: int = 1, id_mode: int = 0, workspace=None,
                            stream=None) -> None:
    """fm_native_topk_paged plus the Level-2 resident mask res_mask
    [rows, mask_ld] int32/uint32 (row qi // mask_group per query, or None) and
    id_mode (0 = logical chunk ids, 1 = reserve cells phys * 64 + o)."""
    Q, n_h, d = q.shape
    R = page_phys.shape[1]
    P = k_pool.shape[0]
    mask_ld = 0 if res_mask is None else res_mask.shape[1]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fm_native_topk_paged_ex(_ptr(q), _ptr(w), _ptr(k_pool), _key_dtype(k_pool), _ptr(k_scale), P,
                                         _ptr(page_phys),
                                         _ptr(page_logical), _ptr(n_res), Q, R, n_h, d, k, _ptr(res_mask), mask_ld,
                                         mask_group, id_mode, _ptr(idx_out), _ptr(score_out), _ptr(workspace),
                                         ws_bytes, _stream(stream)))


def fm_native_topk_paged_noalloc(q, w, k_pool, k_scale, page_phys, page_logical, k: int, idx_out, score_out=None,
                                 n_res=None, stream=None) -> None:
    """fm_native_topk_paged without a workspace, for callers that cannot
    allocate device memory: the scratch is a fixed 16 MiB array inside the
    library (shared by all calls; serialise calls that could overlap)."""
    Q, n_h, d = q.shape
    R = page_phys.shape[1]
    P = k_pool.shape[0]
    _check(lib().fm_native_topk_paged_noalloc(_ptr(q), _ptr(w), _ptr(k_pool), _ptr(k_scale), P, _ptr(page_phys),
                                              _ptr(page_logical), _ptr(n_res), Q, R, n_h, d, k, _ptr(idx_out),
                                              _ptr(score_out), _stream(stream)))


def fm_index_prefill_workspace(T: int, S: int) -> int:
    return lib().fm_index_prefill_workspace(T, S)


def fm_index_prefill_topk(q, w, pos, keys, k: int, idx_out, score_out=None, ratio: int = 4, workspace=None,
                          stream=None) -> None:
    """q [T,64,128] bf16, w [T,64] fp32, pos [T] int64, keys [S,128] bf16,
    idx_out [T,k] int32, score_out [T,k] fp32 or None."""
    T, n_h, d = q.shape
    S = keys.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fm_index_prefill_topk(_ptr(q), _ptr(w), _ptr(pos), _ptr(keys), T, S, n_h, d, ratio, k,
                                       _ptr(idx_out), _ptr(score_out), _ptr(workspace), ws_bytes, _stream(stream)))


def fm_index_prefill_scores(q, w, pos, keys, logits_out, ratio: int = 4, stream=None) -> None:
    """q [T,64,128] bf16, w [T,64] fp32, pos [T] int64, keys [S,128] bf16,
    logits_out [T,S] fp32 (contiguous): the dense scores, -inf past each
    token's causal limit."""
    T, n_h, d = q.shape
    S = keys.shape[0]
    _check(lib().fm_index_prefill_scores(_ptr(q), _ptr(w), _ptr(pos), _ptr(keys), T, S, n_h, d, ratio,
                                         _ptr(logits_out), _stream(stream)))


def fm_page_recall(mask, S: int, kmax: int, pages_out, density_out=None, n_out=None, sink: int = 0, recent: int = 0,
                   stream=None) -> None:
    """mask [B, ceil(S/32)] int32/uint32 (fm_memindex_score_mask's output),
    pages_out [B, kmax] int32, density_out [B, kmax] int32 or None, n_out [B]
    int32 or None."""
    B = mask.shape[0]
    _check(lib().fm_page_recall(_ptr(mask), B, S, sink, recent, kmax, _ptr(pages_out), _ptr(density_out),
                                _ptr(n_out), _stream(stream)))


# The wrappers below check every tensor they are given, on each call; a decode step
# waits for that, so the checks of an accepted tensor are a few attribute reads and
# the reasons are worked out only for a refused one.
# fm_qk_norm_rope_args and fm_csa_attn_args: one argument through ctypes instead of 25
_QK_ARGS = struct.Struct("@P3i5dfPqi3Pqi3P2q2P")
_ATTN_ARGS = struct.Struct("@P3iP2qP2i2PqiP2qPiPfiPi4PNP")
# fm_kv_append_fp8_args, fm_kv_attn_fp8_args, fm_prompt_attn_args
_APPEND_ARGS = struct.Struct("@PqPq4iPqP4P3qP2i2P5diP")
_KV_ATTN_ARGS = struct.Struct("@Pq4i4P3qP2i2PqPf3PNP")
_PROMPT_ARGS = struct.Struct("@PqPqPq6i2PqPf3P")
_NO_WINDOW = (1 << 63) - 1
_BF16 = _BITS = _I32T = _I64T = _F32T = _U8T = _E4M3 = frozenset()  # accepted element types, set by _types()
_current_device = _raw_stream = None


def _types():
    import torch
    global _BF16, _BITS, _I32T, _I64T, _F32T, _U8T, _E4M3, _current_device, _raw_stream
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    # the current stream's handle alone: a tenth of the time of current_stream()
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    _BITS, _I32T, _I64T = frozenset((torch.int32, torch.uint32)), frozenset((torch.int32,)), frozenset((torch.int64,))
    _F32T, _U8T = frozenset((torch.float32,)), frozenset((torch.uint8,))
    _E4M3 = frozenset((torch.uint8, torch.float8_e4m3fn))  # codes, or the values that they are
    _BF16 = frozenset((torch.bfloat16, torch.int16, torch.uint16))  # bf16 tensors, or their bit patterns


def _refuse(t, name, types, shape, dev, rows):
    if t.dtype not in types:
        raise ValueError(f"{name}: dtype {t.dtype}, need {' or '.join(sorted(map(str, types)))}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, need {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the other tensors are on {'cuda:%d' % dev if dev >= 0 else 'cpu'}")
    raise ValueError(f"{name}: strides {t.stride()} of shape {tuple(shape)}: "
                     f"{'all but the first dimension' if rows else 'the tensor'} must be dense")


def _dense(t, name, types, shape, dev):
    """Pointer of a dense tensor of these types, this shape and device (-1: CPU)."""
    if t.dtype in types and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, types, shape, dev, False)


def _rows(t, name, types, shape, dev):
    """Pointer and first stride of a 3-dimensional tensor that is dense but for its
    first dimension (the dense stride where one row or none leaves it open)."""
    if t.dtype in types and t.shape == shape and t.get_device() == dev:
        if t.is_contiguous():
            return t.data_ptr(), shape[1] * shape[2]
        stride = t.stride()
        if (stride[2] == 1 and stride[1] == shape[2]) or (shape[0] and t[0].is_contiguous()):
            return t.data_ptr(), stride[0]
    _refuse(t, name, types, shape, dev, True)


def _device(t, name):
    """The tensor's device index (-1: CPU), which must be the current device: the
    call's stream and kernels are that device's."""
    if not _BF16:
        _types()
    dev = t.get_device()
    if dev >= 0 and dev != _current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{_current_device()}")
    return dev


def _shape(t, name, dims):
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name}: shape {tuple(shape)}, need {dims} dimensions")
    return shape


def fm_qk_norm_rope(pos, q=None, q_gain=None, q_out=None, k=None, k_gain=None, k_out=None, k_pool=None, k_cell=None,
                    rope_dim: int = 64, eps: float = 1e-6, stream=None, rope_base: float = RETRIEVER_ROPE["rope_base"],
                    rope_factor: float = RETRIEVER_ROPE["rope_factor"],
                    rope_orig_len: float = RETRIEVER_ROPE["rope_orig_len"],
                    rope_beta_fast: float = RETRIEVER_ROPE["rope_beta_fast"],
                    rope_beta_slow: float = RETRIEVER_ROPE["rope_beta_slow"]) -> None:
    """pos [T] int64; q [T,n_q,d] bf16 (any token stride) -> q_out [T,n_q,d];
    k [T,n_k,d] bf16 (any token stride) -> k_out [T,n_k,d] and/or rows
    k_cell [T] int32 of k_pool [P,64,n_k*d] (any page stride).  q or k may be
    None.  RMSNorm per head with q_gain / k_gain [d] (None: ones), then the
    rotation of the last rope_dim entries (YaRN; RETRIEVER_ROPE's parameters)."""
    if q is None and k is None:
        raise ValueError("q or k is needed")
    dev = _device(pos, "pos")
    T, _, d = _shape(k, "k", 3) if q is None else _shape(q, "q", 3)
    n_q = n_k = P = q_stride = k_stride = page_stride = 0
    q_p = qg_p = qo_p = k_p = kg_p = ko_p = kp_p = kc_p = 0
    if q is not None:
        if q_out is None:
            raise ValueError("q needs q_out")
        shape = q.shape
        n_q = shape[1]
        q_p, q_stride = _rows(q, "q", _BF16, (T, n_q, d), dev)
        qo_p = _dense(q_out, "q_out", _BF16, shape, dev)
        if q_gain is not None:
            qg_p = _dense(q_gain, "q_gain", _BF16, (d,), dev)
    if k is not None:
        if k_out is None and k_pool is None:
            raise ValueError("k needs k_out or k_pool")
        shape = _shape(k, "k", 3)
        n_k = shape[1]
        k_p, k_stride = _rows(k, "k", _BF16, (T, n_k, d), dev)
        if k_gain is not None:
            kg_p = _dense(k_gain, "k_gain", _BF16, (d,), dev)
        if k_out is not None:
            ko_p = _dense(k_out, "k_out", _BF16, shape, dev)
        if k_pool is not None:
            if k_cell is None:
                raise ValueError("k_pool needs k_cell")
            P = k_pool.shape[0]
            kp_p, page_stride = _rows(k_pool, "k_pool", _BF16, (P, 64, n_k * d), dev)
            kc_p = _dense(k_cell, "k_cell", _I32T, (T,), dev)
    pos_p = _dense(pos, "pos", _I64T, (T,), dev)
    if dev < 0:
        raise ValueError("the tensors are on the CPU")
    try:
        args = _QK_ARGS.pack(pos_p, T, d, rope_dim, rope_base, rope_factor, rope_orig_len, rope_beta_fast, rope_beta_slow,
                             eps, q_p, q_stride, n_q, qg_p, qo_p, k_p, k_stride, n_k, kg_p, ko_p, kp_p, P, page_stride,
                             kc_p, _raw_stream(dev) if stream is None else _stream(stream))
    except (struct.error, OverflowError) as e:
        raise ValueError(f"fm_qk_norm_rope: {e}") from None
    st = lib().fm_qk_norm_rope_packed(args)
    if st:
        _check(st)


def fm_csa_attn_workspace(T: int, n_h: int) -> int:
    return lib().fm_csa_attn_workspace(T, n_h)


def _csa_attn(tree, q, kv_pool, page_table, pos, out, window, n_sink, seq, cell_pool, cells, sink_logit, scale, lse_out,
              workspace, stream):
    dev = _device(q, "q")
    shape = _shape(q, "q", 3)
    T, n_h, d = shape
    P = kv_pool.shape[0]
    kv_p, kv_stride = _rows(kv_pool, "kv_pool", _BF16, (P, 64, d), dev)
    B, R = _shape(page_table, "page_table", 2)
    seq_p = sink_p = lse_p = cp_p = cells_p = 0
    k = Pc = 0
    cp_stride = 64 * d
    if seq is not None:
        seq_p = _dense(seq, "seq", _I32T, (T,), dev)
    if cells is not None:
        if cell_pool is None:
            raise ValueError("cells needs cell_pool")
        k = _shape(cells, "cells", 2)[1]
        Pc = cell_pool.shape[0]
        cp_p, cp_stride = _rows(cell_pool, "cell_pool", _BF16, (Pc, 64, d), dev)
        cells_p = _dense(cells, "cells", _I32T, (T, k), dev)
    elif cell_pool is not None:
        raise ValueError("cell_pool needs cells")
    if sink_logit is not None:
        sink_p = _dense(sink_logit, "sink_logit", _F32T, (n_h,), dev)
    if lse_out is not None:
        lse_p = _dense(lse_out, "lse_out", _F32T, (T, n_h), dev)
    ws_p = ws_bytes = 0
    if workspace is not None:
        ws_bytes = workspace.shape[0]
        ws_p = _dense(workspace, "workspace", _U8T, (ws_bytes,), dev)
    mask_p = base_p = words = 0
    if tree is not None:
        tree_mask, tree_base = tree
        words = _shape(tree_mask, "tree_mask", 2)[1]
        mask_p = _dense(tree_mask, "tree_mask", _BITS, (T, words), dev)
        base_p = _dense(tree_base, "tree_base", _I64T, (B,), dev)
    q_p, out_p = _dense(q, "q", _BF16, shape, dev), _dense(out, "out", _BF16, shape, dev)
    table_p, pos_p = _dense(page_table, "page_table", _I32T, (B, R), dev), _dense(pos, "pos", _I64T, (T,), dev)
    if dev < 0:
        raise ValueError("the tensors are on the CPU")
    try:
        args = _ATTN_ARGS.pack(q_p, T, n_h, d, kv_p, P, kv_stride, table_p, B, R, seq_p, pos_p, window, n_sink, cp_p, Pc,
                               cp_stride, cells_p, k, sink_p, d ** -0.5 if scale is None else scale, tree is not None,
                               mask_p, words, base_p, out_p, lse_p, ws_p, ws_bytes,
                               _raw_stream(dev) if stream is None else _stream(stream))
    except (struct.error, OverflowError) as e:
        raise ValueError(f"fm_csa_attn: {e}") from None
    st = lib().fm_csa_attn_packed(args)
    if st:
        _check(st)


def fm_csa_attn(q, kv_pool, page_table, pos, out, window: int, n_sink: int = 0, seq=None, cell_pool=None, cells=None,
                sink_logit=None, scale=None, lse_out=None, workspace=None, stream=None) -> None:
    """q [T,n_h,512] bf16, kv_pool [P,64,512] bf16 (any page stride), page_table
    [B,R] int32, pos [T] int64, seq [T] int32 (None: token t is row t), cells
    [T,k] int32 rows of cell_pool [Pc,64,512] (both None: none), sink_logit
    [n_h] fp32 or None, scale (None: 512 ** -0.5) -> out [T,n_h,512] bf16,
    lse_out [T,n_h] fp32 or None; workspace uint8 [>= fm_csa_attn_workspace(T,
    n_h)].  A layer without cached tokens passes a kv_pool of no pages and a
    page_table [T,0]."""
    _csa_attn(None, q, kv_pool, page_table, pos, out, window, n_sink, seq, cell_pool, cells, sink_logit, scale, lse_out,
              workspace, stream)


def fm_csa_attn_tree(q, kv_pool, page_table, pos, out, window: int, tree_mask, tree_base, n_sink: int = 0, seq=None,
                     cell_pool=None, cells=None, sink_logit=None, scale=None, lse_out=None, workspace=None,
                     stream=None) -> None:
    """fm_csa_attn for drafted tokens: sequence b's drafted token i is in cache
    slot tree_base[b] + i (tree_base [B] int64); tree_mask [T, words] int32 or
    uint32 has bit i & 31 of word i >> 5 set where token t sees it."""
    _csa_attn((tree_mask, tree_base), q, kv_pool, page_table, pos, out, window, n_sink, seq, cell_pool, cells, sink_logit,
              scale, lse_out, workspace, stream)


def _pages(t, name, types, shape, dev):
    """Pointer and first stride of a 4-dimensional pool that is dense but for its first
    dimension, as _rows."""
    if t.dtype in types and t.shape == shape and t.get_device() == dev:
        if t.is_contiguous():
            return t.data_ptr(), shape[1] * shape[2] * shape[3]
        if shape[0] and t[0].is_contiguous():
            return t.data_ptr(), t.stride(0)
    _refuse(t, name, types, shape, dev, True)


def _cache(k_pool, v_pool, k_scale, v_scale, n_k, d, dev):
    """Pointers and strides of the 8-bit cache's four arrays: (k, v, k_scale, v_scale,
    P, page_stride, scale_stride)."""
    P = k_pool.shape[0]
    k_p, page = _pages(k_pool, "k_pool", _E4M3, (P, n_k, 64, d), dev)
    v_p, v_page = _pages(v_pool, "v_pool", _E4M3, (P, n_k, 64, d), dev)
    ks_p, stride = _rows(k_scale, "k_scale", _F32T, (P, n_k, 4), dev)
    vs_p, v_stride = _rows(v_scale, "v_scale", _F32T, (P, n_k, 4), dev)
    if P > 1 and (page != v_page or stride != v_stride):
        raise ValueError(f"k_pool and v_pool, and k_scale and v_scale, need the same stride from page to page: "
                         f"{page} and {v_page}, {stride} and {v_stride}")
    return k_p, v_p, ks_p, vs_p, P, page, stride


def _packed(T, page_table, start, cu_tokens, dev):
    """(B, R, page_table, start, cu_tokens) of a call over cached sequences."""
    B, R = _shape(page_table, "page_table", 2)
    table_p = _dense(page_table, "page_table", _I32T, (B, R), dev)
    start_p = _dense(start, "start", _I64T, (B,), dev)
    cu_p = 0
    if cu_tokens is not None:
        cu_p = _dense(cu_tokens, "cu_tokens", _I32T, (B + 1,), dev)
    elif T != B:
        raise ValueError(f"without cu_tokens every sequence has one token: {T} tokens, {B} rows of page_table")
    return B, R, table_p, start_p, cu_p


def fm_kv_append_fp8(k, v, k_pool, v_pool, k_scale, v_scale, page_table, start, cu_tokens=None, q=None, q_out=None,
                     rope_dim: int = 64, stream=None, rope_base: float = RETRIEVER_ROPE["rope_base"],
                     rope_factor: float = RETRIEVER_ROPE["rope_factor"],
                     rope_orig_len: float = RETRIEVER_ROPE["rope_orig_len"],
                     rope_beta_fast: float = RETRIEVER_ROPE["rope_beta_fast"],
                     rope_beta_slow: float = RETRIEVER_ROPE["rope_beta_slow"]) -> None:
    """k, v [T,n_k,d] bf16 (any token stride) into the 8-bit cache k_pool, v_pool
    [P,n_k,64,d] uint8 or float8_e4m3fn and k_scale, v_scale [P,n_k,4] fp32 (any page
    stride), a scale for each 16 positions and head; page_table [B,R] int32, start [B]
    int64 the tokens that a sequence has already, cu_tokens [B+1] int32 the packed
    sequences' offsets (None: one token each).  The last rope_dim entries of k are turned by
    their positions on the way (0: none), and those of q [T,n_h,d] into q_out."""
    dev = _device(k, "k")
    T, n_k, d = _shape(k, "k", 3)
    k_p, k_stride = _rows(k, "k", _BF16, (T, n_k, d), dev)
    v_p, v_stride = _rows(v, "v", _BF16, (T, n_k, d), dev)
    n_h = q_p = q_stride = qo_p = 0
    if q is not None:
        if q_out is None:
            raise ValueError("q needs q_out")
        shape = _shape(q, "q", 3)
        n_h = shape[1]
        q_p, q_stride = _rows(q, "q", _BF16, (T, n_h, d), dev)
        qo_p = _dense(q_out, "q_out", _BF16, shape, dev)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    cache = _cache(k_pool, v_pool, k_scale, v_scale, n_k, d, dev)
    B, R, table_p, start_p, cu_p = _packed(T, page_table, start, cu_tokens, dev)
    if dev < 0:
        raise ValueError("the tensors are on the CPU")
    try:
        args = _APPEND_ARGS.pack(k_p, k_stride, v_p, v_stride, T, n_k, d, n_h, q_p, q_stride, qo_p, *cache, table_p, B, R,
                                 start_p, cu_p, rope_base, rope_factor, rope_orig_len, rope_beta_fast, rope_beta_slow,
                                 rope_dim, _raw_stream(dev) if stream is None else _stream(stream))
    except (struct.error, OverflowError) as e:
        raise ValueError(f"fm_kv_append_fp8: {e}") from None
    st = lib().fm_kv_append_fp8(args)
    if st:
        _check(st)


def fm_kv_attn_fp8_workspace(T: int, n_h: int, n_k: int, d: int) -> int:
    return lib().fm_kv_attn_fp8_workspace(T, n_h, n_k, d)


def fm_kv_attn_fp8(q, k_pool, v_pool, k_scale, v_scale, page_table, start, out, cu_tokens=None, window=None,
                   sink_logit=None, scale=None, lse_out=None, workspace=None, stream=None) -> None:
    """q [T,n_h,d] bf16 (any token stride) over the 8-bit cache (fm_kv_append_fp8's
    arrays): token i of sequence b is at position start[b] + i and attends to the cached
    positions up to its own, the last `window` of them (None: all); sink_logit [n_h] fp32
    or None, scale (None: d ** -0.5) -> out [T,n_h,d] bf16, lse_out [T,n_h] fp32 or
    None; workspace uint8 [>= fm_kv_attn_fp8_workspace(T, n_h, n_k, d)]."""
    dev = _device(q, "q")
    shape = _shape(q, "q", 3)
    T, n_h, d = shape
    n_k = _shape(k_pool, "k_pool", 4)[1]
    q_p, q_stride = _rows(q, "q", _BF16, shape, dev)
    out_p = _dense(out, "out", _BF16, shape, dev)
    cache = _cache(k_pool, v_pool, k_scale, v_scale, n_k, d, dev)
    B, R, table_p, start_p, cu_p = _packed(T, page_table, start, cu_tokens, dev)
    sink_p = lse_p = ws_p = ws_bytes = 0
    if sink_logit is not None:
        sink_p = _dense(sink_logit, "sink_logit", _F32T, (n_h,), dev)
    if lse_out is not None:
        lse_p = _dense(lse_out, "lse_out", _F32T, (T, n_h), dev)
    if workspace is not None:
        ws_bytes = workspace.shape[0]
        ws_p = _dense(workspace, "workspace", _U8T, (ws_bytes,), dev)
    if dev < 0:
        raise ValueError("the tensors are on the CPU")
    try:
        args = _KV_ATTN_ARGS.pack(q_p, q_stride, T, n_h, n_k, d, *cache, table_p, B, R, start_p, cu_p,
                                  _NO_WINDOW if window is None else window, sink_p, d ** -0.5 if scale is None else scale,
                                  out_p, lse_p, ws_p, ws_bytes, _raw_stream(dev) if stream is None else _stream(stream))
    except (struct.error, OverflowError) as e:
        raise ValueError(f"fm_kv_attn_fp8: {e}") from None
    st = lib().fm_kv_attn_fp8(args)
    if st:
        _check(st)


def fm_prompt_attn(q, k, v, out, cu_q=None, cu_k=None, window=None, sink_logit=None, scale=None, lse_out=None,
                   stream=None) -> None:
    """Causal attention over whole prompts: q [T,n_h,d], k, v [Tk,n_k,d] bf16 (any token
    strides), packed sequences with offsets cu_q [B+1] int32 (None: one sequence) and cu_k
    (None: cu_q's); a sequence's queries are the last of its keys.  window (None: no
    limit), sink_logit [n_h] fp32 or None, scale (None: d ** -0.5) -> out [T,n_h,d] bf16,
    lse_out [T,n_h] fp32 or None."""
    dev = _device(q, "q")
    shape = _shape(q, "q", 3)
    T, n_h, d = shape
    Tk, n_k, _ = _shape(k, "k", 3)
    q_p, q_stride = _rows(q, "q", _BF16, shape, dev)
    k_p, k_stride = _rows(k, "k", _BF16, (Tk, n_k, d), dev)
    v_p, v_stride = _rows(v, "v", _BF16, (Tk, n_k, d), dev)
    out_p = _dense(out, "out", _BF16, shape, dev)
    B, cuq_p, cuk_p, sink_p, lse_p = 1, 0, 0, 0, 0
    if cu_q is not None:
        B = _shape(cu_q, "cu_q", 1)[0] - 1
        cuq_p = _dense(cu_q, "cu_q", _I32T, (B + 1,), dev)
    if cu_k is not None:
        if cu_q is None:
            raise ValueError("cu_k needs cu_q")
        cuk_p = _dense(cu_k, "cu_k", _I32T, (B + 1,), dev)
    if sink_logit is not None:
        sink_p = _dense(sink_logit, "sink_logit", _F32T, (n_h,), dev)
    if lse_out is not None:
        lse_p = _dense(lse_out, "lse_out", _F32T, (T, n_h), dev)
    if dev < 0:
        raise ValueError("the tensors are on the CPU")
    try:
        args = _PROMPT_ARGS.pack(q_p, q_stride, k_p, k_stride, v_p, v_stride, T, Tk, n_h, n_k, d, B, cuq_p, cuk_p,
                                 _NO_WINDOW if window is None else window, sink_p, d ** -0.5 if scale is None else scale,
                                 out_p, lse_p, _raw_stream(dev) if stream is None else _stream(stream))
    except (struct.error, OverflowError) as e:
        raise ValueError(f"fm_prompt_attn: {e}") from None
    st = lib().fm_prompt_attn(args)
    if st:
        _check(st)
