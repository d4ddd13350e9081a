"""Python binding of libhqq: the C ABI of include/hqq.h, argument marshalling only.

Every compute step runs in the HIP library; this module passes device pointers
(``tensor.data_ptr()``), sizes and the current HIP stream through ctypes. PyTorch provides
device memory and streams. There is no fallback: if the library is missing the import of a
function raises.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libhqq.so")

HQQ_OK, HQQ_ERR_ARG, HQQ_ERR_UNSUPPORTED, HQQ_ERR_WORKSPACE, HQQ_ERR_DEVICE = range(5)
HQQ_F16, HQQ_BF16 = range(2)

# Functions declared in include/hqq.h (checked by the tests against the header).
EXPORTS = ("hqq_packed_bytes", "hqq_workspace_bytes", "hqq_quantize", "hqq_quantize_batch",
           "hqq_solve_batch", "hqq_requant_batch", "hqq_quantize_streamed",
           "hqq_streamed_workspace_bytes", "hqq_dequantize", "hqq_gemm",
           "hqq_gemm_workspace_bytes", "hqq_gemm_f16", "hqq_requant_scales",
           "hqq_dequantize_scales", "hqq_pack", "hqq_unpack", "hqq_status_string",
           "hqq_last_error", "hqq_batch_check", "hqq_debug_solver", "hqq_quantize_noalloc",
           "hqq_gemm_multi", "hqq_cache_write", "hqq_cache_read", "hqq_cache_attention",
           "hqq_cache_attention_prefix", "hqq_cache_attention_workspace")


class HQQError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{msg} (status {status})")
        self.status = status


class hqq_job(C.Structure):
    _fields_ = [("W", C.c_void_p), ("rows", C.c_int64), ("cols", C.c_int64),
                ("nbits", C.c_int), ("group_size", C.c_int), ("axis", C.c_int),
                ("p", C.c_float), ("beta", C.c_float), ("kappa", C.c_float),
                ("iters", C.c_int), ("early_stop", C.c_int), ("zero_bits", C.c_int),
                ("packed", C.c_void_p), ("scale", C.c_void_p), ("zero", C.c_void_p),
                ("zero_meta", C.c_void_p), ("passes", C.c_void_p)]


class hqq_gemm_weight(C.Structure):
    _fields_ = [("packed", C.c_void_p), ("scale", C.c_void_p), ("zero", C.c_void_p),
                ("zero_meta", C.c_void_p), ("N", C.c_int64), ("nbits", C.c_int),
                ("group_size", C.c_int), ("zero_bits", C.c_int), ("Y", C.c_void_p)]


class hqq_cache(C.Structure):
    _fields_ = [("k_codes", C.c_void_p), ("v_codes", C.c_void_p), ("k_meta", C.c_void_p),
                ("v_meta", C.c_void_p), ("n_pages", C.c_int64), ("page_size", C.c_int),
                ("n_heads", C.c_int), ("head_dim", C.c_int), ("nbits", C.c_int),
                ("group_size", C.c_int), ("dtype", C.c_int)]


class hqq_seqs(C.Structure):
    _fields_ = [("table", C.c_void_p), ("lens", C.c_void_p), ("cu_tokens", C.c_void_p),
                ("n_seqs", C.c_int), ("max_pages", C.c_int), ("n_tokens", C.c_int64)]


_L = None


def lib():
    """The loaded library. Raises if it has not been built (no CPU fallback exists)."""
    global _L
    if _L is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = C.CDLL(LIB_PATH)
        vp, i64, i32, f32 = C.c_void_p, C.c_int64, C.c_int, C.c_float
        L.hqq_packed_bytes.restype = C.c_size_t
        L.hqq_packed_bytes.argtypes = [i64, i32]
        L.hqq_workspace_bytes.restype = C.c_size_t
        L.hqq_workspace_bytes.argtypes = [C.POINTER(hqq_job), i32]
        L.hqq_quantize.restype = i32
        L.hqq_quantize.argtypes = [vp, i64, i64, i32, i32, i32, f32, f32, f32, i32, i32, i32,
                                   vp, vp, vp, vp, vp, vp, C.c_size_t, vp]
        L.hqq_quantize_noalloc.restype = i32
        L.hqq_quantize_noalloc.argtypes = [vp, i64, i64, i32, i32, i32, f32, f32, f32, i32, i32,
                                           i32, vp, vp, vp, vp, vp, vp]
        for name in ("hqq_quantize_batch", "hqq_solve_batch", "hqq_requant_batch"):
            getattr(L, name).restype = i32
            getattr(L, name).argtypes = [C.POINTER(hqq_job), i32, vp, C.c_size_t, vp]
        L.hqq_batch_check.restype = i32
        L.hqq_batch_check.argtypes = [C.POINTER(hqq_job), i32, vp, C.c_size_t, vp]
        L.hqq_debug_solver.restype = None
        L.hqq_debug_solver.argtypes = [i64, i32]
        L.hqq_quantize_streamed.restype = i32
        L.hqq_quantize_streamed.argtypes = [C.POINTER(hqq_job), i32, vp, C.c_size_t, vp,
                                            C.c_size_t, vp, vp]
        L.hqq_streamed_workspace_bytes.restype = C.c_size_t
        L.hqq_streamed_workspace_bytes.argtypes = [C.POINTER(hqq_job), i32, C.c_size_t]
        L.hqq_dequantize.restype = i32
        L.hqq_dequantize.argtypes = [vp, vp, vp, vp, i64, i64, i32, i32, i32, i32, vp, vp]
        L.hqq_gemm.restype = i32
        L.hqq_gemm.argtypes = [vp, i64, vp, vp, vp, vp, i64, i64, i32, i32, i32, vp, vp,
                               C.c_size_t, vp]
        L.hqq_gemm_workspace_bytes.restype = C.c_size_t
        L.hqq_gemm_workspace_bytes.argtypes = [i64, i64, i64]
        L.hqq_gemm_multi.restype = i32
        L.hqq_gemm_multi.argtypes = [vp, i64, i64, C.POINTER(hqq_gemm_weight), i32, vp, C.c_size_t, vp]
        L.hqq_gemm_f16.restype = i32
        L.hqq_gemm_f16.argtypes = [vp, i64, vp, i64, i64, vp, vp]
        L.hqq_requant_scales.restype = i32
        L.hqq_requant_scales.argtypes = [vp, i64, i32, vp, vp, vp]
        L.hqq_dequantize_scales.restype = i32
        L.hqq_dequantize_scales.argtypes = [vp, vp, i64, i32, vp, vp]
        L.hqq_pack.restype = i32
        L.hqq_pack.argtypes = [vp, i64, i32, vp, vp]
        L.hqq_unpack.restype = i32
        L.hqq_unpack.argtypes = [vp, i64, i32, vp, vp]
        cp, sp, st = vp, vp, C.c_size_t         # structs: by reference, or packed
        for name in ("hqq_cache_write", "hqq_cache_read"):
            getattr(L, name).restype = i32
            getattr(L, name).argtypes = [cp, sp, vp, i64, i64, vp, i64, i64, vp]
        L.hqq_cache_attention.restype = i32
        L.hqq_cache_attention.argtypes = [cp, sp, vp, i64, i64, i32, f32, vp, i64, i64, vp, vp, st, vp]
        L.hqq_cache_attention_prefix.restype = i32
        L.hqq_cache_attention_prefix.argtypes = [cp, sp, vp, i32, i64, vp, i64, i64, i32, f32, vp,
                                                 i64, i64, vp, vp, st, vp]
        L.hqq_cache_attention_workspace.restype = st
        L.hqq_cache_attention_workspace.argtypes = [cp, sp, i32, i64]
        L.hqq_status_string.restype = C.c_char_p
        L.hqq_status_string.argtypes = [i32]
        L.hqq_last_error.restype = C.c_char_p
        L.hqq_last_error.argtypes = []
        _L = L
    return _L


def _p(t):
    """Device pointer of a tensor (or None)."""
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is not None:
        return C.c_void_p(int(stream))
    import torch
    return C.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(st: int):
    if st != HQQ_OK:
        L = lib()
        raise HQQError(st, f"{L.hqq_status_string(st).decode()}: {L.hqq_last_error().decode()}")


def hqq_status_string(status: int) -> str:
    return lib().hqq_status_string(status).decode()


def hqq_last_error() -> str:
    return lib().hqq_last_error().decode()


def hqq_packed_bytes(n_codes: int, nbits: int) -> int:
    return int(lib().hqq_packed_bytes(n_codes, nbits))


def make_job(W, nbits, group_size, axis, p, beta, kappa, iters, early_stop, zero_bits,
             packed, scale, zero, zero_meta, passes=None) -> hqq_job:
    rows, cols = W.shape
    return hqq_job(_p(W), rows, cols, nbits, group_size, axis, p, beta, kappa, iters,
                   int(early_stop), zero_bits, _p(packed), _p(scale), _p(zero),
                   _p(zero_meta), _p(passes))


def hqq_workspace_bytes(jobs) -> int:
    arr = (hqq_job * len(jobs))(*jobs)
    n = int(lib().hqq_workspace_bytes(arr, len(jobs)))
    if n == (1 << 64) - 1:
        raise HQQError(HQQ_ERR_ARG, "invalid job in workspace query")
    return n


def hqq_quantize(W, nbits, group_size, axis, p, beta, kappa, iters, early_stop, zero_bits,
                 packed, scale, zero, zero_meta, passes, workspace, stream=None) -> None:
    rows, cols = W.shape
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().hqq_quantize(_p(W), rows, cols, nbits, group_size, axis, p, beta, kappa,
                              iters, int(early_stop), zero_bits, _p(packed), _p(scale),
                              _p(zero), _p(zero_meta), _p(passes), _p(workspace), wsb,
                              _stream(stream)))


def hqq_quantize_noalloc(W, nbits, group_size, axis, p, beta, kappa, iters, early_stop,
                         zero_bits, packed, scale, zero, zero_meta, passes, stream=None) -> None:
    """hqq_quantize on the library's static scratch (no workspace argument)."""
    rows, cols = W.shape
    _check(lib().hqq_quantize_noalloc(_p(W), rows, cols, nbits, group_size, axis, p, beta,
                                      kappa, iters, int(early_stop), zero_bits, _p(packed),
                                      _p(scale), _p(zero), _p(zero_meta), _p(passes),
                                      _stream(stream)))


def _batch(fn, jobs, workspace, stream):
    arr = (hqq_job * len(jobs))(*jobs)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(fn(arr, len(jobs), _p(workspace), wsb, _stream(stream)))


def hqq_quantize_batch(jobs, workspace, stream=None) -> None:
    _batch(lib().hqq_quantize_batch, jobs, workspace, stream)


def hqq_solve_batch(jobs, workspace, stream=None) -> None:
    _batch(lib().hqq_solve_batch, jobs, workspace, stream)


def hqq_requant_batch(jobs, workspace, stream=None) -> None:
    _batch(lib().hqq_requant_batch, jobs, workspace, stream)


def hqq_batch_check(jobs, workspace, stream=None) -> None:
    """Waits for `stream`; raises HQQError (HQQ_ERR_DEVICE) if the last solve on this
    workspace left groups unwritten."""
    _batch(lib().hqq_batch_check, jobs, workspace, stream)


def hqq_debug_solver(step_budget: int = 0, pass_layout: int = 0) -> None:
    """Test hook: a fixed solver step budget (0 = default) and the solver kernel (0 = by
    size, 1 = persistent with one lane per group, 2 = persistent with several lanes per
    group, 3 = lockstep)."""
    lib().hqq_debug_solver(int(step_budget), int(pass_layout))


def hqq_streamed_workspace_bytes(jobs, staging_bytes) -> int:
    arr = (hqq_job * len(jobs))(*jobs)
    n = int(lib().hqq_streamed_workspace_bytes(arr, len(jobs), staging_bytes))
    if n == (1 << 64) - 1:
        raise HQQError(HQQ_ERR_ARG, "invalid job, or a tensor larger than half the staging")
    return n


def hqq_quantize_streamed(jobs, staging, workspace, stream=None, copy_stream=None) -> None:
    """jobs[i].W are host pointers (pinned); staging and workspace are device tensors."""
    arr = (hqq_job * len(jobs))(*jobs)
    sb = staging.numel() * staging.element_size()
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    cs = _stream(copy_stream) if copy_stream is not None else _stream(stream)
    _check(lib().hqq_quantize_streamed(arr, len(jobs), _p(staging), sb, _p(workspace), wsb,
                                       _stream(stream), cs))


def hqq_dequantize(packed, scale, zero, zero_meta, rows, cols, nbits, group_size, axis,
                   zero_bits, W_out, stream=None) -> None:
    _check(lib().hqq_dequantize(_p(packed), _p(scale), _p(zero), _p(zero_meta), rows, cols,
                                nbits, group_size, axis, zero_bits, _p(W_out),
                                _stream(stream)))


def hqq_gemm(X, packed, scale, zero, zero_meta, N, K, nbits, group_size, zero_bits, Y,
             workspace=None, stream=None) -> None:
    """Y[M, N] = X[M, K] . W_r^T for a packed axis-1 quantized weight [N, K]; `workspace`
    (optional, at least hqq_gemm_workspace_bytes(M, N, K) bytes) selects the reconstruct-once
    path for M > 64."""
    M = X.shape[0]
    wb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().hqq_gemm(_p(X), M, _p(packed), _p(scale), _p(zero), _p(zero_meta), N, K,
                          nbits, group_size, zero_bits, _p(Y), _p(workspace), wb,
                          _stream(stream)))


def hqq_gemm_multi(X, weights, workspace=None, stream=None) -> None:
    """Several weights [N_i, K] multiplied by the same X: `weights` is a list of dicts with
    packed, scale, zero, zero_meta, N, nbits, group_size, zero_bits and Y (as hqq_gemm's
    arguments); each Y_i gets what hqq_gemm would write."""
    M, K = X.shape
    arr = (hqq_gemm_weight * max(len(weights), 1))()
    for i, w in enumerate(weights):
        arr[i] = hqq_gemm_weight(_p(w["packed"]), _p(w["scale"]), _p(w["zero"]),
                                 _p(w.get("zero_meta")), w["N"], w["nbits"], w["group_size"],
                                 w["zero_bits"], _p(w["Y"]))
    wb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().hqq_gemm_multi(_p(X), M, K, arr, len(weights), _p(workspace), wb,
                                _stream(stream)))


def hqq_gemm_workspace_bytes(M, N, K) -> int:
    return int(lib().hqq_gemm_workspace_bytes(M, N, K))


def hqq_gemm_f16(X, Wr, N, K, Y, stream=None) -> None:
    """Y[M, N] = X[M, K] . Wr^T for a binary16 weight Wr [N, K] (as hqq_dequantize writes it)."""
    _check(lib().hqq_gemm_f16(_p(X), X.shape[0], _p(Wr), N, K, _p(Y), _stream(stream)))


def hqq_requant_scales(scale, n, scale_group, scale_q, scale_meta, stream=None) -> None:
    _check(lib().hqq_requant_scales(_p(scale), n, scale_group, _p(scale_q), _p(scale_meta),
                                    _stream(stream)))


def hqq_dequantize_scales(scale_q, scale_meta, n, scale_group, scale_out, stream=None) -> None:
    _check(lib().hqq_dequantize_scales(_p(scale_q), _p(scale_meta), n, scale_group,
                                       _p(scale_out), _stream(stream)))


def requant_scales(scale, scale_group=128, stream=None):
    """Allocate and fill 8-bit scales for a binary16 scale tensor: (scale_q, scale_meta)."""
    import torch
    n = scale.numel()
    sq = torch.empty(max(n, 1), dtype=torch.uint8, device=scale.device)
    meta = torch.empty(max(2 * ((n + scale_group - 1) // scale_group), 2), dtype=torch.float16,
                       device=scale.device)
    hqq_requant_scales(scale, n, scale_group, sq, meta, stream)
    return sq[:n], meta[:2 * ((n + scale_group - 1) // scale_group)]


def hqq_pack(codes, n_codes, nbits, packed, stream=None) -> None:
    _check(lib().hqq_pack(_p(codes), n_codes, nbits, _p(packed), _stream(stream)))


def hqq_unpack(packed, n_codes, nbits, codes, stream=None) -> None:
    _check(lib().hqq_unpack(_p(packed), n_codes, nbits, _p(codes), _stream(stream)))


# ---- the quantized key/value cache ------------------------------------------------------------
# A cache is a dict of its four tensors and sizes (alloc_cache makes one): k_codes and v_codes,
# uint8 [n_pages, n_heads, page_size*head_dim*nbits/8], k_meta and v_meta, [n_pages, n_heads,
# page_size, head_dim/group_size, 2] of the type of the rows, page_size, n_heads, head_dim,
# nbits, group_size. table: int32 [n_seqs, max_pages]; lens: int32 [n_seqs]; cu_tokens: int32
# [n_seqs + 1] or None. Rows are [n_tokens, heads, head_dim] with contiguous dimensions. The
# calls run on the current stream of the cache's device unless `stream` is given; what they allocate
# then belongs to that stream, as if allocated under it (wait for it before other streams use it, and
# record_stream before they outlive it).
# hqq_cache and hqq_seqs as bytes (a third of the time that a ctypes structure takes to make)
_pack_cache = struct.Struct("@4Pq6i").pack
_pack_seqs = struct.Struct("@3P2iq").pack
_torch = None


def _th():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _bad(msg):
    return HQQError(HQQ_ERR_ARG, msg)


def _cache_struct(cache):
    """The C struct of a cache dict, its GPU's index and its type."""
    T = _torch or _th()
    kc, vc, km, vm = cache["k_codes"], cache["v_codes"], cache["k_meta"], cache["v_meta"]
    page, heads, dim = cache["page_size"], cache["n_heads"], cache["head_dim"]
    nbits, group = cache["nbits"], cache["group_size"]
    codes, meta, dtype, dev = kc.shape, km.shape, km.dtype, kc.get_device()
    n = codes[0]
    if codes != (n, heads, page * dim * nbits // 8) or vc.shape != codes or \
            not kc.dtype == vc.dtype == T.uint8:
        raise _bad("k_codes and v_codes must be uint8 [n_pages, n_heads, page_size*head_dim*nbits/8]")
    if meta != (n, heads, page, dim // max(group, 1), 2) or vm.shape != meta or vm.dtype != dtype or \
            (dtype != T.float16 and dtype != T.bfloat16):
        raise _bad("k_meta and v_meta must be [n_pages, n_heads, page_size, head_dim/group_size, 2] "
                   "of float16 or bfloat16")
    if not (kc.is_contiguous() and vc.is_contiguous() and km.is_contiguous() and vm.is_contiguous()):
        raise _bad("the cache's tensors must be contiguous")
    if dev < 0 or not dev == vc.get_device() == km.get_device() == vm.get_device():
        raise _bad("the cache's tensors must be on one GPU")
    return _pack_cache(kc.data_ptr(), vc.data_ptr(), km.data_ptr(), vm.data_ptr(), n, page, heads,
                       dim, nbits, group, HQQ_BF16 if dtype == T.bfloat16 else HQQ_F16), dev, dtype


def _seqs_struct(table, lens, cu_tokens, n_tokens, dev):
    i32 = _torch.int32
    shape = table.shape
    if len(shape) != 2 or table.dtype != i32 or table.get_device() != dev or not table.is_contiguous():
        raise _bad("table must be a contiguous int32 [n_seqs, max_pages] on the cache's device")
    n = shape[0]
    if lens.shape != (n,) or lens.dtype != i32 or lens.get_device() != dev or not lens.is_contiguous():
        raise _bad("lens must be a contiguous int32 [n_seqs] on the cache's device")
    cu = 0
    if cu_tokens is not None:
        if cu_tokens.shape != (n + 1,) or cu_tokens.dtype != i32 or cu_tokens.get_device() != dev or \
                not cu_tokens.is_contiguous():
            raise _bad("cu_tokens must be a contiguous int32 [n_seqs + 1] on the cache's device")
        cu = cu_tokens.data_ptr()
    return _pack_seqs(table.data_ptr(), lens.data_ptr(), cu, n, shape[1], n_tokens)


def _rows(x, shape, dev, dtype, name):
    """Pointer and strides of rows; a strided dimension of one element may have any stride."""
    if x.shape != shape or x.dtype != dtype or x.get_device() != dev:
        raise _bad(f"{name} must be [n_tokens, heads, head_dim] of the cache's sizes, type and device")
    ts, hs, ds = x.stride()
    if ds != 1:
        raise _bad(f"{name} must have contiguous dimensions")
    return x.data_ptr(), ts if shape[0] > 1 else 0, hs if shape[1] > 1 else 0


def _on(dev, fn, *args):
    """The status of fn(*args) with `dev` as the current GPU."""
    if _torch._C._cuda_getDevice() == dev:
        return fn(*args)
    with _torch.cuda.device(dev):
        return fn(*args)


def _stream_of(dev, stream):
    return int(stream) if stream is not None else _torch._C._cuda_getCurrentRawStream(dev)


def _cache_rows(fn, cache, table, lens, k, v, cu_tokens, stream):
    c, dev, dtype = _cache_struct(cache)
    shape = (k.shape[0], cache["n_heads"], cache["head_dim"])
    s = _seqs_struct(table, lens, cu_tokens, shape[0], dev)
    kp, kt, kh = _rows(k, shape, dev, dtype, "k")
    vp, vt, vh = _rows(v, shape, dev, dtype, "v")
    st = _on(dev, fn, c, s, kp, kt, kh, vp, vt, vh, _stream_of(dev, stream))
    if st:
        _check(st)


def hqq_cache_write(cache, table, lens, k, v, cu_tokens=None, stream=None) -> None:
    """Quantize k and v [n_tokens, n_heads, head_dim] into the cache as the last tokens of
    their sequences (lens counts them)."""
    _cache_rows(lib().hqq_cache_write, cache, table, lens, k, v, cu_tokens, stream)


def hqq_cache_read(cache, table, lens, k, v, cu_tokens=None, stream=None) -> None:
    """Fill k and v with what the cache holds of the last tokens of the sequences."""
    _cache_rows(lib().hqq_cache_read, cache, table, lens, k, v, cu_tokens, stream)


def hqq_cache_attention_workspace(cache, table, lens, n_tokens, n_q_heads, prefix_len=0, cu_tokens=None) -> int:
    """Workspace bytes of an attention call of these sizes."""
    c, dev, _ = _cache_struct(cache)
    s = _seqs_struct(table, lens, cu_tokens, n_tokens, dev)
    n = int(lib().hqq_cache_attention_workspace(c, s, n_q_heads, prefix_len))
    if n == 0 and hqq_last_error():
        raise _bad(hqq_last_error())
    return n


def _on_stream(dev, stream, make):
    """make(), with what it allocates from the allocator's pool of the stream that a call runs on:
    memory of another stream's pool may have work of that stream before it."""
    T = _torch
    if stream is None or dev < 0 or int(stream) == T._C._cuda_getCurrentRawStream(dev):
        return make()
    with T.cuda.stream(T.cuda.ExternalStream(int(stream), device=dev)):
        return make()


def _attention(cache, table, lens, prefix_pages, prefix_len, q, out, lse, scale, cu_tokens, workspace, stream):
    T = _torch or _th()
    c, dev, dtype = _cache_struct(cache)
    shape = q.shape
    if len(shape) != 3 or shape[2] != cache["head_dim"]:
        raise _bad("q must be [n_tokens, n_q_heads, head_dim]")
    n, heads, dim = shape
    s = _seqs_struct(table, lens, cu_tokens, n, dev)
    qp, qt, qh = _rows(q, shape, dev, dtype, "q")
    if out is None:
        out = _on_stream(dev, stream, lambda: T.empty(shape, dtype=dtype, device=q.device))
    op, ot, oh = _rows(out, shape, dev, dtype, "out")
    if lse is not None and (lse.shape != (n, heads) or lse.dtype != T.float32 or lse.get_device() != dev or
                            not lse.is_contiguous()):
        raise _bad("lse must be a contiguous float32 [n_tokens, n_q_heads] on the cache's device")
    pages, n_pages = None, 0
    if prefix_pages is not None:
        if prefix_pages.dim() != 1 or prefix_pages.dtype != T.int32 or prefix_pages.get_device() != dev or \
                not prefix_pages.is_contiguous():
            raise _bad("prefix_pages must be a contiguous int32 vector on the cache's device")
        pages, n_pages = prefix_pages.data_ptr(), prefix_pages.shape[0]
    L = _L or lib()
    if workspace is None:
        need = L.hqq_cache_attention_workspace(c, s, heads, prefix_len)
        if need:
            workspace = _on_stream(dev, stream, lambda: T.empty(need, dtype=T.uint8, device=dev))
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise _bad("workspace must be contiguous, on the cache's device")
    wp, wb = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    st = _on(dev, L.hqq_cache_attention_prefix, c, s, pages, n_pages, prefix_len, qp, qt, qh, heads,
             dim ** -0.5 if scale is None else scale, op, ot, oh, None if lse is None else lse.data_ptr(),
             wp, wb, _stream_of(dev, stream))
    if st:
        _check(st)
    return out


def hqq_cache_attention(cache, table, lens, q, out, lse=None, scale=None, cu_tokens=None,
                        workspace=None, stream=None) -> None:
    """out = attention of q [n_tokens, n_q_heads, head_dim] over the cache: the row at position
    x of its sequence sees positions 0..x. scale: head_dim ** -0.5 unless given. workspace: a
    tensor of hqq_cache_attention_workspace() bytes, allocated when None."""
    _attention(cache, table, lens, None, 0, q, out, lse, scale, cu_tokens, workspace, stream)


def hqq_cache_attention_prefix(cache, table, lens, prefix_pages, prefix_len, q, out, lse=None, scale=None,
                               cu_tokens=None, workspace=None, stream=None) -> None:
    """hqq_cache_attention for sequences that share a prefix of prefix_len tokens, held once in
    prefix_pages (int32 [n]); table and lens are those of what follows it."""
    _attention(cache, table, lens, prefix_pages, prefix_len, q, out, lse, scale, cu_tokens, workspace, stream)


def alloc_cache(n_pages, page_size, n_heads, head_dim, nbits=4, group_size=64, dtype=None, device="cuda"):
    """An empty cache (a dict, see above); its tensors' contents are of no meaning until written."""
    import torch
    dtype = torch.float16 if dtype is None else dtype
    codes = (n_pages, n_heads, page_size * head_dim * nbits // 8)
    meta = (n_pages, n_heads, page_size, head_dim // group_size, 2)
    return dict(k_codes=torch.empty(codes, dtype=torch.uint8, device=device),
                v_codes=torch.empty(codes, dtype=torch.uint8, device=device),
                k_meta=torch.empty(meta, dtype=dtype, device=device),
                v_meta=torch.empty(meta, dtype=dtype, device=device),
                page_size=page_size, n_heads=n_heads, head_dim=head_dim, nbits=nbits,
                group_size=group_size)


def cache_read(cache, table, lens, n_tokens, cu_tokens=None, stream=None):
    """Allocate and fill (k, v) for the last tokens of the sequences, n_tokens in all."""
    T = _torch or _th()
    km = cache["k_meta"]
    both = _on_stream(km.get_device(), stream, lambda: T.empty(
        (2, n_tokens, cache["n_heads"], cache["head_dim"]), dtype=km.dtype, device=km.device))
    k, v = both.unbind(0)
    hqq_cache_read(cache, table, lens, k, v, cu_tokens, stream)
    return k, v


def cache_attention(cache, table, lens, q, cu_tokens=None, scale=None, lse=None, stream=None):
    """Allocate the output (contiguous) and call hqq_cache_attention."""
    return _attention(cache, table, lens, None, 0, q, None, lse, scale, cu_tokens, None, stream)


def cache_attention_prefix(cache, table, lens, prefix_pages, prefix_len, q, cu_tokens=None, scale=None,
                           lse=None, stream=None):
    """Allocate the output (contiguous) and call hqq_cache_attention_prefix."""
    return _attention(cache, table, lens, prefix_pages, prefix_len, q, None, lse, scale, cu_tokens, None, stream)


# ---- allocation helpers (PyTorch device memory for the outputs) -----------------------------
def alloc_outputs(rows, cols, nbits, group_size, zero_bits, device, passes=False):
    """Output tensors of one job: packed (uint8, 16-byte aligned by the allocator), scale,
    zero, zero_meta (or None) and passes (or None)."""
    import torch
    ng = rows * cols // group_size
    out = dict(
        packed=torch.empty(max(hqq_packed_bytes(rows * cols, nbits), 1), dtype=torch.uint8,
                           device=device),
        scale=torch.empty(ng, dtype=torch.float16, device=device),
        zero=torch.empty(ng, dtype=torch.float16 if zero_bits == 16 else torch.uint8,
                         device=device),
        zero_meta=torch.empty(2, dtype=torch.float16, device=device) if zero_bits == 8 else None,
        passes=torch.empty(ng, dtype=torch.uint8, device=device) if passes else None,
    )
    return out


def alloc_workspace(jobs, device):
    import torch
    n = hqq_workspace_bytes(jobs)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device) if n > 0 else None


def quantize(W, nbits, group_size, axis=1, p=0.7, beta=1.0, kappa=1.01, iters=20,
             early_stop=True, zero_bits=16, passes=False, stream=None):
    """Allocate outputs and a workspace, then call hqq_quantize. Returns the output dict."""
    rows, cols = W.shape
    out = alloc_outputs(rows, cols, nbits, group_size, zero_bits, W.device, passes)
    job = make_job(W, nbits, group_size, axis, p, beta, kappa, iters, early_stop, zero_bits,
                   out["packed"], out["scale"], out["zero"], out["zero_meta"], out["passes"])
    ws = alloc_workspace([job], W.device)
    hqq_quantize(W, nbits, group_size, axis, p, beta, kappa, iters, early_stop, zero_bits,
                 out["packed"], out["scale"], out["zero"], out["zero_meta"], out["passes"],
                 ws, stream)
    out["workspace"] = ws
    out["job"] = job
    return out
