"""Thin ctypes binding of liblowbit (include/lowbit.h).

Argument marshalling only: torch tensors are passed as device pointers with
the current HIP stream; every step runs in the library's HIP kernels.  The
library must be built first (``python -m ultra_bit_dit_amd.build``); there is
no fallback.
"""
import ctypes
import os
import sys

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "liblowbit.so")

OK, E_NULL, E_SHAPE, E_ALIGN, E_UNSUPPORTED, E_BADCODE, E_HIP, E_NOMEM = 0, -1, -2, -3, -4, -5, -6, -7
E_TOO_LARGE = -8
BINARY, TERNARY_2BIT, TERNARY_BASE3 = 1, 2, 3
F32, BF16, I8, SIGN1, I32, MXFP4 = 1, 2, 3, 4, 5, 6
EPI_NONE, EPI_SILU_MUL = 0, 1

# every symbol the public header declares
EXPORTS = ("lowbit_abi_version", "lowbit_status_str", "lowbit_packed_bytes", "lowbit_pack",
           "lowbit_unpack", "lowbit_quantize_act_i8", "lowbit_gemv", "lowbit_gemm",
           "lowbit_gemv_noalloc", "lowbit_workspace_bytes", "lowbit_reserve_workspace", "lowbit_release_workspaces",
           "lowbit_chain_create", "lowbit_chain_create_rows", "lowbit_chain_run", "lowbit_chain_status",
           "lowbit_chain_destroy",
           "lowbit_hbm_read_probe", "lowbit_quantize_weights", "lowbit_rotate_act",
           "lowbit_mxfp4_bytes", "lowbit_pack_mxfp4", "lowbit_quantize_mxfp4", "lowbit_gemm_mxfp4",
           "lowbit_kv8_append", "lowbit_attention_kv8", "lowbit_attention_kv8_workspace")


class GemvStage(ctypes.Structure):
    """lowbit_gemv_stage"""
    _fields_ = [("fmt", ctypes.c_int), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("pcodes", ctypes.c_void_p), ("pscales", ctypes.c_void_p),
                ("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("wait_prev", ctypes.c_int),
                ("epilogue", ctypes.c_int)]


class Kv8(ctypes.Structure):
    """lowbit_kv8"""
    _fields_ = [("n_pages", ctypes.c_int64), ("page_tokens", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p)]


class Kv8Batch(ctypes.Structure):
    """lowbit_kv8_batch"""
    _fields_ = [("n_seqs", ctypes.c_int64), ("page_table", ctypes.c_void_p), ("table_width", ctypes.c_int64),
                ("kv_lens", ctypes.c_void_p), ("q_starts", ctypes.c_void_p), ("total_q", ctypes.c_int64),
                ("max_q", ctypes.c_int64), ("max_kv", ctypes.c_int64), ("bad_pages", ctypes.c_void_p)]


class LowbitError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn}: {status_str(status)} ({status})")
        self.status = status


_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"liblowbit is not built ({LIB_PATH} missing); "
                               "run `python -m ultra_bit_dit_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        i64, vp, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        L.lowbit_abi_version.restype = i32
        L.lowbit_status_str.argtypes = [i32]
        L.lowbit_status_str.restype = ctypes.c_char_p
        L.lowbit_packed_bytes.argtypes = [i32, i64, i64, ctypes.POINTER(ctypes.c_size_t),
                                          ctypes.POINTER(ctypes.c_size_t)]
        L.lowbit_pack.argtypes = [i32, i64, i64, vp, vp, vp, vp, vp, vp]
        L.lowbit_unpack.argtypes = [i32, i64, i64, vp, vp, vp, vp, vp, vp]
        L.lowbit_quantize_act_i8.argtypes = [i64, i64, vp, vp, vp, vp]
        L.lowbit_gemv.argtypes = [i32, i64, i64, vp, vp, i32, vp, ctypes.c_float, i32, vp, vp]
        L.lowbit_gemv_noalloc.argtypes = [i32, i64, i64, vp, vp, i32, vp, ctypes.c_float, i32, vp, vp]
        L.lowbit_gemm.argtypes = [i32, i64, i64, i64, vp, vp, i32, vp, vp, i32, vp, vp]
        L.lowbit_workspace_bytes.argtypes = [i32, i64, i64, i64, i32, ctypes.POINTER(ctypes.c_size_t)]
        L.lowbit_reserve_workspace.argtypes = [ctypes.c_size_t, vp]
        L.lowbit_release_workspaces.argtypes = []
        L.lowbit_chain_create.argtypes = [i32, ctypes.POINTER(GemvStage), i32, i32,
                                          ctypes.POINTER(vp)]
        L.lowbit_chain_create_rows.argtypes = [i32, ctypes.POINTER(GemvStage), i64, i32, i32,
                                               ctypes.POINTER(vp)]
        L.lowbit_chain_run.argtypes = [vp, vp]
        L.lowbit_chain_status.argtypes = [vp, ctypes.POINTER(i32)]
        L.lowbit_chain_destroy.argtypes = [vp]
        L.lowbit_hbm_read_probe.argtypes = [vp, i64, vp, vp]
        L.lowbit_quantize_weights.argtypes = [i32, i64, i64, vp, vp, vp, vp, vp]
        L.lowbit_rotate_act.argtypes = [i64, i64, vp, vp, vp, vp]
        szp, kvp, kbp = ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(Kv8), ctypes.POINTER(Kv8Batch)
        L.lowbit_mxfp4_bytes.argtypes = [i64, i64, szp, szp]
        L.lowbit_pack_mxfp4.argtypes = [i64, i64, vp, vp, vp, vp, vp]
        L.lowbit_quantize_mxfp4.argtypes = [i64, i64, i32, vp, i64, vp, vp, vp, vp]
        L.lowbit_gemm_mxfp4.argtypes = [i64, i64, i64, vp, vp, i32, vp, i64, vp, i32, vp, vp]
        L.lowbit_kv8_append.argtypes = [kvp, kbp, i32, vp, vp, i64, i64, vp]
        L.lowbit_attention_kv8.argtypes = [kvp, kbp, i64, vp, i64, ctypes.c_float, i32, i64, vp, i64, vp, vp]
        L.lowbit_attention_kv8_workspace.argtypes = [kvp, kbp, i64, szp]
        for name in EXPORTS[2:]:
            getattr(L, name).restype = i32
        _lib = L
    return _lib


def status_str(status):
    return lib().lowbit_status_str(int(status)).decode()


def _check(fn, status):
    if status != OK:
        raise LowbitError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def packed_bytes(fmt, N, K):
    cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _check("lowbit_packed_bytes", lib().lowbit_packed_bytes(fmt, N, K, ctypes.byref(cb), ctypes.byref(sb)))
    return cb.value, sb.value


def empty_packed(fmt, N, K, device="cuda"):
    import torch
    cb, sb = packed_bytes(fmt, N, K)
    return (torch.empty(cb, dtype=torch.uint8, device=device),
            torch.empty(sb // 2, dtype=torch.int16, device=device))


def pack(fmt, codes, scales, pcodes=None, pscales=None, bad=None, stream=None):
    """codes int8 [N][K], scales fp16 (or int16 bits) [N][K/128] -> packed tensors."""
    N, K = codes.shape
    if pcodes is None:
        pcodes, pscales = empty_packed(fmt, N, K, codes.device)
    _check("lowbit_pack", lib().lowbit_pack(fmt, N, K, _ptr(codes), _ptr(scales), _ptr(pcodes),
                                            _ptr(pscales), _ptr(bad), _stream(stream)))
    return pcodes, pscales


def unpack(fmt, N, K, pcodes, pscales, bad=None, stream=None):
    import torch
    codes = torch.empty((N, K), dtype=torch.int8, device=pcodes.device)
    scales = torch.empty((N, K // 128), dtype=torch.int16, device=pcodes.device)
    _check("lowbit_unpack", lib().lowbit_unpack(fmt, N, K, _ptr(pcodes), _ptr(pscales), _ptr(codes),
                                                _ptr(scales), _ptr(bad), _stream(stream)))
    return codes, scales


def quantize_act_i8(X, Q=None, s_x=None, stream=None):
    """bf16 X [M][K] -> (int8 Q [M][K], fp32 s_x [M]); Q and s_x may be given."""
    import torch
    M, K = X.shape
    if Q is None:
        Q = torch.empty((M, K), dtype=torch.int8, device=X.device)
    if s_x is None:
        s_x = torch.empty(M, dtype=torch.float32, device=X.device)
    sx = s_x
    _check("lowbit_quantize_act_i8", lib().lowbit_quantize_act_i8(M, K, _ptr(X), _ptr(Q), _ptr(sx),
                                                                  _stream(stream)))
    return Q, sx


def _xdt(x, x_dtype):
    import torch
    if x_dtype is not None:
        return x_dtype
    return {torch.float32: F32, torch.bfloat16: BF16, torch.int8: I8, torch.uint8: SIGN1}[x.dtype]


def _ytorch(y_dtype):
    import torch
    return {F32: torch.float32, BF16: torch.bfloat16, I32: torch.int32}[y_dtype]


def gemv(fmt, N, K, pcodes, pscales, x, x_scale=1.0, y_dtype=F32, y=None, x_dtype=None,
         stream=None):
    """y[n] = sum_k W[n][k] x[k] (see lowbit_gemv)."""
    import torch
    if y is None:
        y = torch.empty(N, dtype=_ytorch(y_dtype), device=pcodes.device)
    _check("lowbit_gemv", lib().lowbit_gemv(fmt, N, K, _ptr(pcodes), _ptr(pscales), _xdt(x, x_dtype),
                                            _ptr(x), float(x_scale), y_dtype, _ptr(y), _stream(stream)))
    return y


def gemv_noalloc(fmt, N, K, pcodes, pscales, x, y, x_scale=1.0, y_dtype=F32, x_dtype=None,
                 stream=None):
    """lowbit_gemv through the allocation-free entry point (lowbit_gemv_noalloc):
    the caller passes the output y; nothing is allocated."""
    _check("lowbit_gemv_noalloc",
           lib().lowbit_gemv_noalloc(fmt, N, K, _ptr(pcodes), _ptr(pscales), _xdt(x, x_dtype),
                                     _ptr(x), float(x_scale), y_dtype, _ptr(y), _stream(stream)))
    return y


def gemm(fmt, M, N, K, pcodes, pscales, X, x_scales=None, y_dtype=F32, Y=None, x_dtype=None,
         stream=None):
    """Y[m][n] = sum_k W[n][k] X[m][k] (see lowbit_gemm)."""
    import torch
    if Y is None:
        Y = torch.empty((M, N), dtype=_ytorch(y_dtype), device=pcodes.device)
    _check("lowbit_gemm", lib().lowbit_gemm(fmt, M, N, K, _ptr(pcodes), _ptr(pscales), _xdt(X, x_dtype),
                                            _ptr(X), _ptr(x_scales), y_dtype, _ptr(Y), _stream(stream)))
    return Y


def workspace_bytes(fmt, M, N, K, x_dtype):
    """Workspace bytes lowbit_gemm (or lowbit_gemv, M = 1) needs for these arguments."""
    b = ctypes.c_size_t()
    _check("lowbit_workspace_bytes",
           lib().lowbit_workspace_bytes(fmt, M, N, K, x_dtype, ctypes.byref(b)))
    return b.value


def reserve_workspace(nbytes, stream=None):
    """Grow the stream's workspace to at least nbytes (do it before capturing a graph)."""
    _check("lowbit_reserve_workspace", lib().lowbit_reserve_workspace(int(nbytes), _stream(stream)))


def release_workspaces():
    """Wait for the devices, then free every workspace (no graph using one may be replayed after)."""
    _check("lowbit_release_workspaces", lib().lowbit_release_workspaces())


def quantize_weights(fmt, W, signs=None, stream=None):
    """Dense (codes int8 [N][K], scales int16 fp16 bits [N][K/128]) from bf16
    weights W [N][K] (see lowbit_quantize_weights); signs int8 [K] or None."""
    import torch
    N, K = W.shape
    codes = torch.empty((N, K), dtype=torch.int8, device=W.device)
    scales = torch.empty((N, K // 128), dtype=torch.int16, device=W.device)
    _check("lowbit_quantize_weights",
           lib().lowbit_quantize_weights(fmt, N, K, _ptr(W), _ptr(signs), _ptr(codes),
                                         _ptr(scales), _stream(stream)))
    return codes, scales


def rotate_act(X, signs, stream=None):
    """fp32 X_rot [M][K] from bf16 X [M][K] (see lowbit_rotate_act)."""
    import torch
    M, K = X.shape
    Xr = torch.empty((M, K), dtype=torch.float32, device=X.device)
    _check("lowbit_rotate_act",
           lib().lowbit_rotate_act(M, K, _ptr(X), _ptr(signs), _ptr(Xr), _stream(stream)))
    return Xr


# ---- MXFP4


def _on(device, *tensors):
    """Every given tensor lies on `device`, which has to be the current one (calls run there)."""
    import torch
    if device.index != torch.cuda.current_device():
        raise ValueError(f"tensors on {device}, but the current device is cuda:{torch.cuda.current_device()}")
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"tensors on {device} and {t.device} in one call")


def _want(cond, what):
    if not cond:
        raise ValueError(what)


def _mx_sizes(rows, K):
    if rows < 1 or K < 32 or K % 32:
        raise LowbitError("lowbit_mxfp4_bytes", E_SHAPE)
    nb, g = (rows + 15) // 16, (K + 127) // 128
    return nb * g * 1024, nb * ((g + 3) // 4) * 256


def mxfp4_bytes(rows, K):
    """Bytes of the packed MXFP4 codes and scales of a rows x K matrix."""
    cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _check("lowbit_mxfp4_bytes", lib().lowbit_mxfp4_bytes(rows, K, ctypes.byref(cb), ctypes.byref(sb)))
    return cb.value, sb.value


def empty_mxfp4(rows, K, device="cuda"):
    """Uninitialised packed MXFP4 buffers (codes, scales), both uint8."""
    import torch
    cb, sb = _mx_sizes(rows, K)
    return (torch.empty(cb, dtype=torch.uint8, device=device),
            torch.empty(sb, dtype=torch.uint8, device=device))


def _mx_packed(codes, scales, rows, K, what):
    import torch
    cb, sb = _mx_sizes(rows, K)
    _want(codes.dtype == torch.uint8 and scales.dtype == torch.uint8 and codes.numel() == cb
          and scales.numel() == sb and codes.is_contiguous() and scales.is_contiguous(),
          f"{what}: packed MXFP4 buffers of a {rows} x {K} matrix are {cb} and {sb} contiguous uint8")


def pack_mxfp4(codes, scales, pcodes=None, pscales=None, stream=None):
    """Row-major MXFP4 (uint8 codes [rows][K/2], scales [rows][K/32]) -> packed buffers
    (see lowbit_pack_mxfp4)."""
    import torch
    rows, K = codes.shape[0], 2 * codes.shape[1]
    _want(codes.dtype == torch.uint8 and scales.dtype == torch.uint8 and tuple(scales.shape) == (rows, K // 32)
          and codes.is_contiguous() and scales.is_contiguous(),
          "pack_mxfp4: contiguous uint8 codes [rows][K/2] and scales [rows][K/32]")
    if pcodes is None:
        pcodes, pscales = empty_mxfp4(rows, K, codes.device)
    _mx_packed(pcodes, pscales, rows, K, "pack_mxfp4")
    _on(codes.device, scales, pcodes, pscales)
    _check("lowbit_pack_mxfp4", lib().lowbit_pack_mxfp4(rows, K, _ptr(codes), _ptr(scales), _ptr(pcodes),
                                                        _ptr(pscales), _stream(stream)))
    return pcodes, pscales


def quantize_mxfp4(X, values=False, pcodes=None, pscales=None, stream=None):
    """X [rows][K] (bf16 or fp32, rows may be strided) -> packed (codes, scales);
    values=True (or a tensor): and the numbers they stand for, in X's type (see
    lowbit_quantize_mxfp4)."""
    import torch
    _want(X.dim() == 2 and X.stride(1) == 1, "quantize_mxfp4: X is [rows][K] with contiguous rows")
    rows, K = X.shape
    if pcodes is None:
        pcodes, pscales = empty_mxfp4(rows, K, X.device)
    _mx_packed(pcodes, pscales, rows, K, "quantize_mxfp4")
    vals = None
    if values is not False and values is not None:
        vals = torch.empty((rows, K), dtype=X.dtype, device=X.device) if values is True else values
        _want(tuple(vals.shape) == (rows, K) and vals.dtype == X.dtype and vals.is_contiguous(),
              "quantize_mxfp4: values is contiguous, of X's shape and type")
    _on(X.device, pcodes, pscales, vals)
    _check("lowbit_quantize_mxfp4",
           lib().lowbit_quantize_mxfp4(rows, K, _xfloat(X), _ptr(X), max(X.stride(0), K), _ptr(pcodes),
                                       _ptr(pscales), _ptr(vals), _stream(stream)))
    return (pcodes, pscales) if vals is None else (pcodes, pscales, vals)


def _xfloat(x):
    import torch
    if x.dtype == torch.bfloat16:
        return BF16
    if x.dtype == torch.float32:
        return F32
    raise ValueError(f"bf16 or fp32 expected, got {x.dtype}")


def gemm_mxfp4(M, N, K, pcodes, pscales, X, x_scales=None, y_dtype=F32, Y=None, stream=None):
    """Y[m][n] = sum_k W[n][k] X[m][k] with MXFP4 weights (see lowbit_gemm_mxfp4): X is
    bf16 [M][K] (rows may be strided), or with x_scales the packed MXFP4 codes of
    the activations."""
    import torch
    _mx_packed(pcodes, pscales, N, K, "gemm_mxfp4: weights")
    if x_scales is not None:
        _mx_packed(X, x_scales, M, K, "gemm_mxfp4: activations")
        xd, ld = MXFP4, 0
    else:
        _want(X.dtype == torch.bfloat16 and tuple(X.shape) == (M, K) and X.stride(1) == 1,
              "gemm_mxfp4: X is bf16 [M][K] with contiguous rows, or packed codes with x_scales")
        xd, ld = BF16, max(X.stride(0), K)
    if Y is None:
        Y = torch.empty((M, N), dtype=_ytorch(y_dtype), device=pcodes.device)
    else:
        _want(tuple(Y.shape) == (M, N) and Y.dtype == _ytorch(y_dtype) and Y.is_contiguous(),
              "gemm_mxfp4: Y is contiguous [M][N] of y_dtype")
    _on(pcodes.device, pscales, X, x_scales, Y)
    _check("lowbit_gemm_mxfp4",
           lib().lowbit_gemm_mxfp4(M, N, K, _ptr(pcodes), _ptr(pscales), xd, _ptr(X), ld, _ptr(x_scales),
                                   y_dtype, _ptr(Y), _stream(stream)))
    return Y


# ---- 8-bit paged cache


def empty_kv8(n_pages, page_tokens, kv_heads, head_dim, device="cuda"):
    """A zeroed cache (k_codes, v_codes, k_scales, v_scales) in lowbit_kv8's layout: e4m3 codes
    [n_pages][kv_heads][page_tokens][head_dim] and [..][head_dim][page_tokens], uint8 exponents."""
    import torch
    k = torch.zeros((n_pages, kv_heads, page_tokens, head_dim), dtype=torch.uint8, device=device)
    v = torch.zeros((n_pages, kv_heads, head_dim, page_tokens), dtype=torch.uint8, device=device)
    s = torch.zeros((2, n_pages, kv_heads), dtype=torch.uint8, device=device)
    return k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), s[0], s[1]


def _kv8(cache, page_table, kv_lens, q_starts, total_q, max_q, max_kv, bad_pages):
    import torch
    kc, vc, ks, vs = cache
    _want(kc.dim() == 4 and vc.dim() == 4 and kc.element_size() == 1 and vc.element_size() == 1,
          "cache: 8-bit codes [pages][heads][tokens][dim] and [pages][heads][dim][tokens]")
    n, H, P, D = kc.shape
    _want(tuple(vc.shape) == (n, H, D, P) and tuple(ks.shape) == (n, H) and tuple(vs.shape) == (n, H)
          and ks.dtype == torch.uint8 and vs.dtype == torch.uint8,
          "cache: v_codes [pages][heads][dim][tokens] and uint8 scales [pages][heads] of the same sizes")
    _want(kc.is_contiguous() and vc.is_contiguous() and ks.is_contiguous() and vs.is_contiguous(),
          "cache: contiguous tensors")
    i32 = torch.int32
    _want(page_table.dim() == 2 and page_table.dtype == i32 and page_table.is_contiguous(),
          "page_table: contiguous int32 [sequences][pages]")
    B = page_table.shape[0]
    _want(kv_lens.dtype == i32 and tuple(kv_lens.shape) == (B,) and kv_lens.is_contiguous(),
          "kv_lens: contiguous int32 [sequences]")
    if q_starts is None:
        _want(B > 0 and total_q % B == 0, "without q_starts every sequence has the same number of new tokens")
        if max_q is None:
            max_q = total_q // B
    else:
        _want(q_starts.dtype == i32 and tuple(q_starts.shape) == (B + 1,) and q_starts.is_contiguous(),
              "q_starts: contiguous int32 [sequences + 1]")
        if max_q is None:
            max_q = total_q
    if max_kv is None:
        max_kv = page_table.shape[1] * P
    if bad_pages is not None:
        _want(bad_pages.dtype == i32 and bad_pages.numel() >= 1, "bad_pages: int32")
    _on(kc.device, vc, ks, vs, page_table, kv_lens, q_starts, bad_pages)
    c = Kv8(n, P, H, D, kc.data_ptr(), vc.data_ptr(), ks.data_ptr(), vs.data_ptr())
    b = Kv8Batch(B, page_table.data_ptr(), page_table.shape[1], kv_lens.data_ptr(),
                 None if q_starts is None else q_starts.data_ptr(), total_q, max_q, max_kv,
                 None if bad_pages is None else bad_pages.data_ptr())
    return c, b


def _heads(x, H, D, what):
    """Token stride of a [tokens][heads][dim] tensor whose heads are contiguous."""
    _want(x.dim() == 3 and x.shape[2] == D and (H is None or x.shape[1] == H) and x.stride(2) == 1
          and (x.stride(1) == D or x.shape[1] == 1), f"{what}: [tokens][heads][{D}] with contiguous heads")
    return max(x.stride(0), x.shape[1] * D)


def kv8_append(cache, page_table, kv_lens, K, V, q_starts=None, max_q=None, max_kv=None, bad_pages=None,
               stream=None):
    """Write new keys and values [tokens][kv_heads][dim] (bf16 or fp32, tokens may be strided) into the
    cache (see lowbit_kv8_append).  kv_lens counts them already; q_starts None: every sequence has
    tokens / sequences new ones."""
    H, D = cache[0].shape[1], cache[0].shape[3]
    ks, vs = _heads(K, H, D, "K"), _heads(V, H, D, "V")
    _want(K.shape[0] == V.shape[0] and K.dtype == V.dtype, "K and V: the same tokens and type")
    c, b = _kv8(cache, page_table, kv_lens, q_starts, K.shape[0], max_q, max_kv, bad_pages)
    _on(cache[0].device, K, V)
    _check("lowbit_kv8_append", lib().lowbit_kv8_append(c, b, _xfloat(K), _ptr(K), _ptr(V), ks, vs,
                                                        _stream(stream)))


def attention_kv8(Q, cache, page_table, kv_lens, q_starts=None, max_q=None, max_kv=None, softmax_scale=None,
                  causal=True, window=0, O=None, lse=None, return_lse=False, bad_pages=None, stream=None):
    """Attention of bf16 queries [tokens][q_heads][dim] (tokens may be strided) over the cache (see
    lowbit_attention_kv8); softmax_scale None: 1 / sqrt(dim).  Returns O, or (O, lse) with return_lse."""
    import torch
    D = cache[0].shape[3]
    qs = _heads(Q, None, D, "Q")
    T, Hq = Q.shape[0], Q.shape[1]
    _want(Q.dtype == torch.bfloat16, f"Q: bf16 expected, got {Q.dtype}")
    c, b = _kv8(cache, page_table, kv_lens, q_starts, T, max_q, max_kv, bad_pages)
    if O is None:
        O = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=Q.device)
    else:
        _want(tuple(O.shape) == (T, Hq, D) and O.dtype == torch.bfloat16, "O: bf16 of Q's shape")
    if return_lse and lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=Q.device)
    if lse is not None:
        _want(tuple(lse.shape) == (T, Hq) and lse.dtype == torch.float32 and lse.is_contiguous(),
              "lse: contiguous fp32 [tokens][q_heads]")
    _on(cache[0].device, Q, O, lse)
    _check("lowbit_attention_kv8",
           lib().lowbit_attention_kv8(c, b, Hq, _ptr(Q), qs, float(D ** -0.5 if softmax_scale is None else softmax_scale),
                                      int(bool(causal)), int(window), _ptr(O), _heads(O, Hq, D, "O"), _ptr(lse),
                                      _stream(stream)))
    return (O, lse) if return_lse else O


def attention_kv8_workspace(cache, page_table, kv_lens, q_heads, total_q, q_starts=None, max_q=None, max_kv=None):
    """Workspace bytes lowbit_attention_kv8 needs for these arguments (reserve before a capture)."""
    c, b = _kv8(cache, page_table, kv_lens, q_starts, total_q, max_q, max_kv, None)
    n = ctypes.c_size_t()
    _check("lowbit_attention_kv8_workspace",
           lib().lowbit_attention_kv8_workspace(c, b, q_heads, ctypes.byref(n)))
    return n.value


def hbm_read_probe(src, out, stream=None):
    """Stream-read every byte of device tensor `src` once, XOR-folding the
    data into the int32 device tensor `out` (see lowbit_hbm_read_probe)."""
    nbytes = src.numel() * src.element_size()
    _check("lowbit_hbm_read_probe",
           lib().lowbit_hbm_read_probe(_ptr(src), nbytes, _ptr(out), _stream(stream)))


class Chain:
    """A planned chain of batch-1 products run as one persistent launch
    (lowbit_chain_*).  `stages` is a list of (fmt, N, K, pcodes, pscales, x, y,
    wait_prev[, epilogue]) with device tensors (epilogue EPI_NONE or
    EPI_SILU_MUL); rows > 1: every x is [rows][K] and every y [rows][N]
    (lowbit_chain_create_rows).  The tensors are kept referenced for the
    chain's lifetime."""

    def __init__(self, stages, x_dtype=BF16, y_dtype=F32, rows=1):
        self._keep = [t for st in stages for t in st[3:7]]
        arr = (GemvStage * len(stages))()
        for i, st in enumerate(stages):
            fmt, N, K, pc, ps, x, y, wait = st[:8]
            epi = st[8] if len(st) > 8 else EPI_NONE
            arr[i] = GemvStage(fmt, N, K, pc.data_ptr(), ps.data_ptr(), x.data_ptr(), y.data_ptr(),
                               int(wait), int(epi))
        h = ctypes.c_void_p()
        _check("lowbit_chain_create_rows",
               lib().lowbit_chain_create_rows(len(stages), arr, ctypes.c_int64(rows), x_dtype, y_dtype,
                                              ctypes.byref(h)))
        self._h = h

    def run(self, stream=None):
        _check("lowbit_chain_run", lib().lowbit_chain_run(self._h, _stream(stream)))

    def failed_waits(self):
        v = ctypes.c_int(0)
        _check("lowbit_chain_status", lib().lowbit_chain_status(self._h, ctypes.byref(v)))
        return v.value

    def close(self):
        if self._h:
            _check("lowbit_chain_destroy", lib().lowbit_chain_destroy(self._h))
            self._h = None
            self._keep = []

    def __del__(self):
        # at interpreter exit the HIP runtime may already be torn down: leave
        # the chain's memory to the process exit then
        if sys is None or sys.is_finalizing():
            return
        try:
            self.close()
        except Exception:
            pass
