"""Thin ctypes binding of liblowbit (include/lowbit.h).

Argument marshalling only: torch tensors are passed as device pointers with
the current HIP stream; every step runs in the library's HIP kernels.  The
library must be built first (``python -m ultra_bit_dit_amd.build``); there is
no fallback.
"""
import ctypes
import os
import struct
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
           "lowbit_mxfp4_bytes", "lowbit_pack_mxfp4", "lowbit_quantize_mxfp4", "lowbit_gemm_mxfp4", "lowbit_gemm_mxfp4_workspace",
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
        L.lowbit_gemm_mxfp4_workspace.argtypes = [i64, i64, i64, i32, szp]
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


# ---- MXFP4 and the 8-bit cache.  Single tokens take a few microseconds on the
# device, so these wrappers check with plain comparisons and pass addresses and
# packed structs straight to the library.

_torch = None     # set by the first call
_FLOAT = {}       # torch type -> lowbit_dtype of the float inputs
_fast = None      # the same exports with address-only prototypes
_PACK_KV8 = struct.Struct("@qiiiPPPP").pack        # lowbit_kv8
_PACK_BATCH = struct.Struct("@qPqPPqqqP").pack     # lowbit_kv8_batch


class _Fast:
    def __init__(self):
        L, vp, i64, i32 = lib(), ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        for name, types in (
                ("lowbit_quantize_mxfp4", [i64, i64, i32, vp, i64, vp, vp, vp, vp]),
                ("lowbit_gemm_mxfp4", [i64, i64, i64, vp, vp, i32, vp, i64, vp, i32, vp, vp]),
                ("lowbit_kv8_append", [vp, vp, i32, vp, vp, i64, i64, vp]),
                ("lowbit_attention_kv8", [vp, vp, i64, vp, i64, ctypes.c_float, i32, i64, vp, i64, vp, vp])):
            f = L[name]  # a function object of its own
            f.argtypes, f.restype = types, i32
            setattr(self, name[7:], f)


def _load():
    global _torch, _fast
    import torch
    _FLOAT.update({torch.bfloat16: BF16, torch.float32: F32})
    _fast = _Fast()
    _torch = torch
    return torch


def _device(T, dev, *tensors):
    """The given tensors lie on GPU `dev`, the current one (calls run there)."""
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on {t.device} and GPU {dev} in one call")
    if dev < 0 or dev != T._C._cuda_getDevice():
        raise ValueError(f"tensors on device {dev}: calls take tensors of the current GPU")


def _of_device(stream, dev):
    if stream.device_index != dev:
        raise ValueError(f"a stream of GPU {stream.device_index} for tensors of GPU {dev}")
    return stream


def _raw_stream(T, dev, stream):
    return T._C._cuda_getCurrentRawStream(dev) if stream is None else _of_device(stream, dev).cuda_stream


def _empty(T, shape, dtype, device, stream):
    """An output of a call on `stream`: memory of that stream, which no work still queued
    on the current one uses."""
    if stream is None:
        return T.empty(shape, dtype=dtype, device=device)
    with T.cuda.stream(_of_device(stream, device.index)):
        return T.empty(shape, dtype=dtype, device=device)


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


def _mx_packed(T, codes, scales, rows, K, what):
    cb, sb = _mx_sizes(rows, K)
    u8 = T.uint8
    if (codes.dtype != u8 or scales.dtype != u8 or codes.numel() != cb or scales.numel() != sb
            or not codes.is_contiguous() or not scales.is_contiguous()):
        raise ValueError(f"{what}: packed MXFP4 buffers of a {rows} x {K} matrix are {cb} and {sb} contiguous uint8")


def pack_mxfp4(codes, scales, pcodes=None, pscales=None, stream=None):
    """Row-major MXFP4 (uint8 codes [rows][K/2], scales [rows][K/32]) -> packed buffers
    (see lowbit_pack_mxfp4)."""
    T = _torch or _load()
    rows, K = codes.shape[0], 2 * codes.shape[1]
    if (codes.dtype != T.uint8 or scales.dtype != T.uint8 or tuple(scales.shape) != (rows, K // 32)
            or not codes.is_contiguous() or not scales.is_contiguous()):
        raise ValueError("pack_mxfp4: contiguous uint8 codes [rows][K/2] and scales [rows][K/32]")
    if pcodes is None:
        sizes = _mx_sizes(rows, K)
        _device(T, codes.get_device(), scales)
        pcodes, pscales = (_empty(T, n, T.uint8, codes.device, stream) for n in sizes)
    else:
        _mx_packed(T, pcodes, pscales, rows, K, "pack_mxfp4")
        _device(T, codes.get_device(), scales, pcodes, pscales)
    _check("lowbit_pack_mxfp4", lib().lowbit_pack_mxfp4(rows, K, _ptr(codes), _ptr(scales), _ptr(pcodes), _ptr(pscales),
                                                        _raw_stream(T, codes.get_device(), stream)))
    return pcodes, pscales


def quantize_mxfp4(X, values=False, pcodes=None, pscales=None, stream=None):
    """X [rows][K] (bf16 or fp32, rows may be strided) -> packed (codes, scales);
    values=True (or a tensor): and the numbers they stand for, in X's type (see
    lowbit_quantize_mxfp4)."""
    T = _torch or _load()
    if X.dim() != 2 or X.stride(1) != 1 or X.dtype not in _FLOAT:
        raise ValueError("quantize_mxfp4: X is bf16 or fp32 [rows][K] with contiguous rows")
    rows, K = X.shape
    dev = X.get_device()
    if pcodes is None:
        cb, sb = _mx_sizes(rows, K)
        _device(T, dev)
        pcodes = _empty(T, cb, T.uint8, X.device, stream)
        pscales = _empty(T, sb, T.uint8, X.device, stream)
    else:
        _mx_packed(T, pcodes, pscales, rows, K, "quantize_mxfp4")
        _device(T, dev, pcodes, pscales)
    vals = None
    if values is True:
        vals = _empty(T, (rows, K), X.dtype, X.device, stream)
    elif values is not False and values is not None:
        vals = values
        if vals.shape != X.shape or vals.dtype != X.dtype or not vals.is_contiguous() or vals.get_device() != dev:
            raise ValueError("quantize_mxfp4: values is contiguous, of X's shape, type and device")
    rc = _fast.quantize_mxfp4(rows, K, _FLOAT[X.dtype], X.data_ptr(), X.stride(0) if rows > 1 else K,
                              pcodes.data_ptr(), pscales.data_ptr(), None if vals is None else vals.data_ptr(),
                              _raw_stream(T, dev, stream))
    if rc:
        raise LowbitError("lowbit_quantize_mxfp4", rc)
    return (pcodes, pscales) if vals is None else (pcodes, pscales, vals)


def gemm_mxfp4(M, N, K, pcodes, pscales, X, x_scales=None, y_dtype=F32, Y=None, stream=None):
    """Y[m][n] = sum_k W[n][k] X[m][k] with MXFP4 weights (see lowbit_gemm_mxfp4): X is
    bf16 [M][K] (rows may be strided), or with x_scales the packed MXFP4 codes of
    the activations."""
    T = _torch or _load()
    _mx_packed(T, pcodes, pscales, N, K, "gemm_mxfp4: weights")
    dev = pcodes.get_device()
    if x_scales is not None:
        _mx_packed(T, X, x_scales, M, K, "gemm_mxfp4: activations")
        xd, ld, xs = MXFP4, 0, x_scales.data_ptr()
    else:
        if X.dtype != T.bfloat16 or X.shape != (M, K) or X.stride(1) != 1:
            raise ValueError("gemm_mxfp4: X is bf16 [M][K] with contiguous rows, or packed codes with x_scales")
        xd, ld, xs = BF16, X.stride(0) if M > 1 else K, None
    if Y is not None and (Y.shape != (M, N) or Y.dtype != _ytorch(y_dtype) or not Y.is_contiguous()):
        raise ValueError("gemm_mxfp4: Y is contiguous [M][N] of y_dtype")
    _device(T, dev, pscales, X, x_scales, Y)
    if Y is None:
        Y = _empty(T, (M, N), T.float32 if y_dtype == F32 else _ytorch(y_dtype), pcodes.device, stream)
    rc = _fast.gemm_mxfp4(M, N, K, pcodes.data_ptr(), pscales.data_ptr(), xd, X.data_ptr(), ld, xs, y_dtype,
                          Y.data_ptr(), _raw_stream(T, dev, stream))
    if rc:
        raise LowbitError("lowbit_gemm_mxfp4", rc)
    return Y


def gemm_mxfp4_workspace(M, N, K, x_dtype):
    """Workspace bytes lowbit_gemm_mxfp4 needs for these arguments (BF16 or MXFP4 activations)."""
    n = ctypes.c_size_t()
    _check("lowbit_gemm_mxfp4_workspace",
           lib().lowbit_gemm_mxfp4_workspace(M, N, K, x_dtype, ctypes.byref(n)))
    return n.value


def empty_kv8(n_pages, page_tokens, kv_heads, head_dim, device="cuda"):
    """A zeroed cache (k_codes, v_codes, k_scales, v_scales) in lowbit_kv8's layout: e4m3 codes
    [n_pages][kv_heads][page_tokens][head_dim] and [..][head_dim][page_tokens], uint8 exponents."""
    import torch
    k = torch.zeros((n_pages, kv_heads, page_tokens, head_dim), dtype=torch.uint8, device=device)
    v = torch.zeros((n_pages, kv_heads, head_dim, page_tokens), dtype=torch.uint8, device=device)
    s = torch.zeros((2, n_pages, kv_heads), dtype=torch.uint8, device=device)
    return k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), s[0], s[1]


def _kv8(T, cache, page_table, kv_lens, q_starts, total_q, max_q, max_kv, bad_pages):
    """Checked and packed lowbit_kv8 and lowbit_kv8_batch, and the tensors' device."""
    kc, vc, ks, vs = cache
    n, H, P, D = kc.shape
    if vc.shape != (n, H, D, P) or kc.element_size() != 1 or vc.element_size() != 1:
        raise ValueError("cache: 8-bit codes k [pages][heads][tokens][dim] and v [pages][heads][dim][tokens]")
    if ks.shape != (n, H) or vs.shape != (n, H) or ks.dtype != T.uint8 or vs.dtype != T.uint8:
        raise ValueError("cache: uint8 scales [pages][heads]")
    if not (kc.is_contiguous() and vc.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()):
        raise ValueError("cache: contiguous tensors")
    B, width = page_table.shape
    i32 = T.int32
    if page_table.dtype != i32 or not page_table.is_contiguous():
        raise ValueError("page_table: contiguous int32 [sequences][pages]")
    if kv_lens.dtype != i32 or kv_lens.shape != (B,) or not kv_lens.is_contiguous():
        raise ValueError("kv_lens: contiguous int32 [sequences]")
    dev = kc.get_device()
    starts = bad = 0
    if q_starts is None:
        if B < 1 or total_q % B:
            raise ValueError("without q_starts every sequence has the same number of new tokens")
        if max_q is None:
            max_q = total_q // B
    else:
        if q_starts.dtype != i32 or q_starts.shape != (B + 1,) or not q_starts.is_contiguous():
            raise ValueError("q_starts: contiguous int32 [sequences + 1]")
        starts = q_starts.data_ptr()
        if max_q is None:
            max_q = total_q
    if max_kv is None:
        max_kv = width * P
    if bad_pages is not None:
        if bad_pages.dtype != i32 or bad_pages.numel() < 1:
            raise ValueError("bad_pages: int32")
        bad = bad_pages.data_ptr()
    _device(T, dev, vc, ks, vs, page_table, kv_lens, q_starts, bad_pages)
    return (_PACK_KV8(n, P, H, D, kc.data_ptr(), vc.data_ptr(), ks.data_ptr(), vs.data_ptr()),
            _PACK_BATCH(B, page_table.data_ptr(), width, kv_lens.data_ptr(), starts, total_q, max_q, max_kv, bad), dev)


def _heads(x, H, D, what):
    """Token stride of a [tokens][heads][dim] tensor whose heads are contiguous."""
    shape = x.shape
    if len(shape) != 3 or shape[2] != D or shape[1] != H:
        raise ValueError(f"{what}: [tokens][{H}][{D}] expected, got {list(shape)}")
    s0, s1, s2 = x.stride()
    if s2 != 1 or (s1 != D and H != 1):
        raise ValueError(f"{what}: a token's heads have to be contiguous")
    return s0 if shape[0] > 1 else H * D


def kv8_append(cache, page_table, kv_lens, K, V, q_starts=None, max_q=None, max_kv=None, bad_pages=None,
               stream=None):
    """Write new keys and values [tokens][kv_heads][dim] (bf16 or fp32, tokens may be strided) into the
    cache (see lowbit_kv8_append).  kv_lens counts them already; q_starts None: every sequence has
    tokens / sequences new ones.  max_q and max_kv bound one sequence's new tokens and length and size
    the launch: without them, with q_starts, all the tokens (pass max_q for a batch of sequences), and
    the whole page table."""
    T = _torch or _load()
    _, H, _, D = cache[0].shape
    ks, vs = _heads(K, H, D, "K"), _heads(V, H, D, "V")
    if K.shape[0] != V.shape[0] or K.dtype != V.dtype or K.dtype not in _FLOAT:
        raise ValueError("K and V: the same tokens and type, bf16 or fp32")
    c, b, dev = _kv8(T, cache, page_table, kv_lens, q_starts, K.shape[0], max_q, max_kv, bad_pages)
    if K.get_device() != dev or V.get_device() != dev:
        raise ValueError("K and V lie on another device than the cache")
    rc = _fast.kv8_append(c, b, _FLOAT[K.dtype], K.data_ptr(), V.data_ptr(), ks, vs, _raw_stream(T, dev, stream))
    if rc:
        raise LowbitError("lowbit_kv8_append", rc)


def attention_kv8(Q, cache, page_table, kv_lens, q_starts=None, max_q=None, max_kv=None, softmax_scale=None,
                  causal=True, window=0, O=None, lse=None, return_lse=False, bad_pages=None, stream=None):
    """Attention of bf16 queries [tokens][q_heads][dim] (tokens may be strided) over the cache (see
    lowbit_attention_kv8); softmax_scale None: 1 / sqrt(dim).  Returns O, or (O, lse) with return_lse.
    max_q and max_kv bound one sequence's new tokens and length; they size the launch and choose its
    kernel.  Without them, with q_starts, max_q is all the tokens: single tokens of many sequences
    passed so run as prompts; max_kv is the whole page table."""
    T = _torch or _load()
    D = cache[0].shape[3]
    if Q.dim() != 3 or Q.dtype != T.bfloat16:
        raise ValueError("Q: bf16 [tokens][q_heads][dim]")
    tokens, Hq, _ = Q.shape
    qs = _heads(Q, Hq, D, "Q")
    c, b, dev = _kv8(T, cache, page_table, kv_lens, q_starts, tokens, max_q, max_kv, bad_pages)
    if O is None:
        O = _empty(T, (tokens, Hq, D), T.bfloat16, Q.device, stream)
        os = Hq * D
    else:
        if O.shape != Q.shape or O.dtype != T.bfloat16 or O.get_device() != dev:
            raise ValueError("O: bf16 of Q's shape, on its device")
        os = _heads(O, Hq, D, "O")
    if lse is None:
        if return_lse:
            lse = _empty(T, (tokens, Hq), T.float32, Q.device, stream)
    elif lse.shape != (tokens, Hq) or lse.dtype != T.float32 or not lse.is_contiguous() or lse.get_device() != dev:
        raise ValueError("lse: contiguous fp32 [tokens][q_heads] on Q's device")
    if Q.get_device() != dev:
        raise ValueError("Q lies on another device than the cache")
    rc = _fast.attention_kv8(c, b, Hq, Q.data_ptr(), qs, D ** -0.5 if softmax_scale is None else softmax_scale,
                             1 if causal else 0, window, O.data_ptr(), os, None if lse is None else lse.data_ptr(),
                             _raw_stream(T, dev, stream))
    if rc:
        raise LowbitError("lowbit_attention_kv8", rc)
    return (O, lse) if return_lse else O


def attention_kv8_workspace(cache, page_table, kv_lens, q_heads, total_q, q_starts=None, max_q=None, max_kv=None):
    """Workspace bytes lowbit_attention_kv8 needs for these arguments (reserve before a capture)."""
    T = _torch or _load()
    c, b, _ = _kv8(T, cache, page_table, kv_lens, q_starts, total_q, max_q, max_kv, None)
    n = ctypes.c_size_t()
    _check("lowbit_attention_kv8_workspace",
           lib().lowbit_attention_kv8_workspace(Kv8.from_buffer_copy(c), Kv8Batch.from_buffer_copy(b), q_heads,
                                                ctypes.byref(n)))
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
