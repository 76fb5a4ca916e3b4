"""ctypes binding of libsrftq.so (argument marshalling only).

Every function named ``srftq_*`` here calls the C entry point of the same
name declared in include/srftq.h; the arguments are torch tensors on a CUDA
device (PyTorch provides device memory and streams, nothing else). All of the
codec's work runs in the library's CUDA kernels: there is no fallback, and
loading fails loudly when the library has not been built.

Tensor views are accepted when each row's heads and elements are contiguous;
a slice stride larger than the row count (for example ``cache[:, t0:t1]`` of
a [S, T, H, d] buffer) is passed through as the slice stride in rows.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libsrftq.so")
# the same library built with device-side index checks (SRFTQ_DEBUG_CHECKS)
LIB_DEBUG_PATH = os.path.join(PKG_DIR, "libsrftq_debug.so")

SRFTQ_OK = 0
SRFTQ_ERR_INVALID_ARG = -1
SRFTQ_ERR_UNSUPPORTED = -2
SRFTQ_ERR_MISALIGNED = -3
SRFTQ_ERR_CUDA = -4
SRFTQ_ERR_DEVICE_CHECK = -5

SRFT = 0
SRHT = 1

# Every symbol include/srftq.h declares (checked by the CPU test suite).
EXPORTED = ("srftq_quantize", "srftq_dequantize", "srftq_calibrate_lambda", "srftq_rotate",
            "srftq_dequantize_rotated", "srftq_unrotate", "srftq_decode_attention",
            "srftq_householder_rotation", "srftq_dense_operand", "srftq_calibrate_lambda_dense",
            "srftq_quantize_dense", "srftq_dequantize_dense", "srftq_block_tables",
            "srftq_quantize_paged", "srftq_dequantize_paged", "srftq_prefix_attention",
            "srftq_prefix_attention_workspace", "srftq_status_string",
            "srftq_check_device", "srftq_probe_wait_timeout", "srftq_probe_index_check",
            "srftq_debug_checks", "srftq_version")


class SrftqDesc(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("heads", ctypes.c_int32), ("group", ctypes.c_int32),
                ("bits", ctypes.c_int32), ("rotation", ctypes.c_int32)]


class SrftqError(RuntimeError):
    def __init__(self, fn, status, text):
        super().__init__(f"{fn} failed: status {status} ({text})")
        self.status = status


_libs = {}            # path -> loaded library
_use_debug = False    # set inside debug_checks()


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Loads the in-tree libsrftq.so once (or, inside `debug_checks()`, the
    in-tree libsrftq_debug.so); raises if it is missing (no CPU fallback
    exists)."""
    if path is None:
        path = LIB_DEBUG_PATH if _use_debug else LIB_PATH
    if path in _libs:
        return _libs[path]
    if not os.path.exists(path):
        flag = " --debug" if path == LIB_DEBUG_PATH else ""
        raise FileNotFoundError(
            f"{path} not found: build it with `python -m rotate_then_quantize_b200.build{flag}`")
    lib = ctypes.CDLL(path)
    P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    D = ctypes.POINTER(SrftqDesc)
    lib.srftq_quantize.argtypes = [D, I64, I64, P, I64, P, P, P, P, I64, P]
    lib.srftq_dequantize.argtypes = [D, I64, I64, P, P, I64, P, P, P, I64, P]
    lib.srftq_calibrate_lambda.argtypes = [D, I64, I64, P, I64, P, P, P]
    lib.srftq_rotate.argtypes = [D, I64, I64, P, I64, P, P, P, P]
    lib.srftq_dequantize_rotated.argtypes = [D, I64, I64, P, P, I64, P, P, I64, P]
    lib.srftq_unrotate.argtypes = [D, I64, I64, P, I64, P, P, I64, P]
    lib.srftq_decode_attention.argtypes = [D, I64, I64, I32, P, P, P, P, P, P, P, P, P, I64, I64,
                                           ctypes.c_float, P, P]
    lib.srftq_householder_rotation.argtypes = [D, I64, ctypes.c_int32, P, P, P, P]
    lib.srftq_dense_operand.argtypes = [D, I64, P, P, P]
    lib.srftq_calibrate_lambda_dense.argtypes = [D, I64, I64, P, I64, P, P, P]
    lib.srftq_quantize_dense.argtypes = [D, I64, I64, P, I64, P, P, P, P, I64, P]
    lib.srftq_dequantize_dense.argtypes = [D, I64, I64, P, P, I64, P, P, P, I64, P]
    lib.srftq_block_tables.argtypes = [I64, P, P, I64, P, I64, P, I64, P, I64, P, P, P, P]
    lib.srftq_quantize_paged.argtypes = [D, I64, I64, P, I64, P, P, P, P, P, I64, P]
    lib.srftq_dequantize_paged.argtypes = [D, I64, I64, P, P, I64, P, P, P, P, I64, P]
    lib.srftq_prefix_attention.argtypes = [D, ctypes.c_int32, I64, ctypes.c_int32, P, P, P, P, P,
                                           P, P, P, P, I64, I64, P, I64, P, I64, P,
                                           ctypes.c_float, P, P, P, I64, P]
    lib.srftq_prefix_attention_workspace.argtypes = [D, I64, ctypes.c_int32, I64]
    lib.srftq_status_string.argtypes = [I32]
    lib.srftq_status_string.restype = ctypes.c_char_p
    lib.srftq_check_device.argtypes = [P]
    lib.srftq_probe_wait_timeout.argtypes = [ctypes.c_uint32, P]
    lib.srftq_probe_index_check.argtypes = [I64, I64, P]
    lib.srftq_debug_checks.argtypes = []
    lib.srftq_version.argtypes = []
    for name in EXPORTED:
        if name != "srftq_status_string":
            getattr(lib, name).restype = I32
    lib.srftq_prefix_attention_workspace.restype = I64
    _libs[path] = lib
    return lib


@contextlib.contextmanager
def debug_checks():
    """Within the block every srftq_* call of this module goes to the in-tree
    debug build (libsrftq_debug.so, `python -m rotate_then_quantize_b200.build
    --debug`), whose kernels check every global-memory index against the
    call's extents and record a failure in the device guard word
    (srftq_check_device) instead of making the access."""
    global _use_debug
    load_library(LIB_DEBUG_PATH)
    prev = _use_debug
    _use_debug = True
    try:
        yield
    finally:
        _use_debug = prev


def status_string(status: int) -> str:
    return load_library().srftq_status_string(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != SRFTQ_OK:
        raise SrftqError(fn, status, status_string(status))


def make_desc(d: int, heads: int, group: int, bits: int, rotation: int = SRFT) -> SrftqDesc:
    return SrftqDesc(int(d), int(heads), int(group), int(bits), int(rotation))


def _stream_handle(stream) -> int:
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _rows_layout(t, H: int, row_elems: int, name: str):
    """(pointer, n_slices, n_rows, slice_stride_rows) of a [S, N, H, e] view.

    Each row's heads and elements must be contiguous; slices may sit further
    apart than N rows (a window of a larger cache) but must not overlap, so a
    view whose slice stride is below N rows (an expanded or overlapping
    view) is refused before anything reaches the library."""
    if t.dim() != 4 or t.shape[2] != H or t.shape[3] != row_elems:
        raise ValueError(f"{name}: expected [S, N, {H}, {row_elems}], got {tuple(t.shape)}")
    S, N = t.shape[0], t.shape[1]
    if N > 1 and t.stride(1) != H * row_elems:
        raise ValueError(f"{name}: heads and elements of a row must be contiguous")
    if t.stride(3) != 1 or t.stride(2) != row_elems:
        raise ValueError(f"{name}: heads and elements of a row must be contiguous")
    if S <= 1:
        return t.data_ptr(), S, N, N
    if t.stride(0) % (H * row_elems) != 0:
        raise ValueError(f"{name}: slice stride must be a whole number of rows")
    stride_rows = t.stride(0) // (H * row_elems)
    if stride_rows < N:
        raise ValueError(f"{name}: slices overlap (slice stride {stride_rows} rows < {N} rows)")
    return t.data_ptr(), S, N, stride_rows


def _check_tensor(t, dtype, name: str):
    """t must live on the current CUDA device and have the dtype the C ABI reads."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a torch tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected dtype {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name}: on {t.device}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")


def _rows_view(t, H: int, row_elems: int, name: str, dtype):
    _check_tensor(t, dtype, name)
    return _rows_layout(t, H, row_elems, name)


def _table(t, S: int, H: int, d: int, name: str, dtype):
    _check_tensor(t, dtype, name)
    if tuple(t.shape) != (S, H, d) or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous [{S}, {H}, {d}], got {tuple(t.shape)}")
    return t.data_ptr()


def _dtypes():
    import torch

    return torch.float16, torch.uint8, torch.int8, torch.float32


def srftq_quantize(desc: SrftqDesc, x, signs, lam, codes, scales, stream=None) -> None:
    """x [S,N,H,d] fp16 -> codes [S,N,H,d*bits/8] uint8, scales [S,N,H,d/G] fp16."""
    lib = load_library()
    F16, U8, I8, F32 = _dtypes()
    H, d = desc.heads, desc.d
    px, S, N, xs = _rows_view(x, H, d, "x", F16)
    pc, S2, N2, os_ = _rows_view(codes, H, d * desc.bits // 8, "codes", U8)
    ps, S3, N3, os2 = _rows_view(scales, H, d // desc.group, "scales", F16)
    if (S2, N2) != (S, N) or (S3, N3) != (S, N) or os2 != os_:
        raise ValueError("codes/scales must match x's slices and rows and share a slice stride")
    st = lib.srftq_quantize(ctypes.byref(desc), S, N, px, xs, _table(signs, S, H, d, "signs", I8),
                            _table(lam, S, H, d, "lambda", F32), pc, ps, os_,
                            _stream_handle(stream))
    _check("srftq_quantize", st)


def srftq_dequantize(desc: SrftqDesc, codes, scales, signs, lam, xhat, stream=None) -> None:
    """codes, scales -> xhat [S,N,H,d] fp16 (the inverse of srftq_quantize)."""
    lib = load_library()
    F16, U8, I8, F32 = _dtypes()
    H, d = desc.heads, desc.d
    pc, S, N, is_ = _rows_view(codes, H, d * desc.bits // 8, "codes", U8)
    ps, S2, N2, is2 = _rows_view(scales, H, d // desc.group, "scales", F16)
    px, S3, N3, os_ = _rows_view(xhat, H, d, "xhat", F16)
    if (S2, N2) != (S, N) or (S3, N3) != (S, N) or is2 != is_:
        raise ValueError("codes/scales/xhat shapes disagree")
    st = lib.srftq_dequantize(ctypes.byref(desc), S, N, pc, ps, is_,
                              _table(signs, S, H, d, "signs", I8),
                              _table(lam, S, H, d, "lambda", F32), px, os_,
                              _stream_handle(stream))
    _check("srftq_dequantize", st)


def srftq_calibrate_lambda(desc: SrftqDesc, x, signs, lam_out, n_cal: int, stream=None) -> None:
    """lambda_out [S,H,d] float32 = RMS of the rotated first n_cal rows of x."""
    lib = load_library()
    F16, U8, I8, F32 = _dtypes()
    H, d = desc.heads, desc.d
    px, S, N, xs = _rows_view(x, H, d, "x", F16)
    if n_cal > N:
        raise ValueError("n_cal exceeds the rows of x")
    st = lib.srftq_calibrate_lambda(ctypes.byref(desc), S, int(n_cal), px, xs,
                                    _table(signs, S, H, d, "signs", I8),
                                    _table(lam_out, S, H, d, "lambda_out", F32),
                                    _stream_handle(stream))
    _check("srftq_calibrate_lambda", st)


def srftq_rotate(desc: SrftqDesc, x, signs, y_out, lam=None, stream=None) -> None:
    """y_out [S,N,H,d] float32 (contiguous) = R (s*x), divided by lambda if given."""
    lib = load_library()
    F16, U8, I8, F32 = _dtypes()
    H, d = desc.heads, desc.d
    px, S, N, xs = _rows_view(x, H, d, "x", F16)
    _check_tensor(y_out, F32, "y_out")
    if tuple(y_out.shape) != (S, N, H, d) or not y_out.is_contiguous():
        raise ValueError("y_out must be a contiguous [S, N, H, d] float32 tensor")
    pl = _table(lam, S, H, d, "lambda", F32) if lam is not None else None
    st = lib.srftq_rotate(ctypes.byref(desc), S, N, px, xs, _table(signs, S, H, d, "signs", I8),
                          pl, y_out.data_ptr(), _stream_handle(stream))
    _check("srftq_rotate", st)


def srftq_dequantize_rotated(desc: SrftqDesc, codes, scales, lam, out, stream=None) -> None:
    """codes, scales -> out [S,N,H,d] fp16 = lambda * sigma * q (the rotated domain)."""
    lib = load_library()
    F16, U8, I8, F32 = _dtypes()
    H, d = desc.heads, desc.d
    pc, S, N, is_ = _rows_view(codes, H, d * desc.bits // 8, "codes", U8)
    ps, S2, N2, is2 = _rows_view(scales, H, d // desc.group, "scales", F16)
    po, S3, N3, os_ = _rows_view(out, H, d, "out", F16)
    if (S2, N2) != (S, N) or (S3, N3) != (S, N) or is2 != is_:
        raise ValueError("codes/scales/out shapes disagree")
    st = lib.srftq_dequantize_rotated(ctypes.byref(desc), S, N, pc, ps, is_,
                                      _table(lam, S, H, d, "lambda", F32), po, os_,
                                      _stream_handle(stream))
    _check("srftq_dequantize_rotated", st)


def srftq_unrotate(desc: SrftqDesc, y, signs, x_out, stream=None) -> None:
    """x_out [S,N,H,d] float32 = s * R^T y for y [S,N,H,d] float32."""
    lib = load_library()
    F16, U8, I8, F32 = _dtypes()
    H, d = desc.heads, desc.d
    py, S, N, ys = _rows_view(y, H, d, "y", F32)
    px, S2, N2, xs = _rows_view(x_out, H, d, "x_out", F32)
    if (S2, N2) != (S, N):
        raise ValueError("y/x_out shapes disagree")
    st = lib.srftq_unrotate(ctypes.byref(desc), S, N, py, ys, _table(signs, S, H, d, "signs", I8),
                            px, xs, _stream_handle(stream))
    _check("srftq_unrotate", st)


def _cache_rows(t, H: int, row_elems: int, name: str, dtype):
    """(pointer, rows) of a contiguous [rows, H, e] cache tensor."""
    _check_tensor(t, dtype, name)
    if t.dim() != 3 or t.shape[1] != H or t.shape[2] != row_elems or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous [rows, {H}, {row_elems}], got "
                         f"{tuple(t.shape)}")
    return t.data_ptr(), t.shape[0]


def srftq_decode_attention(desc: SrftqDesc, q, k_codes, k_scales, k_signs, k_lambda, v_codes,
                           v_scales, v_signs, v_lambda, n_ctx: int, tok_stride_rows: int,
                           seq_stride_rows: int, scale: float, out, stream=None) -> None:
    """out [n_seq, H*q_per_kv, d] float32 = softmax(scale q . khat) vhat over n_ctx
    tokens of the quantised K and V caches ([rows, H, ...] tensors; token t of
    sequence b is row t*tok_stride_rows + b*seq_stride_rows). The call makes
    three launches on the stream and uses `out` as their scratch, so `out`
    holds the result once that work is complete."""
    lib = load_library()
    F16, U8, I8, F32 = _dtypes()
    H, d = desc.heads, desc.d
    _check_tensor(q, F16, "q")
    if q.dim() != 3 or q.shape[1] % H or q.shape[2] != d or not q.is_contiguous():
        raise ValueError(f"q: expected contiguous [n_seq, {H}*q_per_kv, {d}]")
    n_seq, q_per_kv = q.shape[0], q.shape[1] // H
    _check_tensor(out, F32, "out")
    if tuple(out.shape) != tuple(q.shape) or not out.is_contiguous():
        raise ValueError("out must be a contiguous float32 tensor shaped like q")
    cb, ng = d * desc.bits // 8, d // desc.group
    pk, rk = _cache_rows(k_codes, H, cb, "k_codes", U8)
    pks, rks = _cache_rows(k_scales, H, ng, "k_scales", F16)
    pv, rv = _cache_rows(v_codes, H, cb, "v_codes", U8)
    pvs, rvs = _cache_rows(v_scales, H, ng, "v_scales", F16)
    need = (n_ctx - 1) * tok_stride_rows + (n_seq - 1) * seq_stride_rows + 1 if n_seq else 0
    if min(rk, rks, rv, rvs) < need:
        raise ValueError(f"the caches hold fewer than the {need} rows addressed")
    for t, name, dt in ((k_signs, "k_signs", I8), (v_signs, "v_signs", I8),
                        (k_lambda, "k_lambda", F32), (v_lambda, "v_lambda", F32)):
        _check_tensor(t, dt, name)
        if tuple(t.shape) != (H, d) or not t.is_contiguous():
            raise ValueError(f"{name}: expected contiguous [{H}, {d}]")
    st = lib.srftq_decode_attention(ctypes.byref(desc), n_seq, int(n_ctx), q_per_kv, q.data_ptr(),
                                    pk, pks, k_signs.data_ptr(), k_lambda.data_ptr(), pv, pvs,
                                    v_signs.data_ptr(), v_lambda.data_ptr(), int(tok_stride_rows),
                                    int(seq_stride_rows), float(scale), out.data_ptr(),
                                    _stream_handle(stream))
    _check("srftq_decode_attention", st)


def _matrices(t, S: int, H: int, shape: tuple, name: str, dtype):
    _check_tensor(t, dtype, name)
    if tuple(t.shape) != (S, H) + tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {(S, H) + tuple(shape)}, "
                         f"got {tuple(t.shape)}")
    return t.data_ptr()


def srftq_householder_rotation(desc: SrftqDesc, reflectors, signs, rot_out, stream=None) -> None:
    """rot_out [S,H,d,d] float32 = H(v_1) ... H(v_k) B (B the signed SRFT/SRHT
    matrix of desc.rotation) for reflectors [S,H,k,d] float32 (None for k = 0)."""
    lib = load_library()
    F16, U8, I8, F32 = _dtypes()
    S, H, d = rot_out.shape[0], desc.heads, desc.d
    po = _matrices(rot_out, S, H, (d, d), "rot_out", F32)
    ps = _table(signs, S, H, d, "signs", I8)
    if reflectors is None:
        k, pr = 0, None
    else:
        if reflectors.dim() != 4:
            raise ValueError("reflectors: expected [S, H, k, d]")
        k = reflectors.shape[2]
        pr = _matrices(reflectors, S, H, (k, d), "reflectors", F32)
    st = lib.srftq_householder_rotation(ctypes.byref(desc), S, int(k), pr, ps, po,
                                        _stream_handle(stream))
    _check("srftq_householder_rotation", st)


def srftq_dense_operand(desc: SrftqDesc, rot, operand_out, stream=None) -> None:
    """operand_out [S,H,2,d,d] fp16 = (fp16(R), fp16(R - hi)) of rot [S,H,d,d] float32."""
    lib = load_library()
    F16, U8, I8, F32 = _dtypes()
    S, H, d = rot.shape[0], desc.heads, desc.d
    pr = _matrices(rot, S, H, (d, d), "rot", F32)
    po = _matrices(operand_out, S, H, (2, d, d), "operand_out", F16)
    st = lib.srftq_dense_operand(ctypes.byref(desc), S, pr, po, _stream_handle(stream))
    _check("srftq_dense_operand", st)


def srftq_calibrate_lambda_dense(desc: SrftqDesc, x, operand, lam_out, n_cal: int,
                                 stream=None) -> None:
    """lam_out [S,H,d] float32 = RMS of R x over the first n_cal rows of x."""
    lib = load_library()
    F16, U8, I8, F32 = _dtypes()
    H, d = desc.heads, desc.d
    px, S, N, xs = _rows_view(x, H, d, "x", F16)
    if n_cal > N:
        raise ValueError("n_cal exceeds the rows of x")
    st = lib.srftq_calibrate_lambda_dense(ctypes.byref(desc), S, int(n_cal), px, xs,
                                          _matrices(operand, S, H, (2, d, d), "operand", F16),
                                          _table(lam_out, S, H, d, "lambda_out", F32),
                                          _stream_handle(stream))
    _check("srftq_calibrate_lambda_dense", st)


def srftq_quantize_dense(desc: SrftqDesc, x, operand, lam, codes, scales, stream=None) -> None:
    """x [S,N,H,d] fp16 -> codes, scales with the dense rotation of `operand`."""
    lib = load_library()
    F16, U8, I8, F32 = _dtypes()
    H, d = desc.heads, desc.d
    px, S, N, xs = _rows_view(x, H, d, "x", F16)
    pc, S2, N2, os_ = _rows_view(codes, H, d * desc.bits // 8, "codes", U8)
    ps, S3, N3, os2 = _rows_view(scales, H, d // desc.group, "scales", F16)
    if (S2, N2) != (S, N) or (S3, N3) != (S, N) or os2 != os_:
        raise ValueError("codes/scales must match x's slices and rows and share a slice stride")
    st = lib.srftq_quantize_dense(ctypes.byref(desc), S, N, px, xs,
                                  _matrices(operand, S, H, (2, d, d), "operand", F16),
                                  _table(lam, S, H, d, "lambda", F32), pc, ps, os_,
                                  _stream_handle(stream))
    _check("srftq_quantize_dense", st)


def srftq_dequantize_dense(desc: SrftqDesc, codes, scales, operand, lam, xhat,
                           stream=None) -> None:
    """codes, scales -> xhat [S,N,H,d] fp16 = R^T (lambda sigma q)."""
    lib = load_library()
    F16, U8, I8, F32 = _dtypes()
    H, d = desc.heads, desc.d
    pc, S, N, is_ = _rows_view(codes, H, d * desc.bits // 8, "codes", U8)
    ps, S2, N2, is2 = _rows_view(scales, H, d // desc.group, "scales", F16)
    px, S3, N3, os_ = _rows_view(xhat, H, d, "xhat", F16)
    if (S2, N2) != (S, N) or (S3, N3) != (S, N) or is2 != is_:
        raise ValueError("codes/scales/xhat shapes disagree")
    st = lib.srftq_dequantize_dense(ctypes.byref(desc), S, N, pc, ps, is_,
                                    _matrices(operand, S, H, (2, d, d), "operand", F16),
                                    _table(lam, S, H, d, "lambda", F32), px, os_,
                                    _stream_handle(stream))
    _check("srftq_dequantize_dense", st)


# The paged calls are made once per layer and step, so what they do on the host
# is kept short: one look at the current device and stream per call, one
# comparison per property of a tensor.
_rt = None


def _runtime():
    """torch and the types of the paged calls, looked up once."""
    global _rt
    if _rt is None:
        import types

        import torch

        _rt = types.SimpleNamespace(
            torch=torch, F16=torch.float16, BF16=torch.bfloat16, F32=torch.float32,
            U8=torch.uint8, I8=torch.int8, I32=torch.int32, I64=torch.int64,
            get_device=getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
            raw_stream=getattr(torch._C, "_cuda_getCurrentRawStream", None))
    return _rt


def _device(r) -> int:
    """The current CUDA device (-2 without one: no tensor is there)."""
    try:
        return r.get_device()
    except (RuntimeError, AssertionError):
        return -2


def _raw_stream(r, stream, dev: int) -> int:
    if stream is not None or r.raw_stream is None:
        return _stream_handle(stream)
    return r.raw_stream(dev)


def _address(t, dtype, shape: tuple, name: str, dev: int) -> int:
    """Address of a contiguous tensor of this type and shape on device `dev`."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == dev
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _check_tensor(t, dtype, name)
    raise ValueError(f"{name}: expected contiguous {list(shape)}, got {tuple(t.shape)} with "
                     f"strides {t.stride()}")


def _dims(t, n: int, name: str):
    """The shape of a tensor of n dimensions."""
    shape = getattr(t, "shape", None)
    if shape is None or len(shape) != n:
        raise ValueError(f"{name}: expected a tensor of {n} dimensions, got "
                         f"{type(t).__name__ if shape is None else tuple(shape)}")
    return shape


def srftq_block_tables(cached_lens, new_lens, free_pages, block_table, page_size: int, slots,
                       seq_lens, row_start, counts, stream=None) -> None:
    """Block tables and slot map of a step from the requests' lengths (see
    include/srftq.h): int32 tensors, slots int64; block_table [n_seq, max_pages]
    is extended in place, the last four are written."""
    lib, r = load_library(), _runtime()
    I32, dev = r.I32, _device(r)
    n_seq = _dims(cached_lens, 1, "cached_lens")[0]
    n_free = _dims(free_pages, 1, "free_pages")[0]
    n_slots = _dims(slots, 1, "slots")[0]
    max_pages = _dims(block_table, 2, "block_table")[1]
    st = lib.srftq_block_tables(
        n_seq, _address(cached_lens, I32, (n_seq,), "cached_lens", dev),
        _address(new_lens, I32, (n_seq,), "new_lens", dev), int(page_size),
        _address(free_pages, I32, (n_free,), "free_pages", dev), n_free,
        _address(block_table, I32, (n_seq, max_pages), "block_table", dev), max_pages,
        _address(slots, r.I64, (n_slots,), "slots", dev), n_slots,
        _address(seq_lens, I32, (n_seq,), "seq_lens", dev),
        _address(row_start, I32, (n_seq + 1,), "row_start", dev),
        _address(counts, I32, (3,), "counts", dev), _raw_stream(r, stream, dev))
    _check("srftq_block_tables", st)


def _window(t, dtype, H: int, d: int, name: str, dev: int):
    """(address, slices, rows, slice stride in rows) of [S, N, H, d] rows, or of a
    window of a larger cache."""
    S, N = _dims(t, 4, name)[:2]
    if t.shape == (S, N, H, d) and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr(), S, N, N
    return _rows_view(t, H, d, name, dtype)


def srftq_quantize_paged(desc: SrftqDesc, x, signs, lam, slots, codes, scales,
                         stream=None) -> None:
    """x [S,N,H,d] fp16 -> rows slots[r] (int64 [N]) of the pools codes
    [S,rows,H,d*bits/8] uint8 and scales [S,rows,H,d/G] fp16."""
    lib, r = load_library(), _runtime()
    H, d, dev = desc.heads, desc.d, _device(r)
    px, S, N, xs = _window(x, r.F16, H, d, "x", dev)
    rows = _dims(codes, 4, "codes")[1]
    st = lib.srftq_quantize_paged(
        ctypes.byref(desc), S, N, px, xs, _address(signs, r.I8, (S, H, d), "signs", dev),
        _address(lam, r.F32, (S, H, d), "lambda", dev), _address(slots, r.I64, (N,), "slots", dev),
        _address(codes, r.U8, (S, rows, H, d * desc.bits // 8), "codes", dev),
        _address(scales, r.F16, (S, rows, H, d // desc.group), "scales", dev), rows,
        _raw_stream(r, stream, dev))
    _check("srftq_quantize_paged", st)


def srftq_dequantize_paged(desc: SrftqDesc, codes, scales, slots, signs, lam, xhat,
                           stream=None) -> None:
    """Rows slots[r] of the pools -> rows r of xhat [S,N,H,d] fp16 (rows with a
    negative slot are left as they were)."""
    lib, r = load_library(), _runtime()
    H, d, dev = desc.heads, desc.d, _device(r)
    px, S, N, xs = _window(xhat, r.F16, H, d, "xhat", dev)
    rows = _dims(codes, 4, "codes")[1]
    st = lib.srftq_dequantize_paged(
        ctypes.byref(desc), S, N,
        _address(codes, r.U8, (S, rows, H, d * desc.bits // 8), "codes", dev),
        _address(scales, r.F16, (S, rows, H, d // desc.group), "scales", dev), rows,
        _address(slots, r.I64, (N,), "slots", dev),
        _address(signs, r.I8, (S, H, d), "signs", dev),
        _address(lam, r.F32, (S, H, d), "lambda", dev), px, xs, _raw_stream(r, stream, dev))
    _check("srftq_dequantize_paged", st)


def srftq_prefix_attention_workspace(desc: SrftqDesc, n_seq: int, q_per_kv: int,
                                     prefix_len: int) -> int:
    """Bytes of workspace that srftq_prefix_attention needs for these sizes."""
    n = load_library().srftq_prefix_attention_workspace(ctypes.byref(desc), int(n_seq),
                                                        int(q_per_kv), int(prefix_len))
    if n < 0:
        _check("srftq_prefix_attention_workspace", n)
    return n


def srftq_prefix_attention(desc: SrftqDesc, q, k_codes, k_scales, k_signs, k_lambda, v_codes,
                           v_scales, v_signs, v_lambda, page_size: int, prefix_table,
                           prefix_len: int, block_table, seq_lens, scale: float, out, lse,
                           workspace, stream=None) -> None:
    """out [n_seq, H*q_per_kv, d] = softmax(scale q . khat) vhat over the pages of
    each sequence, the first prefix_len tokens shared (see include/srftq.h).
    Pools are [rows, H, ...] tensors; prefix_table may be None for prefix_len 0,
    lse None; workspace is a contiguous uint8 tensor."""
    lib, r = load_library(), _runtime()
    H, d, dev = desc.heads, desc.d, _device(r)
    shape = _dims(q, 3, "q")
    dtype = q.dtype
    if dtype is not r.F16 and dtype is not r.BF16:
        raise ValueError(f"q: expected float16 or bfloat16, got {dtype}")
    n_seq, HQ = shape[0], shape[1]
    if HQ % H:
        raise ValueError(f"q: {HQ} heads are no multiple of the cache's {H}")
    rows = _dims(k_codes, 3, "k_codes")[0]
    page_size, prefix_len = int(page_size), int(prefix_len)
    if page_size < 1 or rows % page_size:
        raise ValueError(f"the pools' {rows} rows are no whole pages of {page_size}")
    codes_shape, scales_shape = (rows, H, d * desc.bits // 8), (rows, H, d // desc.group)
    pt = 0
    if prefix_table is not None:
        n_pt = _dims(prefix_table, 1, "prefix_table")[0]
        pt = _address(prefix_table, r.I32, (n_pt,), "prefix_table", dev)
    if prefix_len > 0 and (prefix_table is None or n_pt * page_size < prefix_len):
        raise ValueError(f"prefix_table: too few pages for {prefix_len} tokens")
    max_pages = _dims(block_table, 2, "block_table")[1]
    n_ws = _dims(workspace, 1, "workspace")[0]
    st = lib.srftq_prefix_attention(
        ctypes.byref(desc), 0 if dtype is r.F16 else 1, n_seq, HQ // H,
        _address(q, dtype, (n_seq, HQ, d), "q", dev),
        _address(k_codes, r.U8, codes_shape, "k_codes", dev),
        _address(k_scales, r.F16, scales_shape, "k_scales", dev),
        _address(k_signs, r.I8, (H, d), "k_signs", dev),
        _address(k_lambda, r.F32, (H, d), "k_lambda", dev),
        _address(v_codes, r.U8, codes_shape, "v_codes", dev),
        _address(v_scales, r.F16, scales_shape, "v_scales", dev),
        _address(v_signs, r.I8, (H, d), "v_signs", dev),
        _address(v_lambda, r.F32, (H, d), "v_lambda", dev), rows // page_size, page_size, pt,
        prefix_len, _address(block_table, r.I32, (n_seq, max_pages), "block_table", dev),
        max_pages, _address(seq_lens, r.I32, (n_seq,), "seq_lens", dev), float(scale),
        _address(out, dtype, (n_seq, HQ, d), "out", dev),
        None if lse is None else _address(lse, r.F32, (n_seq, HQ), "lse", dev),
        _address(workspace, r.U8, (n_ws,), "workspace", dev), n_ws, _raw_stream(r, stream, dev))
    _check("srftq_prefix_attention", st)


def srftq_probe_wait_timeout(polls: int, stream=None) -> int:
    """Launches the device-side timeout probe (see include/srftq.h); returns the status."""
    return int(load_library().srftq_probe_wait_timeout(int(polls), _stream_handle(stream)))


def srftq_probe_index_check(index: int, limit: int, stream=None) -> int:
    """Launches the device-side index-check probe (see include/srftq.h); returns the status."""
    return int(load_library().srftq_probe_index_check(int(index), int(limit),
                                                      _stream_handle(stream)))


def srftq_debug_checks() -> bool:
    """Whether the active library was built with the device-side index checks."""
    return bool(load_library().srftq_debug_checks())


def srftq_check_device(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device guard status."""
    return int(load_library().srftq_check_device(_stream_handle(stream)))


def srftq_version() -> int:
    return int(load_library().srftq_version())


# ---------------------------------------------------------------------------
# Allocating conveniences (torch allocates; the library computes)
# ---------------------------------------------------------------------------

def quantize(x, signs, lam, group: int = 16, bits: int = 4, rotation: int = SRFT, stream=None):
    """Returns (codes, scales) for x [S,N,H,d] fp16 on a CUDA device."""
    import torch

    S, N, H, d = x.shape
    desc = make_desc(d, H, group, bits, rotation)
    codes = torch.empty((S, N, H, d * bits // 8), dtype=torch.uint8, device=x.device)
    scales = torch.empty((S, N, H, d // group), dtype=torch.float16, device=x.device)
    srftq_quantize(desc, x, signs, lam, codes, scales, stream)
    return codes, scales


def dequantize(codes, scales, signs, lam, d: int, group: int = 16, bits: int = 4,
               rotation: int = SRFT, stream=None):
    import torch

    S, N, H, _ = codes.shape
    desc = make_desc(d, H, group, bits, rotation)
    xhat = torch.empty((S, N, H, d), dtype=torch.float16, device=codes.device)
    srftq_dequantize(desc, codes, scales, signs, lam, xhat, stream)
    return xhat


def calibrate_lambda(x, signs, n_cal: int = 512, rotation: int = SRFT, stream=None):
    import torch

    S, N, H, d = x.shape
    desc = make_desc(d, H, 8, 4, rotation)
    lam = torch.empty((S, H, d), dtype=torch.float32, device=x.device)
    srftq_calibrate_lambda(desc, x, signs, lam, n_cal, stream)
    return lam


def rotate(x, signs, lam=None, rotation: int = SRFT, stream=None):
    import torch

    S, N, H, d = x.shape
    desc = make_desc(d, H, 8, 4, rotation)
    y = torch.empty((S, N, H, d), dtype=torch.float32, device=x.device)
    srftq_rotate(desc, x, signs, y, lam, stream)
    return y


def dequantize_rotated(codes, scales, lam, d: int, group: int = 16, bits: int = 4, stream=None):
    """Returns lambda * sigma * q [S,N,H,d] fp16: the cache in the rotated domain."""
    import torch

    S, N, H, _ = codes.shape
    desc = make_desc(d, H, group, bits, SRFT)
    out = torch.empty((S, N, H, d), dtype=torch.float16, device=codes.device)
    srftq_dequantize_rotated(desc, codes, scales, lam, out, stream)
    return out


def unrotate(y, signs, rotation: int = SRFT, stream=None):
    """Returns s * R^T y [S,N,H,d] float32 for y [S,N,H,d] float32."""
    import torch

    S, N, H, d = y.shape
    desc = make_desc(d, H, 8, 4, rotation)
    x = torch.empty((S, N, H, d), dtype=torch.float32, device=y.device)
    srftq_unrotate(desc, y, signs, x, stream)
    return x


def decode_attention(q, k_codes, k_scales, k_signs, k_lambda, v_codes, v_scales, v_signs,
                     v_lambda, group: int = 16, bits: int = 4, rotation: int = SRFT,
                     n_ctx: int = None, tok_stride_rows: int = None, seq_stride_rows: int = 1,
                     scale: float = None, stream=None):
    """Fused decode attention over quantised K/V caches (see srftq_decode_attention).
    Defaults follow the decode layout row = token * n_seq + sequence."""
    import math

    import torch

    n_seq, HQ, d = q.shape
    H = k_codes.shape[1]
    if tok_stride_rows is None:
        tok_stride_rows = n_seq
    if n_ctx is None:
        n_ctx = k_codes.shape[0] // tok_stride_rows
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    desc = make_desc(d, H, group, bits, rotation)
    out = torch.empty((n_seq, HQ, d), dtype=torch.float32, device=q.device)
    srftq_decode_attention(desc, q, k_codes, k_scales, k_signs, k_lambda, v_codes, v_scales,
                           v_signs, v_lambda, n_ctx, tok_stride_rows, seq_stride_rows, scale, out,
                           stream)
    return out


def householder_rotation(reflectors, signs, rotation: int = SRFT, stream=None):
    """Returns R [S,H,d,d] float32 = H(v_1) ... H(v_k) B for reflectors
    [S,H,k,d] float32 (or None) on top of the signed SRFT/SRHT base."""
    import torch

    S, H, d = signs.shape
    desc = make_desc(d, H, 8, 4, rotation)
    rot = torch.empty((S, H, d, d), dtype=torch.float32, device=signs.device)
    srftq_householder_rotation(desc, reflectors, signs, rot, stream)
    return rot


def dense_operand(rot, stream=None):
    """Returns the fp16 (hi, lo) operand [S,H,2,d,d] of rotations [S,H,d,d]."""
    import torch

    S, H, d, _ = rot.shape
    desc = make_desc(d, H, 8, 4)
    op = torch.empty((S, H, 2, d, d), dtype=torch.float16, device=rot.device)
    srftq_dense_operand(desc, rot, op, stream)
    return op


def calibrate_lambda_dense(x, operand, n_cal: int = 512, stream=None):
    import torch

    S, N, H, d = x.shape
    desc = make_desc(d, H, 8, 4)
    lam = torch.empty((S, H, d), dtype=torch.float32, device=x.device)
    srftq_calibrate_lambda_dense(desc, x, operand, lam, n_cal, stream)
    return lam


def quantize_dense(x, operand, lam, group: int = 16, bits: int = 4, stream=None):
    """Returns (codes, scales) for x [S,N,H,d] fp16 with the dense rotation."""
    import torch

    S, N, H, d = x.shape
    desc = make_desc(d, H, group, bits)
    codes = torch.empty((S, N, H, d * bits // 8), dtype=torch.uint8, device=x.device)
    scales = torch.empty((S, N, H, d // group), dtype=torch.float16, device=x.device)
    srftq_quantize_dense(desc, x, operand, lam, codes, scales, stream)
    return codes, scales


def dequantize_dense(codes, scales, operand, lam, d: int, group: int = 16, bits: int = 4,
                     stream=None):
    import torch

    S, N, H, _ = codes.shape
    desc = make_desc(d, H, group, bits)
    xhat = torch.empty((S, N, H, d), dtype=torch.float16, device=codes.device)
    srftq_dequantize_dense(desc, codes, scales, operand, lam, xhat, stream)
    return xhat


@functools.lru_cache(maxsize=256)
def _desc_of(d: int, heads: int, group: int, bits: int, rotation: int) -> SrftqDesc:
    return make_desc(d, heads, group, bits, rotation)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(d, heads, group, bits, rotation, n_seq, q_per_kv, prefix_len, device) -> int:
    return srftq_prefix_attention_workspace(_desc_of(d, heads, group, bits, rotation), n_seq,
                                            q_per_kv, prefix_len)


def _empty(like, shape, dtype, stream):
    """Memory for work on `stream`: what the call's end gives back is then reused
    in that stream's order."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with _runtime().torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def block_tables(cached_lens, new_lens, free_pages, block_table, page_size: int, n_slots: int,
                 stream=None):
    """Extends block_table in place by the pages that the new tokens need and
    returns (slots [n_slots] int64, seq_lens [n_seq], row_start [n_seq + 1],
    counts [3]: pages taken, pages wanted, new tokens), the last three int32.
    n_slots is the batch's number of rows: those behind the last sequence's
    have slot -1."""
    r = _runtime()
    n_seq = _dims(cached_lens, 1, "cached_lens")[0]
    if not isinstance(cached_lens, r.torch.Tensor):
        _check_tensor(cached_lens, r.I32, "cached_lens")
    slots = _empty(cached_lens, n_slots, r.I64, stream)
    seq_lens = _empty(cached_lens, n_seq, r.I32, stream)
    row_start = _empty(cached_lens, n_seq + 1, r.I32, stream)
    counts = _empty(cached_lens, 3, r.I32, stream)
    srftq_block_tables(cached_lens, new_lens, free_pages, block_table, page_size, slots, seq_lens,
                       row_start, counts, stream)
    return slots, seq_lens, row_start, counts


def quantize_paged(x, signs, lam, slots, codes, scales, group: int = 16, bits: int = 4,
                   rotation: int = SRFT, stream=None) -> None:
    """Quantises x [S,N,H,d] fp16 into rows slots[r] of the pools codes
    [S,rows,H,d*bits/8] and scales [S,rows,H,d/group] (nowhere for a negative
    slot)."""
    _, _, H, d = _dims(x, 4, "x")
    srftq_quantize_paged(_desc_of(d, H, group, bits, rotation), x, signs, lam, slots, codes,
                         scales, stream)


def dequantize_paged(codes, scales, slots, signs, lam, d: int, group: int = 16, bits: int = 4,
                     rotation: int = SRFT, out=None, stream=None):
    """Returns the rows slots[r] of the pools as fp16 [S,N,H,d]. Rows with a
    negative slot are left as they were in `out`, zero without one."""
    S, _, H, _ = _dims(codes, 4, "codes")
    if out is None:
        r = _runtime()
        _check_tensor(codes, r.U8, "codes")
        n = _dims(slots, 1, "slots")[0]
        with contextlib.nullcontext() if stream is None else r.torch.cuda.stream(stream):
            out = codes.new_zeros((S, n, H, d), dtype=r.F16)
    srftq_dequantize_paged(_desc_of(d, H, group, bits, rotation), codes, scales, slots, signs, lam,
                           out, stream)
    return out


def prefix_attention(q, k_codes, k_scales, k_signs, k_lambda, v_codes, v_scales, v_signs,
                     v_lambda, block_table, seq_lens, prefix_table=None, prefix_len: int = 0,
                     page_size: int = 64, group: int = 16, bits: int = 4, rotation: int = SRFT,
                     scale: float = None, out=None, return_lse: bool = False, workspace=None,
                     stream=None):
    """Decode attention over a paged cache for a batch that shares its first
    prefix_len tokens (see srftq_prefix_attention). Returns out [n_seq,
    H*q_per_kv, d] in q's type, or (out, lse) with the float32 log-sum-exp of
    the scores. Without a workspace it allocates one for the call."""
    r = _runtime()
    n_seq, HQ, d = _dims(q, 3, "q")
    H = _dims(k_codes, 3, "k_codes")[1]
    if scale is None:
        scale = d ** -0.5
    desc = _desc_of(d, H, group, bits, rotation)
    if not isinstance(q, r.torch.Tensor):
        _check_tensor(q, None, "q")
    if out is None:
        out = _empty(q, q.shape, q.dtype, stream)
    lse = _empty(q, (n_seq, HQ), r.F32, stream) if return_lse else None
    if workspace is None:
        need = _workspace_bytes(d, H, group, bits, rotation, n_seq, HQ // H if H else 0,
                                int(prefix_len), _device(r))
        workspace = _empty(q, need, r.U8, stream)
    srftq_prefix_attention(desc, q, k_codes, k_scales, k_signs, k_lambda, v_codes, v_scales,
                           v_signs, v_lambda, page_size, prefix_table, prefix_len, block_table,
                           seq_lens, scale, out, lse, workspace, stream)
    return (out, lse) if return_lse else out
