"""Python binding of libqgemm.so, the block-quantized weight matmul for MI355X (gfx950).

The functions below carry the names of the C entry points declared in include/qgemm.h and only
marshal arguments: torch tensors become device pointers, dtypes become the activation-type enum,
the current torch stream is passed as the hipStream_t, and a non-zero status raises QGError.
Every step of the computation runs in the library's HIP kernels.  There is no fallback: if the
library is not built, loading raises.

Host-side helpers for the packed layout (pack_q4 / pack_q4_blocks, expert tables) live here too;
they only move bytes.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqgemm.so")

QG_OK, QG_EINVAL, QG_EALIGN, QG_ESHAPE, QG_EUNSUPPORTED, QG_ELAUNCH, QG_EPLAN, QG_EWORKSPACE, QG_ESCRATCH = range(9)
QG_NOALLOC_SCRATCH_BYTES = 16 << 20
QG_X_F32, QG_X_F16, QG_X_BF16 = 0, 1, 2
QG_EXACT, QG_FAST, QG_FAST_WEXACT = 0, 1, 2
QG_FMT_Q4, QG_FMT_Q4A, QG_FMT_Q8, QG_FMT_Q8A, QG_FMT_Q8A16 = 0, 1, 2, 3, 4

FMT = {"q4": QG_FMT_Q4, "q4a": QG_FMT_Q4A, "q8": QG_FMT_Q8, "q8a": QG_FMT_Q8A, "q8a16": QG_FMT_Q8A16}
MODE = {"exact": QG_EXACT, "fast": QG_FAST, "fast_wexact": QG_FAST_WEXACT}

# exported symbols of include/qgemm.h, in declaration order
SYMBOLS = [
    "qg_strerror", "qg_abi_version",
    "qgemm_q4", "qgemm_q4a", "qgemm_q8", "qgemm_q8a", "qgemm_q8a16", "qgemm_batch",
    "qgemv_q4", "qgemv_q4a", "qgemv_q8", "qgemv_q8a", "qgemv_q8a16",
    "qg_dequant_dump", "qg_repack_gguf", "qg_repack_gguf_q8a", "qg_repack_gguf_q8a16", "qg_repack_q8f", "qg_col_scale", "qg_conv_stats",
    "qg_conv2d",
    "qg_moe_plan_host", "qg_moe_plan", "qg_x_half", "qg_x_half_guard", "qgemm_moe_grouped", "qg_swiglu", "qg_moe_combine",
    "qg_moe_ffn_workspace", "qg_moe_ffn", "qg_moe_ffn_noalloc",
    "qg_kv8_write", "qg_kv8_read", "qg_attn_kv8_workspace", "qg_attn_kv8", "qgemm_w8a8_workspace", "qgemm_w8a8",
    "qg_rope_freqs", "qg_rope", "qg_kv8_write_rope", "qg_tree_plan", "qg_attn_kv8_tree", "qg_draft_verify_workspace",
    "qg_draft_verify",
]


class QGError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {strerror(status)} (status {status})")


_lib = None
_p, _i, _sz = C.c_void_p, C.c_int, C.c_size_t


def lib() -> C.CDLL:
    """The loaded libqgemm.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; "
                              f"g.build()'` (or block_quantized_weight_affine_amd/build.py)")
        L = C.CDLL(LIB_PATH)
        L.qg_strerror.restype = C.c_char_p
        L.qg_strerror.argtypes = [_i]
        L.qg_abi_version.restype = _i
        L.qg_abi_version.argtypes = []
        sig_dense = [_p, _p, _p, _i, _p, _i, _i, _i, _i, _p]
        L.qgemm_q4.argtypes = sig_dense
        L.qgemm_q8.argtypes = sig_dense
        L.qgemm_q4a.argtypes = [_p, _p, _p, _i, _p, _i, _p, _i, _i, _i, _i, _p]
        sig_gemv = [_p, _p, _p, _i, _p, _i, _i, _i, _p]
        L.qgemv_q4.argtypes = sig_gemv
        L.qgemv_q8.argtypes = sig_gemv
        L.qgemv_q4a.argtypes = [_p, _p, _p, _i, _p, _i, _p, _i, _i, _i, _p]
        L.qgemm_q8a.argtypes = [_p, _p, _p, _p, _i, _p, _i, _i, _i, _i, _p]
        L.qgemv_q8a.argtypes = [_p, _p, _p, _p, _i, _p, _i, _i, _i, _p]
        L.qg_repack_gguf_q8a.argtypes = [_i, _p, _i, _i, _p, _p, _p, _p]
        L.qgemm_q8a16.argtypes = [_p, _p, _p, _p, _i, _p, _i, _i, _i, _i, _p]
        L.qgemv_q8a16.argtypes = [_p, _p, _p, _p, _i, _p, _i, _i, _i, _p]
        L.qg_repack_gguf_q8a16.argtypes = [_i, _p, _i, _i, _p, _p, _p, _p]
        L.qg_repack_q8f.argtypes = [_p, _i, _i, _i, _p, _p, _p]
        L.qg_col_scale.argtypes = [_p, _i, _i, _i, _p, _p, _i, _p]
        L.qg_conv_stats.argtypes = [_p, _i, _i, _i, C.c_float, _p, _p]
        L.qg_conv2d.argtypes = [_i, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _p, _p, _i, _p, _i, _p]
        L.qg_dequant_dump.argtypes = [_i, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _p, _p]
        L.qg_moe_plan_host.argtypes = [_p, _i, _i, _i, _p, _p, _p, _p, _p]
        L.qg_repack_gguf.argtypes = [_i, _p, _i, _i, _p, _p, _p]
        L.qgemm_batch.argtypes = [_i, _i, _p, _i, _p, _i, _i, _i, _i, _p]
        L.qg_moe_plan.argtypes = [_p, _i, _i, _i, _p, _p, _p, _p, _p, _p, _p]
        L.qg_x_half.argtypes = [_p, _i, _p, _i, _i, _p, _p, _p]
        L.qg_x_half_guard.argtypes = [_p, _i, _p, _i, _i, _i, _p, _p, _p]
        L.qgemm_moe_grouped.argtypes = [_i, _p, _i, _p, _p, _i, _p, _i, _p, _p, _i, _i, _i, _i, _i, _p]
        L.qg_swiglu.argtypes = [_p, _i, _i, _p, _i, _p, _p]
        L.qg_moe_combine.argtypes = [_p, _i, _p, _p, _p, _i, _i, _i, _i, _p]
        L.qg_moe_ffn_workspace.restype = _sz
        L.qg_moe_ffn_workspace.argtypes = [_i, _i, _i, _i, _i]
        L.qg_moe_ffn.argtypes = [_i, _p, _p, _i, _i, _i, _i, _p, _i, _i, _p, _p, _p, _p, _p, _i, _i, _p, _sz, _p]
        L.qg_moe_ffn_noalloc.argtypes = [_i, _p, _p, _i, _i, _i, _i, _p, _i, _i, _p, _p, _p, _p, _p, _i, _i, _p]
        _i64 = C.c_int64
        L.qg_kv8_write.argtypes = [_p, _p, _p, _i64, _i64, _p, _i64, _i64, _i, _p]
        L.qg_kv8_read.argtypes = [_p, _p, _p, _i64, _i64, _p, _i64, _i64, _i, _p]
        L.qg_attn_kv8_workspace.argtypes = [_p, _p, _i]
        L.qg_attn_kv8.argtypes = [_p, _p, _p, _i64, _i64, _p, _i64, _i64, _i, _i, C.c_float, _i, _i, _p, _sz, _p]
        L.qgemm_w8a8_workspace.argtypes = [_i, _i, _i]
        L.qgemm_w8a8.argtypes = [_p, _p, _p, _i, _p, _i, _i, _i, _i, _p, _sz, _p]
        _d = C.c_double
        L.qg_rope_freqs.argtypes = [_i, _i, _d, _d, _d, _d, _d, _p, _p]
        L.qg_rope.argtypes = [_p, _p, _p, _i64, _i64, _p, _i64, _i64, _i, _i, _i, _i, _p]
        L.qg_kv8_write_rope.argtypes = [_p, _p, _p, _p, _p, _i64, _i64, _p, _i64, _i64, _p, _i, _p, _i64, _i64, _p, _i64,
                                        _i64, _i, _i, _p]
        L.qg_tree_plan.argtypes = [_p, _p, _p, _i, _p, _i, _p]
        L.qg_attn_kv8_tree.argtypes = [_p, _p, _p, _i, _p, _p, _i64, _i64, _p, _i64, _i64, _i, _i, C.c_float, _i, _p, _sz, _p]
        L.qg_draft_verify_workspace.argtypes = [_p, _i]
        L.qg_draft_verify.argtypes = [_p, _p, _p, _p, _i64, _p, _i64, _i, _i, _p, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p]
        for name in ("qg_attn_kv8_workspace", "qgemm_w8a8_workspace", "qg_draft_verify_workspace"):
            getattr(L, name).restype = _sz
        for name in SYMBOLS:
            if name not in ("qg_strerror", "qg_abi_version") and not name.endswith("_workspace"):
                getattr(L, name).restype = _i
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().qg_strerror(int(status)).decode()


def abi_version() -> int:
    return lib().qg_abi_version()


# ---- marshalling helpers ------------------------------------------------------------------------
def _ptr(t):
    """Device (or host) address of a torch tensor / numpy array / int; None for None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


_XT = {}


def _xt(t) -> int:
    if not _XT:
        import torch
        _XT.update({torch.float32: QG_X_F32, torch.float16: QG_X_F16, torch.bfloat16: QG_X_BF16})
    return _XT[t.dtype]


_raw_stream = None


def _stream(stream):
    if stream is None:
        # the current device's current stream as an address; torch.cuda.current_stream() builds an object
        # around it first, 1 us that a launch of a few does not have, but a torch without the two calls has that
        global _raw_stream
        if _raw_stream is None:
            import torch
            torch.cuda.current_stream()  # initialises the device
            get, device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
            if get and device:
                _raw_stream = lambda: get(device())  # noqa: E731
            else:
                _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
        return _raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != QG_OK:
        raise QGError(status, where)


def _mode(mode):
    return MODE[mode] if isinstance(mode, str) else int(mode)


# ---- dense matmuls ------------------------------------------------------------------------------
def qgemm_q4(codes, scales, X, Y, N, K, T, mode="exact", xt=None, stream=None):
    _check(lib().qgemm_q4(_ptr(codes), _ptr(scales), _ptr(X), _xt(X) if xt is None else xt, _ptr(Y), N, K, T,
                          _mode(mode), _stream(stream)), "qgemm_q4")


def qgemm_q4a(codes, scales, offsets, group, X, Y, N, K, T, mode="exact", xt=None, stream=None):
    _check(lib().qgemm_q4a(_ptr(codes), _ptr(scales), _ptr(offsets), group, _ptr(X), _xt(X) if xt is None else xt,
                           _ptr(Y), N, K, T, _mode(mode), _stream(stream)), "qgemm_q4a")


def qgemm_q8(codes, scales, X, Y, N, K, T, mode="exact", xt=None, stream=None):
    _check(lib().qgemm_q8(_ptr(codes), _ptr(scales), _ptr(X), _xt(X) if xt is None else xt, _ptr(Y), N, K, T,
                          _mode(mode), _stream(stream)), "qgemm_q8")


def qgemm_q8a(codes, scales, offsets, X, Y, N, K, T, mode="exact", xt=None, stream=None):
    _check(lib().qgemm_q8a(_ptr(codes), _ptr(scales), _ptr(offsets), _ptr(X), _xt(X) if xt is None else xt,
                           _ptr(Y), N, K, T, _mode(mode), _stream(stream)), "qgemm_q8a")


def qgemv_q4(codes, scales, X, Y, N, K, T, xt=None, stream=None):
    _check(lib().qgemv_q4(_ptr(codes), _ptr(scales), _ptr(X), _xt(X) if xt is None else xt, _ptr(Y), N, K, T,
                          _stream(stream)), "qgemv_q4")


def qgemv_q4a(codes, scales, offsets, group, X, Y, N, K, T, xt=None, stream=None):
    _check(lib().qgemv_q4a(_ptr(codes), _ptr(scales), _ptr(offsets), group, _ptr(X), _xt(X) if xt is None else xt,
                           _ptr(Y), N, K, T, _stream(stream)), "qgemv_q4a")


def qgemv_q8(codes, scales, X, Y, N, K, T, xt=None, stream=None):
    _check(lib().qgemv_q8(_ptr(codes), _ptr(scales), _ptr(X), _xt(X) if xt is None else xt, _ptr(Y), N, K, T,
                          _stream(stream)), "qgemv_q8")


def qgemm_q8a16(codes, scales, offsets, X, Y, N, K, T, mode="exact", xt=None, stream=None):
    _check(lib().qgemm_q8a16(_ptr(codes), _ptr(scales), _ptr(offsets), _ptr(X), _xt(X) if xt is None else xt,
                             _ptr(Y), N, K, T, _mode(mode), _stream(stream)), "qgemm_q8a16")


def qgemv_q8a16(codes, scales, offsets, X, Y, N, K, T, xt=None, stream=None):
    _check(lib().qgemv_q8a16(_ptr(codes), _ptr(scales), _ptr(offsets), _ptr(X), _xt(X) if xt is None else xt,
                             _ptr(Y), N, K, T, _stream(stream)), "qgemv_q8a16")


def qgemv_q8a(codes, scales, offsets, X, Y, N, K, T, xt=None, stream=None):
    _check(lib().qgemv_q8a(_ptr(codes), _ptr(scales), _ptr(offsets), _ptr(X), _xt(X) if xt is None else xt,
                           _ptr(Y), N, K, T, _stream(stream)), "qgemv_q8a")


def qgemm(fmt, codes, scales, offsets, group, X, Y, N, K, T, mode="exact", stream=None):
    """Dispatch by format name: 'q4' | 'q4a' | 'q8' | 'q8a' | 'q8a16'."""
    if fmt == "q8a16":
        return qgemm_q8a16(codes, scales, offsets, X, Y, N, K, T, mode, stream=stream)
    if fmt == "q4":
        return qgemm_q4(codes, scales, X, Y, N, K, T, mode, stream=stream)
    if fmt == "q4a":
        return qgemm_q4a(codes, scales, offsets, group, X, Y, N, K, T, mode, stream=stream)
    if fmt == "q8a":
        return qgemm_q8a(codes, scales, offsets, X, Y, N, K, T, mode, stream=stream)
    return qgemm_q8(codes, scales, X, Y, N, K, T, mode, stream=stream)


def qgemv(fmt, codes, scales, offsets, group, X, Y, N, K, T, stream=None):
    if fmt == "q8a16":
        return qgemv_q8a16(codes, scales, offsets, X, Y, N, K, T, stream=stream)
    if fmt == "q4":
        return qgemv_q4(codes, scales, X, Y, N, K, T, stream=stream)
    if fmt == "q4a":
        return qgemv_q4a(codes, scales, offsets, group, X, Y, N, K, T, stream=stream)
    if fmt == "q8a":
        return qgemv_q8a(codes, scales, offsets, X, Y, N, K, T, stream=stream)
    return qgemv_q8(codes, scales, X, Y, N, K, T, stream=stream)


def qg_dequant_dump(fmt, codes, scales, offsets, group, N, K, n0, k0, rows, cols, staged, out, stream=None):
    _check(lib().qg_dequant_dump(FMT[fmt] if isinstance(fmt, str) else fmt, _ptr(codes), _ptr(scales),
                                 _ptr(offsets), group, N, K, n0, k0, rows, cols, staged, _ptr(out),
                                 _stream(stream)), "qg_dequant_dump")


class QgJob(C.Structure):
    """qg_job of qgemm.h: one weight matrix of a batched call."""
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("offsets", C.c_void_p), ("Y", C.c_void_p),
                ("N", C.c_int)]


def job_array(jobs):
    """Host array of qg_job from (codes, scales, offsets-or-None, Y, N) tuples of device tensors."""
    arr = (QgJob * len(jobs))()
    for i, (c, s, o, y, n) in enumerate(jobs):
        arr[i] = QgJob(_ptr(c), _ptr(s), _ptr(o), _ptr(y), int(n))
    return arr


def qgemm_batch(fmt, group, jobs, X, K, T, mode="exact", xt=None, stream=None):
    """jobs: list of (codes, scales, offsets-or-None, Y, N) sharing X [T][K]."""
    arr = job_array(jobs)
    _check(lib().qgemm_batch(FMT[fmt] if isinstance(fmt, str) else fmt, group, C.cast(arr, C.c_void_p), len(jobs),
                             _ptr(X), _xt(X) if xt is None else xt, K, T, _mode(mode), _stream(stream)), "qgemm_batch")


QG_GGUF_Q4_0, QG_GGUF_Q4_1, QG_GGUF_Q5_0, QG_GGUF_Q5_1, QG_GGUF_Q8_0, QG_GGUF_Q4_K, QG_GGUF_Q5_K = 2, 3, 6, 7, 8, 12, 13
QG_GGUF_Q2_K, QG_GGUF_Q3_K, QG_GGUF_Q6_K = 10, 11, 14
GGUF = {"q4_0": QG_GGUF_Q4_0, "q4_1": QG_GGUF_Q4_1, "q5_0": QG_GGUF_Q5_0, "q5_1": QG_GGUF_Q5_1,
        "q8_0": QG_GGUF_Q8_0, "q4_k": QG_GGUF_Q4_K, "q5_k": QG_GGUF_Q5_K, "q2_k": QG_GGUF_Q2_K,
        "q3_k": QG_GGUF_Q3_K, "q6_k": QG_GGUF_Q6_K}


def qg_repack_gguf(gtype, src, N, K, codes, scales, stream=None):
    """GGUF Q4_0 / Q8_0 blocks (device uint8 tensor) -> this library's codes and scales (device)."""
    _check(lib().qg_repack_gguf(GGUF[gtype] if isinstance(gtype, str) else gtype, _ptr(src), N, K, _ptr(codes),
                                _ptr(scales), _stream(stream)), "qg_repack_gguf")


def qg_repack_gguf_q8a(gtype, src, N, K, codes, scales, offsets, stream=None):
    """GGUF Q4_1 / Q5_0 / Q5_1 / Q4_K / Q5_K blocks (device uint8 tensor) -> Q8A codes (int8 [N*K]), f32
    scales and f32 offsets ([N*K/32]), all device tensors."""
    _check(lib().qg_repack_gguf_q8a(GGUF[gtype] if isinstance(gtype, str) else gtype, _ptr(src), N, K,
                                    _ptr(codes), _ptr(scales), _ptr(offsets), _stream(stream)),
           "qg_repack_gguf_q8a")


def qg_repack_q8f(blob, N, K, has_col, scales, col=None, stream=None):
    """q8_2f (has_col) / q8_row tensor blob (device uint8: int8 codes [N][K], f16 row scales, f16 column
    field) -> f32 Q8 block scales [N*K/32] and the f32 column field [K]; the blob is the Q8 codes."""
    _check(lib().qg_repack_q8f(_ptr(blob), N, K, int(bool(has_col)), _ptr(scales), _ptr(col), _stream(stream)),
           "qg_repack_q8f")


def qg_col_scale(X, T, K, col, Xs, stream=None):
    """Xs = X * col[k] (types from the tensors' dtypes)."""
    _check(lib().qg_col_scale(_ptr(X), _xt(X), T, K, _ptr(col), _ptr(Xs), _xt(Xs), _stream(stream)), "qg_col_scale")


# ---- convolution ------------------------------------------------------------------------------------
CONV_NORM = {None: 0, "none": 0, "group": 1, "layer": 2}


def conv_out_size(H, W, ksize, stride):
    """(oh, ow) of qg_conv2d: pad = ksize // 2."""
    pad = ksize // 2
    return (H + 2 * pad - ksize) // stride + 1, (W + 2 * pad - ksize) // stride + 1


def qg_conv_stats(X, npix, cin, groups, eps, stats, stream=None):
    """(mean, rstd) f32 pairs of the image X [npix][cin] into stats (device): per group of
    cin / groups channels (groups > 0) or per pixel (groups == 0)."""
    _check(lib().qg_conv_stats(_ptr(X), npix, cin, groups, float(eps), _ptr(stats), _stream(stream)),
           "qg_conv_stats")


def qg_conv2d(fmt, codes, scales, X, H, W, cin, ksize, stride, n_out, Y, norm=None, groups=0, stats=None,
              gamma_beta=None, silu=False, mode="exact", stream=None):
    """Implicit-GEMM convolution of the image X [H][W][cin] (f32) with the quantized weight matrix
    [n_out][ksize * ksize * cin] into Y [oh * ow][n_out] (device tensors)."""
    _check(lib().qg_conv2d(FMT[fmt] if isinstance(fmt, str) else fmt, _ptr(codes), _ptr(scales), _ptr(X), H, W, cin,
                           ksize, stride, n_out, CONV_NORM[norm] if not isinstance(norm, int) else norm, groups,
                           _ptr(stats), _ptr(gamma_beta), int(bool(silu)), _ptr(Y), _mode(mode), _stream(stream)),
           "qg_conv2d")


# ---- MoE ----------------------------------------------------------------------------------------
def qg_moe_plan_host(logits: np.ndarray, T: int, E: int, k: int) -> dict:
    """Routing plan on the host (numpy in, numpy out)."""
    lg = np.ascontiguousarray(logits, dtype=np.float32)
    seg_off = np.empty(E + 1, np.int32)
    row_src = np.empty(T * k, np.int32)
    slot_row = np.empty(T * k, np.int32)
    slot_w = np.empty(T * k, np.float32)
    slot_e = np.empty(T * k, np.int32)
    _check(lib().qg_moe_plan_host(_ptr(lg), T, E, k, _ptr(seg_off), _ptr(row_src), _ptr(slot_row), _ptr(slot_w),
                                  _ptr(slot_e)), "qg_moe_plan_host")
    return {"seg_off": seg_off, "row_src": row_src, "slot_row": slot_row, "slot_w": slot_w, "slot_expert": slot_e}


def qg_moe_plan(logits, T, E, k, seg_off, row_src, slot_row, slot_w, slot_expert=None, status=None, stream=None):
    """Routing plan on the device: every argument a device tensor (int32 / float32) or None."""
    _check(lib().qg_moe_plan(_ptr(logits), T, E, k, _ptr(seg_off), _ptr(row_src), _ptr(slot_row), _ptr(slot_w),
                             _ptr(slot_expert), _ptr(status), _stream(stream)), "qg_moe_plan")


def qg_x_half(X, x_rows, row_src, R, K, Xh, rs, stream=None):
    _check(lib().qg_x_half(_ptr(X), x_rows, _ptr(row_src), R, K, _ptr(Xh), _ptr(rs), _stream(stream)), "qg_x_half")


def qg_x_half_guard(X, x_rows, row_src, R, K, shift, Xh, rs=None, stream=None):
    _check(lib().qg_x_half_guard(_ptr(X), x_rows, _ptr(row_src), R, K, int(shift), _ptr(Xh), _ptr(rs), _stream(stream)),
           "qg_x_half_guard")


def qgemm_moe_grouped(fmt, experts, group, seg_off, row_src, x_rows, X, rs, Y, N, K, R, E, mode="exact", xt=None,
                      stream=None):
    _check(lib().qgemm_moe_grouped(FMT[fmt] if isinstance(fmt, str) else fmt, _ptr(experts), group, _ptr(seg_off),
                                   _ptr(row_src), x_rows, _ptr(X), _xt(X) if xt is None else xt, _ptr(rs), _ptr(Y),
                                   N, K, R, E, _mode(mode), _stream(stream)), "qgemm_moe_grouped")


def qg_swiglu(GU, R, I, A, at, rs=None, stream=None):
    _check(lib().qg_swiglu(_ptr(GU), R, I, _ptr(A), at, _ptr(rs), _stream(stream)), "qg_swiglu")


def qg_moe_combine(O, R, slot_row, slot_w, Y, H, T, k, accumulate=0, stream=None):
    _check(lib().qg_moe_combine(_ptr(O), R, _ptr(slot_row), _ptr(slot_w), _ptr(Y), H, T, k, int(accumulate),
                                _stream(stream)), "qg_moe_combine")


def qg_moe_ffn_workspace(H, I, T, k, mode="exact") -> int:
    return int(lib().qg_moe_ffn_workspace(H, I, T, k, _mode(mode)))


def qg_moe_ffn(fmt, gate_up, down, group, E, H, I, X, T, k, seg_off, row_src, slot_row, slot_w, Y, accumulate,
               mode, workspace, ws_bytes, stream=None):
    _check(lib().qg_moe_ffn(FMT[fmt] if isinstance(fmt, str) else fmt, _ptr(gate_up), _ptr(down), group, E, H, I,
                            _ptr(X), T, k, _ptr(seg_off), _ptr(row_src), _ptr(slot_row), _ptr(slot_w), _ptr(Y),
                            int(accumulate), _mode(mode), _ptr(workspace), int(ws_bytes), _stream(stream)),
           "qg_moe_ffn")


def qg_moe_ffn_noalloc(fmt, gate_up, down, group, E, H, I, X, T, k, seg_off, row_src, slot_row, slot_w, Y,
                       accumulate, mode, stream=None):
    _check(lib().qg_moe_ffn_noalloc(FMT[fmt] if isinstance(fmt, str) else fmt, _ptr(gate_up), _ptr(down), group, E, H,
                                    I, _ptr(X), T, k, _ptr(seg_off), _ptr(row_src), _ptr(slot_row), _ptr(slot_w),
                                    _ptr(Y), int(accumulate), _mode(mode), _stream(stream)),
           "qg_moe_ffn_noalloc")


# ---- 8-bit serving operators ------------------------------------------------------------------------
class QgKv8Cache(C.Structure):
    """qg_kv8_cache of qgemm.h."""
    _fields_ = [("k_codes", C.c_void_p), ("k_scales", C.c_void_p), ("v_codes", C.c_void_p), ("v_scales", C.c_void_p),
                ("pages", C.c_int), ("page", C.c_int), ("heads", C.c_int), ("dim", C.c_int)]


class QgKv8Seqs(C.Structure):
    """qg_kv8_seqs of qgemm.h."""
    _fields_ = [("table", C.c_void_p), ("rows", C.c_void_p), ("kv_len", C.c_void_p), ("seqs", C.c_int),
                ("width", C.c_int), ("T", C.c_int), ("max_new", C.c_int), ("max_kv", C.c_int)]


class _Desc:
    """A C descriptor and the tensors that its addresses point into."""
    __slots__ = ("struct", "ptr", "keep", "T", "heads", "dim")

    def __init__(self, struct, keep, T=0, heads=0, dim=0):
        self.struct, self.keep, self.T, self.heads, self.dim = struct, keep, T, heads, dim
        self.ptr = C.addressof(struct)


def _expect(ok: bool, where: str, status: int = QG_EINVAL):
    if not ok:
        raise QGError(status, where)


def kv8_pages(pages, page, heads, dim, device="cuda"):
    """Empty cache tensors (k_codes, k_scales, v_codes, v_scales) for kv8_cache."""
    import torch
    n = pages * heads * (page // 16)
    return (torch.empty(n * 16 * dim, dtype=torch.int8, device=device), torch.empty(n, device=device),
            torch.empty(n * 16 * dim, dtype=torch.int8, device=device), torch.empty(n, device=device))


def kv8_cache(k_codes, k_scales, v_codes, v_scales, page, heads, dim):
    """Descriptor of an 8-bit key/value cache over contiguous device tensors (int8 codes, f32 scales; layouts
    in qgemm.h); the number of pages follows from their sizes.  Keep it as long as the cache."""
    import torch
    t = (k_codes, k_scales, v_codes, v_scales)
    _expect(page >= 16 and page % 16 == 0 and heads >= 1 and dim >= 1, "kv8_cache", QG_ESHAPE)
    per = heads * (page // 16)
    pages = k_scales.numel() // per
    for x, dtype, n in zip(t, (torch.int8, torch.float32) * 2, (per * 16 * dim, per) * 2):
        _expect(x.dtype == dtype and x.is_contiguous() and x.device == k_codes.device, "kv8_cache")
        _expect(x.numel() == pages * n, "kv8_cache", QG_ESHAPE)
    return _Desc(QgKv8Cache(*(x.data_ptr() for x in t), pages, page, heads, dim), t, heads=heads, dim=dim)


def kv8_seqs(table, rows, kv_len, T, max_new, max_kv):
    """Descriptor of a batch of sequences: int32 device tensors table [seqs][width], rows [seqs + 1] and
    kv_len [seqs], and the host's bounds (qg_kv8_seqs in qgemm.h).  The tensors' contents may change later
    within the bounds."""
    import torch
    t = (table, rows, kv_len)
    for x in t:
        _expect(x.dtype == torch.int32 and x.is_contiguous() and x.device == table.device, "kv8_seqs")
    _expect(table.dim() == 2 and rows.numel() == table.shape[0] + 1 and kv_len.numel() == table.shape[0], "kv8_seqs",
            QG_ESHAPE)
    return _Desc(QgKv8Seqs(*(x.data_ptr() for x in t), table.shape[0], table.shape[1], T, max_new, max_kv), t, T=T)


_entries = {}
_int8 = _int32 = None


def _entry(name):
    """An entry point, looked up once: these calls are made a few at a time for microseconds of work."""
    import torch
    global _int8, _int32
    _int8, _int32 = torch.int8, torch.int32
    _XT.update({torch.float32: QG_X_F32, torch.float16: QG_X_F16, torch.bfloat16: QG_X_BF16})
    _entries[name] = call = getattr(lib(), name)
    return call


def qg_kv8_write(cache, seqs, k, v, stream=None):
    """Codes k, v [T][heads][dim] (any row and head strides) into the cache as their sequences' last tokens."""
    _kv8("qg_kv8_write", cache, seqs, k, v, stream)


def qg_kv8_read(cache, seqs, k_out, v_out, stream=None):
    """Reads the sequences' last tokens back into k_out, v_out [T][heads][dim]."""
    _kv8("qg_kv8_read", cache, seqs, k_out, v_out, stream)


def _kv8(where, cache, seqs, k, v, stream):
    call = _entries.get(where) or _entry(where)
    xt, shape = k.dtype, (seqs.T, cache.heads, cache.dim)
    if xt is not v.dtype or xt not in _XT:
        raise QGError(QG_EINVAL, where)
    if k.shape != shape or v.shape != shape:
        raise QGError(QG_ESHAPE, where)
    k_row, k_head, k_one = k.stride()
    v_row, v_head, v_one = v.stride()
    if k_one != 1 or v_one != 1:
        raise QGError(QG_EALIGN, where)
    status = call(cache.ptr, seqs.ptr, k.data_ptr(), k_row, k_head, v.data_ptr(), v_row, v_head, _XT[xt],
                  _stream(stream))
    if status:
        raise QGError(status, where)


def qg_attn_kv8_workspace(cache, seqs, q_heads) -> int:
    return int(lib().qg_attn_kv8_workspace(cache.ptr, seqs.ptr, q_heads))


def qg_attn_kv8(cache, seqs, q, o, q_heads, scale, causal=True, window=0, workspace=None, stream=None):
    """Attention of q [T][q_heads][dim] over the cache into o (same shape and type); workspace: a device
    tensor of at least qg_attn_kv8_workspace bytes."""
    call = _entries.get("qg_attn_kv8") or _entry("qg_attn_kv8")
    xt, shape = q.dtype, (seqs.T, q_heads, cache.dim)
    if xt is not o.dtype or xt not in _XT:
        raise QGError(QG_EINVAL, "qg_attn_kv8")
    if q.shape != shape or o.shape != shape:
        raise QGError(QG_ESHAPE, "qg_attn_kv8")
    q_row, q_head, q_one = q.stride()
    o_row, o_head, o_one = o.stride()
    if q_one != 1 or o_one != 1:
        raise QGError(QG_EALIGN, "qg_attn_kv8")
    wp, size = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    status = call(cache.ptr, seqs.ptr, q.data_ptr(), q_row, q_head, o.data_ptr(), o_row, o_head, _XT[xt], q_heads, scale,
                  1 if causal else 0, window, wp, size, _stream(stream))
    if status:
        raise QGError(status, "qg_attn_kv8")


def qgemm_w8a8_workspace(N, K, T) -> int:
    return int(lib().qgemm_w8a8_workspace(N, K, T))


def qgemm_w8a8(w_codes, w_scales, X, Y, N, K, T, workspace=None, stream=None):
    """Y [T][N] = X [T][K] times int8 weights [N][K] with a scale an output channel, X coded in 8 bits with a
    scale a token on the way; types from the tensors' dtypes; workspace: a device tensor of at least
    qgemm_w8a8_workspace bytes."""
    call = _entries.get("qgemm_w8a8") or _entry("qgemm_w8a8")
    xt, yt = _XT.get(X.dtype), _XT.get(Y.dtype)
    if xt is None or yt is None or w_codes.dtype is not _int8 or _XT.get(w_scales.dtype) != QG_X_F32:
        raise QGError(QG_EINVAL, "qgemm_w8a8")
    if X.numel() < T * K or Y.numel() < T * N or w_codes.numel() < N * K or w_scales.numel() < N:
        raise QGError(QG_ESHAPE, "qgemm_w8a8")
    if not (X.is_contiguous() and Y.is_contiguous() and w_codes.is_contiguous() and w_scales.is_contiguous()):
        raise QGError(QG_EALIGN, "qgemm_w8a8")
    wp, size = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    status = call(w_codes.data_ptr(), w_scales.data_ptr(), X.data_ptr(), xt, Y.data_ptr(), yt, N, K, T, wp, size,
                  _stream(stream))
    if status:
        raise QGError(status, "qgemm_w8a8")


# ---- drafted tokens over the 8-bit cache ------------------------------------------------------------
ROPE = {None: 0, "plain": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}


class QgRotary(C.Structure):
    """qg_rotary of qgemm.h."""
    _fields_ = [("freqs", C.c_void_p), ("rot", C.c_int), ("interleaved", C.c_int), ("mscale", C.c_float)]


def rope_freqs(rot, base=10000.0, scaling=None, factor=1.0, context=0.0, low=1.0, high=32.0):
    """Frequencies of rotary positions (numpy f64 [rot / 2], radians a position) and the factor mscale; scaling: None,
    "linear", "ntk", "bands" or "yarn" (qg_rope_freqs in qgemm.h)."""
    freqs, mscale = np.empty(max(0, rot // 2), np.float64), C.c_float()
    kind = ROPE.get(scaling, scaling if isinstance(scaling, int) else -1)
    _check(lib().qg_rope_freqs(kind, rot, base, factor, context, low, high, freqs.ctypes.data, C.addressof(mscale)),
           "qg_rope_freqs")
    return freqs, mscale.value


def rotary(freqs, interleaved=False, mscale=1.0):
    """Descriptor of rotary positions over a contiguous f64 device tensor of rot / 2 frequencies (None: nothing is turned).
    Keep it as long as it is used."""
    import torch
    if freqs is None:
        return _Desc(QgRotary(None, 0, 0, 1.0), ())
    _expect(freqs.dtype == torch.float64 and freqs.dim() == 1 and freqs.is_contiguous(), "rotary")
    return _Desc(QgRotary(freqs.data_ptr(), 2 * freqs.numel(), int(bool(interleaved)), mscale), (freqs,))


def _int(where, n, x):
    """A contiguous int32 tensor of at least n values."""
    if x.dtype is not _int32:
        raise QGError(QG_EINVAL, where)
    if x.numel() < n:
        raise QGError(QG_ESHAPE, where)
    if not x.is_contiguous():
        raise QGError(QG_EALIGN, where)


def _float(where, n, x):
    """A contiguous f32 tensor of at least n values."""
    if _XT.get(x.dtype) != QG_X_F32:
        raise QGError(QG_EINVAL, where)
    if x.numel() < n:
        raise QGError(QG_ESHAPE, where)
    if not x.is_contiguous():
        raise QGError(QG_EALIGN, where)


def qg_rope(rot, pos, x, y, stream=None):
    """x [T][heads][dim] (any row and head strides) at positions pos [T] turned into y, which may be x."""
    call = _entries.get("qg_rope") or _entry("qg_rope")
    xt, shape = _XT.get(x.dtype), x.shape
    if x.dtype is not y.dtype or xt is None:
        raise QGError(QG_EINVAL, "qg_rope")
    if len(shape) != 3 or y.shape != shape:
        raise QGError(QG_ESHAPE, "qg_rope")
    T, heads, dim = shape
    _int("qg_rope", T, pos)
    x_row, x_head, x_one = x.stride()
    y_row, y_head, y_one = y.stride()
    if x_one != 1 or y_one != 1:
        raise QGError(QG_EALIGN, "qg_rope")
    status = call(rot.ptr, pos.data_ptr(), x.data_ptr(), x_row, x_head, y.data_ptr(), y_row, y_head, xt, T, heads, dim,
                  _stream(stream))
    if status:
        raise QGError(status, "qg_rope")


def qg_kv8_write_rope(cache, seqs, rot, k, v, q=None, q_out=None, pos=None, src=None, stream=None):
    """qg_kv8_write with K turned on the way; q [T][q_heads][dim] is turned into q_out beside it.  pos [T]: positions other
    than the rows' places; src [T]: row r is row src[r] of k and v, which then have any number of rows."""
    where = "qg_kv8_write_rope"
    call = _entries.get(where) or _entry(where)
    xt, shape, dim, T = _XT.get(k.dtype), k.shape, cache.dim, seqs.T
    if k.dtype is not v.dtype or xt is None:
        raise QGError(QG_EINVAL, where)
    if len(shape) != 3 or shape[1] != cache.heads or shape[2] != dim or v.shape != shape or (src is None and shape[0] != T):
        raise QGError(QG_ESHAPE, where)
    if pos is not None:
        _int(where, T, pos)
    if src is not None:
        _int(where, T, src)
    k_row, k_head, k_one = k.stride()
    v_row, v_head, v_one = v.stride()
    if k_one != 1 or v_one != 1:
        raise QGError(QG_EALIGN, where)
    qs = (None, 0, 0, None, 0, 0, 0)
    if q is not None:
        if q_out is None or q.dtype is not k.dtype or q_out.dtype is not k.dtype:
            raise QGError(QG_EINVAL, where)
        turned = q.shape
        if len(turned) != 3 or q_out.shape != turned or turned[0] != T or turned[2] != dim or turned[1] == 0:
            raise QGError(QG_ESHAPE, where)
        q_row, q_head, q_one = q.stride()
        o_row, o_head, o_one = q_out.stride()
        if q_one != 1 or o_one != 1:
            raise QGError(QG_EALIGN, where)
        qs = (q.data_ptr(), q_row, q_head, q_out.data_ptr(), o_row, o_head, turned[1])
    status = call(cache.ptr, seqs.ptr, rot.ptr, None if pos is None else pos.data_ptr(), k.data_ptr(), k_row, k_head,
                  v.data_ptr(), v_row, v_head, None if src is None else src.data_ptr(), shape[0], *qs, xt, _stream(stream))
    if status:
        raise QGError(status, where)


def _masks(where, seqs, mask):
    """Words of a mask [T][words]."""
    if mask.dtype is not _int32:
        raise QGError(QG_EINVAL, where)
    shape = mask.shape
    if len(shape) != 2 or shape[0] < seqs.T:
        raise QGError(QG_ESHAPE, where)
    if not mask.is_contiguous():
        raise QGError(QG_EALIGN, where)
    return shape[1]


def qg_tree_plan(seqs, parents, mask, pos, window=0, stream=None):
    """Masks (int32 [T][words]) and positions (int32 [T]) of a batch of trees from their parents [T]."""
    call = _entries.get("qg_tree_plan") or _entry("qg_tree_plan")
    words = _masks("qg_tree_plan", seqs, mask)
    _int("qg_tree_plan", seqs.T, parents)
    _int("qg_tree_plan", seqs.T, pos)
    status = call(seqs.ptr, parents.data_ptr(), mask.data_ptr(), words, pos.data_ptr(), window, _stream(stream))
    if status:
        raise QGError(status, "qg_tree_plan")


def qg_attn_kv8_tree(cache, seqs, mask, q, o, q_heads, scale, window=0, pos=None, workspace=None, stream=None):
    """Attention of q [T][q_heads][dim] over the cache into o, the batch's rows seeing each other by mask (int32
    [T][words]); pos [T] is read with a window alone.  Workspace as for qg_attn_kv8."""
    where = "qg_attn_kv8_tree"
    call = _entries.get(where) or _entry(where)
    xt, shape = _XT.get(q.dtype), (seqs.T, q_heads, cache.dim)
    if q.dtype is not o.dtype or xt is None:
        raise QGError(QG_EINVAL, where)
    if q.shape != shape or o.shape != shape:
        raise QGError(QG_ESHAPE, where)
    words = _masks(where, seqs, mask)
    if pos is not None:
        _int(where, shape[0], pos)
    q_row, q_head, q_one = q.stride()
    o_row, o_head, o_one = o.stride()
    if q_one != 1 or o_one != 1:
        raise QGError(QG_EALIGN, where)
    wp, size = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    status = call(cache.ptr, seqs.ptr, mask.data_ptr(), words, None if pos is None else pos.data_ptr(), q.data_ptr(), q_row,
                  q_head, o.data_ptr(), o_row, o_head, xt, q_heads, scale, window, wp, size, _stream(stream))
    if status:
        raise QGError(status, where)


def qg_draft_verify_workspace(seqs, vocab) -> int:
    return int(lib().qg_draft_verify_workspace(seqs.ptr, vocab))


def qg_draft_verify(seqs, tokens, target, accepted, next, rows_out, path, kv_out, sample=None, temps=None, parents=None,
                    draft=None, accept=None, workspace=None, stream=None):
    """Which drafted tokens [T] stay by the logits target [T][vocab], and what follows them: accepted, next and kv_out
    [seqs], rows_out [seqs + 1], path [T] (int32).  draft: the logits that the tokens were drawn from, with accept [T]; None:
    they were chosen.  sample [T] (f32; None: the largest logit throughout), temps [seqs] (f32; None: 1), parents [T] (None:
    chains); workspace: a device tensor of at least qg_draft_verify_workspace bytes."""
    where = "qg_draft_verify"
    call = _entries.get(where) or _entry(where)
    xt, shape, T, n = _XT.get(target.dtype), target.shape, seqs.T, seqs.struct.seqs
    if xt is None or (draft is not None and draft.dtype is not target.dtype):
        raise QGError(QG_EINVAL, where)
    if len(shape) != 2 or shape[0] < T or (draft is not None and draft.shape != shape):
        raise QGError(QG_ESHAPE, where)
    t_row, one = target.stride()
    d_row, d_one = (0, 1) if draft is None else draft.stride()
    if one != 1 or d_one != 1:
        raise QGError(QG_EALIGN, where)
    for x in (tokens, path) if parents is None else (tokens, path, parents):
        _int(where, T, x)
    for x in (accepted, next, kv_out):
        _int(where, n, x)
    _int(where, n + 1, rows_out)
    for x, least in ((sample, T), (accept, T), (temps, n)):
        if x is not None:
            _float(where, least, x)
    wp, size = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    status = call(seqs.ptr, None if parents is None else parents.data_ptr(), tokens.data_ptr(), target.data_ptr(), t_row,
                  None if draft is None else draft.data_ptr(), d_row, xt, shape[1],
                  None if temps is None else temps.data_ptr(), None if accept is None else accept.data_ptr(),
                  None if sample is None else sample.data_ptr(), accepted.data_ptr(), next.data_ptr(), rows_out.data_ptr(),
                  path.data_ptr(), kv_out.data_ptr(), wp, size, _stream(stream))
    if status:
        raise QGError(status, where)


# ---- host layout helpers (byte movement only) ----------------------------------------------------
def pack_q4(nibbles: np.ndarray) -> np.ndarray:
    """Nibble matrix [N][K] (values 0..15, element order) -> packed Q4 codes uint8 [N][K/2] in the
    block layout: byte j of block b holds element 32b+j (low nibble) and 32b+16+j (high nibble)."""
    nb = np.asarray(nibbles, dtype=np.uint8)
    N, K = nb.shape
    if K % 32:
        raise ValueError("K must be a multiple of 32")
    if nb.max(initial=0) > 15:
        raise ValueError("nibbles must be in 0..15")
    b = nb.reshape(N, K // 32, 32)
    return (b[:, :, :16] | (b[:, :, 16:] << 4)).reshape(N, K // 2)


def unpack_q4(codes: np.ndarray, N: int, K: int) -> np.ndarray:
    """Inverse of pack_q4: packed codes -> nibble matrix [N][K]."""
    c = np.asarray(codes, dtype=np.uint8).reshape(N, K // 32, 16)
    return np.concatenate([c & 15, c >> 4], axis=2).reshape(N, K)


def expert_table(experts, device="cuda"):
    """Device array of qg_expert {codes, scales, offsets} (three 64-bit pointers each) for a list of
    (codes, scales, offsets-or-None) device tensors."""
    import torch
    rows = [[_ptr(c), _ptr(s), _ptr(o) if o is not None else 0] for (c, s, o) in experts]
    host = torch.tensor(np.array(rows, dtype=np.uint64).view(np.int64), dtype=torch.int64)
    return host.to(device)


def qg_repack_gguf_q8a16(gtype, src, N, K, codes, scales, offsets, stream=None):
    """GGUF Q6_K / Q3_K / Q2_K super-blocks (device uint8 tensor) -> Q8A16 codes (int8 [N*K]), f32 scales
    and f32 offsets ([N*K/16]; None for the offset-free Q6_K / Q3_K layout), all device tensors."""
    _check(lib().qg_repack_gguf_q8a16(GGUF[gtype] if isinstance(gtype, str) else gtype, _ptr(src), N, K,
                                      _ptr(codes), _ptr(scales), _ptr(offsets), _stream(stream)),
           "qg_repack_gguf_q8a16")
