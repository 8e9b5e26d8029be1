"""Thin ctypes binding of libqmm (include/qmm.h).

Argument marshalling only.  Every step of the computation runs in the CUDA
library.  The functions take torch tensors for device memory and use torch's
current CUDA stream.  Each one raises ``QmmError`` when the C entry point
returns a status other than QMM_OK.  There is no Python fallback: if
libqmm.so is missing, importing this module raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqmm.so")

QMM_OK, QMM_ERR_INVALID_ARG, QMM_ERR_UNSUPPORTED, QMM_ERR_OVERFLOW_BOUND = 0, 1, 2, 3
QMM_ERR_CUDA, QMM_ERR_TIMEOUT, QMM_ERR_BAD_EXPERT_ID, QMM_ERR_WORKSPACE, QMM_ERR_RANGE = 4, 5, 6, 7, 8
QMM_ERR_NO_PAGES = 9
QMM_U8, QMM_S8, QMM_S32, QMM_F32, QMM_BF16 = 1, 2, 3, 4, 5
DTYPES = {"u8": QMM_U8, "s8": QMM_S8, "s32": QMM_S32, "f32": QMM_F32, "bf16": QMM_BF16}
TORCH_OUT = {"s32": torch.int32, "f32": torch.float32, "s8": torch.int8, "u8": torch.uint8}

# exported symbols and their C signatures (restype, argtypes)
_c = ctypes
_vp, _i64, _i32, _sz = _c.c_void_p, _c.c_int64, _c.c_int32, _c.c_size_t
_szp = _c.POINTER(_c.c_size_t)


class QmmEpilogue(ctypes.Structure):
    _fields_ = [("out_type", _c.c_int), ("bias", _vp), ("s_x", _vp), ("s_x_stride", _i64),
                ("s_w", _vp), ("s_y", _c.c_float), ("zp_y", _i32)]


class QmmInt8Problem(ctypes.Structure):
    _fields_ = [("A", _vp), ("a_type", _c.c_int), ("M", _i64), ("K", _i64), ("lda", _i64), ("zA", _i32),
                ("packedB", _vp), ("col_sum", _vp), ("N", _i64), ("b_orig_type", _c.c_int), ("zB", _i32),
                ("ep", QmmEpilogue), ("out", _vp), ("ldo", _i64)]


class QmmQ4GemvProblem(ctypes.Structure):
    _fields_ = [("tiles", _vp), ("N", _i64), ("K", _i64), ("x", _vp), ("y", _vp)]


class QmmKvCache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("type", _c.c_int), ("n_pages", _i64),
                ("page_size", _i64), ("n_heads", _i64), ("head_dim", _i64), ("stride_page", _i64),
                ("stride_token", _i64), ("stride_head", _i64)]


class QmmNorm(ctypes.Structure):
    _fields_ = [("kind", _c.c_int), ("eps", _c.c_float), ("weight", _vp), ("bias", _vp)]


class QmmLoraSet(ctypes.Structure):
    _fields_ = [("A", _vp), ("a_stride_slot", _i64), ("a_stride_rank", _i64), ("B", _vp), ("b_stride_slot", _i64),
                ("b_stride_row", _i64), ("ranks", _vp), ("scales", _vp), ("n_adapters", _i64), ("max_rank", _i64),
                ("K", _i64), ("N", _i64)]


SIGNATURES = {
    "qmm_status_string": (_c.c_char_p, [_c.c_int]),
    "qmm_version": (_c.c_int, []),
    "qmm_pack_b_int8_size": (_c.c_int, [_i64, _i64, _szp]),
    "qmm_pack_b_int8": (_c.c_int, [_vp, _c.c_int, _i64, _i64, _i64, _vp, _sz, _vp, _vp, _vp]),
    "qmm_int8_gemm_workspace_size": (_c.c_int, [_i64, _i64, _i64, _szp]),
    "qmm_int8_gemm": (_c.c_int, [_vp, _c.c_int, _i64, _i64, _i64, _i32, _vp, _vp, _i64, _c.c_int,
                                 _i32, _c.POINTER(QmmEpilogue), _vp, _i64, _vp, _sz, _vp, _vp]),
    "qmm_widen_b_int8_size": (_c.c_int, [_i64, _i64, _szp]),
    "qmm_widen_b_int8": (_c.c_int, [_vp, _i64, _i64, _vp, _sz, _vp, _vp]),
    "qmm_int8_gemm_b16_workspace_size": (_c.c_int, [_i64, _i64, _i64, _szp]),
    "qmm_int8_gemm_b16": (_c.c_int, [_vp, _c.c_int, _i64, _i64, _i64, _i32, _vp, _vp, _vp, _i64, _c.c_int,
                                     _i32, _c.POINTER(QmmEpilogue), _vp, _i64, _vp, _sz, _vp, _vp]),
    "qmm_int8_gemm_group": (_c.c_int, [_c.POINTER(QmmInt8Problem), _i64, _vp, _vp]),
    "qmm_int8_gemm_axis_zp_workspace_size": (_c.c_int, [_i64, _i64, _i64, _szp]),
    "qmm_int8_gemm_axis_zp": (_c.c_int, [_vp, _c.c_int, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _c.c_int,
                                         _vp, _c.POINTER(QmmEpilogue), _vp, _i64, _vp, _sz, _vp, _vp]),
    "qmm_quantize_act_int8_workspace_size": (_c.c_int, [_i64, _i64, _c.c_int, _szp]),
    "qmm_quantize_act_int8": (_c.c_int, [_vp, _c.c_int, _i64, _i64, _i64, _c.c_int, _vp, _i64, _vp, _vp, _sz,
                                         _vp]),
    "qmm_pack_q4_size": (_c.c_int, [_i64, _i64, _szp]),
    "qmm_pack_q4": (_c.c_int, [_vp, _i64, _i64, _i64, _vp, _sz, _vp]),
    "qmm_q4_gemm_workspace_size": (_c.c_int, [_i64, _i64, _i64, _szp]),
    "qmm_q4_gemm": (_c.c_int, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _sz, _vp, _vp]),
    "qmm_q4_gemv_group": (_c.c_int, [_c.POINTER(QmmQ4GemvProblem), _i64, _vp, _vp]),
    "qmm_q4_gemm_id_workspace_size": (_c.c_int, [_i64, _i64, _i64, _i64, _szp]),
    "qmm_q4_gemm_id": (_c.c_int, [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _i64,
                                  _vp, _i64, _i64, _vp, _sz, _vp, _vp]),
    "qmm_q4_gemm_id_pair": (_c.c_int, [_vp, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _vp, _vp,
                                       _i64, _i64, _vp, _sz, _vp, _vp]),
    "qmm_q4_gemm_id_noalloc": (_c.c_int, [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64,
                                          _i64, _vp, _i64, _i64, _vp, _vp]),
    "qmm_pack_w8_size": (_c.c_int, [_i64, _i64, _szp, _szp]),
    "qmm_pack_w8": (_c.c_int, [_vp, _i64, _i64, _i64, _vp, _sz, _vp, _sz, _vp]),
    "qmm_w8_gemm_workspace_size": (_c.c_int, [_i64, _i64, _i64, _szp]),
    "qmm_w8_gemm": (_c.c_int, [_vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _sz, _vp, _vp]),
    "qmm_repack_q4k": (_c.c_int, [_vp, _i64, _i64, _i64, _vp, _sz, _vp]),
    "qmm_pack_q8_size": (_c.c_int, [_i64, _i64, _szp]),
    "qmm_pack_q8": (_c.c_int, [_vp, _i64, _i64, _i64, _c.c_int, _vp, _sz, _vp]),
    "qmm_q8_gemm_workspace_size": (_c.c_int, [_i64, _i64, _i64, _szp]),
    "qmm_q8_gemm": (_c.c_int, [_vp, _c.c_int, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _sz, _vp, _vp]),
    "qmm_kv_plan": (_c.c_int, [_vp, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _i64, _vp, _vp,
                               _vp, _vp, _vp, _vp]),
    "qmm_kv_append": (_c.c_int, [_vp, _i64, _i64, _vp, _i64, _i64, _c.c_int, _i64, _vp, _c.POINTER(QmmKvCache), _vp,
                                 _vp]),
    "qmm_tree_attention_workspace_size": (_c.c_int, [_i64, _i64, _i64, _i64, _szp]),
    "qmm_tree_attention": (_c.c_int, [_vp, _c.c_int, _i64, _i64, _i64, _c.POINTER(QmmKvCache), _vp, _i64, _i64, _vp,
                                      _vp, _i64, _i64, _i64, _vp, _i64, _c.c_float, _vp, _i64, _i64, _vp, _sz, _vp,
                                      _vp]),
    "qmm_block_norm": (_c.c_int, [_vp, _c.c_int, _i64, _vp, _c.c_int, _i64, _c.POINTER(QmmNorm), _vp, _c.c_int, _i64,
                                  _c.c_float, _vp, _i64, _c.POINTER(QmmNorm), _vp, _c.c_int, _i64, _vp, _i64, _i64,
                                  _vp]),
    "qmm_lora_add_workspace_size": (_c.c_int, [_i64, _i64, _i64, _i64, _i64, _szp]),
    "qmm_lora_add": (_c.c_int, [_c.POINTER(QmmLoraSet), _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _sz, _vp,
                                _vp]),
    "qmm_token_logprobs": (_c.c_int, [_vp, _c.c_int, _i64, _i64, _i64, _c.c_float, _vp, _i64, _i64, _vp, _vp, _i64,
                                      _vp, _vp, _vp, _vp]),
    "qmm_token_logprobs_or": (_c.c_int, [_vp, _c.c_int, _i64, _i64, _i64, _c.c_float, _vp, _i64, _i64, _vp, _vp, _i64,
                                         _vp, _vp, _vp, _c.c_float, _vp]),
    "qmm_probe_hbm_read": (_c.c_int, [_vp, _sz, _c.c_int, _vp, _vp, _vp]),
    "qmm_selftest_wait_timeout": (_c.c_int, [_c.c_uint64, _vp, _vp, _vp]),
}
QMM_Q8_LAYOUT_KR, QMM_Q8_LAYOUT_SLAB16 = 0, 1


class QmmError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} returned {status_string(status)} ({status})")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"libqmm.so not built ({path}); run quantized_matmul_qmm_gb300.build.build()")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


lib = load_library()


def status_string(s: int) -> str:
    return lib.qmm_status_string(int(s)).decode()


def _check(fn: str, status: int):
    if status != QMM_OK:
        raise QmmError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # None: torch without CUDA


def _stream_of(t):
    """The handle of torch's current stream on t's device (a decoding step makes
    many small calls: _stream's Stream object alone takes 3 us)."""
    return _raw_stream(t.get_device())


def _size(fn, *args) -> int:
    out = ctypes.c_size_t(0)
    _check(fn, getattr(lib, fn)(*args, ctypes.byref(out)))
    return int(out.value)


# ---------------------------------------------------------------------------
# int8
# ---------------------------------------------------------------------------

def pack_b_int8_size(K: int, N: int) -> int:
    return _size("qmm_pack_b_int8_size", K, N)


def pack_b_int8(B: torch.Tensor, b_type: str):
    """B: device [K][N] (fp32, int8 or uint8).  Returns (packed [N][Kp] int8,
    col_scale [N] fp32 or None, col_sum [N] int32)."""
    K, N = B.shape
    dev = B.device
    nbytes = pack_b_int8_size(K, N)
    packed = torch.empty(nbytes, dtype=torch.int8, device=dev).view(N, nbytes // N)
    col_scale = torch.empty(N, dtype=torch.float32, device=dev) if b_type == "f32" else None
    col_sum = torch.empty(N, dtype=torch.int32, device=dev)
    _check("qmm_pack_b_int8", lib.qmm_pack_b_int8(
        _ptr(B), DTYPES[b_type], K, N, B.stride(0), _ptr(packed), nbytes, _ptr(col_scale),
        _ptr(col_sum), _stream()))
    return packed, col_scale, col_sum


def int8_gemm_workspace_size(M: int, K: int, N: int) -> int:
    return _size("qmm_int8_gemm_workspace_size", M, K, N)


def widen_b_int8(packed: torch.Tensor, K: int, N: int, dev_status=None) -> torch.Tensor:
    """packed [N][Kp] int8 from pack_b_int8 -> its f16 copy [N][Kp] through
    qmm_widen_b_int8 (done once, like the pack)."""
    nbytes = _size("qmm_widen_b_int8_size", K, N)
    b16 = torch.empty(nbytes // 2, dtype=torch.float16, device=packed.device).view(N, nbytes // (2 * N))
    _check("qmm_widen_b_int8", lib.qmm_widen_b_int8(_ptr(packed), K, N, _ptr(b16), nbytes, _ptr(dev_status),
                                                    _stream()))
    return b16


def int8_gemm(A: torch.Tensor, a_type: str, zA: int, packed: torch.Tensor, col_sum: torch.Tensor,
              N: int, b_orig_type: str, zB: int, out_type: str = "s32", bias=None, s_x=None,
              s_x_stride: int = 0, s_w=None, s_y: float = 1.0, zp_y: int = 0, out=None,
              workspace=None, dev_status=None, b16=None):
    """Y = A (x) packB through qmm_int8_gemm, or qmm_int8_gemm_b16 when b16
    (from widen_b_int8) is given.  Returns the output tensor."""
    M, K = A.shape
    if out is None:
        out = torch.empty((M, N), dtype=TORCH_OUT[out_type], device=A.device)
    ws_need = (_size("qmm_int8_gemm_b16_workspace_size", M, K, N) if b16 is not None
               else int8_gemm_workspace_size(M, K, N))
    if workspace is None and ws_need > 0:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=A.device)
    ep = QmmEpilogue(DTYPES[out_type], _ptr(bias), _ptr(s_x), s_x_stride, _ptr(s_w),
                     float(s_y), int(zp_y))
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if b16 is not None:
        _check("qmm_int8_gemm_b16", lib.qmm_int8_gemm_b16(
            _ptr(A), DTYPES[a_type], M, K, A.stride(0), int(zA), _ptr(packed), _ptr(b16), _ptr(col_sum), N,
            DTYPES[b_orig_type], int(zB), ctypes.byref(ep), _ptr(out), out.stride(0), _ptr(workspace), ws_bytes,
            _ptr(dev_status), _stream()))
        return out
    _check("qmm_int8_gemm", lib.qmm_int8_gemm(
        _ptr(A), DTYPES[a_type], M, K, A.stride(0), int(zA), _ptr(packed), _ptr(col_sum), N,
        DTYPES[b_orig_type], int(zB), ctypes.byref(ep), _ptr(out), out.stride(0), _ptr(workspace), ws_bytes,
        _ptr(dev_status), _stream()))
    return out


def int8_gemm_group(problems, dev_status=None):
    """Several small-M int8 GEMMs (M <= 64) in one launch through
    qmm_int8_gemm_group.  problems: list of dicts with int8_gemm's arguments
    (A, a_type, zA, packed, col_sum, N, b_orig_type, zB, out_type, bias, s_x,
    s_x_stride, s_w, s_y, zp_y, out); `out` is created when absent.  Returns
    the list of outputs."""
    arr = (QmmInt8Problem * len(problems))()
    outs = []
    for i, d in enumerate(problems):
        A = d["A"]
        M, K = A.shape
        N, ot = d["N"], d.get("out_type", "s32")
        out = d.get("out")
        if out is None:
            out = torch.empty((M, N), dtype=TORCH_OUT[ot], device=A.device)
        outs.append(out)
        ep = QmmEpilogue(DTYPES[ot], _ptr(d.get("bias")), _ptr(d.get("s_x")), d.get("s_x_stride", 0),
                         _ptr(d.get("s_w")), float(d.get("s_y", 1.0)), int(d.get("zp_y", 0)))
        ptr = lambda t: 0 if t is None else t.data_ptr()
        arr[i] = QmmInt8Problem(ptr(A), DTYPES[d["a_type"]], M, K, A.stride(0), int(d["zA"]), ptr(d["packed"]),
                                ptr(d["col_sum"]), N, DTYPES[d["b_orig_type"]], int(d["zB"]), ep, ptr(out),
                                out.stride(0))
    _check("qmm_int8_gemm_group", lib.qmm_int8_gemm_group(arr, len(problems), _ptr(dev_status), _stream()))
    return outs


def int8_gemm_axis_zp_workspace_size(M: int, K: int, N: int) -> int:
    return _size("qmm_int8_gemm_axis_zp_workspace_size", M, K, N)


def int8_gemm_axis_zp(A: torch.Tensor, a_type: str, zA, packed: torch.Tensor, col_sum: torch.Tensor,
                      N: int, b_orig_type: str, zB, out_type: str = "s32", bias=None, s_x=None,
                      s_x_stride: int = 0, s_w=None, s_y: float = 1.0, zp_y: int = 0, out=None,
                      workspace=None, dev_status=None):
    """qmm_int8_gemm with per-axis zero points: zA a device int32 [M] (or None:
    all 0), zB a device int32 [N] (or None).  Returns the output tensor."""
    M, K = A.shape
    if out is None:
        out = torch.empty((M, N), dtype=TORCH_OUT[out_type], device=A.device)
    if workspace is None:
        workspace = torch.empty(int8_gemm_axis_zp_workspace_size(M, K, N), dtype=torch.uint8, device=A.device)
    ep = QmmEpilogue(DTYPES[out_type], _ptr(bias), _ptr(s_x), s_x_stride, _ptr(s_w),
                     float(s_y), int(zp_y))
    _check("qmm_int8_gemm_axis_zp", lib.qmm_int8_gemm_axis_zp(
        _ptr(A), DTYPES[a_type], M, K, A.stride(0), _ptr(zA), _ptr(packed), _ptr(col_sum), N,
        DTYPES[b_orig_type], _ptr(zB), ctypes.byref(ep), _ptr(out), out.stride(0), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_status), _stream()))
    return out


def quantize_act_int8_workspace_size(M: int, K: int, per_row: bool) -> int:
    return _size("qmm_quantize_act_int8_workspace_size", M, K, int(per_row))


def quantize_act_int8(X: torch.Tensor, per_row: bool = True, A=None, s_x=None, workspace=None):
    """Symmetric int8 codes of X (fp32 or bf16 [M][K] on the device) through
    qmm_quantize_act_int8.  Returns (A int8 [M][K], s_x fp32 [M] or [1])."""
    M, K = X.shape
    x_type = {torch.float32: "f32", torch.bfloat16: "bf16"}[X.dtype]
    if A is None:
        lda = (K + 15) // 16 * 16
        A = torch.empty((M, lda), dtype=torch.int8, device=X.device)[:, :K]
    if s_x is None:
        s_x = torch.empty(M if per_row else 1, dtype=torch.float32, device=X.device)
    ws_need = quantize_act_int8_workspace_size(M, K, per_row)
    if workspace is None and ws_need > 0:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=X.device)
    _check("qmm_quantize_act_int8", lib.qmm_quantize_act_int8(
        _ptr(X), DTYPES[x_type], M, K, X.stride(0), int(per_row), _ptr(A), A.stride(0), _ptr(s_x),
        _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(), _stream()))
    return A, s_x


# ---------------------------------------------------------------------------
# 4-bit
# ---------------------------------------------------------------------------

def pack_q4_size(N: int, K: int) -> int:
    return _size("qmm_pack_q4_size", N, K)


def pack_q4(W: torch.Tensor) -> torch.Tensor:
    """W: device fp32 [N][K].  Returns the tile bytes (uint8)."""
    N, K = W.shape
    nbytes = pack_q4_size(N, K)
    tiles = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    _check("qmm_pack_q4", lib.qmm_pack_q4(_ptr(W), N, K, W.stride(0), _ptr(tiles), nbytes,
                                          _stream()))
    return tiles


def q4_gemm_workspace_size(M: int, K: int, N: int) -> int:
    return _size("qmm_q4_gemm_workspace_size", M, K, N)


def q4_gemm(tiles: torch.Tensor, N: int, K: int, X: torch.Tensor, Y=None, workspace=None, dev_status=None):
    """Y[m][n] = sum_k X[m][k] w[n][k]; X bf16 [M][K] on the device."""
    M = X.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=X.device)
    if workspace is None:
        need = q4_gemm_workspace_size(M, K, N)
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    _check("qmm_q4_gemm", lib.qmm_q4_gemm(
        _ptr(tiles), N, K, _ptr(X), M, X.stride(0), _ptr(Y), Y.stride(0), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _ptr(dev_status), _stream()))
    return Y


def q4_gemv_group(problems, dev_status=None):
    """Grouped decode GEMVs in one launch: problems is a list of
    (tiles, N, K, x, y) with x bf16 [K] and y fp32 [N] on the device;
    y_i = W_i x_i for every i.  Returns the list of y tensors."""
    arr = (QmmQ4GemvProblem * len(problems))()
    for i, (tiles, N, K, x, y) in enumerate(problems):
        arr[i] = QmmQ4GemvProblem(tiles.data_ptr(), N, K, x.data_ptr(), y.data_ptr())
    _check("qmm_q4_gemv_group", lib.qmm_q4_gemv_group(arr, len(problems), _ptr(dev_status), _stream()))
    return [y for (_, _, _, _, y) in problems]


def q4_gemm_id_workspace_size(n_expert: int, n_used: int, T: int, K: int) -> int:
    return _size("qmm_q4_gemm_id_workspace_size", n_expert, n_used, T, K)


def q4_gemm_id(tiles: torch.Tensor, n_expert: int, N: int, K: int, X: torch.Tensor,
               ids: torch.Tensor, ld_ids: int, n_used: int, T: int, Y=None, workspace=None,
               dev_status=None):
    """MUL_MAT_ID.  X is [T][K] (shared src1) or [T][n_used][K] (per-slot src1);
    ids a device int32 buffer read as ids[t*ld_ids + i].  Returns Y [T][n_used][N]."""
    if X.dim() == 2:
        ldx_token, ldx_slot = X.stride(0), 0
    else:
        ldx_token, ldx_slot = X.stride(0), X.stride(1)
    if Y is None:
        Y = torch.empty((T, n_used, N), dtype=torch.float32, device=X.device)
    if workspace is None:
        workspace = torch.empty(q4_gemm_id_workspace_size(n_expert, n_used, T, K), dtype=torch.uint8,
                                device=X.device)
    _check("qmm_q4_gemm_id", lib.qmm_q4_gemm_id(
        _ptr(tiles), n_expert, N, K, _ptr(X), ldx_token, ldx_slot, _ptr(ids), ld_ids, n_used, T,
        _ptr(Y), Y.stride(0), Y.stride(1), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_status), _stream()))
    return Y


def q4_gemm_id_pair(tiles_gate: torch.Tensor, tiles_up: torch.Tensor, n_expert: int, N: int, K: int,
                    X: torch.Tensor, ids: torch.Tensor, ld_ids: int, n_used: int, T: int, Y_gate=None, Y_up=None,
                    workspace=None, dev_status=None):
    """The gate/up pair: both MUL_MAT_IDs over the shared src1 X [T][K] in one
    call.  Returns (Y_gate, Y_up), each [T][n_used][N]."""
    if Y_gate is None:
        Y_gate = torch.empty((T, n_used, N), dtype=torch.float32, device=X.device)
    if Y_up is None:
        Y_up = torch.empty((T, n_used, N), dtype=torch.float32, device=X.device)
    assert Y_gate.stride() == Y_up.stride()
    if workspace is None:
        workspace = torch.empty(q4_gemm_id_workspace_size(n_expert, n_used, T, K), dtype=torch.uint8,
                                device=X.device)
    _check("qmm_q4_gemm_id_pair", lib.qmm_q4_gemm_id_pair(
        _ptr(tiles_gate), _ptr(tiles_up), n_expert, N, K, _ptr(X), X.stride(0), _ptr(ids), ld_ids, n_used, T,
        _ptr(Y_gate), _ptr(Y_up), Y_gate.stride(0), Y_gate.stride(1), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_status), _stream()))
    return Y_gate, Y_up


def q4_gemm_id_noalloc(tiles: torch.Tensor, n_expert: int, N: int, K: int, X: torch.Tensor,
                       ids: torch.Tensor, ld_ids: int, n_used: int, T: int, Y: torch.Tensor,
                       dev_status=None):
    """MUL_MAT_ID through qmm_q4_gemm_id_noalloc: the same result as
    q4_gemm_id, for callers that cannot allocate device memory.  The library
    keeps the routing tables and activation-row scales in its own fixed device
    array (and packs the activation rows there when they fit), so the caller
    passes only inputs and the output Y [T][n_used][N] (preallocated).
    Limits: n_expert <= 1024, T * n_used <= 65536."""
    if X.dim() == 2:
        ldx_token, ldx_slot = X.stride(0), 0
    else:
        ldx_token, ldx_slot = X.stride(0), X.stride(1)
    _check("qmm_q4_gemm_id_noalloc", lib.qmm_q4_gemm_id_noalloc(
        _ptr(tiles), n_expert, N, K, _ptr(X), ldx_token, ldx_slot, _ptr(ids), ld_ids, n_used, T,
        _ptr(Y), Y.stride(0), Y.stride(1), _ptr(dev_status), _stream()))
    return Y


# ---------------------------------------------------------------------------
# W8A16
# ---------------------------------------------------------------------------

def pack_w8_size(N: int, K: int):
    """(code bytes, scale bytes) of an N x K weight."""
    cb, sb = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check("qmm_pack_w8_size", lib.qmm_pack_w8_size(N, K, ctypes.byref(cb), ctypes.byref(sb)))
    return int(cb.value), int(sb.value)


def pack_w8(W: torch.Tensor):
    """W: device fp32 [N][K].  Returns (codes int8 [N][Kp], scales fp32 [N][ceil(K/1024)])."""
    N, K = W.shape
    cb, sb = pack_w8_size(N, K)
    codes = torch.empty((N, cb // N), dtype=torch.int8, device=W.device)
    scales = torch.empty((N, sb // (4 * N)), dtype=torch.float32, device=W.device)
    _check("qmm_pack_w8", lib.qmm_pack_w8(_ptr(W), N, K, W.stride(0), _ptr(codes), cb, _ptr(scales), sb,
                                          _stream()))
    return codes, scales


def w8_gemm_workspace_size(M: int, K: int, N: int) -> int:
    return _size("qmm_w8_gemm_workspace_size", M, K, N)


def w8_gemm(codes: torch.Tensor, scales: torch.Tensor, N: int, K: int, X: torch.Tensor, Y=None, workspace=None,
            dev_status=None):
    """Y[m][n] = sum_b scales[n][b] sum_{k in b} codes[n][k] X[m][k]; X bf16 [M][K] on the device."""
    M = X.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=X.device)
    if workspace is None:
        need = w8_gemm_workspace_size(M, K, N)
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    _check("qmm_w8_gemm", lib.qmm_w8_gemm(
        _ptr(codes), _ptr(scales), N, K, _ptr(X), M, X.stride(0), _ptr(Y), Y.stride(0), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _ptr(dev_status), _stream()))
    return Y


# ---------------------------------------------------------------------------
# More weight formats: Q4_K -> q4_1 tiles, Q8 tiles
# ---------------------------------------------------------------------------

def repack_q4k(q4k: torch.Tensor, N: int, K: int, tiles=None) -> torch.Tensor:
    """q4k: device uint8 [N][row_bytes] of Q4_K super-blocks (row_bytes >= K/256*144).
    Returns q4_1 tile bytes (uint8) for qmm_q4_gemm / qmm_q4_gemm_id."""
    nbytes = pack_q4_size(N, K)
    if tiles is None:
        tiles = torch.empty(nbytes, dtype=torch.uint8, device=q4k.device)
    row_bytes = q4k.stride(0) if q4k.dim() == 2 else K // 256 * 144
    _check("qmm_repack_q4k", lib.qmm_repack_q4k(_ptr(q4k), N, K, row_bytes, _ptr(tiles),
                                                tiles.numel(), _stream()))
    return tiles


def pack_q8_size(N: int, K: int) -> int:
    return _size("qmm_pack_q8_size", N, K)


def pack_q8(W: torch.Tensor, layout: int) -> torch.Tensor:
    """W: device fp32 [N][K].  Returns Q8 tile bytes (uint8) in the given code layout."""
    N, K = W.shape
    nbytes = pack_q8_size(N, K)
    tiles = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    _check("qmm_pack_q8", lib.qmm_pack_q8(_ptr(W), N, K, W.stride(0), int(layout), _ptr(tiles), nbytes,
                                          _stream()))
    return tiles


def q8_gemm_workspace_size(M: int, K: int, N: int) -> int:
    return _size("qmm_q8_gemm_workspace_size", M, K, N)


def q8_gemm(tiles: torch.Tensor, layout: int, N: int, K: int, X: torch.Tensor, Y=None, workspace=None,
            dev_status=None):
    """Y[m][n] = sum_k X[m][k] w[n][k] over Q8 tiles; X bf16 [M][K] on the device."""
    M = X.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=X.device)
    if workspace is None:
        need = q8_gemm_workspace_size(M, K, N)
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    _check("qmm_q8_gemm", lib.qmm_q8_gemm(
        _ptr(tiles), int(layout), N, K, _ptr(X), M, X.stride(0), _ptr(Y), Y.stride(0), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _ptr(dev_status), _stream()))
    return Y


# ---------------------------------------------------------------------------
# Paged key/value cache and tree attention
# ---------------------------------------------------------------------------

_KV_TYPES = {torch.bfloat16: QMM_BF16, torch.int8: QMM_S8}
_ROW_TYPES = {torch.float32: QMM_F32, torch.bfloat16: QMM_BF16}


def _addr(t):
    return None if t is None else t.data_ptr()


_I32, _I64 = torch.int32, torch.int64


def _ints(fn, dtype, *tensors):
    """Lengths, slots and the like are read as plain arrays: refused unless they are."""
    for t in tensors:
        if t.dtype is not dtype or not t.is_contiguous():
            raise ValueError(f"{fn}: not a contiguous {dtype} tensor: {t.dtype}, strides {t.stride()}")


def _status_addr(fn, t):
    if t is None:
        return None
    if t.dtype is not _I32:
        raise ValueError(f"{fn}: dev_status is not contiguous int32: {t.dtype}")
    return t.data_ptr()


def _row_stride(fn, t):
    """Of a block table or mask (of words without a sign, too)."""
    (rows, cols), (ld, inner) = t.shape, t.stride()
    if t.dtype is not _I32 and t.dtype is not torch.uint32 or inner != 1 and cols > 1:
        raise ValueError(f"{fn}: not a 32-bit table of contiguous rows: {t.dtype}, strides {(ld, inner)}")
    return ld if rows > 1 else max(ld, cols)


def _kv_cache(k_cache, v_cache, k_scale, v_scale) -> QmmKvCache:
    n_pages, page_size, n_heads, head_dim = k_cache.shape
    sp, st, sh, sd = strides = k_cache.stride()
    if v_cache.shape != k_cache.shape or v_cache.stride() != strides or v_cache.dtype != k_cache.dtype or sd != 1:
        raise ValueError("k_cache and v_cache must have one shape, type and strides, with contiguous heads")
    if k_cache.dtype == torch.int8:
        for sc in (k_scale, v_scale):
            if sc is None or sc.dtype != torch.float32 or sc.shape != (n_pages, n_heads, page_size) \
                    or not sc.is_contiguous():
                raise ValueError("an int8 cache needs contiguous fp32 scales [pages][heads][page_size]")
    return QmmKvCache(k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale), _addr(v_scale),
                      _KV_TYPES[k_cache.dtype], n_pages, page_size, n_heads, head_dim, sp, st, sh)


def kv_plan(ctx_lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor, block_table: torch.Tensor,
            page_size: int, slots: torch.Tensor, positions: torch.Tensor, cu_new=None, pages_taken=None, parents=None,
            mask=None, dev_status=None):
    """Pages, slots, positions and tree masks of a step through qmm_kv_plan.
    block_table int32 [R][max_blocks] is updated in place; slots int64 and
    positions int32 [max_tokens] are written, and with parents (int32
    [max_tokens]) the mask int32 [max_tokens][words].  Returns (cu_new int32
    [R+1], pages_taken int32 [1])."""
    R, T = ctx_lens.numel(), slots.numel()
    if cu_new is None:
        cu_new = torch.empty(R + 1, dtype=_I32, device=ctx_lens.device)
    if pages_taken is None:
        pages_taken = torch.empty(1, dtype=_I32, device=ctx_lens.device)
    # Checks in line, few calls: a decoding step waits for this code, not for the kernel.
    rows, blocks = block_table.shape
    ld_table, inner = block_table.stride()
    if inner != 1 or rows == 1 or block_table.dtype is not _I32:
        ld_table = _row_stride("kv_plan", block_table)
    agree = rows == R == new_lens.numel() and positions.numel() == T and cu_new.numel() == R + 1
    p_parents = p_mask = p_status = None
    words = ld_mask = 0
    if parents is not None:
        agree = agree and parents.numel() == T
        if parents.dtype is not _I32 or not parents.is_contiguous():
            _ints("kv_plan", _I32, parents)
        p_parents = parents.data_ptr()
    if mask is not None:
        mask_rows, words = mask.shape
        agree = agree and mask_rows == T
        ld_mask, inner = mask.stride()
        if inner != 1 or mask_rows == 1 or mask.dtype is not _I32:
            ld_mask = _row_stride("kv_plan", mask)
        p_mask = mask.data_ptr()
    if not agree:
        raise ValueError("kv_plan: shapes do not agree")
    if dev_status is not None:
        p_status = _status_addr("kv_plan", dev_status)
    if not (ctx_lens.dtype is new_lens.dtype is free_pages.dtype is positions.dtype is cu_new.dtype
            is pages_taken.dtype is _I32 and slots.dtype is _I64 and ctx_lens.is_contiguous()
            and new_lens.is_contiguous() and free_pages.is_contiguous() and positions.is_contiguous()
            and cu_new.is_contiguous() and slots.is_contiguous()):
        raise ValueError("kv_plan: slots must be contiguous int64, the other lists contiguous int32")
    status = lib.qmm_kv_plan(
        ctx_lens.data_ptr(), new_lens.data_ptr(), R, free_pages.data_ptr(), free_pages.numel(),
        block_table.data_ptr(), ld_table, blocks, page_size, p_parents, p_mask,
        ld_mask, words, T, cu_new.data_ptr(), slots.data_ptr(), positions.data_ptr(), pages_taken.data_ptr(),
        p_status, _raw_stream(slots.get_device()))
    if status != QMM_OK:
        _check("qmm_kv_plan", status)
    return cu_new, pages_taken


def kv_append(K: torch.Tensor, V: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              k_scale=None, v_scale=None, dev_status=None):
    """Store the rows K, V (fp32 or bf16 [T][heads][head_dim]) at slots (int64
    [T], -1 skips) of a cache [pages][page_size][heads][head_dim], bf16 or int8
    with scales fp32 [pages][heads][page_size], through qmm_kv_append."""
    cache = _kv_cache(k_cache, v_cache, k_scale, v_scale)
    (kt, kh, kd), (vt, vh, vd) = K.stride(), V.stride()
    T, heads, head_dim = shape = K.shape
    if V.shape != shape or V.dtype != K.dtype or kd != 1 or vd != 1 or T != slots.numel() \
            or heads != cache.n_heads or head_dim != cache.head_dim:
        raise ValueError("kv_append: K, V, slots and the cache do not agree")
    _ints("kv_append", _I64, slots)
    _check("qmm_kv_append", lib.qmm_kv_append(
        K.data_ptr(), kt, kh, V.data_ptr(), vt, vh, _ROW_TYPES[K.dtype], T, slots.data_ptr(),
        cache, _status_addr("kv_append", dev_status), _stream_of(k_cache)))


def tree_attention_workspace_size(n_q_heads: int, n_kv_heads: int, head_dim: int, max_new: int) -> int:
    return _size("qmm_tree_attention_workspace_size", n_q_heads, n_kv_heads, head_dim, max_new)


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                   ctx_lens: torch.Tensor, cu_new: torch.Tensor, max_new: int, mask=None, scale=None, k_scale=None,
                   v_scale=None, out=None, workspace=None, dev_status=None):
    """Attention of a step's tokens q (fp32 or bf16 [T][q heads][head_dim]) over
    the paged cache through qmm_tree_attention; mask int32 [T][words] (kv_plan's)
    or None for causal chunks and plain decoding; scale 1 / sqrt(head_dim) by
    default.  Returns out, bf16 [T][q heads][head_dim]."""
    cache = _kv_cache(k_cache, v_cache, k_scale, v_scale)
    T, heads, head_dim = shape = q.shape
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
    (qt, qh, qd), (ot, oh, od) = q.stride(), out.stride()
    R = ctx_lens.numel()
    rows, blocks = block_table.shape
    if head_dim != cache.head_dim or out.shape != shape or out.dtype != torch.bfloat16 or qd != 1 or od != 1 \
            or cu_new.numel() != R + 1 or rows != R \
            or (mask is not None and (mask.shape[0] != T or mask.shape[1] * 32 < max_new)):
        raise ValueError("tree_attention: shapes do not agree")
    ld_table = _row_stride("tree_attention", block_table)
    ld_mask = 0 if mask is None else _row_stride("tree_attention", mask)
    _ints("tree_attention", _I32, ctx_lens, cu_new)
    if workspace is None:
        workspace = torch.empty(tree_attention_workspace_size(heads, cache.n_heads, head_dim, max_new),
                                dtype=torch.uint8, device=q.device)
    _check("qmm_tree_attention", lib.qmm_tree_attention(
        q.data_ptr(), _ROW_TYPES[q.dtype], qt, qh, heads, cache, block_table.data_ptr(),
        ld_table, blocks, ctx_lens.data_ptr(), cu_new.data_ptr(), R, T,
        max_new, _addr(mask), ld_mask,
        head_dim ** -0.5 if scale is None else scale, out.data_ptr(), ot, oh, workspace.data_ptr(),
        workspace.nbytes, _status_addr("tree_attention", dev_status), _stream_of(q)))
    return out


# ---------------------------------------------------------------------------
# Beside the projections
# ---------------------------------------------------------------------------

_NORM_KINDS = {"rms": 1, "layer": 2}
_OUT_TYPES = {torch.float32: QMM_F32, torch.bfloat16: QMM_BF16, torch.int8: QMM_S8}
_OUT_NAMES = {"bf16": torch.bfloat16, "f32": torch.float32}
_F32, _BF16 = torch.float32, torch.bfloat16
_F32_ONLY, _BF16_ONLY, _INT32_ONLY = (torch.float32,), (torch.bfloat16,), (torch.int32,)
_empty = torch.empty
_NAN = float("nan")
_current_device = getattr(torch._C, "_cuda_getDevice", None)   # None: torch without CUDA

# Every tensor has to lie on the current GPU: an address of another device or of
# the host would reach the kernel as it is.  The checks stand in few calls: a
# decoding step waits for this code, not for the kernels.


def _device_of(fn, t):
    dev = t.get_device()
    if _current_device is None or dev != _current_device():
        raise ValueError(f"{fn}: tensors have to be on the current CUDA device, got {t.device}")
    return dev


def _rows(fn, dev, t, shape, types):
    """Row stride of a [rows][width] tensor with contiguous rows."""
    if t.shape == shape and t.dtype in types and t.get_device() == dev:
        ld, inner = t.stride()
        if inner == 1 or shape[1] <= 1:
            return ld
    raise ValueError(f"{fn}: expected {tuple(shape)} with contiguous rows of {[str(x) for x in types]} on device "
                     f"{dev}, got {tuple(t.shape)} {t.dtype} with strides {t.stride()} on {t.device}")


def _vector(fn, dev, t, size, dtype):
    """Address of `size` contiguous values, or None."""
    if t is None:
        return None
    if t.numel() != size or t.dtype is not dtype or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{fn}: expected {size} contiguous values of {dtype} on device {dev}, got {tuple(t.shape)} "
                         f"{t.dtype} with strides {t.stride()} on {t.device}")
    return t.data_ptr()


def block_norm(residual: torch.Tensor, branch=None, *, norm="rms", weight=None, bias=None, eps=1e-6, branch_norm=None,
               branch_weight=None, branch_bias=None, branch_eps=None, gate=None, scale=1.0, residual_out=None, out=None,
               out_type="bf16", s_x=None):
    """Join a block's output to the residual stream and make the next block's
    input, through qmm_block_norm:

        u = branch_norm(branch); sum = residual + scale * gate * u; out = norm(sum)

    residual and branch fp32 or bf16 [T][D]; norm and branch_norm "rms",
    "layer" or None with fp32 weights and biases [D] (or None); gate fp32 or bf16
    [D] or [T][D].  residual_out takes the sum (the residual itself, in place,
    when a branch is given and residual_out is not); out is "bf16", "f32" or
    "s8", the last with row scales s_x fp32 [T], made when not given (out=False:
    the sum alone).  Returns (sum, out), or (sum, out, s_x) for "s8"."""
    fn = "block_norm"
    dev = _device_of(fn, residual)
    shape = residual.shape
    T, D = shape
    ldr = _rows(fn, dev, residual, shape, _ROW_TYPES)
    r_type = _ROW_TYPES[residual.dtype]
    ldb = ldg = lds = ldo = 0
    p_branch = p_gate = p_sum = p_out = n_branch = n_out = None
    b_type = g_type = QMM_F32
    o_type = QMM_BF16
    if branch is not None:
        ldb, p_branch, b_type = _rows(fn, dev, branch, shape, _ROW_TYPES), branch.data_ptr(), _ROW_TYPES[branch.dtype]
        if branch_norm is not None:
            n_branch = QmmNorm(_NORM_KINDS[branch_norm], eps if branch_eps is None else branch_eps,
                               _vector(fn, dev, branch_weight, D, _F32), _vector(fn, dev, branch_bias, D, _F32))
        if gate is not None:
            if gate.dim() == 1:
                _rows(fn, dev, gate.unsqueeze(0), (1, D), _ROW_TYPES)
            else:
                ldg = _rows(fn, dev, gate, shape, _ROW_TYPES)
            p_gate, g_type = gate.data_ptr(), _ROW_TYPES[gate.dtype]
        if residual_out is None:
            residual_out = residual
    if residual_out is not None:
        lds, p_sum = _rows(fn, dev, residual_out, shape, (residual.dtype,)), residual_out.data_ptr()
    p_sx = None
    if out is not False:
        if out is None:
            if out_type == "s8":       # rows of whole 16 bytes, as the int8 GEMM takes them
                out = torch.empty((T, (D + 15) // 16 * 16), dtype=torch.int8, device=residual.device)[:, :D]
            else:
                out = torch.empty(shape, dtype=_OUT_NAMES[out_type], device=residual.device)
        ldo, p_out, o_type = _rows(fn, dev, out, shape, _OUT_TYPES), out.data_ptr(), _OUT_TYPES[out.dtype]
        if o_type == QMM_S8:
            if s_x is None:
                s_x = torch.empty(T, dtype=_F32, device=residual.device)
            p_sx = _vector(fn, dev, s_x, T, _F32)
        if norm is not None:
            n_out = QmmNorm(_NORM_KINDS[norm], eps, _vector(fn, dev, weight, D, _F32), _vector(fn, dev, bias, D, _F32))
    status = lib.qmm_block_norm(
        residual.data_ptr(), r_type, ldr, p_branch, b_type, ldb, n_branch, p_gate, g_type, ldg, scale, p_sum, lds,
        n_out, p_out, o_type, ldo, p_sx, T, D, _raw_stream(dev))
    if status != QMM_OK:
        _check("qmm_block_norm", status)
    total = residual if residual_out is None else residual_out
    return (total, out, s_x) if o_type == QMM_S8 else (total, None if out is False else out)


def lora_add_workspace_size(M: int, K: int, N: int, n_adapters: int, max_rank: int) -> int:
    return _size("qmm_lora_add_workspace_size", M, K, N, n_adapters, max_rank)


def lora_add(X: torch.Tensor, ids: torch.Tensor, A: torch.Tensor, B: torch.Tensor, base=None, out=None, ranks=None,
             scales=None, workspace=None, dev_status=None):
    """Adapters of many requests beside a shared projection, through qmm_lora_add:
    out[m] = base[m] + scales[a] * B[a] (A[a] X[m]) with a = ids[m] (-1: none).
    X bf16 [M][K], ids int32 [M], A bf16 [adapters][max_rank][K], B bf16
    [adapters][N][max_rank], ranks int32 and scales fp32 [adapters] (or None), base
    fp32 [M][N] (or None for zeros).  out is made when not given; out=base adds in
    place.  X, A and B are read 16 bytes at a time: their data has to begin at 16 bytes,
    the strides of all their dimensions but the last to be multiples of 8 elements (a B
    of another rank is the first columns of one that is wider), and B's last row to be
    readable up to the next multiple of 8.  Returns out."""
    fn = "lora_add"
    dev = _device_of(fn, X)
    M, K = shape = X.shape
    ldx = _rows(fn, dev, X, shape, _BF16_ONLY)
    slots, rank, k = A.shape
    b_slots, N, b_rank = B.shape
    a_slot, a_row, a_in = A.stride()
    b_slot, b_row, b_in = B.stride()
    if k != K or b_slots != slots or b_rank != rank or A.dtype is not _BF16 or B.dtype is not _BF16 \
            or (a_in != 1 and K > 1) or (b_in != 1 and rank > 1) or A.get_device() != dev or B.get_device() != dev:
        raise ValueError("lora_add: A has to be bf16 [adapters][rank][K], B bf16 [adapters][N][rank], with "
                         "contiguous innermost values, for X [M][K], all on one device")
    out_shape = (M, N)
    p_base, ldb = (None, 0) if base is None else (base.data_ptr(), _rows(fn, dev, base, out_shape, _F32_ONLY))
    if out is None:
        out = torch.empty(out_shape, dtype=_F32, device=X.device)
        ldo = N
    else:
        ldo = _rows(fn, dev, out, out_shape, _F32_ONLY)
    weights = QmmLoraSet(A.data_ptr(), a_slot, a_row, B.data_ptr(), b_slot, b_row,
                         _vector(fn, dev, ranks, slots, _I32), _vector(fn, dev, scales, slots, _F32), slots, rank, K, N)
    if workspace is None:
        workspace = torch.empty(lora_add_workspace_size(M, K, N, slots, rank), dtype=torch.uint8, device=X.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("lora_add: workspace has to be contiguous, on X's device")
    status = lib.qmm_lora_add(
        weights, X.data_ptr(), ldx, _vector(fn, dev, ids, M, _I32), M, p_base, ldb, out.data_ptr(), ldo,
        workspace.data_ptr(), workspace.nbytes, _vector(fn, dev, dev_status, 1, _I32), _raw_stream(dev))
    if status != QMM_OK:
        if status == QMM_ERR_INVALID_ARG:
            for name, t in (("X", X), ("A", A), ("B", B)):
                if t.data_ptr() % 16 or any(s % 8 for s, n in zip(t.stride()[:-1], t.shape) if n > 1):
                    raise ValueError(f"{fn}: {name} has to begin at 16 bytes and its strides but the last to be "
                                     f"multiples of 8 elements, got {tuple(t.shape)} with strides {t.stride()}")
        _check("qmm_lora_add", status)
    return out


def token_logprobs(logits: torch.Tensor, tokens=None, top_k: int = 0, scale: float = 1.0, logprobs=None, entropy=None,
                   top_ids=None, top_logprobs=None, dev_status=None):
    """Log probabilities of tokens (int32 [M][G] or [M], -1: none) under
    softmax(scale * logits), logits fp32 or bf16 [M][V], with the entropy fp32 [M]
    (entropy=False: none) and the top_k <= 32 alternatives, through
    qmm_token_logprobs.  A token of -1 (or outside the vocabulary, which dev_status
    tells) leaves its place in a logprobs tensor given as it was; in one made here it
    is NaN.  Returns (logprobs, entropy, top_ids, top_logprobs), None for what was not
    asked for."""
    fn = "token_logprobs"
    dev = _device_of(fn, logits)
    M, V = shape = logits.shape
    ld = _rows(fn, dev, logits, shape, _ROW_TYPES)
    device = logits.device
    G = ldt = 0
    made = False
    p_tokens = p_logprobs = p_ids = p_top = p_entropy = p_status = None
    if tokens is not None:
        if tokens.dim() == 2:
            G = tokens.shape[1]
            ldt = _rows(fn, dev, tokens, (M, G), _INT32_ONLY)
        else:
            if tokens.shape != (M,) or tokens.dtype is not _I32 or tokens.get_device() != dev:
                raise ValueError(f"{fn}: expected int32 tokens [{M}] or [{M}][G] on device {dev}, got "
                                 f"{tuple(tokens.shape)} {tokens.dtype} on {tokens.device}")
            G, ldt = 1, tokens.stride(0)
        p_tokens = tokens.data_ptr()
        if logprobs is None:
            logprobs, made = _empty(tokens.shape, dtype=_F32, device=device), True
            p_logprobs = logprobs.data_ptr()
        else:
            p_logprobs = _vector(fn, dev, logprobs, M * G, _F32)
    if entropy is False:
        entropy = None
    elif entropy is None:
        entropy = _empty(M, dtype=_F32, device=device)
        p_entropy = entropy.data_ptr()
    else:
        p_entropy = _vector(fn, dev, entropy, M, _F32)
    if top_k > 0:
        if top_ids is None:
            top_ids = _empty((M, top_k), dtype=_I32, device=device)
            p_ids = top_ids.data_ptr()
        else:
            p_ids = _vector(fn, dev, top_ids, M * top_k, _I32)
        if top_logprobs is None:
            top_logprobs = _empty((M, top_k), dtype=_F32, device=device)
            p_top = top_logprobs.data_ptr()
        else:
            p_top = _vector(fn, dev, top_logprobs, M * top_k, _F32)
    else:
        top_ids = top_logprobs = None
    if dev_status is not None:
        p_status = _vector(fn, dev, dev_status, 1, _I32)
    if made:
        status = lib.qmm_token_logprobs_or(
            logits.data_ptr(), _ROW_TYPES[logits.dtype], M, V, ld, scale, p_tokens, ldt, G, p_logprobs, p_entropy,
            top_k, p_ids, p_top, p_status, _NAN, _raw_stream(dev))
    else:
        status = lib.qmm_token_logprobs(
            logits.data_ptr(), _ROW_TYPES[logits.dtype], M, V, ld, scale, p_tokens, ldt, G, p_logprobs, p_entropy,
            top_k, p_ids, p_top, p_status, _raw_stream(dev))
    if status != QMM_OK:
        _check("qmm_token_logprobs", status)
    return logprobs, entropy, top_ids, top_logprobs


# ---------------------------------------------------------------------------
# Diagnostics
# ---------------------------------------------------------------------------

def selftest_wait_timeout(limit_ns: int, dev_status: torch.Tensor, out: torch.Tensor):
    """Run the bounded-wait error path on purpose (see qmm_selftest_wait_timeout):
    dev_status (device int32 [1], zeroed by the caller) receives QMM_ERR_TIMEOUT
    and out (device int64 [4]) the wait results and times."""
    _check("qmm_selftest_wait_timeout", lib.qmm_selftest_wait_timeout(int(limit_ns), _ptr(dev_status), _ptr(out),
                                                                      _stream()))
    return out


def probe_hbm_read(buf: torch.Tensor, mode: int, sink: torch.Tensor, dev_status=None):
    """Load-only read of the whole of `buf` (see qmm_probe_hbm_read); sink is a
    device int32/uint32 [1] that normally stays untouched."""
    nbytes = buf.numel() * buf.element_size()
    _check("qmm_probe_hbm_read", lib.qmm_probe_hbm_read(_ptr(buf), nbytes, int(mode), _ptr(sink),
                                                        _ptr(dev_status), _stream()))
