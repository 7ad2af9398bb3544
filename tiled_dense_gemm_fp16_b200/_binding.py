"""ctypes binding of ``libtg_gemm.so`` (the C ABI in ``include/tg_gemm.h``).

Argument marshalling only: every step of C = ReLU(A . B) runs in the CUDA
kernels behind the C ABI.  PyTorch supplies device memory and the current
stream.  There is no fallback: if the library is missing or cannot be loaded,
every call raises.
"""
from __future__ import annotations

import ctypes
import enum
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libtg_gemm.so")


class Status(enum.IntEnum):
    OK = 0
    INVALID_ARG = 1
    UNSUPPORTED_DEVICE = 2
    LAUNCH = 3
    TIMEOUT = 4
    INTERNAL = 5
    TOO_LARGE = 6


class Path(enum.IntEnum):
    INVALID = -2
    NONE = -1
    AUTO = 0
    TC = 1
    TC_EDGE = 2
    SKINNY = 3
    ZERO = 5
    TC_PAIR = 6
    TC_PAIR512 = 7
    REPACK = 8
    RC = 9


class TGError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = Status(status) if status in Status._value2member_map_ else status
        super().__init__(f"{what}: {status_string(status)} ({int(status)})" if what else status_string(status))


A_MK, A_KM = 0, 1
B_KN, B_NK = 0, 1
FP8_E4M3, FP8_E5M2 = 0, 1
TYPE_F16, TYPE_BF16 = 0, 1
ACT_RELU, ACT_SILU, ACT_GELU = 0, 1, 2


class GemmOptions(ctypes.Structure):
    """Mirror of tg_gemm_options (include/tg_gemm.h)."""
    _fields_ = [
        ("lda", ctypes.c_int64),
        ("ldb", ctypes.c_int64),
        ("ldc", ctypes.c_int64),
        ("a_layout", ctypes.c_int32),
        ("b_layout", ctypes.c_int32),
        ("path", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("bias", ctypes.c_void_p),
        ("batch", ctypes.c_int64),
        ("stride_a", ctypes.c_int64),
        ("stride_b", ctypes.c_int64),
        ("stride_c", ctypes.c_int64),
    ]


class GatedOptions(ctypes.Structure):
    """Mirror of tg_gated_options (include/tg_gemm.h)."""
    _fields_ = [
        ("type", ctypes.c_int32),
        ("act", ctypes.c_int32),
        ("ldx", ctypes.c_int64),
        ("ldwg", ctypes.c_int64),
        ("ldwu", ctypes.c_int64),
        ("ldh", ctypes.c_int64),
        ("ldg", ctypes.c_int64),
        ("ldu", ctypes.c_int64),
        ("lddx", ctypes.c_int64),
        ("lddwg", ctypes.c_int64),
        ("lddwu", ctypes.c_int64),
        ("reserved", ctypes.c_int64),
    ]


EXPORTS = (
    "tg_gemm_relu_f16_ex",
    "tg_workspace_size_ex",
    "tg_select_path_ex",
    "tg_gemm_relu_f16",
    "tg_gemm_relu_f16_path",
    "tg_gemm_relu_f16_ws",
    "tg_workspace_size",
    "tg_select_path_ws",
    "tg_gemm_relu_f16_static_ws",
    "tg_select_path",
    "tg_path_supports",
    "tg_device_status",
    "tg_wait_timeout_selftest",
    "tg_status_string",
    "tg_path_name",
    "tg_version",
    "tg_gemm_mxf8_grouped",
    "tg_mx_grouped_rows",
    "tg_mx_scale_bytes",
    "tg_gemm_nvf4_grouped",
    "tg_nvf4_scale_bytes",
    "tg_gemm_relu_w4a16",
    "tg_w4a16_workspace_size",
    "tg_w4a16_kernel",
    "tg_dequant_w4_f16",
    "tg_gated",
    "tg_gated_workspace_size",
    "tg_gated_backward",
    "tg_gated_backward_workspace_size",
    "tg_quantize_rows_i8",
    "tg_gemm_i8",
    "tg_gated_i8",
)

_lib = None
_lock = threading.Lock()


def _bind(lib):
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.tg_gemm_relu_f16.argtypes = [vp, vp, vp, i64, i64, i64, vp]
    lib.tg_gemm_relu_f16.restype = i32
    lib.tg_gemm_relu_f16_path.argtypes = [vp, vp, vp, i64, i64, i64, vp, i32]
    lib.tg_gemm_relu_f16_path.restype = i32
    lib.tg_select_path.argtypes = [vp, vp, vp, i64, i64, i64]
    lib.tg_select_path.restype = i32
    lib.tg_gemm_relu_f16_ws.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, i64]
    lib.tg_gemm_relu_f16_ws.restype = i32
    lib.tg_workspace_size.argtypes = [vp, vp, vp, i64, i64, i64]
    lib.tg_workspace_size.restype = i64
    lib.tg_select_path_ws.argtypes = [vp, vp, vp, i64, i64, i64, i64]
    lib.tg_select_path_ws.restype = i32
    lib.tg_gemm_relu_f16_static_ws.argtypes = [vp, vp, vp, i64, i64, i64, vp]
    lib.tg_gemm_relu_f16_static_ws.restype = i32
    optp = ctypes.POINTER(GemmOptions)
    lib.tg_gemm_relu_f16_ex.argtypes = [vp, vp, vp, i64, i64, i64, optp, vp, vp, i64]
    lib.tg_gemm_relu_f16_ex.restype = i32
    lib.tg_workspace_size_ex.argtypes = [vp, vp, vp, i64, i64, i64, optp]
    lib.tg_workspace_size_ex.restype = i64
    lib.tg_select_path_ex.argtypes = [vp, vp, vp, i64, i64, i64, optp, i64]
    lib.tg_select_path_ex.restype = i32
    lib.tg_path_supports.argtypes = [i32, vp, vp, vp, i64, i64, i64]
    lib.tg_path_supports.restype = i32
    lib.tg_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    lib.tg_device_status.restype = i32
    lib.tg_wait_timeout_selftest.argtypes = [i64, vp]
    lib.tg_wait_timeout_selftest.restype = i32
    lib.tg_status_string.argtypes = [i32]
    lib.tg_status_string.restype = ctypes.c_char_p
    lib.tg_path_name.argtypes = [i32]
    lib.tg_path_name.restype = ctypes.c_char_p
    lib.tg_version.argtypes = []
    lib.tg_version.restype = i32
    i64p = ctypes.POINTER(ctypes.c_int64)
    lib.tg_gemm_mxf8_grouped.argtypes = [vp, vp, vp, vp, vp, i64p, ctypes.c_int32, i64, i64, ctypes.c_int32,
                                         ctypes.c_int32, ctypes.c_int32, vp]
    lib.tg_gemm_mxf8_grouped.restype = i32
    lib.tg_mx_grouped_rows.argtypes = [i64p, ctypes.c_int32]
    lib.tg_mx_grouped_rows.restype = i64
    lib.tg_mx_scale_bytes.argtypes = [i64, i64]
    lib.tg_mx_scale_bytes.restype = i64
    lib.tg_gemm_nvf4_grouped.argtypes = [vp, vp, vp, vp, vp, i64p, ctypes.c_int32, i64, i64, ctypes.c_float,
                                         ctypes.c_int32, vp]
    lib.tg_gemm_nvf4_grouped.restype = i32
    lib.tg_nvf4_scale_bytes.argtypes = [i64, i64]
    lib.tg_nvf4_scale_bytes.restype = i64
    lib.tg_gemm_relu_w4a16.argtypes = [vp, vp, vp, vp, i64, i64, i64, ctypes.c_int32, vp, vp, i64]
    lib.tg_gemm_relu_w4a16.restype = i32
    lib.tg_w4a16_workspace_size.argtypes = [i64, i64, i64, ctypes.c_int32]
    lib.tg_w4a16_workspace_size.restype = i64
    lib.tg_w4a16_kernel.argtypes = [i64, i64, i64, ctypes.c_int32]
    lib.tg_w4a16_kernel.restype = ctypes.c_int
    lib.tg_dequant_w4_f16.argtypes = [vp, vp, vp, i64, i64, ctypes.c_int32, vp]
    lib.tg_dequant_w4_f16.restype = i32
    gop = ctypes.POINTER(GatedOptions)
    lib.tg_gated.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, gop, vp, vp, i64]
    lib.tg_gated.restype = i32
    lib.tg_gated_workspace_size.argtypes = [vp, vp, vp, i64, i64, i64, gop]
    lib.tg_gated_workspace_size.restype = i64
    lib.tg_gated_backward.argtypes = [vp] * 9 + [i64, i64, i64, gop, vp, vp, i64]
    lib.tg_gated_backward.restype = i32
    lib.tg_gated_backward_workspace_size.argtypes = [vp] * 6 + [i64, i64, i64, gop]
    lib.tg_gated_backward_workspace_size.restype = i64
    lib.tg_quantize_rows_i8.argtypes = [vp, vp, vp, i64, i64, i64, i64, ctypes.c_int32, vp]
    lib.tg_quantize_rows_i8.restype = i32
    lib.tg_gemm_i8.argtypes = [vp] * 6 + [i64] * 6 + [ctypes.c_int32, ctypes.c_int32, vp]
    lib.tg_gemm_i8.restype = i32
    lib.tg_gated_i8.argtypes = [vp] * 7 + [i64, i64, i64, gop, vp]
    lib.tg_gated_i8.restype = i32
    return lib


def lib():
    """The loaded C library; raises if ``libtg_gemm.so`` is missing."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise ImportError(
                        f"{LIB_PATH} is not built; run `python -m tiled_dense_gemm_fp16_b200.build` "
                        "(there is no fallback implementation)")
                _lib = _bind(ctypes.CDLL(LIB_PATH))
    return _lib


def status_string(status: int) -> str:
    return lib().tg_status_string(int(status)).decode()


def path_name(path: int) -> str:
    return lib().tg_path_name(int(path)).decode()


def version() -> int:
    return int(lib().tg_version())


def _check(st, what):
    if st != Status.OK:
        raise TGError(st, what)


# ---------------------------------------------------------------------------
# Raw pointer API (mirrors the C ABI one to one)
# ---------------------------------------------------------------------------

def gemm_relu_f16_raw(A: int, B: int, C: int, M: int, N: int, K: int, stream: int = 0, path: int = Path.AUTO) -> int:
    """Call the C ABI on raw device pointers; returns the tg_status value."""
    if int(path) == Path.AUTO:
        return int(lib().tg_gemm_relu_f16(A, B, C, M, N, K, stream))
    return int(lib().tg_gemm_relu_f16_path(A, B, C, M, N, K, stream, int(path)))


def gemm_relu_f16_ws_raw(A: int, B: int, C: int, M: int, N: int, K: int, stream: int, ws: int, ws_bytes: int) -> int:
    """tg_gemm_relu_f16_ws on raw device pointers; returns the tg_status value."""
    return int(lib().tg_gemm_relu_f16_ws(A, B, C, M, N, K, stream, ws, ws_bytes))


def gemm_relu_f16_static_ws_raw(A: int, B: int, C: int, M: int, N: int, K: int, stream: int = 0) -> int:
    """tg_gemm_relu_f16_static_ws on raw device pointers (no allocation anywhere); returns the tg_status."""
    return int(lib().tg_gemm_relu_f16_static_ws(A, B, C, M, N, K, stream))


STATIC_WORKSPACE_BYTES = 16 * 1024 * 1024


def workspace_size(A: int, B: int, C: int, M: int, N: int, K: int) -> int:
    return int(lib().tg_workspace_size(A, B, C, M, N, K))


def options(lda=0, ldb=0, ldc=0, b_layout=B_KN, bias=0, batch=0, stride_a=0, stride_b=0, stride_c=0,
            path=Path.AUTO, a_layout=A_MK, reserved=0) -> GemmOptions:
    """A tg_gemm_options value (zeros mean the dense defaults)."""
    return GemmOptions(lda, ldb, ldc, int(a_layout), int(b_layout), int(path), int(reserved), bias or None, batch,
                       stride_a, stride_b, stride_c)


def gemm_relu_f16_ex_raw(A: int, B: int, C: int, M: int, N: int, K: int, opts: GemmOptions | None = None,
                         stream: int = 0, ws: int = 0, ws_bytes: int = 0) -> int:
    """tg_gemm_relu_f16_ex on raw device pointers; returns the tg_status value."""
    return int(lib().tg_gemm_relu_f16_ex(A, B, C, M, N, K, ctypes.byref(opts) if opts is not None else None,
                                         stream, ws, ws_bytes))


def workspace_size_ex(A: int, B: int, C: int, M: int, N: int, K: int, opts: GemmOptions | None = None) -> int:
    return int(lib().tg_workspace_size_ex(A, B, C, M, N, K, ctypes.byref(opts) if opts is not None else None))


def select_path_ex(A: int, B: int, C: int, M: int, N: int, K: int, opts: GemmOptions | None = None,
                   ws_bytes: int = 0) -> int:
    return int(lib().tg_select_path_ex(A, B, C, M, N, K, ctypes.byref(opts) if opts is not None else None, ws_bytes))


def select_path(A: int, B: int, C: int, M: int, N: int, K: int) -> int:
    return int(lib().tg_select_path(A, B, C, M, N, K))


def select_path_ws(A: int, B: int, C: int, M: int, N: int, K: int, ws_bytes: int) -> int:
    return int(lib().tg_select_path_ws(A, B, C, M, N, K, ws_bytes))


def path_supports(path: int, A: int, B: int, C: int, M: int, N: int, K: int) -> bool:
    return bool(lib().tg_path_supports(int(path), A, B, C, M, N, K))


def device_status():
    """(Status, raw error word) after synchronizing the current device."""
    word = ctypes.c_uint32(0)
    st = int(lib().tg_device_status(ctypes.byref(word)))
    return Status(st), int(word.value)


def wait_timeout_selftest(budget_ns: int, stream: int = 0) -> int:
    return int(lib().tg_wait_timeout_selftest(int(budget_ns), stream))


# ---------------------------------------------------------------------------
# torch tensor API
# ---------------------------------------------------------------------------

def _stream_handle(device):
    import torch
    return torch.cuda.current_stream(device).cuda_stream


def gemm_relu(A, B, out=None, path: int = Path.AUTO, stream=None, workspace="auto"):
    """C = ReLU(A @ B) for row-major fp16 CUDA tensors A (M, K) and B (K, N).

    ``out`` (M, N) fp16 on the same device is written in place if given.
    Runs on ``stream`` (a torch.cuda.Stream) or on the current stream.
    ``workspace``: "auto" lets torch allocate the scratch bytes the repack path
    needs when TMA cannot describe A or B (odd row lengths, unaligned bases);
    None never uses a workspace (edge mode instead); a uint8 CUDA tensor is
    used as given.  The library itself allocates nothing at run time.
    """
    import torch
    if A.dtype != torch.float16 or B.dtype != torch.float16:
        raise TypeError("A and B must be torch.float16")
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[0]:
        raise ValueError(f"shape mismatch: A{tuple(A.shape)} B{tuple(B.shape)}")
    if not (A.is_cuda and B.is_cuda) or A.device != B.device:
        raise ValueError("A and B must be CUDA tensors on the same device")
    if not (A.is_contiguous() and B.is_contiguous()):
        raise ValueError("A and B must be contiguous row-major tensors")
    M, K = A.shape
    N = B.shape[1]
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=A.device)
    elif (out.dtype != torch.float16 or tuple(out.shape) != (M, N) or not out.is_contiguous()
          or out.device != A.device):
        raise ValueError("out must be a contiguous (M, N) float16 tensor on A's device")
    handle = stream.cuda_stream if stream is not None else _stream_handle(A.device)
    a, b, c = A.data_ptr(), B.data_ptr(), out.data_ptr()
    with torch.cuda.device(A.device):
        if int(path) == Path.AUTO and workspace is not None:
            need = workspace_size(a, b, c, M, N, K)
            if need > 0:
                if isinstance(workspace, str):
                    workspace = torch.empty(need, dtype=torch.uint8, device=A.device)
                st = gemm_relu_f16_ws_raw(a, b, c, M, N, K, handle, workspace.data_ptr(), workspace.numel())
                _check(st, "tg_gemm_relu_f16_ws")
                return out
        st = gemm_relu_f16_raw(a, b, c, M, N, K, handle, path)
    _check(st, "tg_gemm_relu_f16")
    return out


def _call_ex(a, b, c, M, N, K, opts, device, stream, workspace):
    import torch
    handle = stream.cuda_stream if stream is not None else _stream_handle(device)
    with torch.cuda.device(device):
        need = workspace_size_ex(a, b, c, M, N, K, opts)
        if need < 0:
            raise TGError(Status.INVALID_ARG, "tg_workspace_size_ex")
        ws_ptr, ws_bytes = 0, 0
        if need > 0 and workspace is not None:
            if isinstance(workspace, str):
                workspace = torch.empty(need, dtype=torch.uint8, device=device)
            ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel()
        st = gemm_relu_f16_ex_raw(a, b, c, M, N, K, opts, handle, ws_ptr, ws_bytes)
    _check(st, "tg_gemm_relu_f16_ex")


def linear_relu(x, weight, bias=None, out=None, stream=None, workspace="auto"):
    """ReLU(x @ weight^T + bias) for fp16 CUDA tensors: x (..., K), weight (N, K) as a
    linear layer stores it, bias (N,) or None.  Leading dimensions of x are flattened
    into M rows (x must be contiguous)."""
    import torch
    if x.dtype != torch.float16 or weight.dtype != torch.float16:
        raise TypeError("x and weight must be torch.float16")
    if weight.dim() != 2 or x.shape[-1] != weight.shape[1]:
        raise ValueError(f"shape mismatch: x{tuple(x.shape)} weight{tuple(weight.shape)}")
    if not (x.is_contiguous() and weight.is_contiguous()):
        raise ValueError("x and weight must be contiguous")
    K = x.shape[-1]
    N = weight.shape[0]
    lead = tuple(x.shape[:-1])
    M = 1
    for d in lead:
        M *= d
    if bias is not None and (bias.dtype != torch.float16 or bias.numel() != N or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous float16 tensor of N elements")
    if out is None:
        out = torch.empty(lead + (N,), dtype=torch.float16, device=x.device)
    opts = options(b_layout=B_NK, bias=bias.data_ptr() if bias is not None else 0)
    _call_ex(x.data_ptr(), weight.data_ptr(), out.data_ptr(), M, N, K, opts, x.device, stream, workspace)
    return out


def bmm_relu(A, B, bias=None, out=None, stream=None, workspace="auto"):
    """ReLU(A[e] @ B[e] + bias) for fp16 CUDA tensors A (b, M, K) and B (b, K, N)."""
    import torch
    if A.dim() != 3 or B.dim() != 3 or A.shape[0] != B.shape[0] or A.shape[2] != B.shape[1]:
        raise ValueError(f"shape mismatch: A{tuple(A.shape)} B{tuple(B.shape)}")
    if A.dtype != torch.float16 or B.dtype != torch.float16 or not (A.is_contiguous() and B.is_contiguous()):
        raise ValueError("A and B must be contiguous float16 tensors")
    nb, M, K = A.shape
    N = B.shape[2]
    if out is None:
        out = torch.empty((nb, M, N), dtype=torch.float16, device=A.device)
    opts = options(bias=bias.data_ptr() if bias is not None else 0, batch=nb, stride_a=M * K, stride_b=K * N,
                   stride_c=M * N)
    _call_ex(A.data_ptr(), B.data_ptr(), out.data_ptr(), M, N, K, opts, A.device, stream, workspace)
    return out


# ---------------------------------------------------------------------------
# MXFP8 grouped GEMM
# ---------------------------------------------------------------------------

def _i64_array(values):
    values = [int(v) for v in values]
    return (ctypes.c_int64 * max(1, len(values)))(*values), len(values)


def mx_grouped_rows(m_sizes) -> int:
    """Stacked rows of A / C for these group sizes (each group padded to 128 rows); -1 if invalid."""
    arr, n = _i64_array(m_sizes)
    return int(lib().tg_mx_grouped_rows(arr, n))


def mx_scale_bytes(rows: int, K: int) -> int:
    """Bytes of one blocked UE8M0 scale array for ``rows`` rows and K elements."""
    return int(lib().tg_mx_scale_bytes(rows, K))


def gemm_mxf8_grouped_raw(A: int, SFA: int, B: int, SFB: int, C: int, m_sizes, N: int, K: int,
                          a_format: int = FP8_E4M3, b_format: int = FP8_E4M3, relu: bool = False,
                          stream: int = 0) -> int:
    arr, n = _i64_array(m_sizes)
    return int(lib().tg_gemm_mxf8_grouped(A, SFA, B, SFB, C, arr, n, N, K, int(a_format), int(b_format),
                                          1 if relu else 0, stream))


def mxf8_grouped(A, SFA, B, SFB, m_sizes, relu=False, a_format=FP8_E4M3, b_format=FP8_E4M3, out=None,
                 stream=None):
    """Grouped MXFP8 GEMM on CUDA tensors (uint8 codes): A (rows, K), B (G, N, K), SFA / SFB in the
    blocked scale layout; returns C (rows, N) bfloat16 (rows outside the groups untouched)."""
    import torch
    if A.dim() != 2 or B.dim() != 3 or A.shape[1] != B.shape[2] or B.shape[0] != len(m_sizes):
        raise ValueError(f"shape mismatch: A{tuple(A.shape)} B{tuple(B.shape)} groups={len(m_sizes)}")
    rows, K = A.shape
    N = B.shape[1]
    if rows != mx_grouped_rows(m_sizes):
        raise ValueError("A must have tg_mx_grouped_rows(m_sizes) rows")
    for t in (A, B, SFA, SFB):
        if t.dtype != torch.uint8 or not t.is_contiguous():
            raise TypeError("operands and scales must be contiguous uint8 tensors")
    if out is None:
        out = torch.empty((rows, N), dtype=torch.bfloat16, device=A.device)
    handle = stream.cuda_stream if stream is not None else _stream_handle(A.device)
    with torch.cuda.device(A.device):
        st = gemm_mxf8_grouped_raw(A.data_ptr(), SFA.data_ptr(), B.data_ptr(), SFB.data_ptr(), out.data_ptr(),
                                   m_sizes, N, K, a_format, b_format, relu, handle)
    _check(st, "tg_gemm_mxf8_grouped")
    return out


# ---------------------------------------------------------------------------
# NVF4 grouped GEMM
# ---------------------------------------------------------------------------

def nvf4_scale_bytes(rows: int, K: int) -> int:
    """Bytes of one blocked UE4M3 scale array for ``rows`` rows and K elements."""
    return int(lib().tg_nvf4_scale_bytes(rows, K))


def gemm_nvf4_grouped_raw(A: int, SFA: int, B: int, SFB: int, C: int, m_sizes, N: int, K: int, alpha: float = 1.0,
                          relu: bool = False, stream: int = 0) -> int:
    arr, n = _i64_array(m_sizes)
    return int(lib().tg_gemm_nvf4_grouped(A, SFA, B, SFB, C, arr, n, N, K, float(alpha), 1 if relu else 0, stream))


def nvf4_grouped(A, SFA, B, SFB, m_sizes, alpha=1.0, relu=False, out=None, stream=None):
    """Grouped NVF4 GEMM on CUDA uint8 tensors: A (rows, K/2) and B (G, N, K/2) packed E2M1, SFA / SFB
    blocked UE4M3 scales; returns C (rows, N) bfloat16 (rows outside the groups untouched)."""
    import torch
    if A.dim() != 2 or B.dim() != 3 or A.shape[1] != B.shape[2] or B.shape[0] != len(m_sizes):
        raise ValueError(f"shape mismatch: A{tuple(A.shape)} B{tuple(B.shape)} groups={len(m_sizes)}")
    rows, K = A.shape[0], 2 * A.shape[1]
    N = B.shape[1]
    if rows != mx_grouped_rows(m_sizes):
        raise ValueError("A must have tg_mx_grouped_rows(m_sizes) rows")
    for t in (A, B, SFA, SFB):
        if t.dtype != torch.uint8 or not t.is_contiguous():
            raise TypeError("operands and scales must be contiguous uint8 tensors")
    if out is None:
        out = torch.empty((rows, N), dtype=torch.bfloat16, device=A.device)
    handle = stream.cuda_stream if stream is not None else _stream_handle(A.device)
    with torch.cuda.device(A.device):
        st = gemm_nvf4_grouped_raw(A.data_ptr(), SFA.data_ptr(), B.data_ptr(), SFB.data_ptr(), out.data_ptr(),
                                   m_sizes, N, K, alpha, relu, handle)
    _check(st, "tg_gemm_nvf4_grouped")
    return out


# ---------------------------------------------------------------------------
# 4-bit weight-only GEMM (W4A16)
# ---------------------------------------------------------------------------

def w4a16_workspace_size(M: int, N: int, K: int, group: int) -> int:
    return int(lib().tg_w4a16_workspace_size(M, N, K, group))


class W4Kernel(enum.IntEnum):
    INVALID = -1
    NONE = 0
    DECODE = 1
    FUSED = 2
    DEQUANT_GEMM = 3


def w4a16_kernel(M: int, N: int, K: int, group: int) -> "W4Kernel":
    """The kernels tg_gemm_relu_w4a16 runs for these sizes (host logic only)."""
    return W4Kernel(int(lib().tg_w4a16_kernel(M, N, K, group)))


def gemm_relu_w4a16_raw(A: int, Wq: int, S: int, C: int, M: int, N: int, K: int, group: int, stream: int = 0,
                        workspace: int = 0, workspace_bytes: int = 0) -> int:
    return int(lib().tg_gemm_relu_w4a16(A, Wq, S, C, M, N, K, group, stream, workspace, workspace_bytes))


def dequant_w4_f16_raw(Wq: int, S: int, W: int, N: int, K: int, group: int, stream: int = 0) -> int:
    return int(lib().tg_dequant_w4_f16(Wq, S, W, N, K, group, stream))


def gemm_relu_w4a16(A, Wq, S, group, out=None, stream=None, workspace="auto"):
    """ReLU(A @ dequant(W)^T) for CUDA tensors: A (M, K) float16, Wq (N, K/2) uint8 packed codes,
    S (N, K/group) float16 scales; returns C (M, N) float16."""
    import torch
    if A.dim() != 2 or Wq.dim() != 2 or S.dim() != 2 or Wq.shape[1] * 2 != A.shape[1] or S.shape[0] != Wq.shape[0]:
        raise ValueError(f"shape mismatch: A{tuple(A.shape)} Wq{tuple(Wq.shape)} S{tuple(S.shape)}")
    if A.dtype != torch.float16 or S.dtype != torch.float16 or Wq.dtype != torch.uint8:
        raise TypeError("A and S must be float16, Wq uint8")
    if not (A.is_contiguous() and Wq.is_contiguous() and S.is_contiguous()):
        raise ValueError("A, Wq and S must be contiguous")
    M, K = A.shape
    N = Wq.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=A.device)
    handle = stream.cuda_stream if stream is not None else _stream_handle(A.device)
    with torch.cuda.device(A.device):
        need = w4a16_workspace_size(M, N, K, group)
        if need < 0:
            raise TGError(Status.INVALID_ARG, "tg_w4a16_workspace_size")
        ws_ptr, ws_bytes = 0, 0
        if need > 0 and workspace is not None:
            if isinstance(workspace, str):
                workspace = torch.empty(need, dtype=torch.uint8, device=A.device)
            ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel()
        st = gemm_relu_w4a16_raw(A.data_ptr(), Wq.data_ptr(), S.data_ptr(), out.data_ptr(), M, N, K, group, handle,
                                 ws_ptr, ws_bytes)
    _check(st, "tg_gemm_relu_w4a16")
    return out


# ---------------------------------------------------------------------------
# Gated feed-forward block and 8-bit integer products
# ---------------------------------------------------------------------------

_ACTS = {"relu": ACT_RELU, "silu": ACT_SILU, "gelu": ACT_GELU}


def gated_options(type=TYPE_F16, act=ACT_RELU, ldx=0, ldwg=0, ldwu=0, ldh=0, ldg=0, ldu=0, lddx=0, lddwg=0, lddwu=0,
                  reserved=0) -> GatedOptions:
    """A tg_gated_options value (zeros mean fp16, ReLU and dense rows)."""
    return GatedOptions(int(type), int(act), ldx, ldwg, ldwu, ldh, ldg, ldu, lddx, lddwg, lddwu, reserved)


def _ref(opts):
    return ctypes.byref(opts) if opts is not None else None


def gated_raw(X: int, Wg: int, Wu: int, H: int, G: int, U: int, M: int, N: int, K: int,
              opts: GatedOptions | None = None, stream: int = 0, ws: int = 0, ws_bytes: int = 0) -> int:
    """tg_gated on raw device pointers; returns the tg_status value."""
    return int(lib().tg_gated(X, Wg, Wu, H, G, U, M, N, K, _ref(opts), stream, ws, ws_bytes))


def gated_workspace_size(X: int, Wg: int, Wu: int, M: int, N: int, K: int, opts: GatedOptions | None = None) -> int:
    return int(lib().tg_gated_workspace_size(X, Wg, Wu, M, N, K, _ref(opts)))


def gated_backward_raw(dH: int, X: int, Wg: int, Wu: int, G: int, U: int, dX: int, dWg: int, dWu: int, M: int, N: int,
                       K: int, opts: GatedOptions | None = None, stream: int = 0, ws: int = 0,
                       ws_bytes: int = 0) -> int:
    """tg_gated_backward on raw device pointers; returns the tg_status value."""
    return int(lib().tg_gated_backward(dH, X, Wg, Wu, G, U, dX, dWg, dWu, M, N, K, _ref(opts), stream, ws, ws_bytes))


def gated_backward_workspace_size(X: int, Wg: int, Wu: int, dX: int, dWg: int, dWu: int, M: int, N: int, K: int,
                                  opts: GatedOptions | None = None) -> int:
    return int(lib().tg_gated_backward_workspace_size(X, Wg, Wu, dX, dWg, dWu, M, N, K, _ref(opts)))


def quantize_rows_i8_raw(X: int, Q: int, scales: int, M: int, K: int, ldx: int = 0, ldq: int = 0,
                         type: int = TYPE_F16, stream: int = 0) -> int:
    return int(lib().tg_quantize_rows_i8(X, Q, scales, M, K, ldx, ldq, int(type), stream))


def gemm_i8_raw(A: int, a_scale: int, W: int, w_scale: int, bias: int, C: int, M: int, N: int, K: int, lda: int = 0,
                ldw: int = 0, ldc: int = 0, relu: bool = False, type: int = TYPE_F16, stream: int = 0) -> int:
    return int(lib().tg_gemm_i8(A, a_scale, W, w_scale, bias, C, M, N, K, lda, ldw, ldc, 1 if relu else 0, int(type),
                                stream))


def gated_i8_raw(A: int, a_scale: int, Wg: int, g_scale: int, Wu: int, u_scale: int, H: int, M: int, N: int, K: int,
                 opts: GatedOptions | None = None, stream: int = 0) -> int:
    return int(lib().tg_gated_i8(A, a_scale, Wg, g_scale, Wu, u_scale, H, M, N, K, _ref(opts), stream))


def _type_code(dtype):
    import torch
    if dtype == torch.float16:
        return TYPE_F16
    if dtype == torch.bfloat16:
        return TYPE_BF16
    raise TypeError(f"expected torch.float16 or torch.bfloat16, got {dtype}")


def _act_code(act):
    try:
        return _ACTS[act]
    except KeyError:
        raise ValueError(f"unknown activation {act!r}; one of {sorted(_ACTS)}") from None


def _row_stride(t, name):
    """Elements between the rows of a 2-D tensor whose columns are adjacent (0: dense or a single row)."""
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have adjacent columns (stride 1), got strides {t.stride()}")
    if rows <= 1 or cols == 0:
        return 0
    if t.stride(0) < cols:
        raise ValueError(f"{name} has overlapping rows: strides {t.stride()} for shape {tuple(t.shape)}")
    return t.stride(0)


def _matrix(t, name, shape, dtype, device):
    """Check a 2-D operand; returns its row stride (0: dense)."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return _row_stride(t, name)


def _vector(t, name, n, dtype, device):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != n or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be {n} contiguous values on {device}")
    return t.data_ptr()


def _flat(t, name):
    """(..., K) as (rows, K), without a copy."""
    if t.dim() < 1 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor with at least one dimension")
    if t.dim() == 2:
        return t
    rows = 1
    for d in t.shape[:-1]:
        rows *= d
    try:
        return t.view(rows, t.shape[-1])
    except RuntimeError:
        raise ValueError(f"{name}: the leading dimensions of shape {tuple(t.shape)} with strides {t.stride()} "
                         "are not evenly spaced rows") from None


def _on(device, stream, *tensors):
    """Context in which a call runs and allocates: `stream`, or the device's current stream.

    Tensors made on another stream are recorded on `stream`, so that their memory is not reused
    before the call's work is done (making the streams wait for each other stays the caller's part)."""
    import contextlib

    import torch
    if stream is None:
        return contextlib.nullcontext() if torch.cuda.current_device() == device.index else torch.cuda.device(device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    if stream != torch.cuda.current_stream(device):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    return torch.cuda.stream(stream)


def _scratch(workspace, need, device):
    """(pointer, bytes) of the workspace of a call that needs `need` bytes, and the tensor that holds it."""
    import torch
    if need < 0:
        raise TGError(Status.INVALID_ARG, "workspace size")
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 CUDA tensor")
        if need == 0:
            return 0, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if workspace is None:
        return 0, 0, None
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != device:
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    return workspace.data_ptr(), workspace.numel(), workspace


def _given(workspace):
    return None if workspace is None or isinstance(workspace, str) else workspace


def gated(x, w_gate, w_up, act="silu", out=None, save=False, stream=None, workspace="auto"):
    """act(x @ w_gate^T) * (x @ w_up^T) for float16 or bfloat16 CUDA tensors: x (..., K), w_gate and
    w_up (N, K) as linear layers store them (the halves of one (2N, K) weight do too).

    ``act``: "silu", "gelu" (tanh form) or "relu".  Returns H (..., N); with ``save`` the tuple
    (H, gate, up) with the two projections, which ``gated_backward`` takes.  ``out`` receives H.
    Rows may have any stride; ``workspace`` (as for ``gemm_relu``) is needed only where a row stride or
    base is off 16 bytes.  ``gated_block`` is the same under autograd.
    """
    import torch
    x2 = _flat(x, "x")
    M, K = x2.shape
    dtype, device = x.dtype, x.device
    code = _type_code(dtype)
    if w_gate.dim() != 2:
        raise ValueError(f"w_gate must be (N, K), got {tuple(w_gate.shape)}")
    N = w_gate.shape[0]
    opts = GatedOptions(code, _act_code(act), _row_stride(x2, "x"), _matrix(w_gate, "w_gate", (N, K), dtype, device),
                        _matrix(w_up, "w_up", (N, K), dtype, device))
    lead = x.shape[:-1]
    out2 = None
    if out is not None:
        if tuple(out.shape) != (*lead, N):
            raise ValueError(f"out must have shape {(*lead, N)}, got {tuple(out.shape)}")
        out2 = _flat(out, "out")
        opts.ldh = _matrix(out2, "out", (M, N), dtype, device)
    with _on(device, stream, x, w_gate, w_up, out, _given(workspace)):
        if out is None:
            out = out2 = torch.empty((M, N), dtype=dtype, device=device)
            if x.dim() != 2:
                out = out2.view(*lead, N)
        gate = up = None
        if save:
            gate, up = torch.empty((2, M, N), dtype=dtype, device=device)
        ptrs = (x2.data_ptr(), w_gate.data_ptr(), w_up.data_ptr())
        ws, ws_bytes, held = _scratch(workspace, gated_workspace_size(*ptrs, M, N, K, opts), device)
        st = gated_raw(*ptrs, out2.data_ptr(), gate.data_ptr() if save else 0, up.data_ptr() if save else 0, M, N, K,
                       opts, _stream_handle(device), ws, ws_bytes)
    _check(st, "tg_gated")
    return (out, gate.view(*lead, N), up.view(*lead, N)) if save else out


def gated_backward(grad, x, w_gate, w_up, gate, up, act="silu", needs=(True, True, True), stream=None,
                   workspace="auto"):
    """Gradients of ``gated`` for grad = dH (..., N), with the projections that ``gated(..., save=True)``
    returned: (dx, dw_gate, dw_up), None where ``needs`` is false.

    ``workspace``: "auto" lets torch allocate the bytes for dG and dU; a uint8 CUDA tensor is used as
    given (calls whose work may overlap need one each).
    """
    import torch
    x2 = _flat(x, "x")
    M, K = x2.shape
    dtype, device = x.dtype, x.device
    code = _type_code(dtype)
    if w_gate.dim() != 2:
        raise ValueError(f"w_gate must be (N, K), got {tuple(w_gate.shape)}")
    N = w_gate.shape[0]
    grad2, gate2, up2 = _flat(grad, "grad"), _flat(gate, "gate"), _flat(up, "up")
    opts = GatedOptions(code, _act_code(act), _row_stride(x2, "x"), _matrix(w_gate, "w_gate", (N, K), dtype, device),
                        _matrix(w_up, "w_up", (N, K), dtype, device), _matrix(grad2, "grad", (M, N), dtype, device),
                        _matrix(gate2, "gate", (M, N), dtype, device), _matrix(up2, "up", (M, N), dtype, device))
    need_x, need_g, need_u = needs
    with _on(device, stream, grad, x, w_gate, w_up, gate, up, _given(workspace)):
        dx = torch.empty((M, K), dtype=dtype, device=device) if need_x else None
        dwg = torch.empty((N, K), dtype=dtype, device=device) if need_g else None
        dwu = torch.empty((N, K), dtype=dtype, device=device) if need_u else None
        grads = [t.data_ptr() if t is not None else 0 for t in (dx, dwg, dwu)]
        ins = (x2.data_ptr(), w_gate.data_ptr(), w_up.data_ptr())
        ws, ws_bytes, held = _scratch(workspace, gated_backward_workspace_size(*ins, *grads, M, N, K, opts), device)
        st = gated_backward_raw(grad2.data_ptr(), *ins, gate2.data_ptr(), up2.data_ptr(), *grads, M, N, K, opts,
                                _stream_handle(device), ws, ws_bytes)
    _check(st, "tg_gated_backward")
    return (dx.view(x.shape) if need_x else None), dwg, dwu


def gated_block(x, w_gate, w_up, act="silu"):
    """``gated`` under autograd: gradients reach x, w_gate and w_up (those that ask for one).

    Runs on the current stream.  Without gradients to take, no projection is stored."""
    from .autograd import gated_block as impl
    return impl(x, w_gate, w_up, act)


def quantize_i8(x, out=None, scales=None, stream=None):
    """Rows of x (..., K), float16 or bfloat16, as 8-bit integers with one scale each: (codes, scales) with
    codes (..., K) int8 and scales (...) float32, scale = max |x| / 127, codes = x / scale rounded to
    nearest even.  Rows of codes that the call allocates start on 16-byte boundaries whatever K is, as
    ``gemm_i8`` and ``gated_i8`` want them.  Serves activations (a row is a token) and weights (a row is
    a channel).  Rows of zeros: scale 0.  Rows with an infinity or a NaN: scale NaN, codes 0."""
    import torch
    x2 = _flat(x, "x")
    M, K = x2.shape
    device, lead = x.device, x.shape[:-1]
    code, ldx = _type_code(x.dtype), _row_stride(x2, "x")
    out2 = None
    if out is not None:
        if out.shape != x.shape:
            raise ValueError(f"out must have shape {tuple(x.shape)}, got {tuple(out.shape)}")
        out2 = _flat(out, "out")
        ldq = _matrix(out2, "out", (M, K), torch.int8, device)
    if scales is not None:
        _vector(scales, "scales", M, torch.float32, device)
    with _on(device, stream, x, out, scales):
        if out is None:
            ldq = (K + 15) // 16 * 16
            stored = torch.empty((M, ldq), dtype=torch.int8, device=device)
            out2 = stored[:, :K] if ldq != K else stored
            out = out2 if x.dim() == 2 else stored.view(*lead, ldq)[..., :K]
        if scales is None:
            scales = torch.empty(lead, dtype=torch.float32, device=device)
        st = quantize_rows_i8_raw(x2.data_ptr(), out2.data_ptr(), scales.data_ptr(), M, K, ldx, ldq, code,
                                  _stream_handle(device))
    _check(st, "tg_quantize_rows_i8")
    return out, scales


def gemm_i8(a, a_scale, w, w_scale, bias=None, relu=False, dtype=None, out=None, stream=None):
    """(a @ w^T) * a_scale * w_scale + bias, with an optional ReLU, for int8 CUDA tensors a (..., K) and
    w (N, K) with a float32 scale for each of their rows; bias (N,) of the result's type.

    Returns (..., N) of ``dtype`` (float16 unless given, or ``out``'s).  The integer sums are exact.
    Rows of a and w must start on 16-byte boundaries (as those of ``quantize_i8`` do)."""
    import torch
    a2 = _flat(a, "a")
    M, K = a2.shape
    device, lead = a.device, a.shape[:-1]
    if w.dim() != 2:
        raise ValueError(f"w must be (N, K), got {tuple(w.shape)}")
    N = w.shape[0]
    lda, ldw = _matrix(a2, "a", (M, K), torch.int8, device), _matrix(w, "w", (N, K), torch.int8, device)
    sa, sw = _vector(a_scale, "a_scale", M, torch.float32, device), _vector(w_scale, "w_scale", N, torch.float32, device)
    out2, ldc, dtype = _result(out, dtype, lead, M, N, device)
    code = _type_code(dtype)
    b = _vector(bias, "bias", N, dtype, device) if bias is not None else 0
    with _on(device, stream, a, a_scale, w, w_scale, bias, out):
        if out is None:
            out2 = torch.empty((M, N), dtype=dtype, device=device)
            out = out2 if a.dim() == 2 else out2.view(*lead, N)
        st = gemm_i8_raw(a2.data_ptr(), sa, w.data_ptr(), sw, b, out2.data_ptr(), M, N, K, lda, ldw, ldc, relu, code,
                         _stream_handle(device))
    _check(st, "tg_gemm_i8")
    return out


def _result(out, dtype, lead, M, N, device):
    """(2-D view of `out` or None, its row stride, result type)."""
    import torch
    if out is None:
        return None, 0, dtype if dtype is not None else torch.float16
    if tuple(out.shape) != (*lead, N):
        raise ValueError(f"out must have shape {(*lead, N)}, got {tuple(out.shape)}")
    if dtype is None:
        dtype = out.dtype
    out2 = _flat(out, "out")
    return out2, _matrix(out2, "out", (M, N), dtype, device), dtype


def gated_i8(a, a_scale, w_gate, gate_scale, w_up, up_scale, act="silu", dtype=None, out=None, stream=None):
    """``gated`` on 8-bit operands: a (..., K) int8 with a scale a row, w_gate and w_up (N, K) int8 with a
    scale a row.  Returns (..., N) of ``dtype`` (float16 unless given, or ``out``'s).  Operands as for
    ``gemm_i8``."""
    import torch
    a2 = _flat(a, "a")
    M, K = a2.shape
    device, lead = a.device, a.shape[:-1]
    if w_gate.dim() != 2:
        raise ValueError(f"w_gate must be (N, K), got {tuple(w_gate.shape)}")
    N = w_gate.shape[0]
    out2, ldh, dtype = _result(out, dtype, lead, M, N, device)
    opts = GatedOptions(_type_code(dtype), _act_code(act), _matrix(a2, "a", (M, K), torch.int8, device),
                        _matrix(w_gate, "w_gate", (N, K), torch.int8, device),
                        _matrix(w_up, "w_up", (N, K), torch.int8, device), ldh)
    sa = _vector(a_scale, "a_scale", M, torch.float32, device)
    sg = _vector(gate_scale, "gate_scale", N, torch.float32, device)
    su = _vector(up_scale, "up_scale", N, torch.float32, device)
    with _on(device, stream, a, a_scale, w_gate, gate_scale, w_up, up_scale, out):
        if out is None:
            out2 = torch.empty((M, N), dtype=dtype, device=device)
            out = out2 if a.dim() == 2 else out2.view(*lead, N)
        st = gated_i8_raw(a2.data_ptr(), sa, w_gate.data_ptr(), sg, w_up.data_ptr(), su, out2.data_ptr(), M, N, K,
                          opts, _stream_handle(device))
    _check(st, "tg_gated_i8")
    return out
