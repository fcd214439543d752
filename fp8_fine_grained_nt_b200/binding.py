"""Python binding over the C-ABI library ``libfp8nt.so`` (declared in include/fp8_nt.h).

Argument marshalling only: each call checks dtypes, devices and shapes, passes
raw device pointers, sizes and the current CUDA stream to the library, and
raises ``Fp8NtError`` on a nonzero status.  Every step of the GEMM runs in the
library's kernels.  The library is loaded on first use; if it is missing or
fails to load, the call raises (there is no fallback).  The grouped operators,
which may take a few microseconds on the GPU, go through the extension module
``_torch_calls``, which makes the same checks faster; a call that fails one (or
names a stream, a workspace or another device) comes back to the code here.
"""

from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import Optional

import torch

__all__ = [
    "Fp8NtError",
    "library_path",
    "load_library",
    "gemm_fp8_fp8_bf16_nt",
    "gemm_fp8_fp8_bf16_nt_per_tensor",
    "quantize_fp8_1x128",
    "m_grouped_gemm_fp8_fp8_bf16_nt_contiguous",
    "m_grouped_gemm_fp8_fp8_bf16_nt_masked",
    "m_grouped_gemm_nt_ragged",
    "m_grouped_gemm_nn_ragged",
    "k_grouped_gemm_tn_ragged",
    "group_rows_by_index",
    "get_row_groups_capacity",
    "get_group_rows_workspace_size",
    "m_grouped_lora_add",
    "get_lora_workspace_size",
    "get_m_alignment_for_contiguous_layout",
    "get_tma_aligned_size",
    "get_col_major_tma_aligned_tensor",
    "set_num_sms",
    "get_num_sms",
    "get_device_status",
    "selftest_wait_timeout",
    "select_config",
    "force_config",
    "force_swap_ab",
    "force_tail_split",
    "force_ragged",
    "status_string",
    "KIND_DENSE",
    "KIND_CONTIGUOUS",
    "KIND_MASKED",
    "KIND_DENSE_PER_TENSOR",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libfp8nt.so"
_lock = threading.Lock()
_lib = None
_calls = None  # the extension module

KIND_DENSE, KIND_CONTIGUOUS, KIND_MASKED, KIND_DENSE_PER_TENSOR = 0, 1, 2, 3


class Fp8NtError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class DgConfig(ctypes.Structure):
    _fields_ = [("block_m", ctypes.c_int), ("block_n", ctypes.c_int),
                ("stages", ctypes.c_int),
                ("num_tiles", ctypes.c_int), ("grid", ctypes.c_int),
                ("smem_bytes", ctypes.c_int), ("tmem_cols", ctypes.c_int),
                ("split", ctypes.c_int), ("cta_pair", ctypes.c_int),
                ("swap_ab", ctypes.c_int), ("tail_tiles", ctypes.c_int)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


def library_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def load_library():
    """Load libfp8nt.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with "
                              "`python -m fp8_fine_grained_nt_b200.build`")
        lib = ctypes.CDLL(path)
        P, I = ctypes.c_void_p, ctypes.c_int
        lib.gemm_fp8_fp8_bf16_nt.argtypes = [P, P, P, P, P, I, I, I, P]
        lib.gemm_fp8_fp8_bf16_nt_per_tensor.argtypes = [P, P, P, P, P, I, I, I, P]
        lib.quantize_fp8_1x128.argtypes = [P, I, P, P, I, I, P]
        lib.dg_selftest_wait_timeout.argtypes = [I, P]
        lib.m_grouped_gemm_fp8_fp8_bf16_nt_contiguous.argtypes = [P, P, P, P, P, P, I, I, I, I, P]
        lib.m_grouped_gemm_fp8_fp8_bf16_nt_masked.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P]
        lib.get_m_alignment_for_contiguous_layout.argtypes = []
        lib.get_tma_aligned_size.argtypes = [I, I]
        lib.set_num_sms.argtypes = [I]
        lib.get_num_sms.argtypes = []
        lib.dg_status_string.argtypes = [I]
        lib.dg_status_string.restype = ctypes.c_char_p
        lib.dg_get_device_status.argtypes = [P]
        lib.dg_select_config.argtypes = [I, I, I, I, I, I, I, ctypes.POINTER(DgConfig)]
        lib.dg_force_config.argtypes = [I, I, I, I]
        lib.dg_force_swap_ab.argtypes = [I]
        lib.dg_force_tail_split.argtypes = [I]
        lib.m_grouped_gemm_nt_ragged.argtypes = [P, P, P, P, I, I, I, I, I, P]
        lib.m_grouped_gemm_nn_ragged.argtypes = [P, P, P, P, I, I, I, I, I, P]
        lib.k_grouped_gemm_tn_ragged.argtypes = [P, P, P, P, I, I, I, I, I, I, I, P]
        Z, L = ctypes.c_size_t, ctypes.c_longlong
        lib.group_rows_by_index.argtypes = [P, I, P, P, P, P, I, I, I, P, Z, P]
        lib.get_row_groups_capacity.argtypes = [I, I, I]
        lib.get_group_rows_workspace_size.argtypes = [I, I]
        lib.get_group_rows_workspace_size.restype = L
        lib.m_grouped_lora_add.argtypes = [P, L, P, P, P, P, L, P, L, P, P, I, I, I, I, I, I, I, P,
                                           Z, P]
        lib.get_lora_workspace_size.argtypes = [I, I, I, I, I]
        lib.get_lora_workspace_size.restype = L
        lib.dg_force_ragged.argtypes = [I, I, I, I]
        _lib = lib
        return lib


def _load_calls():
    """Load the extension module beside libfp8nt.so (raises if it has not been built)."""
    global _calls
    load_library()  # first: it is the library the module is linked to
    try:
        from . import _torch_calls
    except ImportError as e:
        raise ImportError("_torch_calls.so is missing or does not fit this torch: build it with "
                          "`python -m fp8_fine_grained_nt_b200.build`") from e
    _calls = _torch_calls
    return _torch_calls


def status_string(status: int) -> str:
    try:
        return load_library().dg_status_string(status).decode()
    except ImportError:
        return "unknown"


def _check(status: int, where: str):
    if status != 0:
        raise Fp8NtError(status, where)


def _stream_ptr(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _dev(t: torch.Tensor, name: str, dtypes, ndim: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


_FP8 = (torch.float8_e4m3fn, torch.uint8)
_F32 = (torch.float32,)


def gemm_fp8_fp8_bf16_nt(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor,
                         sb: torch.Tensor, d: torch.Tensor, stream=None) -> torch.Tensor:
    """D[M,N] (bf16) = sum_kb (A_kb B_kb^T) sa[m,kb] sb[n/128,kb].

    a: [M,K] E4M3 (or its uint8 bytes); sa: [ceil(K/128), tma_aligned(M)] fp32
    column-major LHS scales; b: [N,K] E4M3; sb: [ceil(N/128), ceil(K/128)] fp32;
    d: [M,N] bf16 output.
    """
    M, K = a.shape
    N = b.shape[0]
    args = (_dev(a, "a", _FP8, 2), _dev(sa, "sa", _F32, 2), _dev(b, "b", _FP8, 2),
            _dev(sb, "sb", _F32, 2), _dev(d, "d", (torch.bfloat16,), 2))
    if tuple(d.shape) != (M, N) or b.shape[1] != K:
        raise ValueError("shape mismatch between a, b and d")
    _check(load_library().gemm_fp8_fp8_bf16_nt(*args, M, N, K, _stream_ptr(stream)),
           "gemm_fp8_fp8_bf16_nt")
    return d


def gemm_fp8_fp8_bf16_nt_per_tensor(a: torch.Tensor, scale_a: torch.Tensor, b: torch.Tensor,
                                    scale_b: torch.Tensor, d: torch.Tensor,
                                    stream=None) -> torch.Tensor:
    """D[M,N] (bf16) = scale_a * scale_b * (A B^T), FP32 accumulation over all of K.

    a: [M,K] E4M3; b: [N,K] E4M3; scale_a, scale_b: one-element fp32 device
    tensors; d: [M,N] bf16 output.
    """
    M, K = a.shape
    N = b.shape[0]
    if scale_a.numel() != 1 or scale_b.numel() != 1:
        raise ValueError("scale_a and scale_b hold one value each")
    args = (_dev(a, "a", _FP8, 2), _dev(scale_a.reshape(1), "scale_a", _F32, 1),
            _dev(b, "b", _FP8, 2), _dev(scale_b.reshape(1), "scale_b", _F32, 1),
            _dev(d, "d", (torch.bfloat16,), 2))
    if tuple(d.shape) != (M, N) or b.shape[1] != K:
        raise ValueError("shape mismatch between a, b and d")
    _check(load_library().gemm_fp8_fp8_bf16_nt_per_tensor(*args, M, N, K, _stream_ptr(stream)),
           "gemm_fp8_fp8_bf16_nt_per_tensor")
    return d


def quantize_fp8_1x128(x: torch.Tensor, q: torch.Tensor, sa: torch.Tensor,
                       stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """1x128 quantiser: x [M,K] fp32 or bf16 -> q [M,K] E4M3 (uint8 or
    float8_e4m3fn) and sa [K/128, get_tma_aligned_size(M, 4)] fp32 column-major."""
    M, K = x.shape
    dtype = {torch.float32: 0, torch.bfloat16: 1}.get(x.dtype)
    if dtype is None:
        raise TypeError(f"x has dtype {x.dtype}, expected float32 or bfloat16")
    args = (_dev(x, "x", (torch.float32, torch.bfloat16), 2), dtype, _dev(q, "q", _FP8, 2),
            _dev(sa, "sa", _F32, 2))
    if tuple(q.shape) != (M, K) or sa.shape[0] != K // 128 or sa.shape[1] != get_tma_aligned_size(M, 4):
        raise ValueError("shape mismatch between x, q and sa")
    _check(load_library().quantize_fp8_1x128(*args, M, K, _stream_ptr(stream)),
           "quantize_fp8_1x128")
    return q, sa


def m_grouped_gemm_fp8_fp8_bf16_nt_contiguous(a, sa, b, sb, d, m_indices, stream=None):
    """Contiguous m-grouped GEMM: row m of A uses expert m_indices[m] (-1 = padding).

    a: [M_sum,K]; sa: [ceil(K/128), M_sum] (M_sum is a multiple of the alignment);
    b: [G,N,K]; sb: [G, ceil(N/128), ceil(K/128)]; d: [M_sum,N] bf16;
    m_indices: [M_sum] int32 on the device.
    """
    M_sum, K = a.shape
    G, N = b.shape[0], b.shape[1]
    args = (_dev(a, "a", _FP8, 2), _dev(sa, "sa", _F32, 2), _dev(b, "b", _FP8, 3),
            _dev(sb, "sb", _F32, 3), _dev(d, "d", (torch.bfloat16,), 2),
            _dev(m_indices, "m_indices", (torch.int32,), 1))
    if tuple(d.shape) != (M_sum, N) or b.shape[2] != K or m_indices.shape[0] != M_sum:
        raise ValueError("shape mismatch between a, b, d and m_indices")
    _check(load_library().m_grouped_gemm_fp8_fp8_bf16_nt_contiguous(
        *args, G, M_sum, N, K, _stream_ptr(stream)), "m_grouped_gemm_fp8_fp8_bf16_nt_contiguous")
    return d


def m_grouped_gemm_fp8_fp8_bf16_nt_masked(a, sa, b, sb, d, masked_m, expected_m: int,
                                          stream=None):
    """Masked m-grouped GEMM: group g computes its first masked_m[g] rows only.

    a: [G,M_max,K]; sa: [G, ceil(K/128), tma_aligned(M_max)]; b: [G,N,K];
    sb: [G, ceil(N/128), ceil(K/128)]; d: [G,M_max,N] bf16; masked_m: [G] int32
    on the device (never read by the host); expected_m: a host hint for the
    typical masked_m, used only to choose the tile configuration.
    """
    G, M_max, K = a.shape
    N = b.shape[1]
    args = (_dev(a, "a", _FP8, 3), _dev(sa, "sa", _F32, 3), _dev(b, "b", _FP8, 3),
            _dev(sb, "sb", _F32, 3), _dev(d, "d", (torch.bfloat16,), 3),
            _dev(masked_m, "masked_m", (torch.int32,), 1))
    if tuple(d.shape) != (G, M_max, N) or tuple(b.shape) != (G, N, K) or masked_m.shape[0] != G:
        raise ValueError("shape mismatch between a, b, d and masked_m")
    _check(load_library().m_grouped_gemm_fp8_fp8_bf16_nt_masked(
        *args, G, M_max, N, K, int(expected_m), _stream_ptr(stream)),
        "m_grouped_gemm_fp8_fp8_bf16_nt_masked")
    return d


_DTYPE_CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_HALF = (torch.bfloat16, torch.float16)


# The checks below run on every call of operators that take a few microseconds
# on the GPU, so they ask each tensor for as little as they can.


def _device_of(t: torch.Tensor, name: str) -> int:
    """Index of the CUDA device that `t` is on."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return index


def _arg(t: torch.Tensor, name: str, dtype, ndim: int, device: int) -> int:
    """Checked pointer of a contiguous tensor on `device`."""
    if isinstance(t, torch.Tensor) and t.get_device() == device and t.dtype is dtype and t.dim() == ndim \
            and t.is_contiguous():
        return t.data_ptr()
    raise _refusal(t, name, dtype, ndim, device, "must be contiguous")


def _rows(t: torch.Tensor, name: str, dtype, device: int) -> int:
    """Checked pointer of a matrix on `device` whose rows are contiguous."""
    if isinstance(t, torch.Tensor) and t.get_device() == device and t.dtype is dtype and t.dim() == 2 \
            and (t.is_contiguous() or t.stride(1) == 1 or t.size(1) == 1):
        return t.data_ptr()
    raise _refusal(t, name, dtype, 2, device, "must have contiguous rows")


def _refusal(t, name: str, dtype, ndim: int, device: int, layout: str) -> Exception:
    if not isinstance(t, torch.Tensor):
        return TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != device:
        return ValueError(f"{name} must be a CUDA tensor on cuda:{device}, not on {t.device}")
    if t.dtype is not dtype:
        return TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.dim() != ndim:
        return ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    return ValueError(f"{name} {layout}")


def _half(t: torch.Tensor, name: str):
    """The 16-bit type of a call, from its first operand."""
    if t.dtype not in _HALF:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {_HALF}")
    return t.dtype


def _call(name: str, stream, device: int, *args) -> None:
    """Call the library on the tensors' own device, on `stream` or that device's current one."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device)
    elif stream.device.index != device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on cuda:{device}")
    else:
        raw = stream.cuda_stream
    fn = getattr(_lib or load_library(), name)
    if torch._C._cuda_getDevice() == device:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            status = fn(*args, raw)
    if status != 0:
        raise Fp8NtError(status, name)


def _ragged(name: str, a, b, d, offsets, G: int, N: int, K: int, stream):
    device, dtype = _device_of(a, "a"), _half(a, "a")
    _call(name, stream, device, _arg(a, "a", dtype, 2, device), _arg(b, "b", dtype, 3, device),
          _arg(d, "d", dtype, 2, device), _arg(offsets, "offsets", torch.int32, 1, device),
          _DTYPE_CODE[dtype], G, a.size(0), N, K)
    return d


def m_grouped_gemm_nt_ragged(a: torch.Tensor, b: torch.Tensor, d: torch.Tensor,
                             offsets: torch.Tensor, stream=None) -> torch.Tensor:
    """Grouped product over ragged segments: d[t] = a[t] b[g]^T for rows t of segment g.

    a: [T,K] bf16 or fp16; b: [G,N,K], d: [T,N] of the same type; offsets: [G+1]
    int32 on the device, segment g being rows offsets[g] to offsets[g+1] (any
    length, no padding).  Rows outside every segment are left as they are.
    """
    if stream is None:
        status = (_calls or _load_calls()).m_grouped_gemm_nt_ragged(a, b, d, offsets)
        if status == 0:
            return d
        if status > 0:
            raise Fp8NtError(status, "m_grouped_gemm_nt_ragged")
    G, N, K = b.shape
    if a.shape[1] != K or tuple(d.shape) != (a.shape[0], N) or offsets.shape[0] != G + 1:
        raise ValueError("shape mismatch between a, b, d and offsets")
    return _ragged("m_grouped_gemm_nt_ragged", a, b, d, offsets, G, N, K, stream)


def m_grouped_gemm_nn_ragged(a: torch.Tensor, b: torch.Tensor, d: torch.Tensor,
                             offsets: torch.Tensor, stream=None) -> torch.Tensor:
    """Input gradient of m_grouped_gemm_nt_ragged: d[t] = a[t] b[g] for rows t of segment g.

    a: [T,N] (gradients of the forward's output); b: [G,N,K] (the forward's
    weights, not transposed); d: [T,K]; offsets as in the forward.
    """
    if stream is None:
        status = (_calls or _load_calls()).m_grouped_gemm_nn_ragged(a, b, d, offsets)
        if status == 0:
            return d
        if status > 0:
            raise Fp8NtError(status, "m_grouped_gemm_nn_ragged")
    G, N, K = b.shape
    if a.shape[1] != N or tuple(d.shape) != (a.shape[0], K) or offsets.shape[0] != G + 1:
        raise ValueError("shape mismatch between a, b, d and offsets")
    return _ragged("m_grouped_gemm_nn_ragged", a, b, d, offsets, G, N, K, stream)


def k_grouped_gemm_tn_ragged(a: torch.Tensor, b: torch.Tensor, d: torch.Tensor,
                             offsets: torch.Tensor, accumulate: bool = False,
                             stream=None) -> torch.Tensor:
    """Weight gradient of m_grouped_gemm_nt_ragged: d[g] = a[segment g]^T b[segment g].

    a: [T,N] (gradients of the forward's output); b: [T,K] (the forward's
    input), both bf16 or fp16; d: [G,N,K] fp32 or their type.  accumulate: add to
    d (fp32 only), else d is written in full (zeros for a group without rows).
    """
    if stream is None:
        status = (_calls or _load_calls()).k_grouped_gemm_tn_ragged(a, b, d, offsets, accumulate)
        if status == 0:
            return d
        if status > 0:
            raise Fp8NtError(status, "k_grouped_gemm_tn_ragged")
    G, N, K = d.shape
    if a.shape[1] != N or b.shape[1] != K or a.shape[0] != b.shape[0] or offsets.shape[0] != G + 1:
        raise ValueError("shape mismatch between a, b, d and offsets")
    device, dtype = _device_of(a, "a"), _half(a, "a")
    d_dtype = torch.float32 if accumulate or d.dtype is torch.float32 else dtype
    _call("k_grouped_gemm_tn_ragged", stream, device, _arg(a, "a", dtype, 2, device),
          _arg(b, "b", dtype, 2, device), _arg(d, "d", d_dtype, 3, device),
          _arg(offsets, "offsets", torch.int32, 1, device), _DTYPE_CODE[dtype], _DTYPE_CODE[d_dtype],
          int(accumulate), G, a.size(0), N, K)
    return d


def _workspace(given, need: int, stream, device: int, like: torch.Tensor):
    """(pointer, bytes, owner) of the caller's workspace, or of one from torch's
    allocator that belongs to the stream the call runs on."""
    if given is not None:
        if given.get_device() != device or not given.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on cuda:{device}")
        return given.data_ptr(), given.numel() * given.element_size(), given
    if need == 0:
        return 0, 0, None
    if stream is None:
        own = like.new_empty(need, dtype=torch.uint8)
    else:
        with torch.cuda.stream(stream):
            own = like.new_empty(need, dtype=torch.uint8)
    return own.data_ptr(), need, own


@functools.lru_cache(maxsize=4096)
def _size(name: str, *args: int) -> int:
    n = getattr(_lib or load_library(), name)(*args)
    if n < 0:
        raise Fp8NtError(-n, name)
    return n


def get_row_groups_capacity(num_rows: int, num_groups: int, alignment: int = 1) -> int:
    """Slots that num_rows rows in num_groups groups can need (length of order and m_indices)."""
    return _size("get_row_groups_capacity", int(num_rows), int(num_groups), int(alignment))


def get_group_rows_workspace_size(num_rows: int, num_groups: int) -> int:
    """Bytes of workspace group_rows_by_index needs (0 for short calls)."""
    return _size("get_group_rows_workspace_size", int(num_rows), int(num_groups))


def group_rows_by_index(index: torch.Tensor, num_groups: int, offsets: torch.Tensor,
                        order: torch.Tensor, slots: Optional[torch.Tensor] = None,
                        m_indices: Optional[torch.Tensor] = None, alignment: int = 1,
                        workspace: Optional[torch.Tensor] = None, stream=None):
    """Rows sorted (stably) by the group each belongs to; the grouped calls' layout.

    index: [R] int32 or int64, the group of each row or -1 for none.  Results
    (int32): offsets [num_groups+1], the first slot of each segment (multiples of
    alignment); order [capacity], the row in each slot or -1; slots [R], the slot
    of each row or -1 (optional); m_indices [capacity], the group of each slot or
    -1 (optional); capacity = get_row_groups_capacity(R, num_groups, alignment).
    Returns (offsets, order, slots, m_indices).
    """
    if stream is None and workspace is None:
        status = (_calls or _load_calls()).group_rows_by_index(index, num_groups, offsets, order, slots, m_indices,
                                                               alignment)
        if status == 0:
            return offsets, order, slots, m_indices
        if status > 0:
            raise Fp8NtError(status, "group_rows_by_index")
    num_groups, alignment = int(num_groups), int(alignment)
    device = _device_of(index, "index")
    if index.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"index has dtype {index.dtype}, expected int32 or int64")
    args = (_arg(index, "index", index.dtype, 1, device), 1 if index.dtype is torch.int64 else 0,
            _arg(offsets, "offsets", torch.int32, 1, device), _arg(order, "order", torch.int32, 1, device),
            None if slots is None else _arg(slots, "slots", torch.int32, 1, device),
            None if m_indices is None else _arg(m_indices, "m_indices", torch.int32, 1, device))
    R = index.size(0)
    cap = _size("get_row_groups_capacity", R, num_groups, alignment)
    if (offsets.size(0) != num_groups + 1 or order.size(0) != cap or (slots is not None and slots.size(0) != R)
            or (m_indices is not None and m_indices.size(0) != cap)):
        raise ValueError(f"offsets must hold {num_groups + 1} values, order and m_indices {cap}, slots {R}")
    ptr, size, _own = _workspace(workspace, _size("get_group_rows_workspace_size", R, num_groups), stream, device, index)
    _call("group_rows_by_index", stream, device, *args, R, num_groups, alignment, ptr, size)
    return offsets, order, slots, m_indices


def get_lora_workspace_size(num_slots: int, num_adapters: int, rank: int, N: int, K: int) -> int:
    """Bytes of workspace m_grouped_lora_add needs (0 for long batches)."""
    return _size("get_lora_workspace_size", int(num_slots), int(num_adapters), int(rank), int(N), int(K))


def m_grouped_lora_add(x: torch.Tensor, lora_a: torch.Tensor, lora_b: torch.Tensor,
                       scales: torch.Tensor, c: torch.Tensor, d: torch.Tensor,
                       m_indices: torch.Tensor, order: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Low-rank adapters of many requests beside a shared projection c:
    d[t] = c[t] + scales[g] (x[t] lora_a[g]^T) lora_b[g]^T.

    x: [T,K]; lora_a: [L,R,K]; lora_b: [L,N,R]; c, d: [T,N] (d may be c), all bf16
    or all fp16; x, c and d may be column ranges of wider tensors; scales: [L] fp32;
    m_indices: [S] int32, adapter g of each slot (-1: none); order: [S] int32, row t
    of each slot (each row at most once; default: slot i is row i).  Rows in no
    slot with an adapter are not written.  Slots sorted by adapter
    (group_rows_by_index) share the reads of its weights.
    """
    if stream is None and workspace is None:
        status = (_calls or _load_calls()).m_grouped_lora_add(x, lora_a, lora_b, scales, c, d, m_indices, order)
        if status == 0:
            return d
        if status > 0:
            raise Fp8NtError(status, "m_grouped_lora_add")
    L, R, K = lora_a.shape
    T, N = d.shape
    S = m_indices.size(0)
    if (x.shape != (T, K) or lora_b.shape != (L, N, R) or c.shape != (T, N) or scales.size(0) != L
            or (order is not None and order.size(0) != S)):
        raise ValueError("shape mismatch between x, lora_a, lora_b, scales, c, d, m_indices and order")
    if order is None and S > T:
        raise ValueError(f"m_indices holds {S} slots for {T} rows")
    device, dtype = _device_of(x, "x"), _half(x, "x")
    args = (_rows(x, "x", dtype, device), x.stride(0) if T > 1 else K,
            _arg(lora_a, "lora_a", dtype, 3, device), _arg(lora_b, "lora_b", dtype, 3, device),
            _arg(scales, "scales", torch.float32, 1, device),
            _rows(c, "c", dtype, device), c.stride(0) if T > 1 else N,
            _rows(d, "d", dtype, device), d.stride(0) if T > 1 else N,
            _arg(m_indices, "m_indices", torch.int32, 1, device),
            None if order is None else _arg(order, "order", torch.int32, 1, device))
    ptr, size, _own = _workspace(workspace, _size("get_lora_workspace_size", S, L, R, N, K), stream, device, x)
    _call("m_grouped_lora_add", stream, device, *args, _DTYPE_CODE[dtype], S, T, L, R, N, K, ptr, size)
    return d


def get_m_alignment_for_contiguous_layout() -> int:
    return load_library().get_m_alignment_for_contiguous_layout()


def get_tma_aligned_size(x: int, element_size: int) -> int:
    r = load_library().get_tma_aligned_size(int(x), int(element_size))
    if r < 0:
        raise Fp8NtError(-r, "get_tma_aligned_size")
    return r


def get_col_major_tma_aligned_tensor(s: torch.Tensor) -> torch.Tensor:
    """[..., M, nkb] per-row scales -> column-major TMA-aligned [..., nkb, ld] storage.

    A layout helper (torch copy ops, not on the GEMM path): the padding columns
    between M and ld are left as zeros.
    """
    *batch, M, nkb = s.shape
    ld = get_tma_aligned_size(M, 4)
    out = torch.zeros((*batch, nkb, ld), dtype=torch.float32, device=s.device)
    out[..., :M] = s.transpose(-1, -2).float()
    return out


def set_num_sms(n: int) -> None:
    _check(load_library().set_num_sms(int(n)), "set_num_sms")


def get_num_sms() -> int:
    return load_library().get_num_sms()


def selftest_wait_timeout(timeout_us: int = 20000, stream=None) -> None:
    """Enqueue the bounded-wait self-test: a device wait that nothing satisfies
    gives up after timeout_us and records DG_ERR_DEVICE_TIMEOUT (read it with
    get_device_status())."""
    _check(load_library().dg_selftest_wait_timeout(int(timeout_us), _stream_ptr(stream)),
           "dg_selftest_wait_timeout")


def get_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device-side status word."""
    return load_library().dg_get_device_status(_stream_ptr(stream))


def select_config(kind: int, M: int, N: int, K: int, num_groups: int = 1,
                  expected_m: int = 0, num_sms: int = 148) -> dict:
    """The tile configuration the library would launch (host logic only, no GPU)."""
    cfg = DgConfig()
    _check(load_library().dg_select_config(kind, M, N, K, num_groups, expected_m, num_sms,
                                           ctypes.byref(cfg)), "dg_select_config")
    return cfg.as_dict()


def force_config(block_m: int = 0, block_n: int = 0, split: int = 0, cta_pair: int = 0) -> None:
    """Pin the tile shape (0, 0 = automatic), split-K factor (0 = automatic)
    and CTA-pair mode (0 = automatic, 1 = one CTA per tile, 2 = CTA pairs)
    for later calls.  For tests."""
    _check(load_library().dg_force_config(int(block_m), int(block_n), int(split),
                                          int(cta_pair)), "dg_force_config")


def force_swap_ab(mode: int = 0) -> None:
    """Small-M kernel choice for later dense calls: 0 = automatic (M <= 256
    uses it), 1 = never, 2 = wherever it applies.  For tests."""
    _check(load_library().dg_force_swap_ab(int(mode)), "dg_force_swap_ab")


def force_tail_split(mode: int = 0) -> None:
    """Split of a dense call's last partial wave onto the small-M kernel:
    0 = automatic (off), 1 = never, 2 = wherever the block layout allows it,
    3 = where the layout allows it and the cycle estimate favours it."""
    _check(load_library().dg_force_tail_split(int(mode)), "dg_force_tail_split")


def force_ragged(swap_ab: int = 0, cta_pair: int = 0, block_n: int = 0, split: int = 0) -> None:
    """Pin the tile form of later ragged grouped calls (0, 0, 0, 0 = automatic):
    swap_ab 1 = weights on the 128-row side and block_n token rows, the reduction
    shared by split CTAs; cta_pair 1 = 256 x 256 by CTA pairs; block_n alone = 128 x
    block_n.  For tests."""
    _check(load_library().dg_force_ragged(int(swap_ab), int(cta_pair), int(block_n), int(split)),
           "dg_force_ragged")
