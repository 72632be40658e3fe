"""Python binding of libresa.so (ReSA decode hot path on B200, sm_100a).

Argument marshalling only: every function below checks tensor shapes, passes
device pointers, sizes and the current CUDA stream to the C ABI declared in
include/resa.h, and raises on a non-zero status. All arithmetic happens in the
library's CUDA kernels. PyTorch provides device memory and streams.

The library must be built (``python block_sparse_attention_quest_b200/build.py``
or ``__graft_entry__.build()``); importing this module fails loudly when
libresa.so is missing. There is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libresa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libresa.so not found at {LIB_PATH}; build it with "
        "`python block_sparse_attention_quest_b200/build.py`")
_lib = ctypes.CDLL(LIB_PATH)

RESA_OK = 0
RESA_ERR_INVALID_ARG = -1
RESA_ERR_UNSUPPORTED = -2
RESA_ERR_CAPACITY = -3
RESA_ERR_WORKSPACE = -4
RESA_ERR_CUDA = -5
RESA_ERR_TIMEOUT = -6
RESA_ERR_BAD_INDEX = -7
RESA_F32 = 0
RESA_BF16 = 1
BLOCK = 16

EXPORTED = ("resa_num_selected", "resa_workspace_bytes", "resa_build_desc",
            "resa_decode_sparse", "resa_select_blocks", "resa_attend_blocks",
            "resa_decode_dense", "resa_rectify",
            "resa_workspace_status", "resa_status_string", "resa_decode_sparse_noalloc",
            "resa_build_desc_varlen", "resa_decode_sparse_varlen", "resa_decode_dense_varlen",
            "resa_rectify_varlen", "resa_prefill", "resa_wait_check", "resa_noalloc_status",
           "resa_kv4_bytes", "resa_kv4_workspace_bytes", "resa_kv4_quantize",
           "resa_kv4_dequantize", "resa_decode_dense_kv4", "resa_decode_sparse_kv4",
           "resa_attend_blocks_kv4", "resa_weights_workspace_bytes",
           "resa_decode_dense_weights", "resa_evict", "resa_prefill_packed")


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("max_len", ctypes.c_int64)]


_P = ctypes.c_void_p
_lib.resa_num_selected.restype = ctypes.c_int32
_lib.resa_num_selected.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_double, ctypes.c_int32]
_lib.resa_workspace_bytes.restype = ctypes.c_size_t
_lib.resa_workspace_bytes.argtypes = [ctypes.POINTER(Dims), ctypes.c_int64, ctypes.c_int32]
_lib.resa_build_desc.restype = ctypes.c_int
_lib.resa_build_desc.argtypes = [ctypes.POINTER(Dims), _P, ctypes.c_int64, _P, _P]
_lib.resa_decode_sparse.restype = ctypes.c_int
_lib.resa_decode_sparse.argtypes = [ctypes.POINTER(Dims), _P, _P, _P, _P, _P, _P, ctypes.c_int64,
                                    ctypes.c_double, ctypes.c_int32, ctypes.c_float, _P, _P, _P,
                                    _P, ctypes.c_size_t, _P]
_lib.resa_select_blocks.restype = ctypes.c_int
_lib.resa_select_blocks.argtypes = [ctypes.POINTER(Dims), _P, _P, _P, _P, _P, _P, ctypes.c_int64,
                                    ctypes.c_double, ctypes.c_int32, _P, _P, ctypes.c_size_t, _P]
_lib.resa_attend_blocks.restype = ctypes.c_int
_lib.resa_attend_blocks.argtypes = [ctypes.POINTER(Dims), _P, _P, _P, ctypes.c_int64, _P,
                                    ctypes.c_int32, ctypes.c_float, _P, _P, _P, ctypes.c_size_t, _P]
_lib.resa_decode_dense.restype = ctypes.c_int
_lib.resa_decode_dense.argtypes = [ctypes.POINTER(Dims), _P, _P, _P, _P, _P, _P, ctypes.c_int64,
                                   ctypes.c_float, _P, _P, _P, ctypes.c_size_t, _P]
_lib.resa_rectify.restype = ctypes.c_int
_lib.resa_rectify.argtypes = [ctypes.POINTER(Dims), _P, _P, _P, _P, _P, _P, ctypes.c_int64,
                              ctypes.c_int32, ctypes.c_float, _P, _P, ctypes.c_size_t, _P]
_lib.resa_decode_sparse_noalloc.restype = ctypes.c_int
_lib.resa_decode_sparse_noalloc.argtypes = [ctypes.POINTER(Dims), _P, _P, _P, _P, _P, _P,
                                            ctypes.c_int64, ctypes.c_double, ctypes.c_int32,
                                            ctypes.c_float, _P, _P, _P, _P]
_lib.resa_build_desc_varlen.restype = ctypes.c_int
_lib.resa_build_desc_varlen.argtypes = [ctypes.POINTER(Dims), _P, _P, ctypes.c_int64, _P, _P]
_lib.resa_decode_sparse_varlen.restype = ctypes.c_int
_lib.resa_decode_sparse_varlen.argtypes = [ctypes.POINTER(Dims), _P, _P, _P, _P, _P, _P, _P,
                                           ctypes.c_int64, ctypes.c_double, ctypes.c_int32,
                                           ctypes.c_float, _P, _P, _P, _P, ctypes.c_size_t, _P]
_lib.resa_decode_dense_varlen.restype = ctypes.c_int
_lib.resa_decode_dense_varlen.argtypes = [ctypes.POINTER(Dims), _P, _P, _P, _P, _P, _P, _P,
                                          ctypes.c_int64, ctypes.c_float, _P, _P, _P,
                                          ctypes.c_size_t, _P]
_lib.resa_rectify_varlen.restype = ctypes.c_int
_lib.resa_rectify_varlen.argtypes = [ctypes.POINTER(Dims), _P, _P, _P, _P, _P, _P, _P, _P,
                                     ctypes.c_int64, ctypes.c_int32, ctypes.c_float, _P, _P,
                                     ctypes.c_size_t, _P]
_lib.resa_prefill.restype = ctypes.c_int
_lib.resa_prefill.argtypes = [ctypes.POINTER(Dims), _P, _P, _P, _P, ctypes.c_int64, ctypes.c_float,
                              _P, _P, ctypes.c_size_t, _P]
_lib.resa_kv4_bytes.restype = ctypes.c_size_t
_lib.resa_kv4_bytes.argtypes = [ctypes.POINTER(Dims)]
_lib.resa_kv4_workspace_bytes.restype = ctypes.c_size_t
_lib.resa_kv4_workspace_bytes.argtypes = [ctypes.POINTER(Dims), ctypes.c_int64]
_lib.resa_kv4_quantize.restype = ctypes.c_int
_lib.resa_kv4_quantize.argtypes = [ctypes.POINTER(Dims), _P, _P, ctypes.c_int64, _P, _P, _P]
_lib.resa_kv4_dequantize.restype = ctypes.c_int
_lib.resa_kv4_dequantize.argtypes = [ctypes.POINTER(Dims), _P, ctypes.c_int64, _P, _P, _P, _P]
_lib.resa_decode_dense_kv4.restype = ctypes.c_int
_lib.resa_decode_dense_kv4.argtypes = [ctypes.POINTER(Dims), _P, _P, _P, _P, _P, ctypes.c_int64,
                                       _P, ctypes.c_float, _P, _P, _P, ctypes.c_size_t, _P]
_lib.resa_decode_sparse_kv4.restype = ctypes.c_int
_lib.resa_decode_sparse_kv4.argtypes = [ctypes.POINTER(Dims), _P, _P, _P, _P, _P, ctypes.c_int64,
                                        _P, ctypes.c_double, ctypes.c_int32, ctypes.c_float, _P,
                                        _P, _P, _P, ctypes.c_size_t, _P]
_lib.resa_attend_blocks_kv4.restype = ctypes.c_int
_lib.resa_attend_blocks_kv4.argtypes = [ctypes.POINTER(Dims), _P, _P, ctypes.c_int64, _P,
                                        ctypes.c_int32, ctypes.c_float, _P, _P, _P,
                                        ctypes.c_size_t, _P]
_lib.resa_weights_workspace_bytes.restype = ctypes.c_size_t
_lib.resa_weights_workspace_bytes.argtypes = [ctypes.POINTER(Dims), ctypes.c_int64]
_lib.resa_decode_dense_weights.restype = ctypes.c_int
_lib.resa_decode_dense_weights.argtypes = [ctypes.POINTER(Dims), _P, _P, _P, _P, _P, _P, _P,
                                           ctypes.c_int64, _P, ctypes.c_float, _P, _P, _P,
                                           ctypes.c_size_t, _P]
_lib.resa_evict.restype = ctypes.c_int
_lib.resa_evict.argtypes = [ctypes.POINTER(Dims), _P, _P, _P, ctypes.c_int64, _P, ctypes.c_int32,
                            ctypes.c_int32, ctypes.c_int64, _P, _P, _P, _P, _P, _P,
                            ctypes.c_size_t, _P]
_lib.resa_prefill_packed.restype = ctypes.c_int
_lib.resa_prefill_packed.argtypes = [ctypes.POINTER(Dims), _P, _P, _P, _P, ctypes.c_int64,
                                     ctypes.c_int64, _P, _P, _P, ctypes.c_float, _P, _P,
                                     ctypes.c_size_t, _P]
_lib.resa_wait_check.restype = ctypes.c_int
_lib.resa_wait_check.argtypes = [_P, ctypes.c_int32, ctypes.c_uint32, _P, _P]
_lib.resa_workspace_status.restype = ctypes.c_int
_lib.resa_workspace_status.argtypes = [_P, _P]
_lib.resa_noalloc_status.restype = ctypes.c_int
_lib.resa_noalloc_status.argtypes = [_P]
_lib.resa_status_string.restype = ctypes.c_char_p
_lib.resa_status_string.argtypes = [ctypes.c_int]


class ResaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


def status_string(status: int) -> str:
    return _lib.resa_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != RESA_OK:
        raise ResaError(status, what)


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return RESA_F32
    if dt == torch.bfloat16:
        return RESA_BF16
    raise ValueError(f"unsupported dtype {dt}")


def dims_for(k_cache: torch.Tensor, n_q_heads: int) -> Dims:
    """Dims of a cache [B, H_kv, max_len, d] serving n_q_heads query heads."""
    B, H, L, d = k_cache.shape
    return Dims(B, int(n_q_heads), H, d, BLOCK, _dtype_code(k_cache.dtype), L)


def num_selected(length: int, r: float, n_min: int) -> int:
    n = _lib.resa_num_selected(int(length), BLOCK, float(r), int(n_min))
    if n < 0:
        raise ResaError(n, "resa_num_selected")
    return n


def workspace_bytes(dims: Dims, length: int, f: int = 0) -> int:
    n = _lib.resa_workspace_bytes(ctypes.byref(dims), int(length), int(f))
    if n == 0:
        raise ResaError(RESA_ERR_INVALID_ARG, "resa_workspace_bytes")
    return n


def alloc_workspace(dims: Dims, length: int, f: int = 0, device=None) -> torch.Tensor:
    """Zero-filled workspace (uint8) of the size the library asks for."""
    n = workspace_bytes(dims, length, f)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def build_desc(k_cache: torch.Tensor, length: int, desc: torch.Tensor, n_q_heads: int,
               stream=None) -> None:
    dims = dims_for(k_cache, n_q_heads)
    _check(_lib.resa_build_desc(ctypes.byref(dims), _ptr(k_cache), int(length), _ptr(desc),
                                _stream(stream)), "resa_build_desc")


def decode_sparse(q, k_new, v_new, k_cache, v_cache, desc, length: int, r: float, n_min: int,
                  softmax_scale: float, out, workspace, lse=None, sel=None, stream=None) -> None:
    dims = dims_for(k_cache, q.shape[1])
    _check(_lib.resa_decode_sparse(
        ctypes.byref(dims), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
        _ptr(desc), int(length), float(r), int(n_min), float(softmax_scale), _ptr(out), _ptr(lse),
        _ptr(sel), _ptr(workspace), workspace.numel(), _stream(stream)), "resa_decode_sparse")


def select_blocks(q, k_new, v_new, k_cache, v_cache, desc, length: int, r: float, n_min: int,
                  sel, workspace, stream=None) -> None:
    dims = dims_for(k_cache, q.shape[1])
    _check(_lib.resa_select_blocks(
        ctypes.byref(dims), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
        _ptr(desc), int(length), float(r), int(n_min), _ptr(sel), _ptr(workspace),
        workspace.numel(), _stream(stream)), "resa_select_blocks")


def attend_blocks(q, k_cache, v_cache, length: int, sel, softmax_scale: float, out, workspace,
                  lse=None, stream=None) -> None:
    dims = dims_for(k_cache, q.shape[1])
    _check(_lib.resa_attend_blocks(
        ctypes.byref(dims), _ptr(q), _ptr(k_cache), _ptr(v_cache), int(length), _ptr(sel),
        int(sel.shape[-1]), float(softmax_scale), _ptr(out), _ptr(lse), _ptr(workspace),
        workspace.numel(), _stream(stream)), "resa_attend_blocks")


def decode_dense(q, k_new, v_new, k_cache, v_cache, desc, length: int, softmax_scale: float, out,
                 workspace, lse=None, stream=None) -> None:
    dims = dims_for(k_cache, q.shape[1])
    _check(_lib.resa_decode_dense(
        ctypes.byref(dims), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
        _ptr(desc), int(length), float(softmax_scale), _ptr(out), _ptr(lse), _ptr(workspace),
        workspace.numel(), _stream(stream)), "resa_decode_dense")


def rectify(q_f, k_f, v_f, k_cache, v_cache, desc, length: int, f: int, softmax_scale: float,
            out_f, workspace, stream=None) -> None:
    dims = dims_for(k_cache, q_f.shape[2])
    _check(_lib.resa_rectify(
        ctypes.byref(dims), _ptr(q_f), _ptr(k_f), _ptr(v_f), _ptr(k_cache), _ptr(v_cache),
        _ptr(desc), int(length), int(f), float(softmax_scale), _ptr(out_f), _ptr(workspace),
        workspace.numel(), _stream(stream)), "resa_rectify")


def decode_sparse_noalloc(q, k_new, v_new, k_cache, v_cache, desc, length: int, r: float,
                          n_min: int, softmax_scale: float, out, lse=None, sel=None,
                          stream=None) -> None:
    """resa_decode_sparse with the library's own fixed scratch (no workspace)."""
    dims = dims_for(k_cache, q.shape[1])
    _check(_lib.resa_decode_sparse_noalloc(
        ctypes.byref(dims), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
        _ptr(desc), int(length), float(r), int(n_min), float(softmax_scale), _ptr(out), _ptr(lse),
        _ptr(sel), _stream(stream)), "resa_decode_sparse_noalloc")


def noalloc_status(stream=None) -> int:
    """Synchronise and read (and clear) the device error flag of the fixed
    scratch that decode_sparse_noalloc uses on the current device."""
    return _lib.resa_noalloc_status(_stream(stream))


def workspace_status(workspace, stream=None) -> int:
    """Synchronise and read (and clear) the device error flag of a workspace.
    After an error the workspace has to be zeroed before its next use."""
    return _lib.resa_workspace_status(_ptr(workspace), _stream(stream))


# ---- variable-length batches: `lens` is an int32 CUDA tensor [batch] of row
# lengths, `len_bound` an upper bound on its entries (sizes grids, workspace and
# the stride of `sel`)


def _lens(lens):
    if lens is None or lens.dtype != torch.int32 or not lens.is_cuda or lens.dim() != 1:
        raise ValueError("lens must be a 1-D int32 CUDA tensor")
    return _ptr(lens)


def build_desc_varlen(k_cache, lens, len_bound: int, desc, n_q_heads: int, stream=None) -> None:
    dims = dims_for(k_cache, n_q_heads)
    _check(_lib.resa_build_desc_varlen(ctypes.byref(dims), _ptr(k_cache), _lens(lens),
                                       int(len_bound), _ptr(desc), _stream(stream)),
           "resa_build_desc_varlen")


def decode_sparse_varlen(q, k_new, v_new, k_cache, v_cache, desc, lens, len_bound: int, r: float,
                         n_min: int, softmax_scale: float, out, workspace, lse=None, sel=None,
                         stream=None) -> None:
    dims = dims_for(k_cache, q.shape[1])
    _check(_lib.resa_decode_sparse_varlen(
        ctypes.byref(dims), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
        _ptr(desc), _lens(lens), int(len_bound), float(r), int(n_min), float(softmax_scale),
        _ptr(out), _ptr(lse), _ptr(sel), _ptr(workspace), workspace.numel(), _stream(stream)),
        "resa_decode_sparse_varlen")


def decode_dense_varlen(q, k_new, v_new, k_cache, v_cache, desc, lens, len_bound: int,
                        softmax_scale: float, out, workspace, lse=None, stream=None) -> None:
    dims = dims_for(k_cache, q.shape[1])
    _check(_lib.resa_decode_dense_varlen(
        ctypes.byref(dims), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
        _ptr(desc), _lens(lens), int(len_bound), float(softmax_scale), _ptr(out), _ptr(lse),
        _ptr(workspace), workspace.numel(), _stream(stream)), "resa_decode_dense_varlen")


def rectify_varlen(q_f, k_f, v_f, k_cache, v_cache, desc, lens, len_bound: int, f: int,
                   softmax_scale: float, out_f, workspace, windows=None, stream=None) -> None:
    """windows: optional int32 CUDA tensor [batch] of per-row windows in [0, f]
    (0 = row not rectified); None = every row uses f."""
    dims = dims_for(k_cache, q_f.shape[2])
    _check(_lib.resa_rectify_varlen(
        ctypes.byref(dims), _ptr(q_f), _ptr(k_f), _ptr(v_f), _ptr(k_cache), _ptr(v_cache),
        _ptr(desc), _lens(lens), None if windows is None else _lens(windows), int(len_bound), int(f), float(softmax_scale), _ptr(out_f),
        _ptr(workspace), workspace.numel(), _stream(stream)), "resa_rectify_varlen")


def prefill(q, k_cache, v_cache, desc, length: int, softmax_scale: float, out, workspace,
            stream=None) -> None:
    """Causal attention of every prompt position (q, out: [B, len, Hq, d]) and
    the descriptors of the prompt's keys, in one pass."""
    dims = dims_for(k_cache, q.shape[2])
    _check(_lib.resa_prefill(ctypes.byref(dims), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(desc),
                             int(length), float(softmax_scale), _ptr(out), _ptr(workspace),
                             workspace.numel(), _stream(stream)), "resa_prefill")


def _ptrs(*tensors) -> list:
    """Addresses of the tensors (None stays None), which have to be contiguous
    and on the current CUDA device."""
    out, dev = [], None
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        at = t.get_device()                       # -1: not a CUDA tensor
        if at != dev:
            if at < 0 or dev is not None or at != torch._C._cuda_getDevice():
                raise ValueError("tensors must be on the current CUDA device")
            dev = at
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        out.append(t.data_ptr())
    return out


@functools.lru_cache(maxsize=256)
def _dims_ref(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int, dtype: torch.dtype,
              max_len: int):
    """Pointer to a Dims of these values, for the library to read."""
    return ctypes.byref(Dims(batch, n_q_heads, n_kv_heads, head_dim, BLOCK, _dtype_code(dtype),
                             max_len))


def _step(q, k_new, v_new, desc, out, lse, lens, B: int, H: int, blocks: int) -> None:
    """Shapes and types of the arguments of one decode step."""
    Bq, Hq, d = q.shape
    if Bq != B or Hq % H or out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("q and out must be [batch, n_q_heads, head_dim] of one dtype")
    for t in (k_new, v_new):
        if t is not None and (t.shape != (B, H, d) or t.dtype != q.dtype):
            raise ValueError("k_new and v_new must be [batch, n_kv_heads, head_dim] in q's dtype")
    if desc is not None and (desc.shape != (B, H, blocks, 2, d) or desc.dtype != q.dtype):
        raise ValueError("desc must be [batch, n_kv_heads, max_len / 16, 2, head_dim] in q's dtype")
    if lse is not None and (lse.dtype != torch.float32 or lse.numel() != B * Hq):
        raise ValueError("lse must be float32 [batch, n_q_heads]")
    _row_lens(lens, B)


def _row_lens(lens, B: int) -> None:
    if lens is not None and (lens.dtype != torch.int32 or lens.shape != (B,)):
        raise ValueError("lens must be int32 [batch]")


def prefill_packed(q, k, v, starts, longest: int, k_cache, v_cache, desc, softmax_scale: float,
                   out, workspace, stream=None) -> None:
    """Causal attention over packed prompts (q, out: [total, Hq, d]; k, v:
    [total, Hkv, d]; starts: int32 CUDA tensor [batch + 1]), which also fills
    rows of k_cache and v_cache [batch, Hkv, max_len, d] (both or neither None)
    and desc (or None)."""
    if (k_cache is None) != (v_cache is None):
        raise ValueError("k_cache and v_cache: both or neither")
    if starts.dtype != torch.int32 or starts.dim() != 1 or starts.numel() < 2:
        raise ValueError("starts must be int32 [batch + 1]")
    B = starts.numel() - 1
    T, Hq, d = q.shape
    H = k.shape[1]
    # without a cache the capacity only sizes desc, or bounds `longest`
    if k_cache is not None:
        L = k_cache.shape[2]
    else:
        L = -(-max(int(longest), 1) // BLOCK) * BLOCK
        if desc is not None and desc.dim() == 5:
            L = desc.shape[2] * BLOCK
    if k.shape != (T, H, d) or v.shape != k.shape or out.shape != q.shape:
        raise ValueError("q, out must be [total, n_q_heads, d] and k, v [total, n_kv_heads, d]")
    if k_cache is not None and (k_cache.shape != (B, H, L, d) or v_cache.shape != k_cache.shape):
        raise ValueError("the caches must be [batch, n_kv_heads, max_len, d]")
    if any(t is not None and t.dtype != q.dtype for t in (k, v, out, k_cache, v_cache)):
        raise ValueError("q, k, v, out and the caches must share a dtype")
    if desc is not None and (desc.shape != (B, H, L // BLOCK, 2, d) or desc.dtype != q.dtype):
        raise ValueError("desc must be [batch, n_kv_heads, max_len / 16, 2, head_dim]")
    pq, pk, pv, ps, pkc, pvc, pd, po, pw = _ptrs(q, k, v, starts, k_cache, v_cache, desc, out,
                                                 workspace)
    _check(_lib.resa_prefill_packed(
        _dims_ref(B, Hq, H, d, q.dtype, L), pq, pk, pv, ps, T, int(longest), pkc, pvc, pd,
        float(softmax_scale), po, pw, workspace.numel(), _stream(stream)), "resa_prefill_packed")


# ---- attention weights (float32 [B, H_kv, max_len] running sums) and eviction


def _weights(weights, B: int, H: int, L: int) -> None:
    if weights.dtype != torch.float32 or weights.shape != (B, H, L):
        raise ValueError("weights must be float32 [batch, n_kv_heads, max_len]")


def weights_workspace_bytes(dims: Dims, length: int) -> int:
    n = _lib.resa_weights_workspace_bytes(ctypes.byref(dims), int(length))
    if n == 0:
        raise ResaError(RESA_ERR_INVALID_ARG, "resa_weights_workspace_bytes")
    return n


def alloc_weights_workspace(dims: Dims, length: int, device=None) -> torch.Tensor:
    """Zero-filled workspace (uint8) for decode_dense_weights."""
    return torch.zeros(weights_workspace_bytes(dims, length), dtype=torch.uint8,
                       device=device or "cuda")


def decode_dense_weights(q, k_new, v_new, k_cache, v_cache, desc, weights, length: int,
                         softmax_scale: float, out, lse, workspace, lens=None,
                         stream=None) -> None:
    """decode_dense that also adds every token's attention weight to `weights`
    (desc and lse may be None)."""
    B, H, L, d = k_cache.shape
    if v_cache.shape != k_cache.shape or q.shape[2] != d or not (
            k_cache.dtype == v_cache.dtype == q.dtype):
        raise ValueError("k_cache and v_cache must be [batch, n_kv_heads, max_len, head_dim] in q's dtype")
    _step(q, k_new, v_new, desc, out, lse, lens, B, H, L // BLOCK)
    _weights(weights, B, H, L)
    pq, pkn, pvn, pk, pv, pd, pwt, po, pl, pn, pw = _ptrs(
        q, k_new, v_new, k_cache, v_cache, desc, weights, out, lse, lens, workspace)
    _check(_lib.resa_decode_dense_weights(
        _dims_ref(B, q.shape[1], H, d, q.dtype, L), pq, pkn, pvn, pk, pv, pd, pwt, int(length), pn,
        float(softmax_scale), po, pl, pw, workspace.numel(), _stream(stream)),
        "resa_decode_dense_weights")


def evict(k_cache, v_cache, weights, length: int, budget: int, n_recent: int, k_out, v_out,
          desc_out, weights_out, kept, n_q_heads: int, workspace, lens=None, stream=None) -> None:
    """Cut every (row, KV head) to its newest n_recent tokens and the
    budget - n_recent others of the largest weight (desc_out and weights_out
    may be None; kept: int32 [B, H_kv, budget])."""
    B, H, L, d = k_cache.shape
    Lo = k_out.shape[2]
    if not (k_out.shape == v_out.shape == (B, H, Lo, d) and v_cache.shape == k_cache.shape
            and k_cache.dtype == v_cache.dtype == k_out.dtype == v_out.dtype):
        raise ValueError("the caches must be [batch, n_kv_heads, max_len, head_dim] of one dtype")
    _weights(weights, B, H, L)
    if weights_out is not None:
        _weights(weights_out, B, H, Lo)
    if desc_out is not None and (desc_out.shape != (B, H, Lo // BLOCK, 2, d)
                                 or desc_out.dtype != k_cache.dtype):
        raise ValueError("desc_out must be [batch, n_kv_heads, out_max_len / 16, 2, head_dim]")
    if kept.dtype != torch.int32 or kept.shape != (B, H, budget):
        raise ValueError("kept must be int32 [batch, n_kv_heads, budget]")
    _row_lens(lens, B)
    pk, pv, pwt, pko, pvo, pdo, pwo, pi, pn, pw = _ptrs(
        k_cache, v_cache, weights, k_out, v_out, desc_out, weights_out, kept, lens, workspace)
    _check(_lib.resa_evict(
        _dims_ref(B, int(n_q_heads), H, d, k_cache.dtype, L), pk, pv, pwt, int(length), pn,
        int(budget), int(n_recent), Lo, pko, pvo, pdo, pwo, pi, pw, workspace.numel(),
        _stream(stream)), "resa_evict")


# ---- the cache in 4 bits: a uint8 tensor [B, H_kv, max_len / 16, record] of
# records that each hold 16 tokens' keys and values (the format is described in
# include/resa.h). lens: optional int32 CUDA tensor [batch] of row lengths, with
# `length` the bound on them.


def kv4_record_bytes(head_dim: int) -> int:
    """Bytes of the record of one 16-token block of one KV head."""
    return BLOCK * (head_dim + 8 * (head_dim // 64))


def dims_kv4(kv4: torch.Tensor, q: torch.Tensor) -> Dims:
    """Dims of a 4-bit cache serving queries like q [B, H_q, d] (or [.., H_q, d])."""
    B, H, M, rec = kv4.shape
    if kv4.dtype != torch.uint8 or rec != kv4_record_bytes(q.shape[-1]):
        raise ValueError(f"kv4 must be uint8 records of {kv4_record_bytes(q.shape[-1])} bytes")
    return Dims(B, int(q.shape[-2]), H, int(q.shape[-1]), BLOCK, _dtype_code(q.dtype), M * BLOCK)


def alloc_kv4(batch: int, n_kv_heads: int, max_len: int, head_dim: int, device=None) -> torch.Tensor:
    """Zero-filled 4-bit cache of max_len tokens (a multiple of 16) per row."""
    return torch.zeros(batch, n_kv_heads, max_len // BLOCK, kv4_record_bytes(head_dim),
                       dtype=torch.uint8, device=device or "cuda")


def kv4_workspace_bytes(dims: Dims, length: int) -> int:
    n = _lib.resa_kv4_workspace_bytes(ctypes.byref(dims), int(length))
    if n == 0:
        raise ResaError(RESA_ERR_INVALID_ARG, "resa_kv4_workspace_bytes")
    return n


def alloc_kv4_workspace(dims: Dims, length: int, device=None) -> torch.Tensor:
    """Zero-filled workspace (uint8) for the 4-bit decode calls."""
    return torch.zeros(kv4_workspace_bytes(dims, length), dtype=torch.uint8,
                       device=device or "cuda")


def _kv4_rows(k_cache, v_cache, kv4, n_q_heads: int, lens):
    """Dims and addresses (k, v, kv4, lens) of a call on whole rows."""
    B, H, L, d = k_cache.shape
    if (kv4.dtype != torch.uint8 or kv4.shape != (B, H, L // BLOCK, kv4_record_bytes(d))
            or v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype):
        raise ValueError("kv4 must be the uint8 records of k_cache's and v_cache's shape")
    _row_lens(lens, B)
    return (_dims_ref(B, int(n_q_heads), H, d, k_cache.dtype, L),
            *_ptrs(k_cache, v_cache, kv4, lens))


def kv4_quantize(k_cache, v_cache, length: int, kv4, n_q_heads: int, lens=None,
                 stream=None) -> None:
    """The first `length` tokens of every row into 4-bit records."""
    dims, pk, pv, p4, pn = _kv4_rows(k_cache, v_cache, kv4, n_q_heads, lens)
    _check(_lib.resa_kv4_quantize(dims, pk, pv, int(length), pn, p4, _stream(stream)),
           "resa_kv4_quantize")


def kv4_dequantize(kv4, length: int, k_cache, v_cache, n_q_heads: int, lens=None,
                   stream=None) -> None:
    """The values the records stand for, into slots [0, length) of the caches."""
    dims, pk, pv, p4, pn = _kv4_rows(k_cache, v_cache, kv4, n_q_heads, lens)
    _check(_lib.resa_kv4_dequantize(dims, p4, int(length), pn, pk, pv, _stream(stream)),
           "resa_kv4_dequantize")


def _kv4_step(q, k_new, v_new, kv4, desc, out, lse, lens, sel, workspace):
    """Dims and addresses of a decode call on a 4-bit cache."""
    B, H, M, rec = kv4.shape
    d = q.shape[-1]
    if kv4.dtype != torch.uint8 or rec != BLOCK * (d + 8 * (d // 64)):
        raise ValueError(f"kv4 must be uint8 records of {kv4_record_bytes(d)} bytes")
    _step(q, k_new, v_new, desc, out, lse, lens, B, H, M)
    return (_dims_ref(B, q.shape[1], H, d, q.dtype, M * BLOCK),
            *_ptrs(q, k_new, v_new, kv4, desc, out, lse, lens, sel, workspace))


def _sel(sel, kv4, n: int) -> None:
    if sel is not None and (sel.dtype != torch.int32
                            or sel.shape != (kv4.shape[0], kv4.shape[1], n)):
        raise ValueError("sel must be int32 [batch, n_kv_heads, n]")


def decode_dense_kv4(q, k_new, v_new, kv4, desc, length: int, softmax_scale: float, out, workspace,
                     lse=None, lens=None, stream=None) -> None:
    """decode_dense on a 4-bit cache (k_new/v_new and desc may be None)."""
    dims, pq, pkn, pvn, p4, pd, po, pl, pn, _, pw = _kv4_step(q, k_new, v_new, kv4, desc, out, lse,
                                                              lens, None, workspace)
    _check(_lib.resa_decode_dense_kv4(
        dims, pq, pkn, pvn, p4, pd, int(length), pn, float(softmax_scale), po, pl, pw,
        workspace.numel(), _stream(stream)), "resa_decode_dense_kv4")


def decode_sparse_kv4(q, k_new, v_new, kv4, desc, length: int, r: float, n_min: int,
                      softmax_scale: float, out, workspace, lse=None, sel=None, lens=None,
                      stream=None) -> None:
    """decode_sparse (with lens: decode_sparse_varlen) on a 4-bit cache."""
    _sel(sel, kv4, num_selected(length, r, n_min))
    dims, pq, pkn, pvn, p4, pd, po, pl, pn, ps, pw = _kv4_step(q, k_new, v_new, kv4, desc, out, lse,
                                                               lens, sel, workspace)
    _check(_lib.resa_decode_sparse_kv4(
        dims, pq, pkn, pvn, p4, pd, int(length), pn, float(r), int(n_min), float(softmax_scale),
        po, pl, ps, pw, workspace.numel(), _stream(stream)), "resa_decode_sparse_kv4")


def attend_blocks_kv4(q, kv4, length: int, sel, softmax_scale: float, out, workspace, lse=None,
                      stream=None) -> None:
    """attend_blocks on a 4-bit cache."""
    n = int(sel.shape[-1])
    _sel(sel, kv4, n)
    dims, pq, _, _, p4, _, po, pl, _, ps, pw = _kv4_step(q, None, None, kv4, None, out, lse, None,
                                                         sel, workspace)
    _check(_lib.resa_attend_blocks_kv4(dims, pq, p4, int(length), ps, n, float(softmax_scale), po,
                                       pl, pw, workspace.numel(), _stream(stream)),
           "resa_attend_blocks_kv4")


def wait_check(flag, target: int, limit_us: int, workspace, stream=None) -> None:
    """Enqueue the device's bounded wait on `flag` (int32 CUDA tensor) reaching
    `target`; a wait that runs out shows as RESA_ERR_TIMEOUT in
    workspace_status()."""
    _check(_lib.resa_wait_check(_ptr(flag), int(target), int(limit_us), _ptr(workspace),
                                _stream(stream)), "resa_wait_check")
