"""ctypes binding of libdevscan.so (include/devscan.h).

Argument marshalling only: every step of a scan, compaction or language-model
operator runs in the HIP kernels of the library. torch provides device memory
and streams. Importing this module fails with ImportError when the library has
not been built; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdevscan.so")

# ds_dtype, ds_cmp, ds_algo, ds_status (include/devscan.h)
DS_INT32, DS_UINT32, DS_FP32, DS_INT64, DS_UINT64, DS_BF16, DS_FP16, DS_FP8_E4M3 = range(8)
CMP = {"<": 0, "<=": 1, ">": 2, ">=": 3, "==": 4, "!=": 5}
ALGO = {"default": 0, "lookback": 1, "three_pass": 2, "lookback_blocked": 3}
DS_OK = 0
DS_ERR_INVALID_VALUE = 1
DS_ERR_UNSUPPORTED_DTYPE = 2
DS_ERR_OVERLAP = 3
DS_ERR_OUT_OF_MEMORY = 4
DS_ERR_HIP = 5
DS_ERR_MISALIGNED = 6
DS_ERR_TOO_LARGE = 7
DS_ERR_STREAM_CAPTURING = 8

EXPORTS = ["scan_exclusive", "scan_inclusive", "ds_scan", "ds_scan_seeded", "ds_scan_noalloc", "compact_if",
           "ds_compact_unordered", "ds_radix_pass", "ds_moe_align", "ds_embedding", "ds_embedding_grad",
           "ds_embedding_grad_scratch", "ds_embedding_grad_scratch_bytes", "ds_moe_experts_scratch",
           "ds_moe_experts_scratch_bytes", "ds_moe_route", "ds_moe_route_grad", "ds_moe_route_grad_biased",
           "ds_moe_experts", "ds_gated_scan", "ds_gated_scan_scratch_bytes", "ds_gated_scan_grad", "ds_gated_step",
           "ds_grouped_matmul", "ds_grouped_matmul_grad", "ds_page_slots", "ds_copy", "ds_bandwidth_pattern", "ds_tile_scan", "ds_tile_pipeline", "ds_tile_elems",
           "ds_scan_tile_elems", "ds_query_timeout", "ds_fail_next_allocations", "ds_set_spin_limit",
           "ds_status_string", "ds_release_workspace", "ds_version"]
TILE_OF = {"scan_exclusive": 0, "scan_inclusive": 1, "three_pass": 2, "compact": 3, "lds_tile_scan": 4,
           "counting_sort": 5, "counting_sort_values": 6, "moe_align": 7}
TILE_VARIANTS = {"tree": 0, "tree_pad1": 1, "tree_pad2": 2, "hillis_steele": 3}
PATTERNS = {"read": 0, "write": 1, "copy": 2, "read_half": 3, "read_half_held": 4, "copy_held": 5}


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python primitives_device_scan_amd/build.py` "
                          "(or __graft_entry__.build()); there is no CPU fallback")
    L = ctypes.CDLL(path)
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    for name in ("scan_exclusive", "scan_inclusive"):
        getattr(L, name).argtypes = [I, P, P, I64, P]
        getattr(L, name).restype = I
    L.ds_scan.argtypes = [I, I, I, P, P, I64, P]
    L.ds_scan.restype = I
    L.ds_scan_seeded.argtypes = [I, I, P, P, I64, P, P]
    L.ds_scan_seeded.restype = I
    L.ds_scan_noalloc.argtypes = [I, I, P, P, I64, P]
    L.ds_scan_noalloc.restype = I
    L.compact_if.argtypes = [I, P, P, P, I64, I, ctypes.c_uint64, P]
    L.compact_if.restype = I
    L.ds_compact_unordered.argtypes = [I, P, P, P, I64, I, ctypes.c_uint64, I, P]
    L.ds_compact_unordered.restype = I
    L.ds_radix_pass.argtypes = [P, P, P, P, I64, I, I, P]
    L.ds_radix_pass.restype = I
    L.ds_moe_align.argtypes = [P, I64, I, I, P, P, P, I64, P]
    L.ds_moe_align.restype = I
    F = ctypes.c_float
    L.ds_embedding.argtypes = [I, P, I64, I64, I64, P, I, I64, F, P, I64, P]
    L.ds_embedding.restype = I
    L.ds_embedding_grad.argtypes = [I, P, I64, P, I, I64, F, I, P, I64, I64, I64, I, P]
    L.ds_embedding_grad.restype = I
    L.ds_embedding_grad_scratch.argtypes = [I, P, I64, P, I, I64, F, I, P, I64, I64, I64, I, P, I64, P]
    L.ds_embedding_grad_scratch.restype = I
    L.ds_embedding_grad_scratch_bytes.argtypes = [I, I64, I64, I64]
    L.ds_embedding_grad_scratch_bytes.restype = I64
    L.ds_moe_route.argtypes = [I, P, I64, I, I64, P, I, I, I, F, P, P, P]
    L.ds_moe_route.restype = I
    L.ds_moe_route_grad.argtypes = [I, P, I64, I, I64, P, P, I, I, I, F, P, I64, P]
    L.ds_moe_route_grad.restype = I
    L.ds_moe_route_grad_biased.argtypes = [I, P, I64, I, I64, P, P, P, I, I, I, F, P, I64, P]
    L.ds_moe_route_grad_biased.restype = I
    L.ds_moe_experts.argtypes = [I, P, I64, I64, I64, I, P, P, P, P, I, I64, P, P, I, P, I64, P]
    L.ds_moe_experts.restype = I
    L.ds_moe_experts_scratch.argtypes = [I, P, I64, I64, I64, I, P, P, P, P, I, I64, P, P, I, P, I64, P, I64, P]
    L.ds_moe_experts_scratch.restype = I
    L.ds_moe_experts_scratch_bytes.argtypes = [I, I64, I64, I, I64, I]
    L.ds_moe_experts_scratch_bytes.restype = I64
    L.ds_gated_scan_scratch_bytes.argtypes = [I, I, I64, I64]
    L.ds_gated_scan_scratch_bytes.restype = I64
    L.ds_gated_scan.argtypes = [I, P, I64, P, I64, I64, I64, P, I64, I, I, P, P, I64, P, P, I64, P]
    L.ds_gated_scan.restype = I
    L.ds_gated_scan_grad.argtypes = [I, P, I64, P, I64, P, I64, P, I64, I64, I64, P, I64, I, I, P, P, P, I64, P, I64, P,
                                     P, I64, P]
    L.ds_gated_scan_grad.restype = I
    L.ds_gated_step.argtypes = [I, P, I64, P, I64, I64, I64, P, P, I64, I64, I, I, P, I64, P]
    L.ds_gated_step.restype = I
    L.ds_grouped_matmul.argtypes = [I, P, I64, I64, P, I, I64, I64, I, P, I64, P, I, P, I64, P]
    L.ds_grouped_matmul.restype = I
    L.ds_grouped_matmul_grad.argtypes = [I, P, I64, I64, P, I64, I64, P, I, P, I, I64, I64, I, P, I, P]
    L.ds_grouped_matmul_grad.restype = I
    L.ds_page_slots.argtypes = [P, P, I64, P, I64, I64, P, I64, P, I, P, P, P, I64, P, P]
    L.ds_page_slots.restype = I
    L.ds_copy.argtypes = [P, P, I64, P]
    L.ds_copy.restype = I
    L.ds_bandwidth_pattern.argtypes = [I, I, I, P, P, I64, P]
    L.ds_bandwidth_pattern.restype = I
    L.ds_tile_scan.argtypes = [I, I, P, P, P, I64, P]
    L.ds_tile_scan.restype = I
    L.ds_tile_pipeline.argtypes = [I, I, P, P, I64, P]
    L.ds_tile_pipeline.restype = I
    L.ds_query_timeout.argtypes = [P, ctypes.POINTER(I)]
    L.ds_query_timeout.restype = I
    L.ds_fail_next_allocations.argtypes = [I]
    L.ds_fail_next_allocations.restype = I
    L.ds_set_spin_limit.argtypes = [ctypes.c_uint32]
    L.ds_set_spin_limit.restype = I
    L.ds_status_string.argtypes = [I]
    L.ds_status_string.restype = ctypes.c_char_p
    L.ds_release_workspace.argtypes = []
    L.ds_release_workspace.restype = None
    L.ds_tile_elems.argtypes = [I, I]
    L.ds_tile_elems.restype = I64
    L.ds_scan_tile_elems.argtypes = [I, I, I64]
    L.ds_scan_tile_elems.restype = I64
    L.ds_version.argtypes = []
    L.ds_version.restype = I
    return L


lib = load_library()


class DevscanError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib.ds_status_string(status).decode()}")


def _check(status: int, what: str):
    if status != DS_OK:
        raise DevscanError(status, what)


_DTYPES = {torch.int32: DS_INT32, torch.float32: DS_FP32, torch.int64: DS_INT64}
if hasattr(torch, "uint32"):
    _DTYPES[torch.uint32] = DS_UINT32
if hasattr(torch, "uint64"):
    _DTYPES[torch.uint64] = DS_UINT64


def dtype_code(dt: torch.dtype) -> int:
    if dt not in _DTYPES:
        raise TypeError(f"unsupported dtype {dt}; one of {list(_DTYPES)}")
    return _DTYPES[dt]


def _stream_handle(x: torch.Tensor, stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(x.device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check_tensor(x: torch.Tensor, name: str):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def scan(x: torch.Tensor, inclusive: bool, out: torch.Tensor | None = None, *, algo: str = "default",
         stream=None) -> torch.Tensor:
    """Exclusive or inclusive scan of the 1-D contiguous GPU tensor x (into out, may be x)."""
    _check_tensor(x, "x")
    code = dtype_code(x.dtype)
    if out is None:
        out = torch.empty_like(x)
    _check_tensor(out, "out")
    if out.dtype != x.dtype or out.numel() != x.numel() or out.device != x.device:
        raise ValueError("out must match x in dtype, size and device")
    with torch.cuda.device(x.device):
        _check(lib.ds_scan(code, int(bool(inclusive)), ALGO[algo], x.data_ptr(), out.data_ptr(), x.numel(),
                           _stream_handle(x, stream)), "ds_scan")
    return out


def scan_seeded(x: torch.Tensor, inclusive: bool, seed: torch.Tensor | None, out: torch.Tensor | None = None, *,
                stream=None) -> torch.Tensor:
    """One shard of a longer scan: the scan of x with every prefix offset by seed
    (a one-element GPU tensor of x's dtype, or None for 0)."""
    _check_tensor(x, "x")
    code = dtype_code(x.dtype)
    if out is None:
        out = torch.empty_like(x)
    _check_tensor(out, "out")
    if out.dtype != x.dtype or out.numel() != x.numel() or out.device != x.device:
        raise ValueError("out must match x in dtype, size and device")
    if seed is not None and (seed.dtype != x.dtype or seed.numel() != 1 or seed.device != x.device):
        raise ValueError("seed must be one element of x's dtype on x's device")
    with torch.cuda.device(x.device):
        _check(lib.ds_scan_seeded(code, int(bool(inclusive)), x.data_ptr(), out.data_ptr(), x.numel(),
                                  None if seed is None else seed.data_ptr(), _stream_handle(x, stream)),
               "ds_scan_seeded")
    return out


def scan_exclusive(x: torch.Tensor, out: torch.Tensor | None = None, *, stream=None) -> torch.Tensor:
    _check_tensor(x, "x")
    if out is None:
        out = torch.empty_like(x)
    _check_tensor(out, "out")
    if out.dtype != x.dtype or out.numel() != x.numel() or out.device != x.device:
        raise ValueError("out must match x in dtype, size and device")
    with torch.cuda.device(x.device):
        _check(lib.scan_exclusive(dtype_code(x.dtype), x.data_ptr(), out.data_ptr(), x.numel(),
                                  _stream_handle(x, stream)), "scan_exclusive")
    return out


def scan_inclusive(x: torch.Tensor, out: torch.Tensor | None = None, *, stream=None) -> torch.Tensor:
    _check_tensor(x, "x")
    if out is None:
        out = torch.empty_like(x)
    _check_tensor(out, "out")
    if out.dtype != x.dtype or out.numel() != x.numel() or out.device != x.device:
        raise ValueError("out must match x in dtype, size and device")
    with torch.cuda.device(x.device):
        _check(lib.scan_inclusive(dtype_code(x.dtype), x.data_ptr(), out.data_ptr(), x.numel(),
                                  _stream_handle(x, stream)), "scan_inclusive")
    return out


def operand_bits(dtype: torch.dtype, value) -> int:
    """The bit pattern compact_if expects for `value` in `dtype`."""
    code = dtype_code(dtype)
    if code == DS_FP32:
        return struct.unpack("<I", struct.pack("<f", float(value)))[0]
    if code in (DS_INT32, DS_UINT32):
        return int(value) & 0xFFFFFFFF
    return int(value) & 0xFFFFFFFFFFFFFFFF


def compact_if(x: torch.Tensor, cmp: str, operand, out: torch.Tensor | None = None,
               num_selected: torch.Tensor | None = None, *, stream=None):
    """Order-preserving compaction of x by (x_i cmp operand).

    Returns (out, num_selected): out holds the kept elements in out[:k], and
    num_selected is a one-element int64 GPU tensor holding k.
    """
    _check_tensor(x, "x")
    code = dtype_code(x.dtype)
    if out is None:
        out = torch.empty_like(x)
    if num_selected is None:
        num_selected = torch.empty(1, dtype=torch.int64, device=x.device)
    _check_tensor(out, "out")
    _check_tensor(num_selected, "num_selected")
    if out.dtype != x.dtype or out.numel() < x.numel() or out.device != x.device:
        raise ValueError("out must match x in dtype and device and hold x.numel() elements")
    if num_selected.dtype != torch.int64 or num_selected.numel() < 1:
        raise ValueError("num_selected must be an int64 tensor of at least one element")
    with torch.cuda.device(x.device):
        _check(lib.compact_if(code, x.data_ptr(), out.data_ptr(), num_selected.data_ptr(), x.numel(), CMP[cmp],
                              operand_bits(x.dtype, operand), _stream_handle(x, stream)), "compact_if")
    return out, num_selected


CLAIM = {"wave": 0, "workgroup": 1}


def compact_unordered(x: torch.Tensor, cmp: str, operand, out: torch.Tensor | None = None,
                      num_selected: torch.Tensor | None = None, *, claim: str = "workgroup", stream=None):
    """Compaction in no particular order (atomic space claims); returns (out, num_selected)."""
    _check_tensor(x, "x")
    code = dtype_code(x.dtype)
    out = torch.empty_like(x) if out is None else out
    num_selected = torch.empty(1, dtype=torch.int64, device=x.device) if num_selected is None else num_selected
    _check_tensor(out, "out")
    _check_tensor(num_selected, "num_selected")
    if out.dtype != x.dtype or out.numel() < x.numel() or num_selected.dtype != torch.int64:
        raise ValueError("out must match x and hold x.numel() elements; num_selected must be int64")
    with torch.cuda.device(x.device):
        _check(lib.ds_compact_unordered(code, x.data_ptr(), out.data_ptr(), num_selected.data_ptr(), x.numel(),
                                        CMP[cmp], operand_bits(x.dtype, operand), CLAIM[claim],
                                        _stream_handle(x, stream)), "ds_compact_unordered")
    return out, num_selected


def radix_pass(keys: torch.Tensor, shift: int, bits: int, vals: torch.Tensor | None = None,
               keys_out: torch.Tensor | None = None, vals_out: torch.Tensor | None = None, *, stream=None):
    """One stable counting-sort pass over the digit (key >> shift) & (2^bits - 1) of 32-bit keys
    (int32 or uint32 storage, compared as unsigned); returns (keys_out, vals_out or None)."""
    _check_tensor(keys, "keys")
    if keys.element_size() != 4 or keys.is_floating_point():
        raise TypeError("keys must be 32-bit integers")
    keys_out = torch.empty_like(keys) if keys_out is None else keys_out
    _check_tensor(keys_out, "keys_out")
    if vals is not None:
        _check_tensor(vals, "vals")
        vals_out = torch.empty_like(vals) if vals_out is None else vals_out
        _check_tensor(vals_out, "vals_out")
        if vals.element_size() != 4 or vals.numel() != keys.numel() or vals_out.numel() < keys.numel():
            raise ValueError("vals must hold one 32-bit value per key")
    if keys_out.numel() < keys.numel():
        raise ValueError("keys_out is too small")
    with torch.cuda.device(keys.device):
        _check(lib.ds_radix_pass(keys.data_ptr(), keys_out.data_ptr(), None if vals is None else vals.data_ptr(),
                                 None if vals is None else vals_out.data_ptr(), keys.numel(), shift, bits,
                                 _stream_handle(keys, stream)), "ds_radix_pass")
    return keys_out, (vals_out if vals is not None else None)


def moe_align(topk_ids: torch.Tensor, num_experts: int, block: int, *, stream=None):
    """MoE alignment of int32 expert ids [tokens, top_k]: returns (counts[E], offsets[E+1],
    sorted_ids[capacity]); the first offsets[E] entries of sorted_ids are written."""
    _check_tensor(topk_ids, "topk_ids")
    if topk_ids.dtype != torch.int32:
        raise TypeError("topk_ids must be int32")
    n = topk_ids.numel()
    cap = max(1, n + num_experts * (block - 1))
    dev = topk_ids.device
    counts = torch.empty(num_experts, dtype=torch.int32, device=dev)
    offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
    sorted_ids = torch.empty(cap, dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        _check(lib.ds_moe_align(topk_ids.data_ptr(), n, num_experts, block, counts.data_ptr(), offsets.data_ptr(),
                                sorted_ids.data_ptr(), cap, _stream_handle(topk_ids, stream)), "ds_moe_align")
    return counts, offsets, sorted_ids


# Language-model operators. Their matrices are 2-D tensors whose rows are contiguous; rows may be any distance apart. They
# record nothing for autograd and refuse tensors that require grad while it is on; the gradients are calls of their own.
# Small calls are bound by this code, not by the GPU, so the checks of what is right ask each tensor a few questions and
# the rest is left to the functions that say what is wrong.
_FLOATS = {torch.float32: DS_FP32, torch.bfloat16: DS_BF16, torch.float16: DS_FP16}
_ID_BYTES = {torch.int32: 4, torch.int64: 8}
SCORES = {"softmax": 0, "sigmoid": 1}
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _float_code(x: torch.Tensor, name: str) -> int:
    code = _FLOATS.get(x.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, not {x.dtype}")
    return code


def _check_rows(x: torch.Tensor, name: str, rows: int | None = None, cols: int | None = None,
                like: torch.Tensor | None = None) -> int:
    """x is a 2-D GPU tensor with contiguous rows, of the given shape and on like's device; returns its row stride."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if x.dim() != 2:
        raise ValueError(f"{name} must be a matrix, not of shape {list(x.shape)}")
    n, m = x.shape
    if (rows is not None and n != rows) or (cols is not None and m != cols):
        raise ValueError(f"{name} must be a matrix of shape [{'*' if rows is None else rows}, "
                         f"{'*' if cols is None else cols}], not {[n, m]}")
    if like is not None and x.get_device() != like.get_device():
        raise ValueError(f"{name} must be on {like.device}")
    if x.is_contiguous():
        return m
    if m > 1 and x.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if n <= 1 or m == 0:
        return m
    if x.stride(0) < m:
        raise ValueError(f"the rows of {name} must not overlap")
    return x.stride(0)


def _check_flat(x: torch.Tensor, name: str, dtype, shape, like: torch.Tensor):
    """x is contiguous, of the dtype (or a key of the dict of them) and shape given, on like's device."""
    _check_tensor(x, name)
    if x.dtype not in dtype if isinstance(dtype, dict) else x.dtype != dtype:
        names = " or ".join(str(d) for d in dtype) if isinstance(dtype, dict) else str(dtype)
        raise TypeError(f"{name} must be {names}, not {x.dtype}")
    if shape is not None and x.shape != shape:
        raise ValueError(f"{name} must have the shape {list(shape)}, not {list(x.shape)}")
    if x.get_device() != like.get_device():
        raise ValueError(f"{name} must be on {like.device}")


def _refuse_history(*tensors):
    """These calls record nothing for autograd: a result that looked like any other would lose its gradient."""
    if torch.is_grad_enabled():
        for t in tensors:
            if getattr(t, "requires_grad", False):
                raise ValueError("a tensor that requires grad: these calls have no autograd history; detach it or call "
                                 "them under torch.no_grad(), and use embedding_grad, moe_route_grad, gated_scan_grad and "
                                 "grouped_matmul_grad for gradients")


def _elsewhere(x: torch.Tensor, stream) -> bool:
    """Whether a call on x runs on another stream than the current one of the current device."""
    return stream is not None or x.get_device() != _current_device()


def _stream_of(x: torch.Tensor) -> int:
    return torch.cuda.current_stream(x.device).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    def _stream_of(x: torch.Tensor) -> int:  # noqa: F811  the same without a Stream object, 2 us less per call
        return torch._C._cuda_getCurrentRawStream(x.get_device())


_recording = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


# A call that is being recorded takes its scratch from the graph's own memory (torch allocates there during a capture, and
# the graph keeps it): the stream's workspace is shared with every other graph recorded on it and with its eager calls.
def _scratch_of(x: torch.Tensor, room: int) -> torch.Tensor | None:
    return x.new_empty(room, dtype=torch.uint8) if room else None


def _call_elsewhere(call, x: torch.Tensor, stream, used):
    """call() with x's device and the stream current: outputs are allocated on the stream that the call runs on, and
    tensors that belong to another stream are kept from reuse until the call has run."""
    if stream is None:
        with torch.cuda.device(x.device):
            return call()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=x.device)
    with torch.cuda.stream(stream):  # also makes the stream's device current
        if _current_device() != x.get_device():
            raise ValueError(f"the stream must be one of {x.device}")
        result = call()
        for t in used:
            if t is not None:
                t.record_stream(stream)
    return result


def embedding(table: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """scale * table[ids] (int32 or int64 ids of any shape); a row of zeros where an id is no row of the table.
    Returns [*ids.shape, dim]; `out`, if given, is a matrix [ids.numel(), dim] and is returned as it is."""
    _refuse_history(table, out)
    code = _float_code(table, "table")
    stride = _check_rows(table, "table")
    _check_flat(ids, "ids", _ID_BYTES, None, table)
    if _elsewhere(table, stream):
        return _call_elsewhere(lambda: embedding(table, ids, scale=scale, out=out), table, stream, (table, ids, out))
    rows, dim = table.shape
    n = ids.numel()
    shaped = None
    if out is None:
        shape = ids.shape
        if len(shape) == 1:
            out = table.new_empty((n, dim))
        else:
            shaped = table.new_empty((*shape, dim))
            out = shaped.view(n, dim)
        out_stride = dim
    else:
        out_stride = _check_rows(out, "out", n, dim, table)
        if out.dtype != table.dtype:
            raise TypeError("out must have the table's dtype")
    _check(lib.ds_embedding(code, table.data_ptr(), rows, dim, stride, ids.data_ptr(), _ID_BYTES[ids.dtype], n, scale,
                            out.data_ptr(), out_stride, _stream_of(table)), "ds_embedding")
    return out if shaped is None else shaped


def embedding_grad(dout: torch.Tensor, ids: torch.Tensor, rows: int, *, scale: float = 1.0,
                   dtype: torch.dtype | None = None, out: torch.Tensor | None = None, accumulate: bool = False,
                   stream=None) -> torch.Tensor:
    """The gradient of embedding's table [rows, dim] from the gradient dout of its output ([*ids.shape, dim], or
    [ids.numel(), dim] with rows any distance apart). `dtype` is dout's (the default) or float32. accumulate: the sums
    are added to `out`; otherwise every row is written, into `out` if it is given."""
    _refuse_history(dout, out)
    if not isinstance(dout, torch.Tensor) or dout.dim() < 1:
        raise ValueError("dout must be a GPU tensor")
    if dout.dim() != 2:
        if dout.shape[:-1] != ids.shape or not dout.is_contiguous():
            raise ValueError("dout must be a matrix, or contiguous of shape [*ids.shape, dim]")
        dout = dout.view(ids.numel(), dout.shape[-1])
    code = _float_code(dout, "dout")
    n = ids.numel()
    stride = _check_rows(dout, "dout", n)
    _check_flat(ids, "ids", _ID_BYTES, None, dout)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if dtype is None:
        dtype = dout.dtype if out is None else out.dtype
    if dtype != dout.dtype and dtype != torch.float32:
        raise TypeError("the gradient's dtype must be dout's or float32")
    if _elsewhere(dout, stream):
        return _call_elsewhere(lambda: embedding_grad(dout, ids, rows, scale=scale, dtype=dtype, out=out,
                                                      accumulate=accumulate), dout, stream, (dout, ids, out))
    dim = dout.shape[1]
    if out is None:
        out = dout.new_empty((rows, dim), dtype=dtype)
        grad_stride = dim
    else:
        grad_stride = _check_rows(out, "out", rows, dim, dout)
        if out.dtype != dtype:
            raise TypeError(f"out must be {dtype}")
    scratch, room = None, 0
    if _recording():
        room = lib.ds_embedding_grad_scratch_bytes(_FLOATS[dtype], n, rows, dim)
        scratch = _scratch_of(dout, room)
    _check(lib.ds_embedding_grad_scratch(code, dout.data_ptr(), stride, ids.data_ptr(), _ID_BYTES[ids.dtype], n, scale,
                                         _FLOATS[dtype], out.data_ptr(), rows, dim, grad_stride, 1 if accumulate else 0,
                                         None if scratch is None else scratch.data_ptr(), room, _stream_of(dout)),
           "ds_embedding_grad")
    return out


def moe_route(logits: torch.Tensor, top_k: int, *, score: str = "softmax", bias: torch.Tensor | None = None,
              renormalize: bool = True, scale: float = 1.0, stream=None):
    """Each token's top_k experts by logit (+ bias, float32 [experts], for the choice alone), ties to the lower index;
    returns (weights float32, ids int32), both [tokens, top_k], best first. weights = scale * score, where score is
    "softmax" over the experts that can be chosen or "sigmoid", with renormalize divided by its sum over the chosen.
    Experts at -inf or NaN cannot be chosen; where fewer than top_k can, the rest is id -1 with weight 0."""
    _refuse_history(logits, bias)
    code = _float_code(logits, "logits")
    stride = _check_rows(logits, "logits")
    tokens, experts = logits.shape
    if bias is not None:
        _check_flat(bias, "bias", torch.float32, (experts,), logits)
    if score not in SCORES:
        raise ValueError(f"score must be one of {list(SCORES)}")
    if not 1 <= top_k <= experts:
        raise ValueError("top_k must be between 1 and the number of experts")
    if _elsewhere(logits, stream):
        return _call_elsewhere(lambda: moe_route(logits, top_k, score=score, bias=bias, renormalize=renormalize,
                                                 scale=scale), logits, stream, (logits, bias))
    weights = logits.new_empty((tokens, top_k), dtype=torch.float32)
    ids = logits.new_empty((tokens, top_k), dtype=torch.int32)
    _check(lib.ds_moe_route(code, logits.data_ptr(), tokens, experts, stride, None if bias is None else bias.data_ptr(),
                            top_k, SCORES[score], 1 if renormalize else 0, scale, weights.data_ptr(), ids.data_ptr(),
                            _stream_of(logits)), "ds_moe_route")
    return weights, ids


def moe_route_grad(logits: torch.Tensor, ids: torch.Tensor, dweights: torch.Tensor, *, score: str = "softmax",
                   bias: torch.Tensor | None = None, renormalize: bool = True, scale: float = 1.0,
                   stream=None) -> torch.Tensor:
    """The gradient of moe_route's weights with respect to its logits, from the ids it chose and the gradient dweights
    (float32 [tokens, top_k]) of the weights, for the score, bias, renormalize and scale that it had; in the logits'
    dtype."""
    _refuse_history(logits, dweights, bias)
    code = _float_code(logits, "logits")
    stride = _check_rows(logits, "logits")
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens, top_k]")
    tokens, experts = logits.shape
    top_k = ids.shape[1]
    _check_flat(ids, "ids", torch.int32, (tokens, top_k), logits)
    _check_flat(dweights, "dweights", torch.float32, (tokens, top_k), logits)
    if bias is not None:
        _check_flat(bias, "bias", torch.float32, (experts,), logits)
    if score not in SCORES:
        raise ValueError(f"score must be one of {list(SCORES)}")
    if _elsewhere(logits, stream):
        return _call_elsewhere(lambda: moe_route_grad(logits, ids, dweights, score=score, bias=bias,
                                                      renormalize=renormalize, scale=scale), logits, stream,
                               (logits, ids, dweights, bias))
    dlogits = logits.new_empty((tokens, experts))
    _check(lib.ds_moe_route_grad_biased(code, logits.data_ptr(), tokens, experts, stride,
                                        None if bias is None else bias.data_ptr(), ids.data_ptr(), dweights.data_ptr(),
                                        top_k, SCORES[score], 1 if renormalize else 0, scale, dlogits.data_ptr(),
                                        experts, _stream_of(logits)), "ds_moe_route_grad")
    return dlogits


def moe_experts(x: torch.Tensor, w_in: torch.Tensor, w_out: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, *,
                w_in_scale: torch.Tensor | None = None, w_out_scale: torch.Tensor | None = None,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The experts of a mixture-of-experts layer for a few tokens (tokens * top_k <= 8192): for each token the sum over
    its choices e = ids[t, j] of weights[t, j] * w_out[e] @ (silu(gate) * up), where gate and up are the first and
    second half of w_in[e] @ x[t]. x [tokens, dim] bfloat16 or float16; w_in [experts, 2 * hidden, dim] and w_out
    [experts, dim, hidden] in x's dtype, or float8_e4m3fn with a float32 scale for every block of 128 x 128
    ([experts, ceil(rows / 128), ceil(columns / 128)]); ids int32, weights float32 [tokens, top_k]. Choices outside
    [0, experts) are left out."""
    _refuse_history(x, w_in, w_out, weights, w_in_scale, w_out_scale, out)
    code = _float_code(x, "x")
    if code == DS_FP32:
        raise TypeError("x must be bfloat16 or float16")
    x_stride = _check_rows(x, "x")
    tokens, dim = x.shape
    if w_in.dim() != 3 or w_in.shape[1] % 2 or ids.dim() != 2:
        raise ValueError("w_in must be [experts, 2 * hidden, dim] and ids [tokens, top_k]")
    experts, both, _ = w_in.shape
    hidden, top_k = both // 2, ids.shape[1]
    eight = w_in.dtype == torch.float8_e4m3fn
    kind = torch.float8_e4m3fn if eight else x.dtype
    _check_flat(w_in, "w_in", kind, (experts, both, dim), x)
    _check_flat(w_out, "w_out", kind, (experts, dim, hidden), x)
    if eight != (w_in_scale is not None) or eight != (w_out_scale is not None):
        raise ValueError("8-bit weights, and only they, need w_in_scale and w_out_scale")
    if eight:
        blocks = [-(-v // 128) for v in (both, dim, hidden)]
        _check_flat(w_in_scale, "w_in_scale", torch.float32, (experts, blocks[0], blocks[1]), x)
        _check_flat(w_out_scale, "w_out_scale", torch.float32, (experts, blocks[1], blocks[2]), x)
    _check_flat(ids, "ids", torch.int32, (tokens, top_k), x)
    _check_flat(weights, "weights", torch.float32, (tokens, top_k), x)
    if _elsewhere(x, stream):
        return _call_elsewhere(lambda: moe_experts(x, w_in, w_out, ids, weights, w_in_scale=w_in_scale,
                                                   w_out_scale=w_out_scale, out=out), x, stream,
                               (x, w_in, w_out, ids, weights, w_in_scale, w_out_scale, out))
    if out is None:
        out = x.new_empty((tokens, dim))
        y_stride = dim
    else:
        y_stride = _check_rows(out, "out", tokens, dim, x)
        if out.dtype != x.dtype:
            raise TypeError("out must have x's dtype")
    weight_code = DS_FP8_E4M3 if eight else code
    scratch, room = None, 0
    if _recording():
        room = lib.ds_moe_experts_scratch_bytes(weight_code, tokens, dim, experts, hidden, top_k)
        scratch = _scratch_of(x, room)
    _check(lib.ds_moe_experts_scratch(code, x.data_ptr(), tokens, dim, x_stride, weight_code, w_in.data_ptr(),
                                      w_in_scale.data_ptr() if eight else None, w_out.data_ptr(),
                                      w_out_scale.data_ptr() if eight else None, experts, hidden, ids.data_ptr(),
                                      weights.data_ptr(), top_k, out.data_ptr(), y_stride,
                                      None if scratch is None else scratch.data_ptr(), room, _stream_of(x)),
           "ds_moe_experts")
    return out


# Operators on ragged batches. Offsets and lengths stay on the GPU: no call waits for the host.
GATES = {"decay": 0, "log": 1, "sigmoid": 2}


def _ptr(x: torch.Tensor | None):
    return None if x is None else x.data_ptr()


def _check_like(x: torch.Tensor, name: str, like: torch.Tensor, what: str) -> int:
    """x is a matrix of like's shape, dtype and device, with contiguous rows; returns its row stride."""
    stride = _check_rows(x, name, like.shape[0], like.shape[1], like)
    if x.dtype != like.dtype:
        raise TypeError(f"{name} must have {what}'s dtype")
    return stride


def _check_sequences(offsets: torch.Tensor | None, like: torch.Tensor) -> int:
    if offsets is None:
        return 1
    _check_flat(offsets, "offsets", torch.int32, None, like)
    if offsets.dim() != 1 or offsets.numel() < 1:
        raise ValueError("offsets must hold one entry more than there are sequences")
    return offsets.numel() - 1


def gated_scan(gate: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor | None = None, *, form: str = "sigmoid",
               mix: bool = False, initial: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None):
    """A gated linear recurrence over packed sequences: h_t = a_t h_{t-1} + x_t, with mix a_t h_{t-1} + (1 - a_t) x_t.
    gate and x are [tokens, dim]; a_t is the gate ("decay"), its exponential ("log", gates at most 0) or its sigmoid. (Gates
    have x's dtype: between 1 - 2^-8 and 1 bfloat16 holds no number, float16 from 1 - 2^-11 on, so that memories of more
    than some 256 or 2,048 steps need "log" or "sigmoid" there.)
    Sequence s holds the rows offsets[s] to offsets[s + 1] (int32 [sequences + 1]; None: all rows are one sequence) and
    starts from initial[s] (float32 [sequences, dim], or None for 0). Returns (h, final): h [tokens, dim] in x's dtype,
    into `out` if it is given (rows outside the sequences are not written), and final float32 [sequences, dim], the
    states after each sequence's last row."""
    _refuse_history(gate, x, initial, out)
    code = _float_code(x, "x")
    x_stride = _check_rows(x, "x")
    gate_stride = _check_like(gate, "gate", x, "x")
    if form not in GATES:
        raise ValueError(f"form must be one of {list(GATES)}")
    sequences = _check_sequences(offsets, x)
    tokens, dim = x.shape
    if initial is not None:
        _check_flat(initial, "initial", torch.float32, (sequences, dim), x)
    if _elsewhere(x, stream):
        return _call_elsewhere(lambda: gated_scan(gate, x, offsets, form=form, mix=mix, initial=initial, out=out), x,
                               stream, (gate, x, offsets, initial, out))
    if out is None:
        out = x.new_empty((tokens, dim))
        stride = dim
    else:
        stride = _check_like(out, "out", x, "x")
    final = x.new_empty((sequences, dim), dtype=torch.float32)
    scratch, room = None, 0
    if _recording():
        room = lib.ds_gated_scan_scratch_bytes(code, 0, tokens, dim)
        scratch = _scratch_of(x, room)
    _check(lib.ds_gated_scan(code, gate.data_ptr(), gate_stride, x.data_ptr(), x_stride, tokens, dim, _ptr(offsets),
                             sequences, GATES[form], 1 if mix else 0, _ptr(initial), out.data_ptr(), stride,
                             final.data_ptr(), _ptr(scratch), room, _stream_of(x)), "ds_gated_scan")
    return out, final


def gated_scan_grad(gate: torch.Tensor, h: torch.Tensor, dh: torch.Tensor, offsets: torch.Tensor | None = None, *,
                    x: torch.Tensor | None = None, form: str = "sigmoid", mix: bool = False,
                    initial: torch.Tensor | None = None, dfinal: torch.Tensor | None = None, stream=None):
    """The gradients of gated_scan's gate, x and initial states, from its gate, the h that it gave, the gradient dh of h
    and dfinal of the final states (float32 [sequences, dim], or None for 0). With mix it needs x too. Returns (dgate,
    dx, dinitial), the first two in h's dtype (rows outside the sequences are not written), dinitial float32."""
    _refuse_history(gate, h, dh, x, initial, dfinal)
    code = _float_code(h, "h")
    h_stride = _check_rows(h, "h")
    gate_stride = _check_like(gate, "gate", h, "h")
    dh_stride = _check_like(dh, "dh", h, "h")
    if mix and x is None:
        raise ValueError("with mix the gradient needs x")
    x_stride = _check_like(x, "x", h, "h") if mix else 0
    if form not in GATES:
        raise ValueError(f"form must be one of {list(GATES)}")
    sequences = _check_sequences(offsets, h)
    tokens, dim = h.shape
    for name, t in (("initial", initial), ("dfinal", dfinal)):
        if t is not None:
            _check_flat(t, name, torch.float32, (sequences, dim), h)
    if _elsewhere(h, stream):
        return _call_elsewhere(lambda: gated_scan_grad(gate, h, dh, offsets, x=x, form=form, mix=mix, initial=initial,
                                                       dfinal=dfinal), h, stream,
                               (gate, h, dh, offsets, x, initial, dfinal))
    dgate, dx = h.new_empty((tokens, dim)), h.new_empty((tokens, dim))
    dinitial = h.new_empty((sequences, dim), dtype=torch.float32)
    scratch, room = None, 0
    if _recording():
        room = lib.ds_gated_scan_scratch_bytes(code, 1, tokens, dim)
        scratch = _scratch_of(h, room)
    _check(lib.ds_gated_scan_grad(code, gate.data_ptr(), gate_stride, h.data_ptr(), h_stride, dh.data_ptr(), dh_stride,
                                  x.data_ptr() if mix else None, x_stride, tokens, dim, _ptr(offsets), sequences,
                                  GATES[form], 1 if mix else 0, _ptr(initial), _ptr(dfinal), dgate.data_ptr(), dim,
                                  dx.data_ptr(), dim, dinitial.data_ptr(), _ptr(scratch), room, _stream_of(h)),
           "ds_gated_scan_grad")
    return dgate, dx, dinitial


def gated_step(gate: torch.Tensor, x: torch.Tensor, state: torch.Tensor, slots: torch.Tensor | None = None, *,
               form: str = "sigmoid", mix: bool = False, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gated_scan's step for one token of each of several sequences, their states held in a pool: state[slots[i]]
    (float32 [pool, dim]; slots int32 [rows], None: row i's slot is i) takes row i of gate and x [rows, dim], in place,
    and the new state is returned in x's dtype. A row whose slot is none of the pool's is zeros; rows of one slot are its
    tokens in their order."""
    _refuse_history(gate, x, state, out)
    code = _float_code(x, "x")
    x_stride = _check_rows(x, "x")
    gate_stride = _check_like(gate, "gate", x, "x")
    rows, dim = x.shape
    state_stride = _check_rows(state, "state", None, dim, x)
    if state.dtype != torch.float32:
        raise TypeError("state must be float32")
    pool = state.shape[0]
    if slots is not None:
        _check_flat(slots, "slots", torch.int32, (rows,), x)
    elif pool < rows:
        raise ValueError("without slots every row needs a state of its own")
    if form not in GATES:
        raise ValueError(f"form must be one of {list(GATES)}")
    if _elsewhere(x, stream):
        return _call_elsewhere(lambda: gated_step(gate, x, state, slots, form=form, mix=mix, out=out), x, stream,
                               (gate, x, state, slots, out))
    if out is None:
        out = x.new_empty((rows, dim))
        stride = dim
    else:
        stride = _check_like(out, "out", x, "x")
    _check(lib.ds_gated_step(code, gate.data_ptr(), gate_stride, x.data_ptr(), x_stride, rows, dim, _ptr(slots),
                             state.data_ptr(), pool, state_stride, GATES[form], 1 if mix else 0, out.data_ptr(), stride,
                             _stream_of(x)), "ds_gated_step")
    return out


def _check_batch(x: torch.Tensor, offsets: torch.Tensor, index: torch.Tensor | None, top_k: int):
    """(experts, rows of the batch) that offsets and index give."""
    _check_flat(offsets, "offsets", torch.int32, None, x)
    if offsets.dim() != 1 or offsets.numel() < 1:
        raise ValueError("offsets must hold one entry more than there are experts")
    if index is None:
        return offsets.numel() - 1, x.shape[0]
    _check_flat(index, "index", torch.int32, None, x)
    if not 1 <= top_k < 1 << 31:  # 32 bits in the library
        raise ValueError("top_k must be at least 1 and below 2^31")
    return offsets.numel() - 1, index.numel()


def _sixteen_bit(x: torch.Tensor, name: str) -> int:
    code = _float_code(x, name)
    if code == DS_FP32:
        raise TypeError(f"{name} must be bfloat16 or float16")
    return code


def grouped_matmul(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, *, index: torch.Tensor | None = None,
                   top_k: int = 1, transposed: bool = False, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Products grouped by expert: rows offsets[e] to offsets[e + 1] of the batch (int32 [experts + 1], of moe_align or
    an exclusive scan of counts) are multiplied by w[e] (w [experts, rows, cols], bfloat16 or float16): y = x @ w[e].T,
    with transposed y = x @ w[e], the gradient of the inputs. The batch is x, or with index (int32, moe_align's
    sorted_ids) the rows index // top_k of x, zeros where there is no such row. Returns y [rows of the batch, rows]
    ([.., cols] with transposed), into `out` if it is given; rows outside the groups are not written."""
    _refuse_history(x, w, out)
    code = _sixteen_bit(x, "x")
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("w must be [experts, rows, cols]")
    experts, m = _check_batch(x, offsets, index, top_k)
    rows, cols = w.shape[1:]
    _check_flat(w, "w", x.dtype, (experts, rows, cols), x)
    x_stride = _check_rows(x, "x", None, rows if transposed else cols)
    width = cols if transposed else rows
    if _elsewhere(x, stream):
        return _call_elsewhere(lambda: grouped_matmul(x, w, offsets, index=index, top_k=top_k, transposed=transposed,
                                                      out=out), x, stream, (x, w, offsets, index, out))
    if out is None:
        out = x.new_empty((m, width))
        stride = width
    else:
        stride = _check_rows(out, "out", m, width, x)
        if out.dtype != x.dtype:
            raise TypeError("out must have x's dtype")
    _check(lib.ds_grouped_matmul(code, x.data_ptr(), x.shape[0], x_stride, w.data_ptr(), experts, rows, cols,
                                 1 if transposed else 0, offsets.data_ptr(), m, _ptr(index), top_k, out.data_ptr(),
                                 stride, _stream_of(x)), "ds_grouped_matmul")
    return out


def grouped_matmul_grad(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, *, index: torch.Tensor | None = None,
                        top_k: int = 1, dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                        accumulate: bool = False, stream=None) -> torch.Tensor:
    """The gradient of grouped_matmul's w [experts, rows, cols]: for each expert dy.T @ x over its rows of the batch,
    from the gradient dy [rows of the batch, rows] of the products and the x, offsets, index and top_k that they had (rows
    for which the index names none of x are left out, whatever dy holds there).
    `dtype` is x's (the default) or float32. accumulate: added to `out`; otherwise all of it is written, zeros for an
    expert without rows, into `out` if it is given."""
    _refuse_history(dy, x, out)
    code = _sixteen_bit(x, "x")
    x_stride = _check_rows(x, "x")
    experts, m = _check_batch(x, offsets, index, top_k)
    dy_stride = _check_rows(dy, "dy", m, None, x)
    if dy.dtype != x.dtype:
        raise TypeError("dy must have x's dtype")
    rows, cols = dy.shape[1], x.shape[1]
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if dtype is None:
        dtype = x.dtype if out is None else out.dtype
    if dtype != x.dtype and dtype != torch.float32:
        raise TypeError("the gradient's dtype must be x's or float32")
    if _elsewhere(x, stream):
        return _call_elsewhere(lambda: grouped_matmul_grad(dy, x, offsets, index=index, top_k=top_k, dtype=dtype,
                                                           out=out, accumulate=accumulate), x, stream,
                               (dy, x, offsets, index, out))
    if out is None:
        out = x.new_empty((experts, rows, cols), dtype=dtype)
    else:
        _check_flat(out, "out", dtype, (experts, rows, cols), x)
    _check(lib.ds_grouped_matmul_grad(code, dy.data_ptr(), m, dy_stride, x.data_ptr(), x.shape[0], x_stride,
                                      offsets.data_ptr(), experts, _ptr(index), top_k, rows, cols, _FLOATS[dtype],
                                      out.data_ptr(), 1 if accumulate else 0, _stream_of(x)), "ds_grouped_matmul_grad")
    return out


def page_slots(context: torch.Tensor, new: torch.Tensor, tables: torch.Tensor, free: torch.Tensor, count: torch.Tensor,
               page: int, tokens: int, *, stream=None):
    """Page tables and slot maps of a step. Request r has context[r] tokens in a cache held in pages of `page` tokens,
    listed in tables[r] (int32 [requests, width], rows any distance apart), and new[r] tokens now. Pages that they need
    are taken from the end of the free list (free int32 [capacity], its first count[0] entries) and entered into tables
    in place, -1 where none is left. Returns (offsets int32 [requests + 1], the packed batch's; slots int64 [tokens],
    where each of its tokens is to be kept, -1 for one without a page and for the rest of the batch; positions int32
    [tokens], 0 there; left int32 [1], the count for the next step, negative if pages were missing). All arguments but
    page and tokens, the size of the batch, are on the GPU."""
    _check_flat(context, "context", torch.int32, None, context)
    if context.dim() != 1:
        raise ValueError("context must be [requests]")
    requests = context.numel()
    _check_flat(new, "new", torch.int32, (requests,), context)
    stride = _check_rows(tables, "tables", requests, None, context)
    if tables.dtype != torch.int32:
        raise TypeError("tables must be int32")
    _check_flat(free, "free", torch.int32, None, context)
    _check_flat(count, "count", torch.int32, (1,), context)
    if not 1 <= page < 1 << 31 or tokens < 0:  # 32 bits in the library
        raise ValueError("page must be at least 1 and below 2^31, and tokens at least 0")
    if _elsewhere(context, stream):
        return _call_elsewhere(lambda: page_slots(context, new, tables, free, count, page, tokens), context, stream,
                               (context, new, tables, free, count))
    offsets = context.new_empty(requests + 1)
    slots = context.new_empty(tokens, dtype=torch.int64)
    positions = context.new_empty(tokens)
    left = context.new_empty(1)
    _check(lib.ds_page_slots(context.data_ptr(), new.data_ptr(), requests, tables.data_ptr(), tables.shape[1], stride,
                             free.data_ptr(), free.numel(), count.data_ptr(), page, offsets.data_ptr(), slots.data_ptr(),
                             positions.data_ptr(), tokens, left.data_ptr(), _stream_of(context)), "ds_page_slots")
    return offsets, slots, positions, left


def copy(src: torch.Tensor, dst: torch.Tensor, *, stream=None) -> torch.Tensor:
    """The copy kernel with the scan's access pattern (bandwidth ceiling)."""
    _check_tensor(src, "src")
    _check_tensor(dst, "dst")
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() < nbytes:
        raise ValueError("dst too small")
    with torch.cuda.device(src.device):
        _check(lib.ds_copy(src.data_ptr(), dst.data_ptr(), nbytes, _stream_handle(src, stream)), "ds_copy")
    return dst


def tile_scan(x: torch.Tensor, variant: str, out: torch.Tensor | None = None,
              tile_sums: torch.Tensor | None = None, *, stream=None):
    """Block-level exclusive scan of every 4,096-element tile of x in LDS; returns (out, tile_sums)."""
    _check_tensor(x, "x")
    code = dtype_code(x.dtype)
    out = torch.empty_like(x) if out is None else out
    tiles = (x.numel() + 4095) // 4096
    tile_sums = torch.empty(tiles, dtype=x.dtype, device=x.device) if tile_sums is None else tile_sums
    _check_tensor(out, "out")
    _check_tensor(tile_sums, "tile_sums")
    if tile_sums.numel() < tiles or tile_sums.dtype != x.dtype or out.numel() != x.numel() or out.dtype != x.dtype:
        raise ValueError("out must match x; tile_sums must hold ceil(n/4096) elements of x's dtype")
    with torch.cuda.device(x.device):
        _check(lib.ds_tile_scan(code, TILE_VARIANTS[variant], x.data_ptr(), out.data_ptr(), tile_sums.data_ptr(),
                                x.numel(), _stream_handle(x, stream)), "ds_tile_scan")
    return out, tile_sums


def tile_pipeline(x: torch.Tensor, variant: str, out: torch.Tensor | None = None, *, stream=None) -> torch.Tensor:
    """Device-wide exclusive scan by the three-kernel pipeline over LDS tile scans."""
    _check_tensor(x, "x")
    code = dtype_code(x.dtype)
    out = torch.empty_like(x) if out is None else out
    _check_tensor(out, "out")
    if out.numel() != x.numel() or out.dtype != x.dtype:
        raise ValueError("out must match x")
    with torch.cuda.device(x.device):
        _check(lib.ds_tile_pipeline(code, TILE_VARIANTS[variant], x.data_ptr(), out.data_ptr(), x.numel(),
                                    _stream_handle(x, stream)), "ds_tile_pipeline")
    return out


def query_timeout(device=None, stream=None) -> bool:
    """Waits for the stream; True if a look-back wait gave up since the last query (of gated_scan and its gradient on any
    stream of the device)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        s = torch.cuda.current_stream(dev) if stream is None else stream
        flag = ctypes.c_int(0)
        _check(lib.ds_query_timeout(s.cuda_stream if hasattr(s, "cuda_stream") else int(s), ctypes.byref(flag)),
               "ds_query_timeout")
    return bool(flag.value)


def set_spin_limit(polls: int):
    _check(lib.ds_set_spin_limit(int(polls)), "ds_set_spin_limit")


def release_workspace():
    lib.ds_release_workspace()
