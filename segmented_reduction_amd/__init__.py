"""Segmented reduction over offset-delimited segments on AMD MI355X (gfx950).

A thin ctypes binding over the C ABI in ``include/segred.h`` (libsegred.so,
built from ``csrc/`` with hipcc).  Every step of the computation runs in the
library's HIP kernels; this module only checks tensors, allocates outputs
with PyTorch and passes device pointers and PyTorch's current HIP stream.
There is no CPU fallback: if the library is missing, calls raise.

    out, arg = reduce(values, offsets, "max")        # values [N] or [N, F] on the GPU
    values, lengths, offsets, count = offsets_from_rle(sorted_keys)
    out, arg = scatter(values, index, dim_size, "max")  # unsorted int64 index [N]
    offsets = offsets_from_index(sorted_index, dim_size)
    prefix = scan(values, offsets, "sum", exclusive=False)  # segmented scan
    pos, word = galloping_search(values, queries, segments)  # lower bounds per segment
    values, count = unique(keys)                       # distinct adjacent values
    offsets, count = offsets_from_flags(start_flags)   # uint32 flags, nonzero = start

Operators over ragged groups of rows (float32, bfloat16, float16):

    order, position, offsets = group(choice, groups)   # choice int64 [N] or [T, k]
    h = matmul(x, weights, offsets, rows=order)        # each group's rows by its own weights
    y = combine(h, position, prob)                     # the weighted join per token
    dh, dprob = combine_grad(dy, h, position, prob)
    dw = outer(x, dh, offsets, left_rows=order)        # the gradient of the weights
    y = adapter(x, weights, offsets, which, down, up)  # shared projection + low-rank adapter per request
    h = gated(x, weights, offsets, rows=order)         # act(x gate^T) * (x up^T) per group
    dpair = gated_grad(dh, x, weights, offsets, rows=order)   # of both projections; then matmul and outer

Around them in a training step:

    y = norm(x, weight, bias)                          # layer norm of rows, or by the root mean square
    dx, dweight, dbias = norm_grad(dy, x, weight, want_bias=True)
    loss, lse, picked = cross_entropy(x, vocabulary, target)  # the logits are never kept
    dx, dvocabulary = cross_entropy_grad(dloss, x, vocabulary, target, lse, picked)

No call records a gradient: a result does not require one whatever its inputs
do, and a model that is trained through these operators calls the gradients'
operators itself, as above (torch.autograd.Function is the place).
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libsegred.so")

SUM, MIN, MAX, MEAN = 0, 1, 2, 3
OPS = {"sum": SUM, "min": MIN, "max": MAX, "mean": MEAN}
DTYPES = {torch.uint32: 0, torch.int32: 1, torch.float32: 2}
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
FLOATS = {torch.float32: 2, torch.bfloat16: 3, torch.float16: 4}  # the products, combine calls, norms and cross entropy
STATUS = {0: "SEGRED_OK", 1: "SEGRED_ERR_INVALID_ARGUMENT", 2: "SEGRED_ERR_UNSUPPORTED",
          3: "SEGRED_ERR_OUT_OF_MEMORY", 4: "SEGRED_ERR_HIP", 5: "SEGRED_ERR_SCRATCH_LIMIT"}


class SegredError(RuntimeError):
    """A non-zero status returned by the C ABI."""

    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({status_string(status)})")


_lock = threading.Lock()
_lib = None


def library(path: str | None = None):
    """Load libsegred.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(f"libsegred.so not found at {p}; build it with "
                                   "`python -m segmented_reduction_amd.build_lib`")
            lib = ctypes.CDLL(p)
            vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
            lib.segred_reduce.argtypes = [vp, i32, i64, vp, i64, i32, vp, vp, vp]
            lib.segred_reduce.restype = ctypes.c_int
            lib.segred_reduce_noalloc.argtypes = [vp, i32, i64, vp, i64, i32, vp, vp, vp]
            lib.segred_reduce_noalloc.restype = ctypes.c_int
            lib.segred_reduce_device_count.argtypes = [vp, i32, i64, vp, vp, i64, i32, vp, vp, vp]
            lib.segred_reduce_device_count.restype = ctypes.c_int
            lib.segred_offsets_from_rle.argtypes = [vp, i64, vp, vp, vp, vp, vp]
            lib.segred_offsets_from_rle.restype = ctypes.c_int
            lib.segred_scatter_reduce.argtypes = [vp, i32, i64, i64, vp, i64, i32, vp, vp, vp]
            lib.segred_scatter_reduce.restype = ctypes.c_int
            lib.segred_offsets_from_index.argtypes = [vp, i64, i64, vp, vp]
            lib.segred_offsets_from_index.restype = ctypes.c_int
            lib.segred_scan.argtypes = [vp, i32, i64, vp, i64, i32, i32, vp, vp]
            lib.segred_scan.restype = ctypes.c_int
            lib.segred_galloping_search.argtypes = [vp, i32, i64, i64, vp, i64, vp, i64, vp, i64, i64, i32, vp,
                                                    vp, i32, vp]
            lib.segred_galloping_search.restype = ctypes.c_int
            lib.segred_unique.argtypes = [vp, i64, vp, vp, vp]
            lib.segred_unique.restype = ctypes.c_int
            lib.segred_offsets_from_flags.argtypes = [vp, i64, vp, vp, vp]
            lib.segred_offsets_from_flags.restype = ctypes.c_int
            lib.segred_matmul.argtypes = [vp, i32, i64, vp, i64, vp, i32, i64, vp, i64, i64, vp, vp]
            lib.segred_matmul.restype = ctypes.c_int
            lib.segred_outer.argtypes = [vp, vp, i64, i64, vp, vp, i64, i64, i32, vp, i64, i64, vp, i32, vp, i64, vp]
            lib.segred_outer.restype = ctypes.c_int
            lib.segred_outer_mixed.argtypes = [vp, i32, vp, i64, i64, vp, i32, vp, i64, i64, vp, i64, i64, vp, i32, vp,
                                               i64, vp]
            lib.segred_outer_mixed.restype = ctypes.c_int
            lib.segred_outer_workspace.argtypes = [i64, i64, i64, i64]
            lib.segred_outer_workspace.restype = i64
            lib.segred_group.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, i64, vp]
            lib.segred_group.restype = ctypes.c_int
            lib.segred_group_workspace.argtypes = [i64, i64]
            lib.segred_group_workspace.restype = i64
            lib.segred_combine.argtypes = [vp, i32, i64, i64, vp, vp, i64, i64, vp, vp]
            lib.segred_combine.restype = ctypes.c_int
            lib.segred_combine_grad.argtypes = [vp, vp, i32, i64, i64, vp, vp, i64, i64, vp, vp, vp]
            lib.segred_combine_grad.restype = ctypes.c_int
            lib.segred_combine_grad_repeated.argtypes = [vp, vp, i32, i64, i64, vp, vp, i64, i64, vp, vp, vp, i64, vp]
            lib.segred_combine_grad_repeated.restype = ctypes.c_int
            lib.segred_combine_grad_repeated_workspace.argtypes = [i64, i64, i64]
            lib.segred_combine_grad_repeated_workspace.restype = i64
            lib.segred_adapter.argtypes = [vp, i32, i64, vp, i64, vp, vp, i64, i64, vp, vp, vp, i64, i64, i32, vp, vp,
                                           vp, i64, vp]
            lib.segred_adapter.restype = ctypes.c_int
            lib.segred_adapter_mixed.argtypes = [vp, i32, i64, vp, i64, vp, vp, i64, i64, vp, vp, vp, i64, i64, i32, vp,
                                                 vp, i32, vp, i64, vp]
            lib.segred_adapter_mixed.restype = ctypes.c_int
            lib.segred_adapter_workspace.argtypes = [i32, i64, i64, i64, i64]
            lib.segred_adapter_workspace.restype = i64
            f32 = ctypes.c_float
            lib.segred_gated.argtypes = [vp, i32, i64, vp, i64, vp, i64, i32, vp, i64, i64, vp, vp]
            lib.segred_gated.restype = ctypes.c_int
            lib.segred_gated_grad.argtypes = [vp, vp, i32, i64, vp, i64, vp, i64, i32, vp, i64, i64, vp, vp]
            lib.segred_gated_grad.restype = ctypes.c_int
            lib.segred_norm.argtypes = [vp, i32, i64, i64, vp, vp, i32, f32, i32, vp, vp]
            lib.segred_norm.restype = ctypes.c_int
            lib.segred_norm_grad.argtypes = [vp, vp, i32, i64, i64, vp, i32, f32, i32, vp, vp, vp, vp, i64, vp]
            lib.segred_norm_grad.restype = ctypes.c_int
            lib.segred_norm_grad_workspace.argtypes = [i64, i64]
            lib.segred_norm_grad_workspace.restype = i64
            lib.segred_cross_entropy.argtypes = [vp, i32, i64, i64, vp, i64, vp, vp, i64, f32, vp, vp, vp, vp, i64, vp]
            lib.segred_cross_entropy.restype = ctypes.c_int
            lib.segred_cross_entropy_workspace.argtypes = [i32, i64, i64, i64]
            lib.segred_cross_entropy_workspace.restype = i64
            lib.segred_cross_entropy_grad.argtypes = [vp, vp, i32, i64, i64, vp, i64, vp, vp, i64, f32, vp, vp, vp, vp,
                                                      i32, vp, i64, vp]
            lib.segred_cross_entropy_grad.restype = ctypes.c_int
            lib.segred_cross_entropy_grad_workspace.argtypes = [i32, i64, i64, i64, i64]
            lib.segred_cross_entropy_grad_workspace.restype = i64
            lib.segred_status_string.argtypes = [ctypes.c_int]
            lib.segred_status_string.restype = ctypes.c_char_p
            lib.segred_set_shares.argtypes = [i64]
            lib.segred_set_shares.restype = ctypes.c_int
            lib.segred_get_shares.argtypes = [i32, i32, i64]
            lib.segred_get_shares.restype = i64
            lib.segred_resident_waves.argtypes = [i32, i32, i64]
            lib.segred_resident_waves.restype = i64
            lib.segred_timing_enable.argtypes = [ctypes.c_int]
            lib.segred_timing_enable.restype = ctypes.c_int
            lib.segred_timing_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i64),
                                              ctypes.POINTER(ctypes.c_float), i64]
            lib.segred_timing_read.restype = ctypes.c_int
            lib.segred_probe_stream.argtypes = [vp, i64, vp, i32, vp, i32, vp]
            lib.segred_probe_stream.restype = ctypes.c_int
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return library().segred_status_string(int(status)).decode()


def _check(rc: int, what: str):
    if rc != 0:
        raise SegredError(rc, what)


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def reduce(values: torch.Tensor, offsets: torch.Tensor, op: str, *, want_arg: bool = True,
           out: torch.Tensor | None = None, arg: torch.Tensor | None = None,
           num_segments: torch.Tensor | None = None):
    """Segmented ``op`` ("sum", "min", "max", "mean") of ``values`` over ``offsets``.

    values  [N] or [N, ...] uint32 / int32 / float32 on a GPU, contiguous;
            trailing dimensions are flattened into F features per row.
    offsets int64 [S + 1] on the same GPU; segment s is rows offsets[s]..offsets[s+1]-1.
    num_segments  optional one-element int64 GPU tensor: the segment count is
            then read on the device (segred_reduce_device_count); offsets
            and the outputs are its capacity and rows past the count are
            left as they were.
    Returns (out [S, ...], arg [S, ...] int64 or None).  arg is the row of
    the extremum for min/max (lowest on ties, -1 for empty segments).
    """
    if op not in OPS:
        raise ValueError(f"op must be one of {sorted(OPS)}")
    if not (values.is_cuda and offsets.is_cuda):
        raise ValueError("values and offsets must be GPU tensors")
    if values.dtype not in DTYPES:
        raise TypeError(f"values dtype {values.dtype} is not uint32, int32 or float32")
    if offsets.dtype != torch.int64 or offsets.dim() != 1 or offsets.numel() < 1:
        raise ValueError("offsets must be a 1-D int64 tensor with S + 1 entries")
    if values.device != offsets.device:
        raise ValueError("values and offsets must be on the same device")
    if not values.is_contiguous() or not offsets.is_contiguous():
        raise ValueError("values and offsets must be contiguous")
    if values.dim() == 0:
        raise ValueError("values needs at least one dimension")
    s = offsets.numel() - 1
    feat_shape = tuple(values.shape[1:])
    feat = 1
    for d in feat_shape:
        feat *= d
    if feat < 1:
        raise ValueError("values has an empty feature dimension")
    odt = torch.float32 if op == "mean" else values.dtype
    if out is None:
        out = torch.empty((s,) + feat_shape, dtype=odt, device=values.device)
    want = op in ("min", "max") and want_arg
    if want and arg is None:
        arg = torch.empty((s,) + feat_shape, dtype=torch.int64, device=values.device)
    if not want:
        arg = None
    if num_segments is not None:
        if (not num_segments.is_cuda or num_segments.dtype != torch.int64 or num_segments.numel() != 1
                or num_segments.device != values.device):
            raise ValueError("num_segments must be a one-element int64 tensor on the values' device")
        with torch.cuda.device(values.device):
            rc = library().segred_reduce_device_count(
                values.data_ptr(), DTYPES[values.dtype], feat, offsets.data_ptr(), num_segments.data_ptr(), s,
                OPS[op], out.data_ptr(), arg.data_ptr() if arg is not None else None, _stream(values.device))
        _check(rc, "segred_reduce_device_count")
        return out, arg
    with torch.cuda.device(values.device):
        rc = library().segred_reduce(values.data_ptr(), DTYPES[values.dtype], feat, offsets.data_ptr(), s,
                                     OPS[op], out.data_ptr(), arg.data_ptr() if arg is not None else None,
                                     _stream(values.device))
    _check(rc, "segred_reduce")
    return out, arg


def offsets_from_rle(keys: torch.Tensor):
    """Run-length encode uint32 ``keys`` (adjacent runs) on the GPU.

    Returns (values [n], lengths [n], offsets [n + 1], count [1] int64), all on
    the GPU and written asynchronously; only values[:count], lengths[:count]
    and offsets[:count + 1] are meaningful.
    """
    if not keys.is_cuda or keys.dtype != torch.uint32 or keys.dim() != 1 or not keys.is_contiguous():
        raise ValueError("keys must be a contiguous 1-D uint32 GPU tensor")
    n = keys.numel()
    dev = keys.device
    values = torch.empty(max(n, 1), dtype=torch.uint32, device=dev)
    lengths = torch.empty(max(n, 1), dtype=torch.uint32, device=dev)
    offsets = torch.empty(n + 1, dtype=torch.int64, device=dev)
    count = torch.empty(1, dtype=torch.int64, device=dev)
    with torch.cuda.device(dev):
        rc = library().segred_offsets_from_rle(keys.data_ptr() if n else None, n, values.data_ptr(),
                                               lengths.data_ptr(), offsets.data_ptr(), count.data_ptr(),
                                               _stream(dev))
    _check(rc, "segred_offsets_from_rle")
    return values, lengths, offsets, count


def rle(keys: torch.Tensor):
    """``offsets_from_rle`` followed by the one 8-byte readback of the count:
    returns (values[:count], lengths[:count], offsets[:count + 1], count)."""
    values, lengths, offsets, count = offsets_from_rle(keys)
    c = int(count.item())
    return values[:c], lengths[:c], offsets[: c + 1], c


def scatter(values: torch.Tensor, index: torch.Tensor, dim_size: int, op: str, *, want_arg: bool = True,
            out: torch.Tensor | None = None, arg: torch.Tensor | None = None):
    """Scatter ``op`` ("sum", "min", "max", "mean"): row r of ``values`` goes
    to output ``index[r]`` (segred_scatter_reduce).

    values  [N] or [N, ...] uint32 / int32 / float32 on a GPU, contiguous.
    index   int64 [N] on the same GPU, any order; entries outside
            [0, dim_size) are ignored.
    Returns (out [dim_size, ...], arg [dim_size, ...] int64 or None).  Float
    sums use atomic additions and may differ in the last bits run to run.
    """
    if op not in OPS:
        raise ValueError(f"op must be one of {sorted(OPS)}")
    if not (values.is_cuda and index.is_cuda) or values.device != index.device:
        raise ValueError("values and index must be tensors on the same GPU")
    if values.dtype not in DTYPES:
        raise TypeError(f"values dtype {values.dtype} is not uint32, int32 or float32")
    if values.dim() == 0 or not values.is_contiguous():
        raise ValueError("values must be contiguous with at least one dimension")
    if index.dtype != torch.int64 or index.dim() != 1 or not index.is_contiguous():
        raise ValueError("index must be a contiguous 1-D int64 tensor")
    n = values.shape[0]
    if index.numel() != n:
        raise ValueError("index needs one entry per row of values")
    dim_size = int(dim_size)
    if dim_size < 0:
        raise ValueError("dim_size must be >= 0")
    feat_shape = tuple(values.shape[1:])
    feat = 1
    for d in feat_shape:
        feat *= d
    if feat < 1:
        raise ValueError("values has an empty feature dimension")
    odt = torch.float32 if op == "mean" else values.dtype
    if out is None:
        out = torch.empty((dim_size,) + feat_shape, dtype=odt, device=values.device)
    want = op in ("min", "max") and want_arg
    if want and arg is None:
        arg = torch.empty((dim_size,) + feat_shape, dtype=torch.int64, device=values.device)
    if not want:
        arg = None
    with torch.cuda.device(values.device):
        rc = library().segred_scatter_reduce(values.data_ptr() if n else None, DTYPES[values.dtype], feat, n,
                                             index.data_ptr() if n else None, dim_size, OPS[op],
                                             out.data_ptr() if dim_size else None,
                                             arg.data_ptr() if (arg is not None and dim_size) else None,
                                             _stream(values.device))
    _check(rc, "segred_scatter_reduce")
    return out, arg


def offsets_from_index(index: torch.Tensor, dim_size: int) -> torch.Tensor:
    """CSR offsets [dim_size + 1] of an int64 GPU ``index``: offsets[s] = rows
    with index in [0, s) (segred_offsets_from_index)."""
    if not index.is_cuda or index.dtype != torch.int64 or index.dim() != 1 or not index.is_contiguous():
        raise ValueError("index must be a contiguous 1-D int64 GPU tensor")
    dim_size = int(dim_size)
    if dim_size < 0:
        raise ValueError("dim_size must be >= 0")
    n = index.numel()
    offsets = torch.empty(dim_size + 1, dtype=torch.int64, device=index.device)
    with torch.cuda.device(index.device):
        rc = library().segred_offsets_from_index(index.data_ptr() if n else None, n, dim_size,
                                                 offsets.data_ptr(), _stream(index.device))
    _check(rc, "segred_offsets_from_index")
    return offsets


def scan(values: torch.Tensor, offsets: torch.Tensor, op: str, *, exclusive: bool = False,
         out: torch.Tensor | None = None) -> torch.Tensor:
    """Segmented inclusive / exclusive ``op`` ("sum", "min", "max") scan of
    ``values`` over ``offsets`` (segred_scan).

    Returns ``out`` with the shape and dtype of ``values``; rows outside
    [offsets[0], offsets[-1]) are left as they were in ``out`` (uninitialised
    when ``out`` is not given)."""
    if op not in ("sum", "min", "max"):
        raise ValueError("op must be one of ['max', 'min', 'sum']")
    if not (values.is_cuda and offsets.is_cuda) or values.device != offsets.device:
        raise ValueError("values and offsets must be tensors on the same GPU")
    if values.dtype not in DTYPES:
        raise TypeError(f"values dtype {values.dtype} is not uint32, int32 or float32")
    if offsets.dtype != torch.int64 or offsets.dim() != 1 or offsets.numel() < 1:
        raise ValueError("offsets must be a 1-D int64 tensor with S + 1 entries")
    if values.dim() == 0 or not values.is_contiguous() or not offsets.is_contiguous():
        raise ValueError("values and offsets must be contiguous; values needs a row dimension")
    feat = 1
    for d in values.shape[1:]:
        feat *= d
    if feat < 1:
        raise ValueError("values has an empty feature dimension")
    if out is None:
        out = torch.empty_like(values)
    elif out.shape != values.shape or out.dtype != values.dtype or not out.is_contiguous():
        raise ValueError("out must be contiguous with the shape and dtype of values")
    s = offsets.numel() - 1
    with torch.cuda.device(values.device):
        rc = library().segred_scan(values.data_ptr(), DTYPES[values.dtype], feat, offsets.data_ptr(), s, OPS[op],
                                   int(bool(exclusive)), out.data_ptr(), _stream(values.device))
    _check(rc, "segred_scan")
    return out


def galloping_search(values: torch.Tensor, queries: torch.Tensor, segments: torch.Tensor, *,
                     value_order: torch.Tensor | None = None, value_stride: int = 1, value_count: int | None = None,
                     max_query_count: int | None = None, queries_per_tile: int = 32,
                     out: torch.Tensor | None = None, validation: torch.Tensor | None = None,
                     preserve_validation: bool = False):
    """Lower bounds of ``queries`` over segmented sorted ``values``
    (segred_galloping_search).  ``values`` and ``queries`` are uint32 or
    float32 GPU tensors of one dtype; ``segments`` int64 [S, 4] records
    (vo, vc, qo, qc) on the GPU.  ``max_query_count`` defaults to the
    queries' length (no host read of the records).  Returns (out int64
    [len(queries)], validation uint32 [1]), both on the GPU."""
    if values.dtype not in (torch.uint32, torch.float32) or queries.dtype != values.dtype:
        raise TypeError("values and queries must both be uint32 or both float32")
    for t in (values, queries, segments):
        if not t.is_cuda or t.device != values.device or not t.is_contiguous():
            raise ValueError("values, queries and segments must be contiguous tensors on one GPU")
    if segments.dtype != torch.int64 or segments.dim() != 2 or segments.shape[1] != 4:
        raise ValueError("segments must be an int64 [S, 4] tensor")
    if value_order is not None and (value_order.dtype != torch.uint32 or not value_order.is_cuda
                                    or value_order.device != values.device or not value_order.is_contiguous()):
        raise ValueError("value_order must be a contiguous uint32 tensor on the values' GPU")
    n = values.numel()
    vcount = value_count if value_count is not None else (n + value_stride - 1) // value_stride
    qn = queries.numel()
    mq = qn if max_query_count is None else int(max_query_count)
    dev = values.device
    if out is None:
        out = torch.empty(qn, dtype=torch.int64, device=dev)
    if validation is None:
        validation = torch.zeros(1, dtype=torch.int32, device=dev).view(torch.uint32)
    with torch.cuda.device(dev):
        rc = library().segred_galloping_search(
            values.data_ptr() if n else None, DTYPES[values.dtype], vcount, value_stride,
            value_order.data_ptr() if value_order is not None else None,
            value_order.numel() if value_order is not None else 0,
            queries.data_ptr() if qn else None, qn, segments.data_ptr() if segments.numel() else None,
            segments.shape[0], mq, queries_per_tile, out.data_ptr() if qn else None, validation.data_ptr(),
            int(bool(preserve_validation)), _stream(dev))
    _check(rc, "segred_galloping_search")
    return out, validation


def unique(keys: torch.Tensor):
    """Distinct adjacent values of uint32 ``keys`` (segred_unique).

    Returns (values [n], count [1] int64) on the GPU, written asynchronously;
    only values[:count] is meaningful."""
    if not keys.is_cuda or keys.dtype != torch.uint32 or keys.dim() != 1 or not keys.is_contiguous():
        raise ValueError("keys must be a contiguous 1-D uint32 GPU tensor")
    n = keys.numel()
    values = torch.empty(max(n, 1), dtype=torch.uint32, device=keys.device)
    count = torch.empty(1, dtype=torch.int64, device=keys.device)
    with torch.cuda.device(keys.device):
        rc = library().segred_unique(keys.data_ptr() if n else None, n, values.data_ptr(), count.data_ptr(),
                                     _stream(keys.device))
    _check(rc, "segred_unique")
    return values, count


def offsets_from_flags(flags: torch.Tensor):
    """Offsets of the segments that uint32 start ``flags`` open (nonzero =
    start; segred_offsets_from_flags).

    Returns (offsets [n + 1], count [1] int64) on the GPU, written
    asynchronously; only offsets[:count + 1] is meaningful."""
    if not flags.is_cuda or flags.dtype != torch.uint32 or flags.dim() != 1 or not flags.is_contiguous():
        raise ValueError("flags must be a contiguous 1-D uint32 GPU tensor")
    n = flags.numel()
    offsets = torch.empty(n + 1, dtype=torch.int64, device=flags.device)
    count = torch.empty(1, dtype=torch.int64, device=flags.device)
    with torch.cuda.device(flags.device):
        rc = library().segred_offsets_from_flags(flags.data_ptr() if n else None, n, offsets.data_ptr(),
                                                 count.data_ptr(), _stream(flags.device))
    _check(rc, "segred_offsets_from_flags")
    return offsets, count


def _launch(fn, what: str, index: int, *args):
    """Call ``fn`` with ``args`` and the current stream of GPU ``index``, on that GPU.

    The decoding calls take a few microseconds on the GPU, so the host side is
    kept short: the device is switched only where it is not the current one,
    and the stream handle is asked for without building a Stream object (0.1
    us instead of 1.9)."""
    if index == torch._C._cuda_getDevice():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc != 0:
        raise SegredError(rc, what)


def _floats(name: str, t: torch.Tensor):
    """(GPU index, dtype code) of a contiguous [*, features] tensor of the products' types."""
    index = t.get_device()
    if index < 0 or t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D GPU tensor")
    code = FLOATS.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} dtype {t.dtype} is not float32, bfloat16 or float16")
    return index, code


def _beside(index: int, name: str, t: torch.Tensor):
    """Raise unless ``t`` is contiguous and on GPU ``index``."""
    if t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on the GPU of the other inputs")


def _rows(index: int, name: str, t: torch.Tensor):
    """Raise unless ``t`` is a contiguous 1-D int64 tensor on GPU ``index``."""
    if t.get_device() != index or t.dtype != torch.int64 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D int64 tensor on the GPU of the other inputs")


def matmul(values: torch.Tensor, weights: torch.Tensor, offsets: torch.Tensor, *, transpose: bool = False,
           rows: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """The matrix product of each segment's rows with weights of its own
    (segred_matmul): ``out[r] = values[r] @ weights[s]`` for the rows r of
    segment s, with ``weights[s]`` transposed first where ``transpose`` is set.

    values   [N, K] float32 / bfloat16 / float16 on a GPU, contiguous.
    weights  [S, K, M], or [S, M, K] with ``transpose``, of the same type.
    offsets  int64 [S + 1] on the same GPU.
    rows     optional int64 [R]: row r of the product is then made from
             ``values[rows[r]]`` (``group``'s order); an entry outside the
             values stands for a row of zeros.
    Returns out [N or R, M]; rows of no segment are left as they were
    (uninitialised when ``out`` is not given).  The gradient of the (gathered)
    rows is ``matmul(grad, weights, offsets, transpose=not transpose)``, that
    of the weights ``outer``.
    """
    dev, code = _floats("values", values)
    if weights.dtype != values.dtype:
        raise TypeError("weights must have the dtype of values")
    _beside(dev, "weights", weights)
    _rows(dev, "offsets", offsets)
    count, k = values.shape
    s = offsets.shape[0] - 1
    if rows is None:
        n = count
    else:
        _rows(dev, "rows", rows)
        n = rows.shape[0]
    if s < 0 or weights.dim() != 3 or weights.shape[0] != s:
        raise ValueError("weights must be [S, K, M] (or [S, M, K] with transpose) with S + 1 offsets")
    m, kw = (weights.shape[1], weights.shape[2]) if transpose else (weights.shape[2], weights.shape[1])
    if kw != k:
        raise ValueError(f"values have {k} features and weights take {kw}")
    if out is None:
        out = torch.empty((n, m), dtype=values.dtype, device=values.device)
    else:
        _beside(dev, "out", out)
        if out.shape != (n, m) or out.dtype != values.dtype:
            raise ValueError("out must be [rows, M] of the dtype of values")
    _launch((_lib or library()).segred_matmul, "segred_matmul", dev, values.data_ptr(), code, k,
            rows.data_ptr() if rows is not None else None, count, weights.data_ptr(), 1 if transpose else 0, m,
            offsets.data_ptr(), s, n, out.data_ptr())
    return out


def outer(left: torch.Tensor, right: torch.Tensor, offsets: torch.Tensor, *, left_rows: torch.Tensor | None = None,
          right_rows: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
          out: torch.Tensor | None = None) -> torch.Tensor:
    """The sum of outer products of each segment's rows (segred_outer):
    ``out[s] = sum over r of left[r].T @ right[r]``, [S, K, M].

    left, right  [*, K] and [*, M] float32 / bfloat16 / float16 on a GPU,
                 contiguous and of one type; or, where ``out_dtype`` (or
                 ``out``) says what the sums are, one of a 16-bit type, which
                 enters exactly, and one float32 (an adapter's low-rank rows).
    offsets      int64 [S + 1] on the same GPU; an empty segment gives zeros.
    left_rows, right_rows  optional int64 [R]: gather that side's rows.
    out_dtype    the inputs' type (default; either of two) or float32.
    """
    dev, code = _floats("left", left)
    odt = out_dtype or (left.dtype if out is None else out.dtype)
    if right.dtype != left.dtype:
        if torch.float32 not in (left.dtype, right.dtype):
            raise TypeError("right must have the dtype of left, or one of the two float32")
        if out_dtype is None and out is None:
            raise TypeError("right must have the dtype of left where neither out_dtype nor out is given")
    right_code = _floats("right", right)[1]
    _beside(dev, "right", right)
    _rows(dev, "offsets", offsets)
    for name, index in (("left_rows", left_rows), ("right_rows", right_rows)):
        if index is not None:
            _rows(dev, name, index)
    s = offsets.shape[0] - 1
    n = (left if left_rows is None else left_rows).shape[0]
    if (right if right_rows is None else right_rows).shape[0] != n or s < 0:
        raise ValueError("left and right need the same number of rows, and offsets S + 1 entries")
    k, m = left.shape[1], right.shape[1]
    if odt not in (left.dtype, right.dtype, torch.float32):
        raise TypeError("out_dtype must be the dtype of left or right or float32")
    if out is None:
        out = torch.empty((s, k, m), dtype=odt, device=left.device)
    else:
        _beside(dev, "out", out)
        if out.shape != (s, k, m) or out.dtype != odt:
            raise ValueError("out must be [S, K, M] of out_dtype")
    lib = _lib or library()
    need = lib.segred_outer_workspace(k, m, s, n)
    work = torch.empty(need, dtype=torch.uint8, device=left.device) if need else None
    _launch(lib.segred_outer_mixed, "segred_outer", dev, left.data_ptr(), code,
            left_rows.data_ptr() if left_rows is not None else None, left.shape[0], k, right.data_ptr(), right_code,
            right_rows.data_ptr() if right_rows is not None else None, right.shape[0], m, offsets.data_ptr(), s, n,
            out.data_ptr(), FLOATS[odt], work.data_ptr() if need else None, need)
    return out


def group(index: torch.Tensor, dim_size: int):
    """Rows grouped by an index (segred_group).

    index  int64 [N], or [T, k] where each row names k groups.
    Returns (order, position, offsets), all int64: ``order`` [N] or [T * k]
    holds the rows of group 0, then of group 1, and so on, each group's in
    increasing order; ``position``, shaped as ``index``, the place of each
    entry in ``order``; ``offsets`` [dim_size + 1] where each group begins.
    Entries outside [0, dim_size) come behind the last group, at position -1.
    """
    dev = index.get_device()
    if dev < 0 or index.dtype != torch.int64 or index.dim() not in (1, 2) or not index.is_contiguous():
        raise ValueError("index must be a contiguous 1-D or 2-D int64 GPU tensor")
    dim_size = int(dim_size)
    if dim_size < 0:
        raise ValueError("dim_size must be >= 0")
    n, device = index.numel(), index.device
    fanout = max(index.shape[1], 1) if index.dim() == 2 else 1
    order = torch.empty(n, dtype=torch.int64, device=device)
    position = torch.empty_like(index)
    offsets = torch.empty(dim_size + 1, dtype=torch.int64, device=device)
    lib = _lib or library()
    need = lib.segred_group_workspace(n, dim_size)
    work = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _launch(lib.segred_group, "segred_group", dev, index.data_ptr(), n, fanout, dim_size, order.data_ptr(),
            position.data_ptr(), offsets.data_ptr(), work.data_ptr() if need else None, need)
    return order, position, offsets


def _check_combine(values, position, weights):
    """(GPU index, dtype code) of the tensors that both combine calls take."""
    dev, code = _floats("values", values)
    if position.get_device() != dev or position.dtype != torch.int64 or position.dim() != 2 or not position.is_contiguous():
        raise ValueError("position must be a contiguous int64 [T, k] tensor on the GPU of values")
    if (weights.get_device() != dev or weights.dtype != torch.float32 or weights.shape != position.shape
            or not weights.is_contiguous()):
        raise ValueError("weights must be a contiguous float32 tensor of the shape of position, on its GPU")
    return dev, code


def combine(values: torch.Tensor, position: torch.Tensor, weights: torch.Tensor, *,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """The weighted join of the rows a token was sent to (segred_combine):
    ``out[t] = sum over j of weights[t, j] * values[position[t, j]]``.

    values    [N, M] float32 / bfloat16 / float16 on a GPU, contiguous.
    position  int64 [T, k] (``group``'s); entries outside the values take no part.
    weights   float32 [T, k].
    Returns out [T, M] of the values' type.
    """
    dev, code = _check_combine(values, position, weights)
    (n, m), (t, k) = values.shape, position.shape
    if out is None:
        out = torch.empty((t, m), dtype=values.dtype, device=values.device)
    else:
        _beside(dev, "out", out)
        if out.shape != (t, m) or out.dtype != values.dtype:
            raise ValueError("out must be [T, M] of the dtype of values")
    _launch((_lib or library()).segred_combine, "segred_combine", dev, values.data_ptr(), code, m, n,
            position.data_ptr(), weights.data_ptr(), t, k, out.data_ptr())
    return out


def combine_grad(grad: torch.Tensor, values: torch.Tensor, position: torch.Tensor, weights: torch.Tensor, *,
                 repeated: bool = False, out: torch.Tensor | None = None):
    """The gradient of ``combine`` (segred_combine_grad) from ``grad`` [T, M].

    Returns (grad_values [N, M], grad_weights float32 [T, k]).  Each row may be
    named once only, as ``group``'s positions do, which is not checked; rows that
    ``position`` does not name are left as they were (uninitialised when ``out``
    is not given).  With ``repeated`` rows may be named any number of times: the
    entries are sorted by row first, and a row that none names gets zeros."""
    dev, code = _check_combine(values, position, weights)
    _beside(dev, "grad", grad)
    (n, m), (t, k) = values.shape, position.shape
    if grad.shape != (t, m) or grad.dtype != values.dtype:
        raise ValueError("grad must be [T, M] of the dtype of values")
    if out is None:
        out = torch.empty_like(values)
    else:
        _beside(dev, "out", out)
        if out.shape != values.shape or out.dtype != values.dtype:
            raise ValueError("out must have the shape and dtype of values")
    grad_weights = torch.empty_like(weights)
    lib = _lib or library()
    args = (grad.data_ptr(), values.data_ptr(), code, m, n, position.data_ptr(), weights.data_ptr(), t, k,
            out.data_ptr(), grad_weights.data_ptr())
    if repeated:
        need = lib.segred_combine_grad_repeated_workspace(n, t, k)
        work = torch.empty(need, dtype=torch.uint8, device=values.device) if need else None
        _launch(lib.segred_combine_grad_repeated, "segred_combine_grad_repeated", dev, *args,
                work.data_ptr() if need else None, need)
    else:
        _launch(lib.segred_combine_grad, "segred_combine_grad", dev, *args)
    return out, grad_weights


def adapter(values: torch.Tensor, weights: torch.Tensor, offsets: torch.Tensor, which: torch.Tensor,
            down: torch.Tensor, up: torch.Tensor, *, scale: torch.Tensor | None = None, transpose: bool = False,
            want_low: bool | torch.dtype = False, out: torch.Tensor | None = None):
    """A projection that all rows share with a low-rank adapter per segment
    beside it (segred_adapter): for the rows of segment s and a = which[s],
    ``x @ weights.T + scale[a] * (x @ down[a].T) @ up[a].T``, or with
    ``transpose`` (the gradient of x, from that of the output)
    ``x @ weights + scale[a] * (x @ up[a]) @ down[a]``.

    values    [N, K] ([N, M] with ``transpose``) float32 / bfloat16 / float16
              on a GPU, contiguous.
    weights   [M, K]; down [L, r, K]; up [L, M, r], of the same type.
    offsets   int64 [S + 1]; which int64 [S], outside [0, L): no adapter.
    scale     optional float32 [L].
    want_low  also return the low-rank rows [N, r], of this type (float32 or
              the values'; ``True``: the values'): ``outer`` of the output's
              gradient and these gives the gradient of up, ``outer`` of the
              transposed call's and x that of down (rows grouped by adapter).
              Rows of a 16-bit type are rounded, and the gradients once more;
              ask for ``torch.float32`` to round the gradients alone.
    Rows of no segment are left as they were in ``out`` (uninitialised when it
    is not given; likewise the low-rank rows).
    """
    dev, code = _floats("values", values)
    if weights.dtype != values.dtype or down.dtype != values.dtype or up.dtype != values.dtype:
        raise TypeError("weights, down and up must have the dtype of values")
    _beside(dev, "weights", weights)
    _beside(dev, "down", down)
    _beside(dev, "up", up)
    _rows(dev, "offsets", offsets)
    _rows(dev, "which", which)
    if weights.dim() != 2 or down.dim() != 3 or up.dim() != 3:
        raise ValueError("weights must be [M, K], down [L, r, K] and up [L, M, r]")
    (m, k), (count, r, kd) = weights.shape, down.shape
    if kd != k or up.shape != (count, m, r):
        raise ValueError("weights must be [M, K], down [L, r, K] and up [L, M, r]")
    s, (n, width) = offsets.shape[0] - 1, values.shape
    if s < 0 or which.shape[0] != s:
        raise ValueError("which needs one entry per segment and offsets one more")
    if scale is not None:
        _beside(dev, "scale", scale)
        if scale.dtype != torch.float32 or scale.shape != (count,):
            raise ValueError("scale must be a float32 [L] tensor")
    have, give = (m, k) if transpose else (k, m)
    if width != have:
        raise ValueError(f"values have {width} features and the projection takes {have}")
    device = values.device
    if out is None:
        out = torch.empty((n, give), dtype=values.dtype, device=device)
    else:
        _beside(dev, "out", out)
        if out.shape != (n, give) or out.dtype != values.dtype:
            raise ValueError("out must be [N, outputs] of the dtype of values")
    low_dtype = want_low if isinstance(want_low, torch.dtype) else values.dtype
    if low_dtype not in (values.dtype, torch.float32):
        raise TypeError("want_low must be float32 or the dtype of values")
    low = torch.empty((n, r), dtype=low_dtype, device=device) if want_low else None
    lib = _lib or library()
    need = lib.segred_adapter_workspace(code, m, count, r, n)
    work = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _launch(lib.segred_adapter_mixed, "segred_adapter", dev, values.data_ptr(), code, k, weights.data_ptr(), m,
            offsets.data_ptr(), which.data_ptr(), s, n, down.data_ptr(), up.data_ptr(),
            scale.data_ptr() if scale is not None else None, count, r, 1 if transpose else 0, out.data_ptr(),
            low.data_ptr() if want_low else None, FLOATS[low_dtype], work.data_ptr() if need else None, need)
    return (out, low) if want_low else out


def _check_gated(values, weights, offsets, activation, rows):
    """(GPU index, dtype code, activation code, S, N, K, M) of the tensors that both gated calls take."""
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    dev, code = _floats("values", values)
    if weights.dtype != values.dtype:
        raise TypeError("weights must have the dtype of values")
    _beside(dev, "weights", weights)
    _rows(dev, "offsets", offsets)
    n, k = values.shape
    s = offsets.shape[0] - 1
    if rows is not None:
        _rows(dev, "rows", rows)
        n = rows.shape[0]
    if s < 0 or weights.dim() != 3 or weights.shape[0] != s or weights.shape[1] % 2 or weights.shape[2] != k:
        raise ValueError("weights must be [S, 2 * M, K] with S + 1 offsets and the features of values")
    return dev, code, act, s, n, k, weights.shape[1] // 2


def gated(values: torch.Tensor, weights: torch.Tensor, offsets: torch.Tensor, *, activation: str = "silu",
          rows: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """The gated pair of projections of each segment's rows (segred_gated):
    ``out[r] = act(values[r] @ gate[s].T) * (values[r] @ up[s].T)`` for the rows r
    of segment s, ``gate[s], up[s] = weights[s, :M], weights[s, M:]``.

    values      [N, K] float32 / bfloat16 / float16 on a GPU, contiguous.
    weights     [S, 2 * M, K] of the same type.
    offsets     int64 [S + 1] on the same GPU.
    activation  "silu", "gelu" (by the normal distribution), "gelu_tanh" or "relu".
    rows        optional int64 [R]: row r is then made from ``values[rows[r]]``, as
                in ``matmul``.
    Returns out [N or R, M]; rows of no segment are left as they were
    (uninitialised when ``out`` is not given).
    """
    dev, code, act, s, n, k, m = _check_gated(values, weights, offsets, activation, rows)
    if out is None:
        out = torch.empty((n, m), dtype=values.dtype, device=values.device)
    else:
        _beside(dev, "out", out)
        if out.shape != (n, m) or out.dtype != values.dtype:
            raise ValueError("out must be [rows, M] of the dtype of values")
    _launch((_lib or library()).segred_gated, "segred_gated", dev, values.data_ptr(), code, k,
            rows.data_ptr() if rows is not None else None, values.shape[0], weights.data_ptr(), m, act,
            offsets.data_ptr(), s, n, out.data_ptr())
    return out


def gated_grad(grad: torch.Tensor, values: torch.Tensor, weights: torch.Tensor, offsets: torch.Tensor, *,
               activation: str = "silu", rows: torch.Tensor | None = None,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of ``gated``'s two projections from that of its output,
    ``grad`` [N or R, M] (segred_gated_grad): [N or R, 2 * M], the gate's, then the
    other's.  Both projections are formed again from ``values`` and ``weights``.

    ``matmul(pair, weights, offsets)`` is then the gradient of the (gathered)
    rows, ``outer(pair, values, offsets, right_rows=rows)`` that of the weights.
    The pair is rounded to the values' type; where that is too coarse for the two
    products, make all of these calls in float32.  Rows of no segment are left as
    they were.
    """
    dev, code, act, s, n, k, m = _check_gated(values, weights, offsets, activation, rows)
    _beside(dev, "grad", grad)
    if grad.shape != (n, m) or grad.dtype != values.dtype:
        raise ValueError("grad must be [rows, M] of the dtype of values")
    if out is None:
        out = torch.empty((n, 2 * m), dtype=values.dtype, device=values.device)
    else:
        _beside(dev, "out", out)
        if out.shape != (n, 2 * m) or out.dtype != values.dtype:
            raise ValueError("out must be [rows, 2 * M] of the dtype of values")
    _launch((_lib or library()).segred_gated_grad, "segred_gated_grad", dev, grad.data_ptr(), values.data_ptr(), code, k,
            rows.data_ptr() if rows is not None else None, values.shape[0], weights.data_ptr(), m, act,
            offsets.data_ptr(), s, n, out.data_ptr())
    return out


def _check_norm(values, weight, bias):
    """(GPU index, dtype code, type of the parameters) of the tensors that both norm calls take."""
    dev, code = _floats("values", values)
    kind = values.dtype if weight is None and bias is None else (weight if weight is not None else bias).dtype
    if kind not in (values.dtype, torch.float32):
        raise TypeError("weight and bias must be float32 or have the dtype of values")
    for name, p in (("weight", weight), ("bias", bias)):
        if p is None:
            continue
        _beside(dev, name, p)
        if p.dtype != kind:
            raise TypeError("weight and bias must have one dtype")
        if p.shape != (values.shape[1],):
            raise ValueError(f"{name} must have one entry per feature of values")
    return dev, code, kind


def norm(values: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *,
         eps: float = 1e-5, center: bool = True, out: torch.Tensor | None = None) -> torch.Tensor:
    """Layer norm of each row (segred_norm): ``(x - mean) / sqrt(mean((x - mean)**2)
    + eps) * weight + bias``; without ``center`` the mean is taken as 0 (the norm by
    the root mean square).

    values  [N, K] float32 / bfloat16 / float16 on a GPU, contiguous.
    weight, bias  optional [K], both float32 or both of the values' type.
    Returns out [N, K] of the values' type; ``out`` may be ``values`` itself.
    """
    dev, code, kind = _check_norm(values, weight, bias)
    n, k = values.shape
    if out is None:
        out = torch.empty_like(values)
    else:
        _beside(dev, "out", out)
        if out.shape != values.shape or out.dtype != values.dtype:
            raise ValueError("out must have the shape and dtype of values")
    _launch((_lib or library()).segred_norm, "segred_norm", dev, values.data_ptr(), code, k, n,
            weight.data_ptr() if weight is not None else None, bias.data_ptr() if bias is not None else None,
            FLOATS[kind], eps, 1 if center else 0, out.data_ptr())
    return out


def norm_grad(grad: torch.Tensor, values: torch.Tensor, weight: torch.Tensor | None = None, *, eps: float = 1e-5,
              center: bool = True, want_weight: bool | None = None, want_bias: bool = False,
              dtype: torch.dtype | None = None, out: torch.Tensor | None = None):
    """The gradients of ``norm`` from that of its output, ``grad`` [N, K]
    (segred_norm_grad); the rows' statistics are found again.

    want_weight, want_bias  which parameters' gradients to form (the weight's by
            default where there is one): sums over the rows in a fixed order.
    dtype   their type where there is no ``weight`` to go by: float32 or the values'.
    Returns (grad_values [N, K], grad_weight [K] or None, grad_bias [K] or None).
    """
    dev, code, kind = _check_norm(values, weight, None)
    if dtype is not None:
        if dtype not in (values.dtype, torch.float32) or (weight is not None and dtype != weight.dtype):
            raise TypeError("dtype must be the weight's, or without one float32 or the dtype of values")
        kind = dtype
    _beside(dev, "grad", grad)
    if grad.shape != values.shape or grad.dtype != values.dtype:
        raise ValueError("grad must have the shape and dtype of values")
    n, k = values.shape
    if out is None:
        out = torch.empty_like(values)
    else:
        _beside(dev, "out", out)
        if out.shape != values.shape or out.dtype != values.dtype:
            raise ValueError("out must have the shape and dtype of values")
    if want_weight is None:
        want_weight = weight is not None
    grad_weight = torch.empty(k, dtype=kind, device=values.device) if want_weight else None
    grad_bias = torch.empty(k, dtype=kind, device=values.device) if want_bias else None
    lib = _lib or library()
    need = lib.segred_norm_grad_workspace(k, n) if want_weight or want_bias else 0
    work = torch.empty(need, dtype=torch.uint8, device=values.device) if need else None
    _launch(lib.segred_norm_grad, "segred_norm_grad", dev, grad.data_ptr(), values.data_ptr(), code, k, n,
            weight.data_ptr() if weight is not None else None, FLOATS[kind], eps, 1 if center else 0, out.data_ptr(),
            grad_weight.data_ptr() if want_weight else None, grad_bias.data_ptr() if want_bias else None,
            work.data_ptr() if need else None, need)
    return out, grad_weight, grad_bias


def _check_entropy(values, weights, target, probs):
    """(GPU index, dtype code, targets per row) of the tensors that both cross entropy calls take."""
    dev, code = _floats("values", values)
    if weights.dtype != values.dtype:
        raise TypeError("weights must have the dtype of values")
    _beside(dev, "weights", weights)
    if weights.dim() != 2 or weights.shape[1] != values.shape[1] or weights.shape[0] < 1:
        raise ValueError("weights must be [V, K] with the features of values")
    if target.get_device() != dev or target.dtype != torch.int64 or not target.is_contiguous():
        raise ValueError("target must be a contiguous int64 tensor on the GPU of the other inputs")
    if target.dim() not in (1, 2) or target.shape[0] != values.shape[0] or (target.dim() == 2 and target.shape[1] < 1):
        raise ValueError("target must be [N] or [N, k] with a row per row of values")
    if probs is not None:
        _beside(dev, "probs", probs)
        if probs.dtype != torch.float32 or probs.shape != target.shape:
            raise ValueError("probs must be float32 of the shape of target")
    return dev, code, target.shape[1] if target.dim() == 2 else 1


def cross_entropy(values: torch.Tensor, weights: torch.Tensor, target: torch.Tensor, *,
                  probs: torch.Tensor | None = None, scale: float = 1.0):
    """The softmax cross entropy of each row against a vocabulary's weights, whose
    logits ``scale * values @ weights.T`` are never kept (segred_cross_entropy).

    values   [N, K] float32 / bfloat16 / float16 on a GPU, contiguous.
    weights  [V, K] of the same type.
    target   int64 [N], or [N, k]: the entries that a teacher holds most likely,
             with their ``probs`` float32 [N, k] (1 each if not given).  Entries
             outside [0, V) take no part; a row without any has loss 0.
    Returns (loss [N], lse [N], picked, shaped as target), all float32: the
    logarithms of the sums of exponentials and the targets' logits are what
    ``cross_entropy_grad`` goes on from.
    """
    dev, code, picks = _check_entropy(values, weights, target, probs)
    (n, k), v, device = values.shape, weights.shape[0], values.device
    loss = torch.empty(n, dtype=torch.float32, device=device)
    lse = torch.empty(n, dtype=torch.float32, device=device)
    picked = torch.empty(target.shape, dtype=torch.float32, device=device)
    lib = _lib or library()
    need = lib.segred_cross_entropy_workspace(code, k, n, v)
    work = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _launch(lib.segred_cross_entropy, "segred_cross_entropy", dev, values.data_ptr(), code, k, n, weights.data_ptr(), v,
            target.data_ptr(), probs.data_ptr() if probs is not None else None, picks, scale, loss.data_ptr(),
            lse.data_ptr(), picked.data_ptr(), work.data_ptr() if need else None, need)
    return loss, lse, picked


def cross_entropy_grad(grad: torch.Tensor, values: torch.Tensor, weights: torch.Tensor, target: torch.Tensor,
                       lse: torch.Tensor, picked: torch.Tensor, *, probs: torch.Tensor | None = None,
                       scale: float = 1.0, want_values: bool = True, want_weights: bool = True,
                       weights_dtype: torch.dtype | None = None):
    """The gradients of ``cross_entropy``'s loss from ``grad`` float32 [N]
    (segred_cross_entropy_grad), by pieces of the vocabulary.

    lse, picked    what ``cross_entropy`` returned for the same arguments.
    weights_dtype  type of the weights' gradient: theirs (default) or float32.
    The logits' gradient is rounded to the values' type before both products; with
    ``values.float()`` and ``weights.float()`` nothing is.
    Returns (grad_values [N, K] or None, grad_weights [V, K] or None).
    """
    dev, code, picks = _check_entropy(values, weights, target, probs)
    (n, k), v, device = values.shape, weights.shape[0], values.device
    for name, t, shape in (("grad", grad, (n,)), ("lse", lse, (n,)), ("picked", picked, target.shape)):
        _beside(dev, name, t)
        if t.dtype != torch.float32 or t.shape != shape:
            raise ValueError(f"{name} must be float32 {list(shape)}")
    kind = weights_dtype or weights.dtype
    if kind not in (weights.dtype, torch.float32):
        raise TypeError("weights_dtype must be float32 or the dtype of weights")
    grad_values = torch.empty_like(values) if want_values else None
    grad_weights = torch.empty((v, k), dtype=kind, device=device) if want_weights else None
    lib = _lib or library()
    need = lib.segred_cross_entropy_grad_workspace(code, k, n, v, picks)
    work = torch.empty(need, dtype=torch.uint8, device=device)
    _launch(lib.segred_cross_entropy_grad, "segred_cross_entropy_grad", dev, grad.data_ptr(), values.data_ptr(), code, k, n,
            weights.data_ptr(), v, target.data_ptr(), probs.data_ptr() if probs is not None else None, picks, scale,
            lse.data_ptr(), picked.data_ptr(), grad_values.data_ptr() if want_values else None,
            grad_weights.data_ptr() if want_weights else None, FLOATS[kind], work.data_ptr(), need)
    return grad_values, grad_weights


def set_shares(shares: int):
    """Override the work partition (0 = default); see segred_set_shares."""
    _check(library().segred_set_shares(int(shares)), "segred_set_shares")


def get_shares(dtype=torch.float32, op: str = "sum", feat: int = 1) -> int:
    return int(library().segred_get_shares(DTYPES[dtype], OPS[op], int(feat)))


def timing_enable(enable: bool = True):
    _check(library().segred_timing_enable(1 if enable else 0), "segred_timing_enable")


def timing_read(capacity: int = 8192):
    """(total ms, launches, per-launch ms list) of the streaming kernels since the last read:
    each is the kernel's own stop event minus its own start event."""
    ms = ctypes.c_double(0.0)
    n = ctypes.c_int64(0)
    each = (ctypes.c_float * max(capacity, 1))()
    _check(library().segred_timing_read(ctypes.byref(ms), ctypes.byref(n), each, capacity), "segred_timing_read")
    return ms.value, n.value, [each[i] for i in range(min(n.value, capacity))]


def probe_stream(src: torch.Tensor, write_every: int = 0, waves: int = 4096,
                 dst: torch.Tensor | None = None):
    """Streaming-rate probe (measurement context, see segred_probe_stream).

    src  contiguous float32 GPU tensor whose size in bytes is a multiple of
         1,024, read once by `waves` waves over contiguous shares.
    write_every  0 (read only) or 1..1024: one 1 KB block is written per
         `write_every` blocks read, to `dst` (float32, at least
         floor(blocks / write_every) * 256 elements; allocated when None).
    Returns (wave_sums [waves] float32, dst or None).
    """
    if not src.is_cuda or src.dtype != torch.float32 or not src.is_contiguous():
        raise ValueError("src must be a contiguous float32 GPU tensor")
    nbytes = src.numel() * 4
    if write_every > 0 and dst is None:
        dst = torch.empty((nbytes // 1024 // write_every) * 256, dtype=torch.float32, device=src.device)
    if dst is not None and (not dst.is_cuda or dst.dtype != torch.float32 or not dst.is_contiguous()
                            or dst.device != src.device):
        raise ValueError("dst must be a contiguous float32 tensor on the device of src")
    if write_every > 0 and dst.numel() < (nbytes // 1024 // write_every) * 256:
        raise ValueError("dst is smaller than one 1 KB block per write_every blocks of src")
    sums = torch.empty(max(int(waves), 1), dtype=torch.float32, device=src.device)
    _check(library().segred_probe_stream(
        ctypes.c_void_p(src.data_ptr()), nbytes,
        ctypes.c_void_p(dst.data_ptr() if dst is not None and write_every > 0 else 0),
        int(write_every), ctypes.c_void_p(sums.data_ptr()), int(waves),
        ctypes.c_void_p(_stream(src.device))), "segred_probe_stream")
    return sums, (dst if write_every > 0 else None)
