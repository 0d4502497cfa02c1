"""Python binding of libsgmv: SGMV expand-slice on MI355X (gfx950).

Argument marshalling only.  Every step of the operation runs in the HIP
kernels of ``libsgmv.so`` (built in-tree by ``build.py``); PyTorch supplies
device memory and the current stream.  There is no CPU or PyTorch fallback:
if the library is missing, importing this package raises.

Names and argument order follow the wiki page "Implementation: Predibase
Lorax SGMV Expand Slice Kernel" (Signature; I/O Contract):

    sgmv_expand_slice(inputs, lora_b_weights, output_tensor, b_seq_start_loc,
                      seq_len_tensor, lora_indices_tensor, batches,
                      max_seq_length, slice_offset, slice_size, add_inputs=False)

plus the LoRA-A projection that produces those inputs (sgmv_shrink), the
per-token and multi-slice forms, and the two steps fused in one launch
(sgmv_fused_shrink_expand); and the operators a serving step runs beside them:
a shared projection with the adapters (sgmv_lora_linear), products grouped by
expert (sgmv_grouped_gemm), the routing that lays out their segments
(sgmv_route) and the sum of a token's expert rows (sgmv_combine); and both
products with microscaled 4-bit weights (sgmv_mx_lora_linear,
sgmv_mx_grouped_gemm), which sgmv_mx_quantize makes and sgmv_mx_dequantize
reads back.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_HERE, "libsgmv.so")

SGMV_OK, SGMV_ERR_INVALID_ARGUMENT, SGMV_ERR_UNSUPPORTED, SGMV_ERR_HIP = range(4)
MAX_SLICES = 8
MAX_FUSED_SLICES = 3

# Every symbol include/sgmv.h declares.
EXPORTED_SYMBOLS = ("sgmv_expand_slice", "sgmv_expand_multi_slice", "sgmv_bgmv_expand_slice",
                    "sgmv_shrink", "sgmv_shrink_multi_slice", "sgmv_shrink_workspace_bytes",
                    "sgmv_shrink_multi_slice_noalloc",
                    "sgmv_fused_shrink_expand", "sgmv_lora_linear",
                    "sgmv_lora_linear_workspace_bytes", "sgmv_grouped_gemm", "sgmv_route",
                    "sgmv_route_workspace_bytes", "sgmv_combine", "sgmv_mx_quantize",
                    "sgmv_mx_dequantize", "sgmv_mx_lora_linear",
                    "sgmv_mx_lora_linear_workspace_bytes", "sgmv_mx_grouped_gemm",
                    "sgmv_mx_grouped_gemm_workspace_bytes", "sgmv_last_error",
                    "sgmv_abi_version")


class Matrix(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("row_stride", ctypes.c_int64)]


class Stack(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("num", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class SliceDesc(ctypes.Structure):
    _fields_ = [("inputs", Matrix), ("lora_b", Stack), ("slice_offset", ctypes.c_int64),
                ("slice_size", ctypes.c_int64)]


class ShrinkSliceDesc(ctypes.Structure):
    _fields_ = [("lora_a", Stack), ("out", Matrix)]


class FusedSliceDesc(ctypes.Structure):
    _fields_ = [("lora_a", Stack), ("lora_b", Stack), ("slice_offset", ctypes.c_int64)]


class MxStack(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("num", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("code_stride", ctypes.c_int64),
                ("scale_stride", ctypes.c_int64)]


def _hip_runtimes_mapped():
    """Distinct HIP runtime files mapped into this process."""
    found = set()
    try:
        with open("/proc/self/maps") as f:
            for line in f:
                path = line.split()[-1] if line.strip() else ""
                if "libamdhip64.so" in os.path.basename(path):
                    found.add(os.path.realpath(path))
    except OSError:
        pass
    return found


def _load_library() -> ctypes.CDLL:
    # PyTorch ships its own HIP runtime.  Load it first so that libsgmv's
    # dependency on libamdhip64.so.7 resolves to that same, already mapped
    # runtime: two HIP runtimes in one process do not share devices, streams
    # or allocations.
    import torch  # noqa: F401
    if not os.path.exists(LIBRARY_PATH):
        raise ImportError(
            f"{LIBRARY_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; "
            f"g.build()'` (or python segmented_gather_gemm_amd/build.py). There is no fallback.")
    lib = ctypes.CDLL(LIBRARY_PATH)
    runtimes = _hip_runtimes_mapped()
    if len(runtimes) > 1:
        raise ImportError(f"two HIP runtimes are mapped into this process: {sorted(runtimes)}")
    i64, p = ctypes.c_int64, ctypes.c_void_p
    lib.sgmv_expand_slice.argtypes = [Matrix, Stack, Matrix, p, p, p, i64, i64, i64, i64,
                                      ctypes.c_int, p]
    lib.sgmv_expand_slice.restype = ctypes.c_int
    lib.sgmv_expand_multi_slice.argtypes = [ctypes.POINTER(SliceDesc), ctypes.c_int, Matrix, p, p,
                                            p, i64, i64, ctypes.c_int, p]
    lib.sgmv_expand_multi_slice.restype = ctypes.c_int
    lib.sgmv_bgmv_expand_slice.argtypes = [Matrix, Stack, Matrix, p, i64, i64, ctypes.c_int, p]
    lib.sgmv_bgmv_expand_slice.restype = ctypes.c_int
    lib.sgmv_shrink.argtypes = [Matrix, Stack, Matrix, p, p, p, i64, i64, ctypes.c_float, p,
                                ctypes.c_size_t, p]
    lib.sgmv_shrink.restype = ctypes.c_int
    lib.sgmv_shrink_multi_slice.argtypes = [Matrix, ctypes.POINTER(ShrinkSliceDesc), ctypes.c_int,
                                            p, p, p, i64, i64, ctypes.c_float, p,
                                            ctypes.c_size_t, p]
    lib.sgmv_shrink_multi_slice.restype = ctypes.c_int
    lib.sgmv_shrink_workspace_bytes.argtypes = [ctypes.POINTER(ctypes.c_size_t)]
    lib.sgmv_shrink_workspace_bytes.restype = ctypes.c_int
    lib.sgmv_shrink_multi_slice_noalloc.argtypes = [Matrix, ctypes.POINTER(ShrinkSliceDesc),
                                                    ctypes.c_int, p, p, p, i64, i64,
                                                    ctypes.c_float, p]
    lib.sgmv_shrink_multi_slice_noalloc.restype = ctypes.c_int
    lib.sgmv_fused_shrink_expand.argtypes = [Matrix, ctypes.POINTER(FusedSliceDesc), ctypes.c_int,
                                             Matrix, p, p, p, i64, i64, ctypes.c_float,
                                             ctypes.c_int, p]
    lib.sgmv_fused_shrink_expand.restype = ctypes.c_int
    lib.sgmv_lora_linear.argtypes = [Matrix, Matrix, p, ctypes.POINTER(FusedSliceDesc),
                                     ctypes.c_int, Matrix, p, p, p, i64, i64, ctypes.c_float,
                                     ctypes.c_int, p, ctypes.c_size_t, p]
    lib.sgmv_lora_linear.restype = ctypes.c_int
    lib.sgmv_lora_linear_workspace_bytes.argtypes = [i64, ctypes.c_int, i64,
                                                     ctypes.POINTER(ctypes.c_size_t)]
    lib.sgmv_lora_linear_workspace_bytes.restype = ctypes.c_int
    lib.sgmv_grouped_gemm.argtypes = [Matrix, Stack, Matrix, p, p, p, p, i64, i64, ctypes.c_int,
                                      p]
    lib.sgmv_grouped_gemm.restype = ctypes.c_int
    lib.sgmv_route.argtypes = [Matrix, i64, ctypes.c_int, p, p, p, p, p, p, p, ctypes.c_size_t, p]
    lib.sgmv_route.restype = ctypes.c_int
    lib.sgmv_route_workspace_bytes.argtypes = [i64, i64, i64, ctypes.POINTER(ctypes.c_size_t)]
    lib.sgmv_route_workspace_bytes.restype = ctypes.c_int
    lib.sgmv_combine.argtypes = [Matrix, p, p, i64, Matrix, ctypes.c_int, p]
    lib.sgmv_combine.restype = ctypes.c_int
    lib.sgmv_mx_quantize.argtypes = [Matrix, MxStack, p]
    lib.sgmv_mx_quantize.restype = ctypes.c_int
    lib.sgmv_mx_dequantize.argtypes = [MxStack, p, Matrix, p]
    lib.sgmv_mx_dequantize.restype = ctypes.c_int
    lib.sgmv_mx_lora_linear.argtypes = [Matrix, MxStack, p, ctypes.POINTER(FusedSliceDesc),
                                        ctypes.c_int, Matrix, p, p, p, i64, i64, ctypes.c_float,
                                        ctypes.c_int, p, ctypes.c_size_t, p]
    lib.sgmv_mx_lora_linear.restype = ctypes.c_int
    lib.sgmv_mx_lora_linear_workspace_bytes.argtypes = [i64, i64, ctypes.c_int, i64,
                                                        ctypes.POINTER(ctypes.c_size_t)]
    lib.sgmv_mx_lora_linear_workspace_bytes.restype = ctypes.c_int
    lib.sgmv_mx_grouped_gemm.argtypes = [Matrix, MxStack, Matrix, p, p, p, p, i64, i64,
                                         ctypes.c_int, p, ctypes.c_size_t, p]
    lib.sgmv_mx_grouped_gemm.restype = ctypes.c_int
    lib.sgmv_mx_grouped_gemm_workspace_bytes.argtypes = [i64, i64, ctypes.POINTER(ctypes.c_size_t)]
    lib.sgmv_mx_grouped_gemm_workspace_bytes.restype = ctypes.c_int
    lib.sgmv_last_error.argtypes = []
    lib.sgmv_last_error.restype = ctypes.c_char_p
    lib.sgmv_abi_version.argtypes = []
    lib.sgmv_abi_version.restype = ctypes.c_int
    return lib


lib = _load_library()

import torch as _torch  # noqa: E402  (loaded by _load_library before the library)

_DTYPE_CODES = {_torch.float16: 0, _torch.bfloat16: 1, _torch.float32: 2}
# The current stream's raw handle without building a Stream object (a
# measurable part of a call's host time); the public route where absent.
_RAW_STREAM = getattr(_torch._C, "_cuda_getCurrentRawStream", None)
_CURRENT_DEVICE = getattr(_torch._C, "_cuda_getDevice", _torch.cuda.current_device)


def _stream(device) -> int:
    if _RAW_STREAM is not None:
        return _RAW_STREAM(device.index)
    return _torch.cuda.current_stream(device).cuda_stream


def _call_on(device, fn, *args):
    """fn(*args) with `device` current (made current only when it is not)."""
    if _CURRENT_DEVICE() == device.index:
        return fn(*args)
    with _torch.cuda.device(device):
        return fn(*args)


class SgmvError(RuntimeError):
    """A HIP runtime failure reported by libsgmv."""


def _raise(status: int):
    msg = lib.sgmv_last_error().decode(errors="replace")
    if status == SGMV_ERR_INVALID_ARGUMENT:
        raise ValueError(msg)
    if status == SGMV_ERR_UNSUPPORTED:
        raise NotImplementedError(msg)
    raise SgmvError(msg)


def _dtype_code(t) -> int:
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _matrix(t, what: str) -> Matrix:
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must be 2-D, got shape {tuple(shape)}")
    rows, cols = shape
    s0, s1 = t.stride()
    if cols > 1 and s1 != 1:
        raise ValueError(f"{what} must have unit column stride")
    return Matrix(t.data_ptr(), _dtype_code(t), rows, cols, s0 if rows > 1 else max(cols, s0))


def _stack(w, what: str) -> Stack:
    if w.dim() == 4:
        if w.shape[1] != 1:
            raise ValueError(f"{what}: a 4-D lora_b must be (lora_num, 1, slice_size, rank)")
        w = w.squeeze(1)
    shape = w.shape
    if len(shape) != 3:
        raise ValueError(f"{what} must be (lora_num, slice_size, rank), got {tuple(shape)}")
    if not w.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return Stack(w.data_ptr(), _dtype_code(w), shape[0], shape[1], shape[2])


def _meta(t, what: str, device):
    if t.dim() != 1:
        raise ValueError(f"{what} must be 1-D")
    if t.device != device:
        raise ValueError(f"{what} must be on {device}")
    if t.dtype is not _torch.int64 or not t.is_contiguous():
        t = t.to(_torch.int64).contiguous()   # documented marshalling copy
    return t


def _common(output_tensor, metas):
    device = output_tensor.device
    if device.type != "cuda":
        raise ValueError("output_tensor must be a GPU tensor")
    kept = [_meta(m, n, device) for m, n in metas]
    return device, kept


def sgmv_expand_slice(inputs, lora_b_weights, output_tensor, b_seq_start_loc, seq_len_tensor,
                      lora_indices_tensor, batches: int, max_seq_length: int, slice_offset: int,
                      slice_size: int, add_inputs: bool = False):
    """In place: output_tensor[start_b + m, slice_offset:slice_offset + slice_size]
    (+)= inputs[start_b + m] @ lora_b_weights[lora_indices[b]].T for every
    segment b with index != -1.  Enqueued on the current stream."""
    device, (start, lens, idx) = _common(output_tensor, [
        (b_seq_start_loc, "b_seq_start_loc"), (seq_len_tensor, "seq_len_tensor"),
        (lora_indices_tensor, "lora_indices_tensor")])
    for t, n in ((inputs, "inputs"), (lora_b_weights, "lora_b_weights")):
        if t.device != device:
            raise ValueError(f"{n} must be on {device}")
    if start.shape[0] < batches or lens.shape[0] < batches or idx.shape[0] < batches:
        raise ValueError("segment metadata shorter than batches")
    x = _matrix(inputs, "inputs")
    w = _stack(lora_b_weights, "lora_b_weights")
    out = _matrix(output_tensor, "output_tensor")
    stream = _stream(device)
    st = _call_on(device, lib.sgmv_expand_slice, x, w, out, start.data_ptr(), lens.data_ptr(),
                  idx.data_ptr(), int(batches), int(max_seq_length), int(slice_offset),
                  int(slice_size), int(bool(add_inputs)), stream)
    if st != SGMV_OK:
        _raise(st)
    return output_tensor


def sgmv_expand_multi_slice(slices: Sequence[Tuple[object, object, int]], output_tensor,
                            b_seq_start_loc, seq_len_tensor, lora_indices_tensor, batches: int,
                            max_seq_length: int, add_inputs: bool = False):
    """Several slices of one fused output (e.g. Q, K, V) in one launch.

    ``slices``: sequence of (inputs, lora_b_weights, slice_offset); each
    slice's size is its lora_b_weights.size(-2).  Bit-identical to one
    sgmv_expand_slice call per slice."""
    if not 1 <= len(slices) <= MAX_SLICES:
        raise ValueError(f"1..{MAX_SLICES} slices, got {len(slices)}")
    device, (start, lens, idx) = _common(output_tensor, [
        (b_seq_start_loc, "b_seq_start_loc"), (seq_len_tensor, "seq_len_tensor"),
        (lora_indices_tensor, "lora_indices_tensor")])
    if start.shape[0] < batches or lens.shape[0] < batches or idx.shape[0] < batches:
        raise ValueError("segment metadata shorter than batches")
    arr = (SliceDesc * len(slices))()
    for i, (x, w, off) in enumerate(slices):
        if x.device != device or w.device != device:
            raise ValueError(f"slice {i} must be on {device}")
        st = _stack(w, f"slice {i} lora_b")
        arr[i] = SliceDesc(_matrix(x, f"slice {i} inputs"), st, int(off), st.rows)
    out = _matrix(output_tensor, "output_tensor")
    stream = _stream(device)
    rc = _call_on(device, lib.sgmv_expand_multi_slice, arr, len(slices), out, start.data_ptr(),
                  lens.data_ptr(), idx.data_ptr(), int(batches), int(max_seq_length),
                  int(bool(add_inputs)), stream)
    if rc != SGMV_OK:
        _raise(rc)
    return output_tensor


def bgmv_expand_slice(inputs, lora_b_weights, output_tensor, lora_indices_tensor, slice_offset: int,
                      slice_size: int, add_inputs: bool = False):
    """Per-token form: output_tensor[t, slice_offset:slice_offset + slice_size]
    (+)= inputs[t] @ lora_b_weights[lora_indices[t]].T for every token t with
    index != -1.  Enqueued on the current stream."""
    device, (idx,) = _common(output_tensor, [(lora_indices_tensor, "lora_indices_tensor")])
    for t, n in ((inputs, "inputs"), (lora_b_weights, "lora_b_weights")):
        if t.device != device:
            raise ValueError(f"{n} must be on {device}")
    if idx.shape[0] < output_tensor.shape[0]:
        raise ValueError("lora_indices_tensor shorter than the number of tokens")
    x = _matrix(inputs, "inputs")
    w = _stack(lora_b_weights, "lora_b_weights")
    out = _matrix(output_tensor, "output_tensor")
    stream = _stream(device)
    st = _call_on(device, lib.sgmv_bgmv_expand_slice, x, w, out, idx.data_ptr(),
                  int(slice_offset), int(slice_size), int(bool(add_inputs)), stream)
    if st != SGMV_OK:
        _raise(st)
    return output_tensor


def _stack_a(w, what: str) -> Stack:
    if w.dim() != 3:
        raise ValueError(f"{what} must be (lora_num, rank, hidden), got {tuple(w.shape)}")
    if not w.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return Stack(w.data_ptr(), _dtype_code(w), w.shape[0], w.shape[1], w.shape[2])


def shrink_workspace_bytes(device=None) -> int:
    """Bytes of the workspace the shrink calls take on `device` (default:
    the current one)."""
    device = _torch.device("cuda", _torch.cuda.current_device()) if device is None else \
        _torch.device(device)
    n = ctypes.c_size_t()
    rc = _call_on(device, lib.sgmv_shrink_workspace_bytes, ctypes.byref(n))
    if rc != SGMV_OK:
        _raise(rc)
    return n.value


# One zero-filled shrink workspace per device, made on first use.
_WORKSPACES = {}


def _workspace(device, workspace):
    """(pointer, bytes) for a shrink call's `workspace` argument: True = this
    device's shared buffer (made and zero-filled on first use; a first use
    inside a graph capture runs without one, since the fill would run only at
    replay), None or False = none, a uint8 tensor = the caller's buffer (zero
    before its first use)."""
    if workspace is None or workspace is False:
        return None, 0
    if workspace is True:
        ws = _WORKSPACES.get(device.index)
        if ws is None:
            if _torch.cuda.is_current_stream_capturing():
                return None, 0
            ws = _torch.zeros(shrink_workspace_bytes(device), dtype=_torch.uint8, device=device)
            _torch.cuda.synchronize(device)
            _WORKSPACES[device.index] = ws
        return ws.data_ptr(), ws.numel()
    if not _torch.is_tensor(workspace) or workspace.device != device or \
            workspace.dtype != _torch.uint8 or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    return workspace.data_ptr(), workspace.numel()


def sgmv_shrink(inputs, lora_a_weights, output_tensor, b_seq_start_loc, seq_len_tensor,
                lora_indices_tensor, batches: int, max_seq_length: int, scaling: float = 1.0,
                workspace=True):
    """LoRA-A projection, in place: output_tensor[start_b + m] =
    scaling * inputs[start_b + m] @ lora_a_weights[lora_indices[b]].T for every
    segment b with index != -1 (other rows untouched); lora_a_weights is
    (lora_num, rank, hidden).  Enqueued on the current stream.  `workspace`:
    True (the device's shared buffer: calls that may run concurrently on
    other streams pass buffers of their own), None (large batches run
    unbalanced) or a zero-initialised uint8 tensor of shrink_workspace_bytes()."""
    return sgmv_shrink_multi_slice(inputs, [(lora_a_weights, output_tensor)], b_seq_start_loc,
                                   seq_len_tensor, lora_indices_tensor, batches, max_seq_length,
                                   scaling, workspace)


def _shrink_args(inputs, slices, b_seq_start_loc, seq_len_tensor, lora_indices_tensor,
                 batches):
    """(device, inputs matrix, slice descriptors, start, lens, idx) of a shrink call."""
    if not 1 <= len(slices) <= MAX_SLICES:
        raise ValueError(f"1..{MAX_SLICES} slices, got {len(slices)}")
    device, (start, lens, idx) = _common(inputs, [
        (b_seq_start_loc, "b_seq_start_loc"), (seq_len_tensor, "seq_len_tensor"),
        (lora_indices_tensor, "lora_indices_tensor")])
    if start.shape[0] < batches or lens.shape[0] < batches or idx.shape[0] < batches:
        raise ValueError("segment metadata shorter than batches")
    arr = (ShrinkSliceDesc * len(slices))()
    for i, (w, o) in enumerate(slices):
        if w.device != device or o.device != device:
            raise ValueError(f"slice {i} must be on {device}")
        arr[i] = ShrinkSliceDesc(_stack_a(w, f"slice {i} lora_a"), _matrix(o, f"slice {i} output"))
    return device, _matrix(inputs, "inputs"), arr, start, lens, idx


def sgmv_shrink_multi_slice(inputs, slices: Sequence[Tuple[object, object]], b_seq_start_loc,
                            seq_len_tensor, lora_indices_tensor, batches: int,
                            max_seq_length: int, scaling: float = 1.0, workspace=True):
    """Several LoRA-A projections of the same inputs (e.g. Q, K, V) reading
    the inputs once.  ``slices``: sequence of (lora_a_weights, output_tensor).
    Bit-identical to one sgmv_shrink call per slice with the same
    `workspace` choice."""
    device, x, arr, start, lens, idx = _shrink_args(inputs, slices, b_seq_start_loc,
                                                    seq_len_tensor, lora_indices_tensor, batches)
    ws, ws_bytes = _workspace(device, workspace)
    stream = _stream(device)
    rc = _call_on(device, lib.sgmv_shrink_multi_slice, x, arr, len(slices), start.data_ptr(),
                  lens.data_ptr(), idx.data_ptr(), int(batches), int(max_seq_length),
                  float(scaling), ws, ws_bytes, stream)
    if rc != SGMV_OK:
        _raise(rc)
    return [o for _, o in slices]


def sgmv_shrink_multi_slice_noalloc(inputs, slices: Sequence[Tuple[object, object]],
                                    b_seq_start_loc, seq_len_tensor, lora_indices_tensor,
                                    batches: int, max_seq_length: int, scaling: float = 1.0):
    """sgmv_shrink_multi_slice on the library's static workspace (for callers
    that cannot allocate; calls that may overlap on one device race on it).
    Equal bit for bit to sgmv_shrink_multi_slice with a workspace."""
    device, x, arr, start, lens, idx = _shrink_args(inputs, slices, b_seq_start_loc,
                                                    seq_len_tensor, lora_indices_tensor, batches)
    stream = _stream(device)
    rc = _call_on(device, lib.sgmv_shrink_multi_slice_noalloc, x, arr, len(slices),
                  start.data_ptr(), lens.data_ptr(), idx.data_ptr(), int(batches),
                  int(max_seq_length), float(scaling), stream)
    if rc != SGMV_OK:
        _raise(rc)
    return [o for _, o in slices]


def sgmv_fused_shrink_expand(inputs, slices: Sequence[Tuple[object, object, int]], output_tensor,
                             b_seq_start_loc, seq_len_tensor, lora_indices_tensor, batches: int,
                             max_seq_length: int, scaling: float = 1.0,
                             add_inputs: bool = False):
    """The LoRA-A projection and the expand of its result in one launch, for
    the slices of a fused layer: for each (lora_a_weights (lora_num, rank,
    hidden), lora_b_weights (lora_num, slice_size, rank), slice_offset),
    output_tensor[start_b + m, off:off + slice_size] (+)= rne_w(scaling *
    inputs[start_b + m] @ lora_a[idx].T) @ lora_b[idx].T, the projection
    rounded to the weights' 16-bit dtype and never stored.  Equal to
    sgmv_shrink_multi_slice into weight-dtype outputs followed by
    sgmv_expand_multi_slice.  Enqueued on the current stream."""
    if not 1 <= len(slices) <= MAX_FUSED_SLICES:
        raise ValueError(f"1..{MAX_FUSED_SLICES} slices, got {len(slices)}")
    device, (start, lens, idx) = _common(output_tensor, [
        (b_seq_start_loc, "b_seq_start_loc"), (seq_len_tensor, "seq_len_tensor"),
        (lora_indices_tensor, "lora_indices_tensor")])
    if inputs.device != device:
        raise ValueError(f"inputs must be on {device}")
    if start.shape[0] < batches or lens.shape[0] < batches or idx.shape[0] < batches:
        raise ValueError("segment metadata shorter than batches")
    arr = (FusedSliceDesc * len(slices))()
    for i, (a, w, off) in enumerate(slices):
        if a.device != device or w.device != device:
            raise ValueError(f"slice {i} must be on {device}")
        arr[i] = FusedSliceDesc(_stack_a(a, f"slice {i} lora_a"), _stack(w, f"slice {i} lora_b"),
                                int(off))
    x = _matrix(inputs, "inputs")
    out = _matrix(output_tensor, "output_tensor")
    stream = _stream(device)
    rc = _call_on(device, lib.sgmv_fused_shrink_expand, x, arr, len(slices), out,
                  start.data_ptr(), lens.data_ptr(), idx.data_ptr(), int(batches),
                  int(max_seq_length), float(scaling), int(bool(add_inputs)), stream)
    if rc != SGMV_OK:
        _raise(rc)
    return output_tensor


def _bytes_of(fn, *args) -> int:
    n = ctypes.c_size_t()
    rc = fn(*args, ctypes.byref(n))
    if rc != SGMV_OK:
        _raise(rc)
    return n.value


def lora_linear_workspace_bytes(tokens: int, num_slices: int, rank: int) -> int:
    """Bytes of the workspace sgmv_lora_linear takes."""
    return _bytes_of(lib.sgmv_lora_linear_workspace_bytes, int(tokens), int(num_slices), int(rank))


def route_workspace_bytes(tokens: int, experts: int, top_k: int) -> int:
    """Bytes of the workspace sgmv_route takes (0 for small batches)."""
    return _bytes_of(lib.sgmv_route_workspace_bytes, int(tokens), int(experts), int(top_k))


def _scratch(device, workspace, need: int):
    """(tensor to keep alive, pointer, bytes) of a call's scratch memory: the
    caller's uint8 tensor, or None = taken from torch's allocator for this
    call (it is stream-ordered, so the next user of the memory on this stream
    comes after the call's kernels)."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = _torch.empty(need, dtype=_torch.uint8, device=device)
    elif not _torch.is_tensor(workspace) or workspace.device != device or \
            workspace.dtype != _torch.uint8 or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    return workspace, workspace.data_ptr(), workspace.numel()


def _bias(bias, cols: int, dtype, device):
    if bias is None:
        return None
    if bias.device != device or bias.dim() != 1 or bias.shape[0] != cols or \
            bias.dtype != dtype or not bias.is_contiguous():
        raise ValueError(f"bias must be a contiguous ({cols},) {dtype} tensor on {device}")
    return bias.data_ptr()


def _fused_slices(slices, device):
    arr = (FusedSliceDesc * max(1, len(slices)))()
    for i, (a, b, off) in enumerate(slices):
        if a.device != device or b.device != device:
            raise ValueError(f"slice {i} must be on {device}")
        arr[i] = FusedSliceDesc(_stack_a(a, f"slice {i} lora_a"), _stack(b, f"slice {i} lora_b"),
                                int(off))
    return arr


def sgmv_lora_linear(inputs, weight, slices: Sequence[Tuple[object, object, int]], output_tensor,
                     b_seq_start_loc, seq_len_tensor, lora_indices_tensor, batches: int,
                     max_seq_length: int, scaling: float = 1.0, bias=None,
                     add_inputs: bool = False, workspace=None):
    """A shared projection with the adapters of many requests beside it:
    output_tensor (+)= inputs @ weight.T + bias for every row, plus, for each
    (lora_a_weights (lora_num, rank, hidden), lora_b_weights (lora_num,
    slice_size, rank), slice_offset) in ``slices`` and every segment b with
    index != -1, scaling * (inputs[rows] @ lora_a[idx].T) @ lora_b[idx].T in
    the columns [slice_offset, slice_offset + slice_size).  One rounding;
    ``slices`` may be empty.  Enqueued on the current stream.  `workspace`:
    a uint8 tensor of lora_linear_workspace_bytes(), or None (taken from
    torch's allocator for the call)."""
    if len(slices) > MAX_SLICES:
        raise ValueError(f"at most {MAX_SLICES} slices, got {len(slices)}")
    device, (start, lens, idx) = _common(output_tensor, [
        (b_seq_start_loc, "b_seq_start_loc"), (seq_len_tensor, "seq_len_tensor"),
        (lora_indices_tensor, "lora_indices_tensor")])
    if inputs.device != device or weight.device != device:
        raise ValueError(f"inputs and weight must be on {device}")
    if start.shape[0] < batches or lens.shape[0] < batches or idx.shape[0] < batches:
        raise ValueError("segment metadata shorter than batches")
    x = _matrix(inputs, "inputs")
    w = _matrix(weight, "weight")
    out = _matrix(output_tensor, "output_tensor")
    bias_ptr = _bias(bias, w.rows, weight.dtype, device)
    arr = _fused_slices(slices, device)
    need = 0
    if slices and batches > 0 and workspace is None:
        need = lora_linear_workspace_bytes(x.rows, len(slices), arr[0].lora_a.rows)
    keep, ws, ws_bytes = _scratch(device, workspace, need)
    rc = _call_on(device, lib.sgmv_lora_linear, x, w, bias_ptr, arr, len(slices), out,
                  start.data_ptr(), lens.data_ptr(), idx.data_ptr(), int(batches),
                  int(max_seq_length), float(scaling), int(bool(add_inputs)), ws, ws_bytes,
                  _stream(device))
    if rc != SGMV_OK:
        _raise(rc)
    return output_tensor


def sgmv_grouped_gemm(inputs, expert_weights, output_tensor, b_seq_start_loc, seq_len_tensor,
                      expert_indices_tensor, batches: int, max_seq_length: int,
                      row_indices_tensor=None, gated: bool = False):
    """Products grouped by expert, in place: for every row r of segment b with
    expert e = expert_indices[b] (None: b itself), output_tensor[r] =
    inputs[row_indices[r]] (None: inputs[r]) @ expert_weights[e].T;
    expert_weights is (experts, columns, hidden).  ``gated``: the weights hold
    2 * columns rows, gate first, and output_tensor[r] = silu(gate) * other.
    Rows outside the segments and of index -1 ones are untouched.  Enqueued on
    the current stream."""
    metas = [(b_seq_start_loc, "b_seq_start_loc"), (seq_len_tensor, "seq_len_tensor")]
    if expert_indices_tensor is not None:
        metas.append((expert_indices_tensor, "expert_indices_tensor"))
    device, kept = _common(output_tensor, metas)
    if any(m.shape[0] < batches for m in kept):
        raise ValueError("segment metadata shorter than batches")
    if inputs.device != device or expert_weights.device != device:
        raise ValueError(f"inputs and expert_weights must be on {device}")
    x = _matrix(inputs, "inputs")
    if expert_weights.dim() != 3 or not expert_weights.is_contiguous():
        raise ValueError("expert_weights must be contiguous (experts, columns, hidden), got "
                         f"{tuple(expert_weights.shape)}")
    w = Stack(expert_weights.data_ptr(), _dtype_code(expert_weights), *expert_weights.shape)
    out = _matrix(output_tensor, "output_tensor")
    rows = None
    if row_indices_tensor is not None:
        rows = _meta(row_indices_tensor, "row_indices_tensor", device)
        if rows.shape[0] < out.rows:
            raise ValueError("row_indices_tensor shorter than the number of output rows")
    rc = _call_on(device, lib.sgmv_grouped_gemm, x, w, out,
                  None if rows is None else rows.data_ptr(), kept[0].data_ptr(),
                  kept[1].data_ptr(), kept[2].data_ptr() if len(kept) > 2 else None, int(batches),
                  int(max_seq_length), int(bool(gated)), _stream(device))
    if rc != SGMV_OK:
        _raise(rc)
    return output_tensor


def _flat(t, what: str, device, dtype, shape):
    if t.device != device or t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {shape} {dtype} tensor on {device}, got "
                         f"{tuple(t.shape)} {t.dtype}")
    return t.data_ptr()


def sgmv_route(logits, weights, experts, slots, row_indices_tensor, b_seq_start_loc,
               seq_len_tensor, renormalize: bool = False, workspace=None):
    """Choose each token's experts and lay the choices out as the segments
    sgmv_grouped_gemm takes, all on the device.  logits is (tokens, experts);
    weights (float32), experts and slots (int64) are (tokens, top_k), written;
    row_indices_tensor (tokens * top_k,), b_seq_start_loc and seq_len_tensor
    (experts,) are int64, written.  Largest logits first, ties to the lowest
    expert; softmax over all experts, or over the choices (``renormalize``);
    -inf and NaN logits are closed, missing choices are -1 with weight 0.
    Enqueued on the current stream.  `workspace`: a uint8 tensor of
    route_workspace_bytes(), or None (taken from torch's allocator)."""
    device = logits.device
    if device.type != "cuda":
        raise ValueError("logits must be a GPU tensor")
    x = _matrix(logits, "logits")
    if weights.dim() != 2 or weights.shape[0] != x.rows:
        raise ValueError(f"weights must be ({x.rows}, top_k), got {tuple(weights.shape)}")
    T, k, E = x.rows, weights.shape[1], x.cols
    i64 = _torch.int64
    ptrs = (_flat(weights, "weights", device, _torch.float32, (T, k)),
            _flat(experts, "experts", device, i64, (T, k)),
            _flat(slots, "slots", device, i64, (T, k)),
            _flat(row_indices_tensor, "row_indices_tensor", device, i64, (T * k,)),
            _flat(b_seq_start_loc, "b_seq_start_loc", device, i64, (E,)),
            _flat(seq_len_tensor, "seq_len_tensor", device, i64, (E,)))
    need = route_workspace_bytes(T, E, k) if workspace is None else 0
    keep, ws, ws_bytes = _scratch(device, workspace, need)
    rc = _call_on(device, lib.sgmv_route, x, k, int(bool(renormalize)), *ptrs, ws, ws_bytes,
                  _stream(device))
    if rc != SGMV_OK:
        _raise(rc)
    return weights, experts


def sgmv_combine(expert_rows, weights, slots, output_tensor, add_inputs: bool = False):
    """output_tensor[t] (+)= sum over j of weights[t, j] * expert_rows[slots[t, j]]
    (slots outside expert_rows, such as -1, add nothing); weights float32 and
    slots int64, both (tokens, top_k).  Enqueued on the current stream."""
    device = output_tensor.device
    if device.type != "cuda":
        raise ValueError("output_tensor must be a GPU tensor")
    if expert_rows.device != device:
        raise ValueError(f"expert_rows must be on {device}")
    rows = _matrix(expert_rows, "expert_rows")
    out = _matrix(output_tensor, "output_tensor")
    if weights.dim() != 2 or weights.shape[0] != out.rows:
        raise ValueError(f"weights must be ({out.rows}, top_k), got {tuple(weights.shape)}")
    k = weights.shape[1]
    wp = _flat(weights, "weights", device, _torch.float32, (out.rows, k))
    sp = _flat(slots, "slots", device, _torch.int64, (out.rows, k))
    rc = _call_on(device, lib.sgmv_combine, rows, wp, sp, k, out, int(bool(add_inputs)),
                  _stream(device))
    if rc != SGMV_OK:
        _raise(rc)
    return output_tensor


def mx_row_bytes(hidden: int) -> Tuple[int, int]:
    """Bytes of codes and of scales that a row of `hidden` values takes in
    microscaled 4-bit form: 64 and 4 for every group of 128."""
    groups = -(-int(hidden) // 128)
    return 64 * groups, 4 * groups


def _mx_rows(t, what: str, device, dims: int, need: int):
    """(matrices, rows, bytes from row to row) of codes or scales, `need` bytes a row."""
    shape = t.shape
    if t.device != device:
        raise ValueError(f"{what} must be on {device}")
    if len(shape) != dims or shape[-1] != need or t.dtype is not _torch.uint8:
        raise ValueError(f"{what} must be {dims}-D uint8 with {need} bytes a row, got {tuple(shape)} "
                         f"{t.dtype}")
    if dims == 3:
        if not t.is_contiguous():
            raise ValueError(f"{what} must have contiguous matrices")
        return shape[0], shape[1], need
    stride, one = t.stride()
    if one != 1:
        raise ValueError(f"{what} must have contiguous rows")
    return 1, shape[0], stride if shape[0] > 1 else need


def _mx_stack(codes, scales, hidden: int, what: str, device, dims: int) -> MxStack:
    """codes and scales, (rows, bytes) or (matrices, rows, bytes) of uint8, as
    rows of `hidden` values."""
    groups = (hidden + 127) // 128
    num, rows, code_stride = _mx_rows(codes, what + " codes", device, dims, 64 * groups)
    num2, rows2, scale_stride = _mx_rows(scales, what + " scales", device, dims, 4 * groups)
    if rows != rows2 or num != num2:
        raise ValueError(f"{what}: codes {tuple(codes.shape)} and scales {tuple(scales.shape)} differ "
                         "in rows")
    return MxStack(codes.data_ptr(), scales.data_ptr(), num, rows, hidden, code_stride, scale_stride)


def _row_indices(t, rows: int, device):
    if t is None:
        return None
    t = _meta(t, "row_indices_tensor", device)
    if t.shape[0] < rows:
        raise ValueError("row_indices_tensor shorter than the number of output rows")
    return t


def _gpu(t, what: str):
    device = t.device
    if device.type != "cuda":
        raise ValueError(f"{what} must be a GPU tensor")
    return device


def sgmv_mx_quantize(inputs, codes, scales):
    """Rows as microscaled 4-bit values, in place: codes (rows, 64 G) and scales
    (rows, 4 G), uint8, G = ceil(hidden / 128) (mx_row_bytes), from inputs
    (rows, hidden) float16, bfloat16 or float32.  32 values of a row share the
    scale 2^(floor(log2 of the largest) - 2), byte exponent + 127, and take the
    nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 of it (ties to the even code, the even
    value in a byte's low half); 255 marks a block with an infinity or NaN.
    Enqueued on the current stream."""
    device = _gpu(inputs, "inputs")
    x = _matrix(inputs, "inputs")
    q = _mx_stack(codes, scales, x.cols, "output", device, 2)
    rc = _call_on(device, lib.sgmv_mx_quantize, x, q, _stream(device))
    if rc != SGMV_OK:
        _raise(rc)
    return codes, scales


def sgmv_mx_dequantize(codes, scales, output_tensor, row_indices_tensor=None):
    """output_tensor[t] = the values of row row_indices_tensor[t] (None: row t)
    of codes and scales; indices outside their rows give rows of zeros.
    Enqueued on the current stream."""
    device = _gpu(output_tensor, "output_tensor")
    out = _matrix(output_tensor, "output_tensor")
    rows = _row_indices(row_indices_tensor, out.rows, device)
    q = _mx_stack(codes, scales, out.cols, "input", device, 2)
    rc = _call_on(device, lib.sgmv_mx_dequantize, q, None if rows is None else rows.data_ptr(), out,
                  _stream(device))
    if rc != SGMV_OK:
        _raise(rc)
    return output_tensor


def _mx_bytes(rows: int, hidden: int) -> int:
    """The quantised inputs' part of a workspace (as the library sizes it)."""
    groups = (hidden + 127) // 128
    return -(-rows * 64 * groups // 256) * 256 + -(-rows * 4 * groups // 256) * 256


def mx_lora_linear_workspace_bytes(tokens: int, hidden: int, num_slices: int = 0, rank: int = 0) -> int:
    """Bytes of the workspace sgmv_mx_lora_linear takes."""
    return _bytes_of(lib.sgmv_mx_lora_linear_workspace_bytes, int(tokens), int(hidden), int(num_slices),
                     int(rank))


def mx_grouped_gemm_workspace_bytes(input_rows: int, hidden: int) -> int:
    """Bytes of the workspace sgmv_mx_grouped_gemm takes."""
    return _bytes_of(lib.sgmv_mx_grouped_gemm_workspace_bytes, int(input_rows), int(hidden))


def sgmv_mx_lora_linear(inputs, weight_codes, weight_scales, slices: Sequence[Tuple[object, object, int]],
                        output_tensor, b_seq_start_loc, seq_len_tensor, lora_indices_tensor,
                        batches: int, max_seq_length: int, scaling: float = 1.0, bias=None,
                        add_inputs: bool = False, workspace=None):
    """sgmv_lora_linear with a microscaled 4-bit weight (sgmv_mx_quantize's
    codes (columns, 64 G) and scales (columns, 4 G)): the shared projection
    multiplies the 4-bit values of the inputs, quantised within the call, with
    those of the weight; the adapters read the inputs as they are.  Enqueued on
    the current stream.  `workspace`: a uint8 tensor of
    mx_lora_linear_workspace_bytes(), or None (taken from torch's allocator for
    the call)."""
    if len(slices) > MAX_SLICES:
        raise ValueError(f"at most {MAX_SLICES} slices, got {len(slices)}")
    device = _gpu(output_tensor, "output_tensor")
    start = _meta(b_seq_start_loc, "b_seq_start_loc", device)
    lens = _meta(seq_len_tensor, "seq_len_tensor", device)
    idx = _meta(lora_indices_tensor, "lora_indices_tensor", device)
    if inputs.device != device:
        raise ValueError(f"inputs must be on {device}")
    if start.shape[0] < batches or lens.shape[0] < batches or idx.shape[0] < batches:
        raise ValueError("segment metadata shorter than batches")
    x = _matrix(inputs, "inputs")
    w = _mx_stack(weight_codes, weight_scales, x.cols, "weight", device, 2)
    out = _matrix(output_tensor, "output_tensor")
    bias_ptr = _bias(bias, w.rows, inputs.dtype, device)
    arr = _fused_slices(slices, device)
    need = 0
    if workspace is None:
        need = _mx_bytes(x.rows, x.cols)
        if slices and batches > 0:
            need += len(slices) * (-(-x.rows * -(-arr[0].lora_a.rows // 8) * 32 // 256) * 256)
    keep, ws, ws_bytes = _scratch(device, workspace, need)
    rc = _call_on(device, lib.sgmv_mx_lora_linear, x, w, bias_ptr, arr, len(slices), out,
                  start.data_ptr(), lens.data_ptr(), idx.data_ptr(), int(batches),
                  int(max_seq_length), float(scaling), int(bool(add_inputs)), ws, ws_bytes,
                  _stream(device))
    if rc != SGMV_OK:
        _raise(rc)
    return output_tensor


def sgmv_mx_grouped_gemm(inputs, expert_codes, expert_scales, output_tensor, b_seq_start_loc,
                         seq_len_tensor, expert_indices_tensor, batches: int, max_seq_length: int,
                         row_indices_tensor=None, gated: bool = False, workspace=None):
    """sgmv_grouped_gemm with microscaled 4-bit experts, expert_codes (experts,
    columns, 64 G) and expert_scales (experts, columns, 4 G); the inputs are
    quantised within the call.  Enqueued on the current stream.  `workspace`:
    a uint8 tensor of mx_grouped_gemm_workspace_bytes(), or None (taken from
    torch's allocator for the call)."""
    device = _gpu(output_tensor, "output_tensor")
    start = _meta(b_seq_start_loc, "b_seq_start_loc", device)
    lens = _meta(seq_len_tensor, "seq_len_tensor", device)
    idx = None if expert_indices_tensor is None else \
        _meta(expert_indices_tensor, "expert_indices_tensor", device)
    if start.shape[0] < batches or lens.shape[0] < batches or \
            (idx is not None and idx.shape[0] < batches):
        raise ValueError("segment metadata shorter than batches")
    if inputs.device != device:
        raise ValueError(f"inputs must be on {device}")
    x = _matrix(inputs, "inputs")
    w = _mx_stack(expert_codes, expert_scales, x.cols, "expert", device, 3)
    out = _matrix(output_tensor, "output_tensor")
    rows = _row_indices(row_indices_tensor, out.rows, device)
    need = _mx_bytes(x.rows, x.cols) if workspace is None else 0
    keep, ws, ws_bytes = _scratch(device, workspace, need)
    rc = _call_on(device, lib.sgmv_mx_grouped_gemm, x, w, out,
                  None if rows is None else rows.data_ptr(), start.data_ptr(), lens.data_ptr(),
                  None if idx is None else idx.data_ptr(), int(batches),
                  int(max_seq_length), int(bool(gated)), ws, ws_bytes, _stream(device))
    if rc != SGMV_OK:
        _raise(rc)
    return output_tensor


def abi_version() -> int:
    return lib.sgmv_abi_version()


__all__ = ["sgmv_expand_slice", "sgmv_expand_multi_slice", "bgmv_expand_slice", "sgmv_shrink",
           "shrink_workspace_bytes", "sgmv_shrink_multi_slice_noalloc",
           "sgmv_shrink_multi_slice", "sgmv_fused_shrink_expand", "sgmv_lora_linear", "lora_linear_workspace_bytes",
           "sgmv_grouped_gemm", "sgmv_route", "route_workspace_bytes", "sgmv_combine",
           "mx_row_bytes", "sgmv_mx_quantize", "sgmv_mx_dequantize", "sgmv_mx_lora_linear",
           "mx_lora_linear_workspace_bytes", "sgmv_mx_grouped_gemm",
           "mx_grouped_gemm_workspace_bytes", "abi_version", "SgmvError",
           "lib", "MxStack", "Matrix", "Stack", "SliceDesc", "ShrinkSliceDesc", "FusedSliceDesc",
           "EXPORTED_SYMBOLS", "LIBRARY_PATH"]
