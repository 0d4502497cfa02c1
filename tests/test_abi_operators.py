"""The entry points of the shared projection with adapters, the grouped
products, the routing and the weighted row sum, without a GPU: every
host-checkable violation is rejected before any HIP call, empty calls return
without one.  No compute call is made here."""
import ctypes

import pytest

import segmented_gather_gemm_amd as sg
from segmented_gather_gemm_amd import FusedSliceDesc, Matrix, Stack

F16, BF16, F32 = 0, 1, 2
OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = 0x10000  # never dereferenced: every case below fails (or no-ops) before a launch


def error():
    return sg.lib.sgmv_last_error().decode()


def slice_(K=8, n=64, off=0, L=2, dt=BF16, H=64, a=FAKE, b=FAKE, Lb=None, Kb=None):
    return FusedSliceDesc(Stack(a, dt, L, K, H), Stack(b, dt, Lb or L, n, Kb or K), off)


def lora(x=None, w=None, out=None, slices=None, meta=(FAKE, FAKE, FAKE), batches=2, max_len=5, ws=FAKE,
         ws_bytes=1 << 20, bias=None, n=None):
    x = x or Matrix(FAKE, BF16, 10, 64, 64)
    w = w or Matrix(FAKE, BF16, 128, 64, 64)
    out = out or Matrix(FAKE, BF16, 10, 128, 128)
    slices = [slice_()] if slices is None else slices
    arr = (FusedSliceDesc * max(1, len(slices)))(*slices)
    st = sg.lib.sgmv_lora_linear(x, w, bias, arr, len(slices) if n is None else n, out, *meta, batches,
                                 max_len, 1.0, 0, ws, ws_bytes, None)
    return st, error()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(x=Matrix(FAKE, 9, 10, 64, 64)), INVALID, "dtype"),
    (dict(out=Matrix(FAKE, 9, 10, 128, 128)), INVALID, "dtype"),
    (dict(w=Matrix(FAKE, 9, 128, 64, 64)), INVALID, "dtype"),
    (dict(x=Matrix(FAKE, F32, 10, 64, 64)), UNSUPPORTED, "16-bit"),
    (dict(x=Matrix(FAKE, F16, 10, 64, 64)), UNSUPPORTED, "16-bit"),
    (dict(w=Matrix(FAKE, F32, 128, 64, 64)), UNSUPPORTED, "16-bit"),
    (dict(x=Matrix(FAKE, BF16, 10, 64, 63)), INVALID, "row stride"),
    (dict(x=Matrix(FAKE, BF16, -1, 64, 64)), INVALID, "inputs shape"),
    (dict(x=Matrix(FAKE, BF16, 10, 0, 0)), INVALID, "inputs shape"),
    (dict(out=Matrix(FAKE, BF16, 10, 128, 127)), INVALID, "row stride"),
    (dict(out=Matrix(FAKE, BF16, 9, 128, 128)), INVALID, "rows"),
    (dict(w=Matrix(FAKE, BF16, 127, 64, 64)), INVALID, "weight"),
    (dict(w=Matrix(FAKE, BF16, 128, 63, 64)), INVALID, "weight"),
    (dict(w=Matrix(FAKE, BF16, 128, 64, 60)), INVALID, "weight"),
    (dict(batches=-1), INVALID, "batches"),
    (dict(batches=4001), UNSUPPORTED, "batches"),
    (dict(max_len=-1), INVALID, "max_seq_len"),
    (dict(n=-1), INVALID, "num_slices"),
    (dict(n=9), INVALID, "num_slices"),
    (dict(slices=[slice_(dt=F16)]), UNSUPPORTED, "dtype"),
    (dict(slices=[slice_(dt=7)]), INVALID, "dtype"),
    (dict(slices=[slice_(H=32)]), INVALID, "lora_a"),
    (dict(slices=[slice_(Lb=3)]), INVALID, "lora_b"),
    (dict(slices=[slice_(Kb=16)]), INVALID, "lora_b"),
    (dict(slices=[slice_(off=65)]), INVALID, "window"),
    (dict(slices=[slice_(off=-1)]), INVALID, "window"),
    (dict(slices=[slice_(), slice_(off=32)]), INVALID, "overlap"),
    (dict(slices=[slice_(), slice_(K=16, off=64)]), INVALID, "slice 0"),
    (dict(slices=[slice_(), slice_(L=3, off=64)]), INVALID, "slice 0"),
    (dict(slices=[slice_(K=257)]), UNSUPPORTED, "rank"),
    (dict(x=Matrix(0, BF16, 10, 64, 64)), INVALID, "null"),
    (dict(w=Matrix(0, BF16, 128, 64, 64)), INVALID, "null"),
    (dict(out=Matrix(0, BF16, 10, 128, 128)), INVALID, "null"),
    (dict(slices=[slice_(a=0)]), INVALID, "null"),
    (dict(slices=[slice_(b=0)]), INVALID, "null"),
    (dict(meta=(FAKE, 0, FAKE)), INVALID, "metadata"),
    (dict(ws=None), INVALID, "workspace"),
    (dict(ws=FAKE + 8), INVALID, "workspace"),
    (dict(ws_bytes=10 * 8 * 4), INVALID, "workspace"),  # a slice's rows take whole 256-byte blocks
    (dict(x=Matrix(FAKE, BF16, 1 << 31, 64, 64), out=Matrix(FAKE, BF16, 1 << 31, 128, 128)), UNSUPPORTED, "rows"),
])
def test_lora_linear_rejects(kw, status, frag):
    st, msg = lora(**kw)
    assert st == status and frag in msg, msg


@pytest.mark.parametrize("kw", [dict(x=Matrix(0, BF16, 0, 64, 64), out=Matrix(0, BF16, 0, 128, 128)),
                                dict(w=Matrix(0, BF16, 0, 64, 64), out=Matrix(0, BF16, 10, 0, 0), slices=[])])
def test_lora_linear_empty_calls(kw):
    assert lora(**kw) == (OK, "")


def test_lora_linear_workspace_bytes():
    n = ctypes.c_size_t()
    f = sg.lib.sgmv_lora_linear_workspace_bytes
    assert f(10, 3, 8, ctypes.byref(n)) == OK and n.value == 3 * 512
    assert f(10, 3, 9, ctypes.byref(n)) == OK and n.value == 3 * 768
    assert f(10, 0, 0, ctypes.byref(n)) == OK and n.value == 0
    assert f(-1, 1, 8, ctypes.byref(n)) == INVALID
    assert f(1, 9, 8, ctypes.byref(n)) == INVALID
    assert f(1, 1, 257, ctypes.byref(n)) == UNSUPPORTED
    assert f(1, 1, 8, None) == INVALID
    assert sg.lora_linear_workspace_bytes(10, 3, 8) == 1536


def grouped(x=None, w=None, out=None, rows=None, meta=(FAKE, FAKE, None), batches=3, max_len=5, gated=0):
    x = x or Matrix(FAKE, BF16, 10, 64, 64)
    w = w or Stack(FAKE, BF16, 3, 32, 64)
    out = out or Matrix(FAKE, BF16, 10, 32, 32)
    st = sg.lib.sgmv_grouped_gemm(x, w, out, rows, *meta, batches, max_len, gated, None)
    return st, error()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(x=Matrix(FAKE, 5, 10, 64, 64)), INVALID, "dtype"),
    (dict(w=Stack(FAKE, 5, 3, 32, 64)), INVALID, "dtype"),
    (dict(w=Stack(FAKE, F16, 3, 32, 64)), UNSUPPORTED, "16-bit"),
    (dict(x=Matrix(FAKE, F32, 10, 64, 64)), UNSUPPORTED, "16-bit"),
    (dict(w=Stack(FAKE, BF16, 3, 32, 32)), INVALID, "weights"),
    (dict(w=Stack(FAKE, BF16, 3, 64, 64)), INVALID, "weights"),
    (dict(gated=1), INVALID, "weights"),
    (dict(w=Stack(FAKE, BF16, -1, 32, 64)), INVALID, "weights"),
    (dict(x=Matrix(FAKE, BF16, 9, 64, 64)), INVALID, "row_indices"),
    (dict(batches=-1), INVALID, "batches"),
    (dict(batches=4001), UNSUPPORTED, "batches"),
    (dict(max_len=-2), INVALID, "max_seq_len"),
    (dict(x=Matrix(0, BF16, 10, 64, 64)), INVALID, "null"),
    (dict(w=Stack(0, BF16, 3, 32, 64)), INVALID, "null"),
    (dict(out=Matrix(0, BF16, 10, 32, 32)), INVALID, "null"),
    (dict(meta=(0, FAKE, None)), INVALID, "metadata"),
    (dict(out=Matrix(FAKE, BF16, 10, 32, 31)), INVALID, "row stride"),
])
def test_grouped_gemm_rejects(kw, status, frag):
    st, msg = grouped(**kw)
    assert st == status and frag in msg, msg


@pytest.mark.parametrize("kw", [dict(batches=0), dict(w=Stack(0, BF16, 0, 32, 64)),
                                dict(x=Matrix(0, BF16, 0, 64, 64), out=Matrix(0, BF16, 0, 32, 32)),
                                dict(w=Stack(0, BF16, 3, 0, 64), out=Matrix(0, BF16, 10, 0, 0))])
def test_grouped_gemm_empty_calls(kw):
    assert grouped(**kw) == (OK, "")


def route(x=None, k=2, ptrs=(FAKE,) * 6, ws=None, ws_bytes=0):
    st = sg.lib.sgmv_route(x or Matrix(FAKE, F32, 10, 16, 16), k, 0, *ptrs, ws, ws_bytes, None)
    return st, error()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(x=Matrix(FAKE, 4, 10, 16, 16)), INVALID, "dtype"),
    (dict(x=Matrix(FAKE, F32, 10, 16, 15)), INVALID, "row stride"),
    (dict(k=0), INVALID, "top_k"),
    (dict(k=17), INVALID, "top_k"),
    (dict(x=Matrix(FAKE, F32, -1, 16, 16)), INVALID, "tokens"),
    (dict(x=Matrix(FAKE, F32, 10, 0, 0), k=1), INVALID, "experts"),
    (dict(x=Matrix(FAKE, F32, 10, 1025, 1025)), UNSUPPORTED, "experts"),
    (dict(x=Matrix(FAKE, F32, 10, 64, 64), k=33), UNSUPPORTED, "choices"),
    (dict(x=Matrix(FAKE, F32, 1 << 30, 16, 16), k=2), UNSUPPORTED, "choices"),
    (dict(x=Matrix(0, F32, 10, 16, 16)), INVALID, "null"),
    (dict(ptrs=(FAKE, 0, FAKE, FAKE, FAKE, FAKE)), INVALID, "null"),
    (dict(ptrs=(FAKE, FAKE, FAKE, FAKE, 0, FAKE)), INVALID, "metadata"),
    (dict(x=Matrix(FAKE, F32, 5000, 16, 16)), INVALID, "workspace"),
    (dict(x=Matrix(FAKE, F32, 5000, 16, 16), ws=FAKE, ws_bytes=16), INVALID, "workspace"),
])
def test_route_rejects(kw, status, frag):
    st, msg = route(**kw)
    assert st == status and frag in msg, msg


def test_route_workspace_bytes():
    n = ctypes.c_size_t()
    assert sg.lib.sgmv_route_workspace_bytes(10, 16, 2, ctypes.byref(n)) == OK and n.value == 0
    assert sg.lib.sgmv_route_workspace_bytes(1 << 20, 16, 2, ctypes.byref(n)) == OK
    assert 0 < n.value <= 256 * 16 * 4
    assert sg.lib.sgmv_route_workspace_bytes(10, 16, 17, ctypes.byref(n)) == INVALID
    assert sg.lib.sgmv_route_workspace_bytes(10, 16, 2, None) == INVALID


def combine(rows=None, w=FAKE, slots=FAKE, k=2, out=None):
    st = sg.lib.sgmv_combine(rows or Matrix(FAKE, BF16, 20, 64, 64), w, slots, k,
                             out or Matrix(FAKE, BF16, 10, 64, 64), 0, None)
    return st, error()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(rows=Matrix(FAKE, 6, 20, 64, 64)), INVALID, "dtype"),
    (dict(rows=Matrix(FAKE, BF16, -1, 64, 64)), INVALID, "rows shape"),
    (dict(rows=Matrix(FAKE, BF16, 20, 64, 60)), INVALID, "row stride"),
    (dict(out=Matrix(FAKE, BF16, 10, 63, 64)), INVALID, "columns"),
    (dict(out=Matrix(FAKE, BF16, 10, 64, 63)), INVALID, "row stride"),
    (dict(k=-1), INVALID, "top_k"),
    (dict(w=0), INVALID, "null"),
    (dict(slots=0), INVALID, "null"),
    (dict(rows=Matrix(0, BF16, 20, 64, 64)), INVALID, "null"),
    (dict(out=Matrix(0, BF16, 10, 64, 64)), INVALID, "null"),
])
def test_combine_rejects(kw, status, frag):
    st, msg = combine(**kw)
    assert st == status and frag in msg, msg


def test_combine_empty_calls():
    assert combine(out=Matrix(0, BF16, 0, 64, 64)) == (OK, "")
    assert combine(rows=Matrix(FAKE, BF16, 20, 0, 0), out=Matrix(0, BF16, 10, 0, 0)) == (OK, "")


def test_python_wrappers_reject_host_tensors():
    import torch
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        sg.sgmv_lora_linear(x, x, [], x, i, i, i, 1, 1)
    with pytest.raises(ValueError, match="GPU"):
        sg.sgmv_grouped_gemm(x, x[None], x, i, i, None, 1, 1)
    with pytest.raises(ValueError, match="GPU"):
        sg.sgmv_route(x, x, i, i, i, i, i)
    with pytest.raises(ValueError, match="GPU"):
        sg.sgmv_combine(x, x, i, x)


@pytest.mark.parametrize("rows,status", [(1 << 30, UNSUPPORTED), ((1 << 30) + 5, UNSUPPORTED)])
def test_products_of_more_threads_than_a_launch_holds(rows, status):
    """2^36 results and more in 64 x 64 tiles of 256 threads (hidden 65: no other kernel takes it) are
    refused before the adapters' projection is launched."""
    st, msg = lora(x=Matrix(FAKE, BF16, rows, 65, 65), w=Matrix(FAKE, BF16, 64, 65, 65), out=Matrix(FAKE, BF16, rows, 64, 64),
                   slices=[slice_(H=65)], ws_bytes=1 << 62)
    assert st == status and "threads" in msg
    st = sg.lib.sgmv_grouped_gemm(Matrix(FAKE, BF16, rows, 65, 65), Stack(FAKE, BF16, 2, 64, 65), Matrix(FAKE, BF16, rows, 64, 64),
                                  None, FAKE, FAKE, None, 2, 5, 0, None)
    assert st == status and "threads" in error()
