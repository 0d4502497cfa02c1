"""The entry points of microscaled 4-bit rows without a GPU: every
host-checkable violation is rejected before any HIP call, empty calls return
without one.  No compute call is made here."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import segmented_gather_gemm_amd as sg
from segmented_gather_gemm_amd import FusedSliceDesc, Matrix, MxStack, Stack

F16, BF16, F32 = 0, 1, 2
OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = 0x10000  # never dereferenced: every case below fails (or no-ops) before a launch
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "segmented_gather_gemm_amd", "csrc")


def error():
    return sg.lib.sgmv_last_error().decode()


def mx(rows=10, cols=200, num=1, codes=FAKE, scales=FAKE, cs=128, ss=8):
    return MxStack(codes, scales, num, rows, cols, cs, ss)


def x_(rows=10, cols=200, dt=BF16, stride=None, data=FAKE):
    return Matrix(data, dt, rows, cols, cols if stride is None else stride)


BAD_MX = [
    (dict(cols=199), INVALID, "values"),
    (dict(cols=201), INVALID, "values"),
    (dict(cs=112), INVALID, "strides"),
    (dict(ss=4), INVALID, "strides"),
    (dict(cs=136), INVALID, "aligned"),
    (dict(ss=10), INVALID, "aligned"),
    (dict(codes=FAKE + 8), INVALID, "aligned"),
    (dict(scales=FAKE + 2), INVALID, "aligned"),
    (dict(rows=-1), INVALID, "rows"),
    (dict(num=-1), INVALID, "rows"),
    (dict(codes=0), INVALID, "null"),
    (dict(scales=0), INVALID, "null"),
]


@pytest.mark.parametrize("kw,status,frag", BAD_MX + [
    (dict(rows=9), INVALID, "rows"), (dict(rows=5, num=3), INVALID, "rows"), (dict(rows=1 << 40, num=1 << 40), INVALID, "rows")])
def test_quantize_rejects_outputs(kw, status, frag):
    assert sg.lib.sgmv_mx_quantize(x_(), mx(**kw), None) == status and frag in error()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(dt=5), INVALID, "dtype"), (dict(stride=199), INVALID, "row stride"), (dict(rows=-1), INVALID, "shape"),
    (dict(cols=0), INVALID, "shape"), (dict(data=0), INVALID, "null"), (dict(rows=1 << 30), UNSUPPORTED, "2^28")])
def test_quantize_rejects_inputs(kw, status, frag):
    assert sg.lib.sgmv_mx_quantize(x_(**kw), mx(), None) == status and frag in error()


@pytest.mark.parametrize("kw,status,frag", BAD_MX + [(dict(rows=9), INVALID, "rows"), (dict(rows=1 << 31), UNSUPPORTED, "2^31")])
def test_dequantize_rejects_inputs(kw, status, frag):
    assert sg.lib.sgmv_mx_dequantize(mx(**kw), None, x_(), None) == status and frag in error()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(dt=5), INVALID, "dtype"), (dict(stride=199), INVALID, "row stride"), (dict(data=0), INVALID, "null"),
    (dict(rows=1 << 30), UNSUPPORTED, "2^28")])
def test_dequantize_rejects_outputs(kw, status, frag):
    assert sg.lib.sgmv_mx_dequantize(mx(), FAKE, x_(**kw), None) == status and frag in error()


def test_empty_calls():
    assert sg.lib.sgmv_mx_quantize(x_(rows=0, data=0), mx(rows=0, codes=0, scales=0), None) == OK
    assert sg.lib.sgmv_mx_dequantize(mx(rows=0, codes=0, scales=0), None, x_(rows=0, data=0), None) == OK
    assert linear(x=x_(rows=0), out=Matrix(FAKE, BF16, 0, 64, 64), ws=None)[0] == OK
    assert linear(w=mx(rows=0), out=Matrix(FAKE, BF16, 10, 0, 0), slices=[], ws=None)[0] == OK
    assert experts(batches=0, ws=None)[0] == OK
    assert experts(w=mx(rows=64, num=0), ws=None)[0] == OK


def slice_(K=8, n=64, off=0, L=2, dt=BF16, H=200, a=FAKE, b=FAKE, Lb=None, Kb=None):
    return FusedSliceDesc(Stack(a, dt, L, K, H), Stack(b, dt, Lb or L, n, Kb or K), off)


def linear(x=None, w=None, out=None, slices=None, meta=(FAKE, FAKE, FAKE), batches=2, max_len=5, ws=FAKE, ws_bytes=1 << 20, n=None):
    slices = [slice_()] if slices is None else slices
    arr = (FusedSliceDesc * max(1, len(slices)))(*slices)
    st = sg.lib.sgmv_mx_lora_linear(x or x_(), w or mx(rows=64), None, arr, len(slices) if n is None else n,
                                    out or Matrix(FAKE, BF16, 10, 64, 64), *meta, batches, max_len, 1.0, 0, ws, ws_bytes, None)
    return st, error()


@pytest.mark.parametrize("kw,status,frag", [(dict(w=mx(**{"rows": 64, **k})), s, f) for k, s, f in BAD_MX] + [
    (dict(x=x_(dt=F32)), UNSUPPORTED, "16-bit"),
    (dict(x=x_(dt=7)), INVALID, "dtype"),
    (dict(x=x_(stride=100)), INVALID, "row stride"),
    (dict(x=x_(data=0)), INVALID, "null"),
    (dict(out=Matrix(FAKE, 9, 10, 64, 64)), INVALID, "dtype"),
    (dict(out=Matrix(FAKE, BF16, 9, 64, 64)), INVALID, "rows"),
    (dict(out=Matrix(0, BF16, 10, 64, 64)), INVALID, "null"),
    (dict(w=mx(rows=63)), INVALID, "64 rows"),
    (dict(w=mx(rows=64, num=2)), INVALID, "one matrix"),
    (dict(batches=-1), INVALID, "batches"),
    (dict(batches=4001), UNSUPPORTED, "batches"),
    (dict(max_len=-1), INVALID, "max_seq_len"),
    (dict(n=9), INVALID, "num_slices"),
    (dict(slices=[slice_(dt=F16)]), UNSUPPORTED, "dtype"),
    (dict(slices=[slice_(H=128)]), INVALID, "lora_a"),
    (dict(slices=[slice_(off=1)]), INVALID, "window"),
    (dict(slices=[slice_(K=257)]), UNSUPPORTED, "rank"),
    (dict(slices=[slice_(a=0)]), INVALID, "null"),
    (dict(meta=(0, FAKE, FAKE)), INVALID, "metadata"),
    (dict(ws=None), INVALID, "workspace"),
    (dict(ws=None, slices=[]), INVALID, "workspace"),
    (dict(ws=FAKE + 4), INVALID, "workspace"),
    (dict(ws_bytes=10 * 136 + 10 * 32), INVALID, "workspace"),
])
def test_lora_linear_rejects(kw, status, frag):
    st, msg = linear(**kw)
    assert st == status and frag in msg


def experts(x=None, w=None, out=None, rows=FAKE, meta=(FAKE, FAKE, None), batches=2, max_len=5, gated=0, ws=FAKE, ws_bytes=1 << 20):
    st = sg.lib.sgmv_mx_grouped_gemm(x or x_(), w or mx(rows=64, num=3), out or Matrix(FAKE, BF16, 20, 64, 64), rows, *meta, batches, max_len,
                                     gated, ws, ws_bytes, None)
    return st, error()


@pytest.mark.parametrize("kw,status,frag", [(dict(w=mx(**{"rows": 64, "num": 3, **k})), s, f) for k, s, f in BAD_MX] + [
    (dict(x=x_(dt=F32)), UNSUPPORTED, "16-bit"),
    (dict(x=x_(data=0)), INVALID, "null"),
    (dict(out=Matrix(FAKE, 9, 20, 64, 64)), INVALID, "dtype"),
    (dict(out=Matrix(0, BF16, 20, 64, 64)), INVALID, "null"),
    (dict(w=mx(rows=63, num=3)), INVALID, "64 rows"),
    (dict(gated=1), INVALID, "128 rows"),
    (dict(rows=None), INVALID, "row_indices"),
    (dict(w=mx(rows=64, num=1 << 31)), UNSUPPORTED, "experts"),
    (dict(batches=4001), UNSUPPORTED, "batches"),
    (dict(meta=(FAKE, None, None)), INVALID, "metadata"),
    (dict(ws=None), INVALID, "workspace"),
    (dict(ws_bytes=1500), INVALID, "workspace"),
])
def test_grouped_rejects(kw, status, frag):
    st, msg = experts(**kw)
    assert st == status and frag in msg


def test_workspace_sizes():
    """Codes and scales of the inputs, each in whole 256-byte blocks, then the adapters' rows."""
    assert sg.mx_row_bytes(1) == (64, 4) and sg.mx_row_bytes(128) == (64, 4) and sg.mx_row_bytes(129) == (128, 8)
    assert sg.mx_grouped_gemm_workspace_bytes(10, 200) == 1280 + 256
    assert sg.mx_grouped_gemm_workspace_bytes(0, 200) == 0
    assert sg.mx_lora_linear_workspace_bytes(10, 200) == 1536
    assert sg.mx_lora_linear_workspace_bytes(10, 200, 2, 8) == 1536 + sg.lora_linear_workspace_bytes(10, 2, 8)
    # what the wrappers take when no workspace is given
    for rows, hidden, slices, rank in ((1, 1, 0, 0), (10, 200, 2, 8), (77, 4104, 3, 13), (0, 64, 1, 16), (2501, 2056, 1, 24)):
        assert sg._mx_bytes(rows, hidden) == sg.mx_grouped_gemm_workspace_bytes(rows, hidden)
        assert sg.mx_lora_linear_workspace_bytes(rows, hidden, slices, rank) - sg._mx_bytes(rows, hidden) == \
            slices * (-(-rows * -(-rank // 8) * 32 // 256) * 256) == sg.lora_linear_workspace_bytes(rows, slices, rank)
    for bad in ((-1, 8), (1, 0)):
        with pytest.raises(ValueError):
            sg.mx_grouped_gemm_workspace_bytes(*bad)
    with pytest.raises(NotImplementedError):
        sg.mx_grouped_gemm_workspace_bytes(1 << 30, 129)
    with pytest.raises(NotImplementedError):
        sg.mx_lora_linear_workspace_bytes(10, 200, 1, 257)
    with pytest.raises(ValueError):
        sg.mx_lora_linear_workspace_bytes(10, 200, 9, 8)
    assert sg.lib.sgmv_mx_grouped_gemm_workspace_bytes(1, 1, None) == INVALID
    assert sg.lib.sgmv_mx_lora_linear_workspace_bytes(1, 1, 0, 0, None) == INVALID


def test_wrappers_check_their_tensors():
    cpu = torch.zeros(4, 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        sg.sgmv_mx_quantize(torch.zeros(4, 128), cpu, cpu)
    with pytest.raises(ValueError, match="GPU"):
        sg.sgmv_mx_dequantize(cpu, cpu, torch.zeros(4, 128))
    dev = cpu.device
    good = dict(hidden=200, what="weight", device=dev, dims=2)
    codes, scales = torch.zeros(6, 128, dtype=torch.uint8), torch.zeros(6, 8, dtype=torch.uint8)
    q = sg._mx_stack(codes, scales, **good)
    assert (q.num, q.rows, q.cols, q.code_stride, q.scale_stride) == (1, 6, 200, 128, 8)
    one = sg._mx_stack(codes[:1].expand(1, 128), scales[:1], **good)
    assert (one.rows, one.code_stride, one.scale_stride) == (1, 128, 8)
    for bad in ((codes[:, :64], scales), (codes, scales[:, :4]), (codes.int(), scales), (codes[:5], scales), (codes[None], scales[None]),
                (codes.t().contiguous().t(), scales)):
        with pytest.raises(ValueError):
            sg._mx_stack(*bad, **good)
    three = sg._mx_stack(codes.view(2, 3, 128), scales.view(2, 3, 8), 200, "expert", dev, 3)
    assert (three.num, three.rows, three.code_stride, three.scale_stride) == (2, 3, 128, 8)
    with pytest.raises(ValueError, match="contiguous"):
        sg._mx_stack(codes.view(3, 2, 128).transpose(0, 1), scales.view(3, 2, 8).transpose(0, 1), 200, "expert", dev, 3)


DIVIDE = r"""
#include <stdio.h>
#include <stdlib.h>
#include "sgmv_limits.h"
using namespace sgmv::limits;
int main() {
  uint32_t ds[] = {1, 2, 3, 5, 7, 8, 32, 33, 100, 127, 128, 641, 1000, 65535, 65536, 65537, 6700417, 16777216, 1073741823, 1073741824,
                   2147483646, 2147483647};
  uint64_t r = 88172645463325252ull, bad = 0;
  for (uint32_t d : ds) {
    const Divisor m = divisor(d);
    for (int i = 0; i < 200000; ++i) {
      r ^= r << 13; r ^= r >> 7; r ^= r << 17;
      uint32_t n = i < 64 ? (uint32_t)i : i < 128 ? 2147483647u - (i - 64) : i < 50000 ? (uint32_t)((r >> 33) / d * d) - (i & 1) : (uint32_t)(r >> 33);
      n &= 2147483647u;
      if (divide(n, m) != n / d) ++bad;
    }
  }
  printf("%llu %lld\n", (unsigned long long)bad, (long long)(mx_groups(1) * 100 + mx_groups(128) * 10 + mx_groups(129)));
}
"""


def test_division_by_an_invariant(tmp_path):
    src = tmp_path / "divide.cpp"
    src.write_text(DIVIDE)
    exe = str(tmp_path / "divide")
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{CSRC}", str(src), "-o", exe], check=True)
    assert subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split() == ["0", "112"]


def test_the_definition_itself():
    """mx_util on values worked out by hand: a block of 6, 5 (a tie, to 4), 7 (cut to 6), 0.25 (a tie,
    to 0), -0.0, and its scale of 1 (7 lies in [4, 8))."""
    import mx_util as M
    x = torch.zeros(1, 40)
    x[0, :8] = torch.tensor([6.0, 5.0, 7.0, 0.25, -0.0, -0.75, 1.75, 2.5])
    x[0, 32] = 12.0
    codes, scales = M.quantize(x)
    assert scales.tolist() == [[127, 128, 0, 0]]
    assert codes[0, :4].tolist() == [7 | 6 << 4, 7 | 0 << 4, 8 | 10 << 4, 4 | 4 << 4] and codes[0, 16] == 7
    assert M.values(codes, scales, 40)[0, [0, 1, 2, 3, 5, 6, 7, 32]].tolist() == [6, 4, 6, 0, -1, 2, 2, 12]
    nan = torch.full((1, 32), float("nan"))
    codes, scales = M.quantize(nan)
    assert scales[0, 0] == 255 and not codes.any() and bool(M.values(codes, scales, 32).isnan().all())
    assert ctypes.sizeof(MxStack) == 56 and np.array_equal(M.GRID[:3], [0, .5, 1])


STACK = r"""
#include <stdio.h>
#include "sgmv_limits.h"
int main() {
  const int32_t e = 1 << 30, n = 1 << 29;  // as the kernels hold them
  printf("%lld %lld\n", (long long)sgmv::limits::stack_row(e, 2 * (int64_t)1, 1), (long long)sgmv::limits::stack_row(7, 2 * (int64_t)n, n));
}
"""


def test_rows_of_a_stack_past_32_bits(tmp_path):
    """A stack of 2^30 experts of two rows (the gate's and the other factor's) is 137 GB of codes: its last rows' numbers."""
    src, exe = tmp_path / "stack.cpp", str(tmp_path / "stack")
    src.write_text(STACK)
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{CSRC}", str(src), "-o", exe], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in out] == [2 ** 31 + 1, 7 * 2 ** 30 + 2 ** 29]
