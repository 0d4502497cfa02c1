"""Each form of the kernels on microscaled weights at sizes that take it: the
256 x 256 tiles, the 128 x 128 tiles with adapters, the few-row kernel with 64
rows and with long contractions, and the generic kernel, against the
definitions in 64 bits (mx_util).  KERNELS names the form that every case
takes; test_mx_kernel_choice.py holds the library's choice against it."""
import pytest
import torch

import matmul_util as U
import mx_choice as C
import mx_util as M
import test_gpu_mx as X
from test_gpu_matmul import scaled_bound

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
FAR = 1 << 22  # elements from row to row of results that 256 rows' 32-bit offsets do not reach

# (kernel, T, H, N, results' row stride or 0)
DENSE = [("large_dense", 3100, 2056, 4100, 0), ("large_dense", 3000, 2312, 4104, 0), ("medium_dense", 2900, 1032, 4104, 0),
         ("few_dense64", 33, 136, 8200, 0), ("few_dense64", 64, 264, 8203, 0), ("few_dense64", 50, 8192, 8200, 0), ("few_dense64", 40, 8200, 8200, 0),
         ("few_dense16", 1, 6200, 72, 0), ("few_dense16", 1, 14336, 67, 0), ("few_dense16", 16, 8192, 200, 0), ("few_dense16", 9, 8200, 4101, 0),
         ("few_dense16", 16, 20000, 40, 0), ("few_dense32", 17, 6200, 72, 0), ("few_dense32", 32, 8192, 67, 0), ("few_dense32", 29, 8200, 4104, 0),
         ("few_dense32", 32, 14336, 200, 0), ("few_dense32", 20, 20000, 40, 0), ("generic", 70, 392, 72, FAR), ("generic", 3, 136, 67, FAR)]
# (kernel, T, H, widths, rank)
ADAPTED = [("medium_adapted", T, H, [136, 24], K) for T in (257, 390) for H, K in ((2056, 8), (2056, 16), (2312, 24), (2056, 32), (2056, 64), (4104, 128))] + \
          [("large_adapted", 300, 264, [136, 24], 24), ("large_adapted", 600, 520, [520], 64)] + \
          [("few_adapted64", T, 264, [4104], 8) for T in (100, 130)] + [("few_adapted64", 64, 8200, [8200, 24], 8)] + \
          [("few_adapted16", T, H, [136, 72], K) for T in (1, 5, 16) for H, K in ((6200, 8), (8200, 16), (14336, 64))] + \
          [("few_adapted32", 32, H, [136, 67], K) for H, K in ((8192, 8), (14336, 16))]
# (kernel, segments' lengths, H, N, gated, gathered input rows or 0, results' row stride or 0)
GROUPED = [("large_grouped", [700, 0, 1, 1300, 997], 2312, 4100, False, 0, 0), ("large_grouped", [700, 0, 1, 1300, 997], 2312, 4104, False, 500, 0),
           ("large_gated", [700, 0, 1, 1300, 997], 2312, 2100, True, 0, 0), ("large_gated", [1000, 385, 0, 1300, 313], 2312, 2104, True, 500, 0),
           ("medium_grouped", [400, 1, 129], 1032, 264, False, 50, 0), ("medium_gated", [400, 1, 129], 1032, 264, True, 50, 0),
           ("few_grouped16", [2, 1, 3], 8192, 200, False, 9, 0), ("few_grouped16", [1, 1], 6200, 67, False, 0, 0),
           ("few_gated16", [2, 1, 3], 8192, 200, True, 9, 0), ("few_gated16", [1, 1], 6200, 67, True, 0, 0),
           ("generic", [20, 0, 47], 392, 72, False, 9, FAR), ("generic_gated", [20, 0, 47], 392, 72, True, 9, FAR), ("generic_gated", [1, 2], 136, 67, True, 0, FAR)]
# Tiles of 128 x 128 with adapters whatever the ranks, types and segments: T, H, columns.
MEDIUM = [(300, 2056, 200), (513, 2056, 320)]
# (kernel, T, H) of projected values and of scales at their types' ends.
SCALED = [("medium_adapted", 300, 2056), ("large_adapted", 300, 264), ("few_adapted32", 60, 264), ("few_adapted16", 2, 264)]
ENDS = [("few_dense16", 5), ("few_dense32", 20), ("medium_dense", 300)]


def calls():
    """(kernel, the call as mx_choice takes it) of every case."""
    out = [(k, C.linear(T, H, [N], out_stride=s)) for k, T, H, N, s in DENSE]
    out += [(k, C.linear(T, H, w, K, 3, 3)) for k, T, H, w, K in ADAPTED]
    out += [(k, C.grouped(sum(lens) + 2, H, N, len(lens), gated, X_, out_stride=s)) for k, lens, H, N, gated, X_, s in GROUPED]
    out += [("medium_adapted", C.linear(T, H, [N], K, L, B)) for T, H, N in MEDIUM for K in (8, 24, 64) for L in (1, 24) for B in (1, T)]
    out += [(k, C.linear(T, H, [136, 64], 24, 3, 3)) for k, T, H in SCALED]
    return out + [(k, C.linear(T, 264, [96])) for k, T in ENDS]


def weights(gen, rows, hidden, low=118, high=122):
    G = M.groups(hidden)
    codes = torch.randint(0, 256, (*rows, 64 * G), dtype=torch.uint8, generator=gen)
    scales = torch.randint(low, high, (*rows, 4 * G), dtype=torch.uint8, generator=gen)
    past = torch.arange(128 * G) >= hidden                        # what lies past the row's end holds codes 0
    mask = (~past).view(-1, 2).to(torch.uint8)
    codes &= mask[:, 0] * 15 + mask[:, 1] * 240
    return codes.cuda(), scales.cuda()


def results(rows, cols, stride, dtype):
    full = torch.full((rows, stride or cols + 3), 7.0, dtype=dtype, device="cuda")
    return full, full[:, :cols]


def product(xr, wv):
    """(result, error) of rounded rows with weights in 64 bits, on the device."""
    xr, wv = xr.cuda(), wv.cuda()
    return xr @ wv.t(), U.sum_error(xr.shape[1]) * (xr.abs() @ wv.abs().t())


def values(codes, scales, hidden):
    return M.values(codes.cpu().numpy(), scales.cpu().numpy(), hidden)


def within(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} values off, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("kernel,T,H,N,stride", DENSE)
def test_dense(kernel, T, H, N, stride, dtype, out):
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(T + N)
    x = X.normal(gen, T, H, dtype=dtype).cuda()
    codes, scales = weights(gen, (N,), H)
    full, o = results(T, N, stride, out)
    print(f"{kernel} T={T} H={H} N={N} {dtype}->{out}", flush=True)
    none = torch.zeros(1, dtype=torch.int64, device="cuda")
    sg.sgmv_mx_lora_linear(x, codes, scales, [], o, none, none, none, 0, 0)
    torch.cuda.synchronize()
    y, err = product(M.rounded(x), values(codes, scales, H))
    within(o, y, U.rounded(y, err, out), kernel)
    assert bool((full[:, N:] == 7.0).all())


def moved(t, by):
    """The same values, contiguous, `by` elements behind a 16-byte block."""
    if by == 0:
        return t
    flat = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)[by:]
    flat.copy_(t.reshape(-1))
    return flat.view(t.shape)


def adapted(T, H, widths, K, L=3, lens=None, idx=None, start=None, dtype=BF16, out=None, bias=False, add=False, scale=0.5, seed=0, zero=False,
            spoil=None, offset=0, behind=(0, 0)):
    """`zero`: weights of zeros, so that the adapters' share stands alone; `offset`: elements by which the inputs' rows start
    behind a 16-byte block, `behind`: the stacks of lora_A and of lora_B."""
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(seed)
    N, out = sum(widths), out or dtype
    if lens is None:
        third = T // 3
        lens, idx = [third, third, T - 2 * third], [1, -1, 0]
    start = X.starts(lens) if start is None else start
    x = X.normal(gen, T, H + offset, dtype=dtype).cuda()[:, offset:]
    codes, scales = weights(gen, (N,), H)
    if zero:
        codes.zero_()
    b = X.normal(gen, N, dtype=dtype).cuda() if bias else None
    slices, at = [], 0
    for n in widths:
        la, lb = X.normal(gen, L, K, H, sigma=H ** -0.5, dtype=dtype).cuda(), X.normal(gen, L, n, K, dtype=dtype).cuda()
        slices.append((moved(la, behind[0]), moved(lb, behind[1]), at))
        at += n
    if spoil:
        spoil(slices)
    full, o = results(T, N, 0, out)
    o.copy_(torch.randn(T, N, generator=gen).to(out))
    o0 = o.clone()
    print(f"adapted T={T} H={H} widths={widths} K={K} L={L} segments={len(lens)} {dtype}->{out}", flush=True)
    sg.sgmv_mx_lora_linear(x, codes, scales, slices, o, X.i64(start), X.i64(lens), X.i64(idx), len(lens), max(lens), scaling=scale, bias=b,
                           add_inputs=add)
    torch.cuda.synchronize()
    assert bool((full[:, N:] == 7.0).all())
    if spoil:
        return o, lens, start, idx
    if zero:
        want, bound = scaled_bound(x, torch.zeros(N, H), slices, start, lens, idx, scale, 2.0 ** -22)
    else:
        want, bound = M.lora_linear(x, values(codes, scales, H), b, slices, start, lens, idx, scale, o0, add, out)
    U.assert_within(o, want, bound)


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F32), (BF16, F32)])
@pytest.mark.parametrize("kernel,T,H,widths,K", ADAPTED)
def test_adapted(kernel, T, H, widths, K, dtype, out):
    lens = [T // 3, T // 3, T - 2 * (T // 3)] if T > 2 else [T]
    adapted(T, H, widths, K, lens=lens, idx=[1, -1, 0][-len(lens):], dtype=dtype, out=out, seed=T + K)


@pytest.mark.parametrize("T,H,N", MEDIUM)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("out", [BF16, F16, F32])
@pytest.mark.parametrize("add", [False, True])
def test_medium_types(T, H, N, dtype, out, add):
    adapted(T, H, [N - 72, 72], 24, dtype=dtype, out=out, bias=True, add=add)


@pytest.mark.parametrize("T,H,N", MEDIUM)
@pytest.mark.parametrize("K", [8, 16, 24, 64])
@pytest.mark.parametrize("dtype,out", [(BF16, F32), (F16, F16)])
def test_medium_many_adapters(T, H, N, K, dtype, out):
    gen = torch.Generator().manual_seed(T)
    adapted(T, H, [N], K, L=24, lens=[1] * T, idx=torch.randint(-1, 24, (T,), generator=gen).tolist(), dtype=dtype, out=out, seed=K)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_medium_segment_layouts(dtype):
    T = 300
    adapted(T, 2056, [200], 16, lens=[5, 0, 0, 3, 1, 2, 3, 0, -2, 140], idx=[1, 0, 1, 2, -1, 1, 1, 7, 1, 0],
            start=[T - 5, 5, 20, 0, 4, T - 1, -1, 30, 30, 100], dtype=dtype)


@pytest.mark.parametrize("kernel,T,H", SCALED)
@pytest.mark.parametrize("scale", [2.0 ** e for e in (-40, -20, -8, 14, 20, 40)])
def test_projected_values_of_every_size(kernel, T, H, scale):
    """float16 adapters whose projected values lie far outside the type's range keep 22 bits of the largest of a row
    and slice; weights of zeros."""
    adapted(T, H, [136, 64], 24, dtype=F16, out=F32, scale=scale, zero=True,
            lens=[T // 2, T - T // 2], idx=[1, 0])


@pytest.mark.parametrize("T,H,N", MEDIUM)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_medium_adapters_that_are_not_finite(T, H, N, dtype):
    """An infinity and a NaN in two adapters' weights, each in one slice, reach the rows and columns they belong to."""
    args = dict(widths=[N - 80, 80], K=16, lens=[T // 3, T // 3, T - 2 * (T // 3)], idx=[0, 2, 1], dtype=dtype, out=F32, seed=T)

    def spoil(slices):
        slices[0][1][2, 5, 3] = float("inf")
        slices[1][1][1, 0, 7] = float("nan")
    clean = adapted(T, H, **args, spoil=lambda slices: None)[0]
    o, lens, start, idx = adapted(T, H, **args, spoil=spoil)
    odd = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    odd[start[1]:start[2], 5] = True
    odd[start[2]:, N - 80] = True
    assert torch.equal(o[~odd], clean[~odd]) and bool((~o[odd].isfinite()).all())


@pytest.mark.parametrize("T", [1, 20, 300])
@pytest.mark.parametrize("H", [264, 263])
@pytest.mark.parametrize("offset,behind", [(1, (0, 0)), (0, (1, 0)), (0, (0, 1)), (3, (5, 7))])
def test_operands_that_start_between_blocks(T, H, offset, behind):
    adapted(T, H, [72], 16, lens=[T], idx=[2], offset=offset, behind=behind)


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("kernel,lens,H,N,gated,gathered,stride", GROUPED)
def test_grouped(kernel, lens, H, N, gated, gathered, stride, dtype, out):
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(sum(lens) + H)
    R, E = sum(lens) + 2, len(lens)
    x = X.normal(gen, gathered or R, H, dtype=dtype).cuda()
    rows = torch.randint(-1, gathered + 1, (R,), generator=gen) if gathered else None
    codes, scales = weights(gen, (E, 2 * N if gated else N), H, 116, 119)
    full, o = results(R, N, stride, out)
    print(f"{kernel} lens={lens} H={H} N={N} gathered={gathered} {dtype}->{out}", flush=True)
    start = X.starts(lens)
    sg.sgmv_mx_grouped_gemm(x, codes, scales, o, X.i64(start), X.i64(lens), None, E, max(lens),
                            row_indices_tensor=None if rows is None else rows.cuda(), gated=gated)
    torch.cuda.synchronize()
    xr = M.rounded(x)
    for e, (st, n) in enumerate(zip(start, lens)):
        src = torch.arange(st, st + n) if rows is None else rows[st:st + n]
        ok = (src >= 0) & (src < x.shape[0])
        xs = torch.zeros(n, H, dtype=torch.float64)
        xs[ok] = xr[src[ok]]
        y, err = product(xs, values(codes[e], scales[e], H))
        if gated:
            # |silu'| < 1.1; the exponential's own error, as in matmul_util
            g, u, eg, eu = y[:, :N], y[:, N:], err[:, :N], err[:, N:]
            s = g / (1 + torch.exp(-g))
            es = 1.1 * eg + s.abs() * (2.0 ** -20 + g.abs() * 2.0 ** -23)
            y, err = s * u, es * (u.abs() + eu) + s.abs() * eu
        within(o[st:st + n], y, U.rounded(y, err, out), f"{kernel} expert {e}")
    assert bool((full[:, N:] == 7.0).all()) and bool((full[R - 2:] == 7.0).all())


@pytest.mark.parametrize("kernel,T", ENDS)
@pytest.mark.parametrize("low,high", [(225, 229), (16, 20)])
def test_scales_at_both_ends(kernel, T, low, high):
    """Inputs of the smallest scales with weights of large ones, and the reverse: sums near one."""
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(T)
    x = torch.randn(T, 264, generator=gen) * 2.0 ** (122 - high)
    x[1] *= 2.0 ** (-20 if low > 127 else 24)                     # subnormals, of scale byte 0, or values near the largest
    x = x.to(BF16).cuda()
    codes, scales = weights(gen, (96,), 264, low, high)
    full, o = results(T, 96, 0, F32)
    none = torch.zeros(1, dtype=torch.int64, device="cuda")
    print(f"{kernel} T={T} scales {low}..{high}", flush=True)
    sg.sgmv_mx_lora_linear(x, codes, scales, [], o, none, none, none, 0, 0)
    torch.cuda.synchronize()
    y, err = product(M.rounded(x), values(codes, scales, 264))
    within(o, y, U.rounded(y, err, F32), kernel)
