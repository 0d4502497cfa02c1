"""The shared projection with adapters and the grouped products on the GPU,
against their plain 64-bit forms (matmul_util)."""
import numpy as np
import pytest
import torch

import matmul_util as U

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def normal(gen, *shape, sigma=1.0, dtype=BF16):
    return (torch.randn(*shape, generator=gen) * sigma).to(dtype).cuda()


def i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


def guarded(T, N, dtype, pad=0, gen=None):
    """An output of N columns inside wider rows, all set to a known value."""
    full = torch.full((T, N + pad), 7.0, dtype=dtype, device="cuda")
    if gen is not None:
        full[:, :N] = torch.randn(T, N, generator=gen).to(dtype).cuda()
    return full, full[:, :N]


def lora_case(T, H, widths, K, L, lens, idx, dtype=BF16, out=None, bias=False, add=False, scale=0.5,
              start=None, seed=0, pad_x=0, pad_out=0, gaps=()):
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(seed)
    N = sum(widths) + sum(gaps)
    out = out or dtype
    x = normal(gen, T, H + pad_x, dtype=dtype)[:, :H]
    w = normal(gen, N, H, sigma=H ** -0.5, dtype=dtype)
    b = normal(gen, N, dtype=dtype) if bias else None
    slices, at = [], 0
    for i, n in enumerate(widths):
        slices.append((normal(gen, L, K, H, sigma=H ** -0.5, dtype=dtype),
                       normal(gen, L, n, K, sigma=0.3, dtype=dtype), at))
        at += n + (gaps[i] if i < len(gaps) else 0)
    if start is None:
        start = np.concatenate([[0], np.cumsum(lens)[:-1]]).astype(int).tolist() if lens else []
    full, o = guarded(T, N, out, pad_out, gen)
    o0 = o.clone()
    print(f"lora_linear T={T} H={H} N={N} K={K} L={L} segments={len(lens)} {dtype}->{out}", flush=True)
    sg.sgmv_lora_linear(x, w, slices, o, i64(start), i64(lens), i64(idx), len(lens),
                        max(lens, default=0), scaling=scale, bias=b, add_inputs=add)
    torch.cuda.synchronize()
    want, bound = U.lora_linear(x, w, b, slices, start, lens, idx, scale, o0, add, out)
    U.assert_within(o, want, bound)
    assert pad_out == 0 or bool((full[:, N:] == 7.0).all())


# Sizes around the tiles' edges (16, 64, 128 and 256 rows and columns, 64-wide steps), one token
# to several tiles.
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 65, 127, 130, 257, 520])
def test_lora_linear_rows(T):
    half = max(1, T // 2)
    lens = [half, T - half] if T > 1 else [1]
    lora_case(T, 256, [320], 16, 3, lens, [2, -1][:len(lens)] if T % 2 else [1, 2][:len(lens)], seed=T)


@pytest.mark.parametrize("H", [8, 24, 32, 64, 72, 136, 200, 512, 1032])
@pytest.mark.parametrize("T", [5, 150])
def test_lora_linear_hidden(T, H):
    lora_case(T, H, [128], 8, 2, [T], [1], dtype=F16, seed=H)


@pytest.mark.parametrize("widths", [[8], [16], [24], [72], [128, 64, 64], [264], [520], [40, 8, 136]])
@pytest.mark.parametrize("T", [3, 140, 300])
def test_lora_linear_widths(T, widths):
    lora_case(T, 192, widths, 16, 4, [T - 2, 2], [3, 0], bias=True, seed=sum(widths))


@pytest.mark.parametrize("K", [1, 8, 13, 16, 24, 32, 64, 100, 128, 256])
@pytest.mark.parametrize("T", [4, 200])
def test_lora_linear_ranks(T, K):
    lora_case(T, 320, [192], K, 3, [T // 2, T // 2], [0, 2], seed=K)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("out", [BF16, F16, F32])
@pytest.mark.parametrize("T,add", [(7, False), (7, True), (190, False), (190, True), (400, True)])
def test_lora_linear_types(dtype, out, T, add):
    lora_case(T, 264, [136, 200], 24, 3, [T - 3, 3], [1, 2], dtype=dtype, out=out, bias=True, add=add)


@pytest.mark.parametrize("T,H,N,pad_x,pad_out", [(9, 130, 67, 3, 5), (150, 130, 67, 3, 5), (9, 128, 66, 0, 1),
                                                 (300, 66, 131, 8, 0), (70, 7, 1, 1, 0), (1, 1, 1, 0, 0)])
def test_lora_linear_odd_sizes_and_strides(T, H, N, pad_x, pad_out):
    lora_case(T, H, [N], 5, 2, [T], [1], pad_x=pad_x, pad_out=pad_out, bias=True)


@pytest.mark.parametrize("T", [40, 64, 300, 513])
def test_lora_linear_many_adapters(T):
    """One token a segment, many adapters inside every tile, some rows without one."""
    rng = np.random.default_rng(T)
    lora_case(T, 256, [256, 64], 16, 24, [1] * T, rng.integers(-1, 24, T).tolist(), seed=T)


@pytest.mark.parametrize("T", [50, 300])
def test_lora_linear_segment_layouts(T):
    """Unsorted starts, gaps, empty segments, and segments that break a precondition: those get the
    shared projection alone."""
    start = [T - 10, 5, 20, 0, 12, T - 1, -1, 30, 30]
    lens = [10, 4, 0, 3, 6, 2, 3, 5, -2]
    idx = [1, 0, 1, 2, -1, 1, 1, 7, 1]
    lora_case(T, 128, [192], 16, 3, lens, idx, start=start)


@pytest.mark.parametrize("T", [6, 210])
def test_lora_linear_without_adapters(T):
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(T)
    x, w = normal(gen, T, 256), normal(gen, 192, 256, sigma=1 / 16)
    o = torch.empty(T, 192, dtype=F32, device="cuda")
    none = i64([])
    sg.sgmv_lora_linear(x, w, [], o, none, none, none, 0, 0)
    want, bound = U.lora_linear(x, w, None, [], [], [], [], 1.0, o, False, F32)
    U.assert_within(o, want, bound)


@pytest.mark.parametrize("T", [20, 280])
def test_lora_linear_windows_with_gaps(T):
    """Columns between and after the slices' windows get the shared projection alone."""
    lora_case(T, 136, [40, 24], 8, 2, [T], [1], gaps=(72, 104), seed=T)


@pytest.mark.parametrize("T,K,widths,gaps", [(130, 8, [40, 24], (500, 400)), (300, 40, [16], (1000,)),
                                             (3900, 16, [40, 24], (2000, 2032)), (3900, 80, [64], (4032,))])
def test_lora_linear_windows_that_leave_tiles_without_a_slice(T, K, widths, gaps):
    """Whole tiles of columns (128 and 256 wide) that no slice covers, under rows with adapters, after a
    call whose weights are not finite in every tile."""
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(T + K)
    N = sum(widths) + sum(gaps)
    lb = torch.full((2, N, 8), float("nan"), dtype=BF16, device="cuda")
    o = torch.zeros(T, N, dtype=BF16, device="cuda")
    sg.sgmv_lora_linear(normal(gen, T, 64), normal(gen, N, 64), [(normal(gen, 2, 8, 64), lb, 0)], o, i64([0]), i64([T]),
                        i64([1]), 1, T)
    lora_case(T, 136, widths, K, 3, [T // 2, 5, T // 3], [2, -1, 0], gaps=gaps, seed=T + K)


@pytest.mark.parametrize("T", [12, 260])
def test_lora_linear_nan_rows_stay_where_they_are(T):
    """NaN and infinities of one row reach that row alone; rows of the workspace that no segment
    wrote are never used."""
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(1)
    H, N, K, L = 200, 144, 16, 2
    x, w = normal(gen, T, H), normal(gen, N, H, sigma=H ** -0.5)
    la, lb = normal(gen, L, K, H, sigma=H ** -0.5), normal(gen, L, N, K)
    bad = [3, T - 1]
    x[3, 5], x[T - 1, H - 1] = float("nan"), float("inf")
    ws = torch.full((sg.lora_linear_workspace_bytes(T, 1, K),), 255, dtype=torch.uint8, device="cuda")
    o = torch.zeros(T, N, dtype=BF16, device="cuda")
    start, lens, idx = [0, 6], [5, T - 8], [1, -1]
    sg.sgmv_lora_linear(x, w, [(la, lb, 0)], o, i64(start), i64(lens), i64(idx), 2, T, workspace=ws)
    keep = [t for t in range(T) if t not in bad]
    want, bound = U.lora_linear(x, w, None, [(la, lb, 0)], start, lens, idx, 1.0, o, False, BF16)
    U.assert_within(o[keep], want[keep], bound[keep])
    assert not torch.isfinite(o[bad].float()).any()


@pytest.mark.parametrize("T", [12, 100, 260])
@pytest.mark.parametrize("K", [8, 40])
def test_lora_linear_nan_adapters_reach_their_own_rows_alone(T, K):
    """An adapter whose weights hold NaN and infinities, between rows of other requests."""
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(2)
    H, N, L = 136, 152, 3
    x, w = normal(gen, T, H), normal(gen, N, H, sigma=H ** -0.5)
    la, lb = normal(gen, L, K, H, sigma=H ** -0.5), normal(gen, L, N, K)
    la[1, 0, 0], lb[1, :, K - 1] = float("inf"), float("nan")
    idx = [(t * 7) % 4 - 1 for t in range(T)]
    o = torch.zeros(T, N, dtype=BF16, device="cuda")
    sg.sgmv_lora_linear(x, w, [(la, lb, 0)], o, i64(list(range(T))), i64([1] * T), i64(idx), T, 1)
    keep = [t for t in range(T) if idx[t] != 1]
    la, lb = la.clone(), lb.clone()
    la[1], lb[1] = 0, 0
    want, bound = U.lora_linear(x, w, None, [(la, lb, 0)], list(range(T)), [1] * T, idx, 1.0, o, False, BF16)
    U.assert_within(o[keep], want[keep], bound[keep])
    assert torch.isnan(o[[t for t in range(T) if idx[t] == 1]].float()).all()


def grouped_case(lens, H, N, E=None, idx=None, rows=None, X=None, gated=False, dtype=BF16, out=None,
                 start=None, T=None, seed=0, pad_x=0, pad_out=0):
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(seed)
    E = E or len(lens)
    if start is None:
        start = np.concatenate([[0], np.cumsum(lens)[:-1]]).astype(int).tolist()
    T = sum(lens) if T is None else T
    X = T if X is None else X
    x = normal(gen, X, H + pad_x, dtype=dtype)[:, :H]
    w = normal(gen, E, 2 * N if gated else N, H, sigma=2 * H ** -0.5, dtype=dtype)
    full, o = guarded(T, N, out or dtype, pad_out, gen)
    o0 = o.clone()
    print(f"grouped_gemm T={T} H={H} N={N} E={E} gated={gated} {dtype}->{o.dtype}", flush=True)
    sg.sgmv_grouped_gemm(x, w, o, i64(start), i64(lens), None if idx is None else i64(idx), len(lens),
                         max(lens), row_indices_tensor=None if rows is None else i64(rows), gated=gated)
    torch.cuda.synchronize()
    want, bound, written = U.grouped(x, w, start, lens, idx, rows, gated, o0)
    U.assert_within(o[written.cuda()], want[written], bound[written])
    assert torch.equal(o[~written.cuda()], o0[~written.cuda()])
    assert pad_out == 0 or bool((full[:, N:] == 7.0).all())


LENS = [[1], [0, 1, 0, 2], [16, 17, 15, 64, 65], [3, 300, 0, 129, 1], [1] * 40, [255, 256, 257],
        [600, 0, 0, 5]]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("lens", LENS)
def test_grouped_rows(lens, gated):
    grouped_case(lens, 192, 160, gated=gated, seed=len(lens))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("H,N", [(8, 8), (64, 24), (72, 136), (200, 40), (328, 264), (1032, 72)])
@pytest.mark.parametrize("lens", [[2, 0, 5], [70, 130, 300]])
def test_grouped_sizes(lens, H, N, gated):
    grouped_case(lens, H, N, gated=gated, dtype=F16, seed=H)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("out", [BF16, F16, F32])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("lens", [[4, 1, 9], [140, 30, 200]])
def test_grouped_types(dtype, out, gated, lens):
    grouped_case(lens, 136, 152, dtype=dtype, out=out, gated=gated)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("lens", [[4, 1, 9], [140, 30, 200], [300, 100, 270]])
def test_grouped_gathered_rows(lens, gated):
    """Rows picked from fewer inputs, repeated and in any order; an index outside the inputs is a row
    of zeros."""
    rng = np.random.default_rng(3)
    T = sum(lens)
    rows = rng.integers(0, 37, T)
    rows[[1, T - 1]] = [-1, 37]
    grouped_case(lens, 264, 136, rows=rows.tolist(), X=37, gated=gated)


@pytest.mark.parametrize("T", [60, 400])
def test_grouped_segment_layouts(T):
    """Unsorted starts, gaps, repeated and missing experts; rows outside the segments stay."""
    grouped_case([10, 0, T // 2, 3, 5, 6, -1], 128, 96, E=3, idx=[2, 1, 2, -1, 0, 3, 1],
                 start=[T - 10, 4, 8, 0, 3, T - 20, 2], T=T)


@pytest.mark.parametrize("H,N,pad_x,pad_out", [(129, 67, 2, 3), (66, 9, 6, 1), (5, 3, 0, 0), (64, 33, 0, 0)])
@pytest.mark.parametrize("gated", [False, True])
def test_grouped_odd_sizes_and_strides(H, N, pad_x, pad_out, gated):
    grouped_case([3, 90, 0, 20], H, N, gated=gated, pad_x=pad_x, pad_out=pad_out)


def test_grouped_many_segments():
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 3, 900)
    grouped_case(lens.tolist(), 64, 32, E=5, idx=rng.integers(-1, 5, 900).tolist())


# Enough tiles for the 256 x 256 kernel (its choice goes by the tile counts), with a last row tile
# of less and of more than half, steps that end inside a block of 64, and columns that are no
# multiple of eight.
@pytest.mark.parametrize("T,H,N,dtype,out", [(4000, 136, 4000, BF16, BF16), (3900, 64, 4090, F16, F32),
                                             (3850, 200, 4001, BF16, F16)])
def test_lora_linear_large_tiles_without_adapters(T, H, N, dtype, out):
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(T)
    x, w = normal(gen, T, H, dtype=dtype), normal(gen, N, H, sigma=H ** -0.5, dtype=dtype)
    b = normal(gen, N, dtype=dtype)
    full, o = guarded(T, N, out, 6, gen)
    o0 = o.clone()
    none = i64([])
    sg.sgmv_lora_linear(x, w, [], o, none, none, none, 0, 0, bias=b, add_inputs=True)
    want, bound = U.lora_linear(x, w, b, [], [], [], [], 1.0, o0, True, out)
    U.assert_within(o, want, bound)
    assert bool((full[:, N:] == 7.0).all())


@pytest.mark.parametrize("K", [8, 16, 32, 64, 104, 256])
def test_lora_linear_large_tiles(K):
    lens = [1, 700, 0, 259, 1024, 300, 17, 1, 1, 1300]
    T = sum(lens) + 300
    lora_case(T, 72, [2048, 1000, 950], K, 4, lens, [0, 1, 2, -1, 3, 2, 0, 1, 3, 2], dtype=F16 if K == 32 else BF16,
              out=F32 if K == 64 else None, bias=True, seed=K)


@pytest.mark.parametrize("K", [8, 16, 24, 40])
def test_lora_linear_large_tiles_of_single_tokens(K):
    T = 3900
    rng = np.random.default_rng(K)
    lora_case(T, 64, [4096], K, 40, [1] * T, rng.integers(-1, 40, T).tolist(), seed=K)


@pytest.mark.parametrize("T,N", [(100, 152), (3900, 4096)])
def test_lora_linear_odd_weights_in_tiles(T, N):
    """Infinities and NaN among one adapter's weights: its rows get what IEEE arithmetic gives, other
    rows nothing of it."""
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(4)
    H, K, L = 72, 16, 3
    x, w = normal(gen, T, H), normal(gen, N, H, sigma=H ** -0.5)
    la, lb = normal(gen, L, K, H, sigma=H ** -0.5), normal(gen, L, N, K)
    lb[1, 5, 3], lb[1, 9, 0], lb[1, 130, 2], lb[1, 130, 7] = float("inf"), float("nan"), float("-inf"), float("inf")
    lens = [T // 3, T // 3, T - 2 * (T // 3)]
    start, idx = [0, lens[0], 2 * lens[0]], [0, 1, 2]
    o = torch.zeros(T, N, dtype=BF16, device="cuda")
    sg.sgmv_lora_linear(x, w, [(la, lb, 0)], o, i64(start), i64(lens), i64(idx), 3, T)
    y = x.double().cpu() @ w.double().cpu().t()
    for st, n, a in zip(start, lens, idx):
        v = x[st:st + n].double().cpu() @ la[a].double().cpu().t()
        y[st:st + n] += (v[:, None, :] * lb[a].double().cpu()[None]).sum(dim=2) if T < 200 else v @ lb[a].double().cpu().t()
    odd = ~torch.isfinite(y)
    got = o.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(y)) and torch.equal(got[odd & ~torch.isnan(y)], y[odd & ~torch.isnan(y)])
    clean = lb.clone()
    clean[1] = torch.where(torch.isfinite(lb[1].float()), lb[1], torch.zeros_like(lb[1]))
    want, bound = U.lora_linear(x, w, None, [(la, clean, 0)], start, lens, idx, 1.0, o, False, BF16)
    U.assert_within(got[~odd], want[~odd], bound[~odd])


@pytest.mark.parametrize("lens,H,N,gated,gather", [([1200, 0, 1100, 1400], 136, 4096, False, False),
                                                   ([300, 1300, 1029, 1190], 72, 2040, True, True),
                                                   ([3841], 64, 4001, False, True)])
def test_grouped_large_tiles(lens, H, N, gated, gather):
    rng = np.random.default_rng(H)
    rows = rng.integers(-1, 500, sum(lens)).tolist() if gather else None
    grouped_case(lens, H, N, rows=rows, X=499 if gather else None, gated=gated, dtype=F16 if gated else BF16,
                 out=F32 if H == 64 else None, pad_out=5)


@pytest.mark.parametrize("gated", [False, True])
def test_grouped_few_rows_and_columns(gated):
    """Too few tiles for the tiled kernels: the contraction is split over the waves."""
    grouped_case([3, 0, 16, 1, 20], 1032, 136, gated=gated)


@pytest.mark.parametrize("T", [70, 300])
def test_lora_linear_columns_not_a_multiple_of_eight(T):
    lora_case(T, 136, [131], 16, 2, [T], [1], bias=True, pad_out=3)


@pytest.mark.parametrize("T", [9, 150, 3900])
def test_lora_linear_slices_without_columns(T):
    """A slice of width 0 (whose weights have no memory) among others, and alone."""
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(T)
    H, N, K, L = 64, 4096 if T > 1000 else 160, 16, 2
    x, w = normal(gen, T, H), normal(gen, N, H, sigma=1 / 8)
    la, lb = normal(gen, L, K, H, sigma=1 / 8), normal(gen, L, N, K)
    none = (la, torch.empty(L, 0, K, dtype=BF16, device="cuda"), 50)
    for slices in ([none, (la, lb, 0)], [none]):
        o = torch.zeros(T, N, dtype=BF16, device="cuda")
        sg.sgmv_lora_linear(x, w, slices, o, i64([0]), i64([T]), i64([1]), 1, T)
        want, bound = U.lora_linear(x, w, None, [s for s in slices if s[1].shape[1]], [0], [T], [1], 1.0, o, False, BF16)
        U.assert_within(o, want, bound)


def ieee_adapters(x, w, slices, start, lens, idx):
    """The 64-bit sum with every product of a projected value and a weight taken by itself, so that
    infinities and NaN come out as IEEE arithmetic gives them."""
    y = x.double().cpu() @ w.double().cpu().t()
    for st, n, a in zip(start, lens, idx):
        for la, lb, off in slices if a >= 0 else ():
            A, B = la[a].double().cpu(), lb[a].double().cpu()
            v = (x[st:st + n].double().cpu()[:, None, :] * A[None]).sum(dim=2)
            y[st:st + n, off:off + B.shape[0]] += (v[:, None, :] * B[None]).sum(dim=2)
    return y


def check_against_ieee(o, x, w, slices, start, lens, idx):
    """Values that are not finite as in ieee_adapters; the others within the bound of the sums with the
    weights that are not finite taken as zeros (they are multiplied by nothing there)."""
    want = ieee_adapters(x, w, slices, start, lens, idx)
    got, odd = o.double().cpu(), ~torch.isfinite(want)
    clean = [(torch.nan_to_num(la, nan=0, posinf=0, neginf=0), torch.nan_to_num(lb, nan=0, posinf=0, neginf=0), off)
             for la, lb, off in slices]
    _, bound = U.lora_linear(x, w, None, clean, start, lens, idx, 1.0, o, False, o.dtype)
    U.assert_within(got[~odd], want[~odd], bound[~odd])
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf = odd & ~torch.isnan(want)
    assert torch.equal(got[inf], want[inf])
    return odd


# Few-row kernels (1 to 64 rows), both tiles, and the generic kernel (rank 13).
ODD_SHAPES = [(1, 16), (5, 16), (16, 40), (27, 8), (50, 16), (64, 72), (5, 13), (100, 13), (100, 16), (300, 40), (3900, 16)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,K", ODD_SHAPES)
def test_lora_linear_odd_weights_as_in_ieee(T, K, dtype):
    """Infinities and NaN among one adapter's lora_B: an infinity times a finite value is an infinity,
    whichever way a kernel splits the value."""
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(T + K)
    H, N, L = 72, 4096 if T > 1000 else 152, 3
    x, w = normal(gen, T, H, dtype=dtype), normal(gen, N, H, sigma=H ** -0.5, dtype=dtype)
    la, lb = normal(gen, L, K, H, sigma=H ** -0.5, dtype=dtype), normal(gen, L, N, K, dtype=dtype)
    inf, nan = float("inf"), float("nan")
    lb[1, 5, 3], lb[1, 9, 0], lb[1, 130, 2], lb[1, 130, 7], lb[1, 17, K - 1] = inf, nan, -inf, inf, -inf
    x[T // 2], la[1, 3] = 1.0, 2.0 ** -3  # a value that one part of the split holds whole, the other is zero
    start, lens, idx = [0, T // 3], [T // 3, T - T // 3], [0, 1]
    o = torch.zeros(T, N, dtype=dtype, device="cuda")
    sg.sgmv_lora_linear(x, w, [(la, lb, 0)], o, i64(start), i64(lens), i64(idx), 2, T)
    odd = check_against_ieee(o, x, w, [(la, lb, 0)], start, lens, idx)
    assert odd[T // 3:, [5, 9, 17, 130]].all() and int(odd.sum()) == 4 * (T - T // 3)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,K", ODD_SHAPES)
def test_lora_linear_odd_projections_stay_in_their_window(T, K, dtype):
    """Projected values that are not finite (from lora_A) in the first of three slices: they reach its
    columns, in the rows that have the adapter, as IEEE arithmetic says (times 0: NaN), and neither the
    other slices' columns nor the gap between them, which lie in the same tile."""
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(T + K)
    H, L = 72, 3
    widths, offs, N = [40, 24, 32], [0, 40, 80], 4096 if T > 1000 else 152
    x, w = normal(gen, T, H, dtype=dtype), normal(gen, N, H, sigma=H ** -0.5, dtype=dtype)
    slices = [(normal(gen, L, K, H, sigma=H ** -0.5, dtype=dtype), normal(gen, L, n, K, dtype=dtype), off)
              for n, off in zip(widths, offs)]
    la, lb, _ = slices[0]
    inf, nan = float("inf"), float("nan")
    la[1, 0, 7], la[2, K - 1, 3] = inf, nan
    x[:, 7] = x[:, 7].abs() + 0.5
    lb[1, 3, 0], lb[1, 11, 0], lb[1, 12, 0] = 0.0, inf, -inf
    lens = [T // 4, T // 4, T // 4, T - 3 * (T // 4)]
    start, idx = [0, lens[0], 2 * lens[0], 3 * lens[0]], [0, 2, -1, 1]
    o = torch.zeros(T, N, dtype=dtype, device="cuda")
    sg.sgmv_lora_linear(x, w, slices, o, i64(start), i64(lens), i64(idx), 4, T)
    odd = check_against_ieee(o, x, w, slices, start, lens, idx)
    rows = list(range(start[1], start[2])) + list(range(start[3], T))
    assert odd[rows, :40].all() and int(odd.sum()) == 40 * len(rows)


def scaled_bound(x, w, slices, start, lens, idx, scale, left):
    """(exact result, error bound) of a float32 result whose values v = scale A x each keep an error of
    `left` of the largest one of their row and slice, whatever its size (down to 2^-65 itself)."""
    x, w = x.double().cpu(), w.double().cpu()
    e = U.sum_error(x.shape[1])
    y, mag = x @ w.t(), x.abs() @ w.abs().t()
    err = e * mag
    for st, n, a in zip(start, lens, idx):
        for la, lb, off in slices if a >= 0 else ():
            A, B, r, c = la[a].double().cpu(), lb[a].double().cpu(), slice(st, st + n), slice(off, off + lb.shape[1])
            v = scale * (x[r] @ A.t())
            ev = scale * e * (x[r].abs() @ A.abs().t()) + left * v.abs().amax(dim=1, keepdim=True) + 2.0 ** -65
            y[r, c] += v @ B.t()
            m = (v.abs() + ev) @ B.abs().t()
            mag[r, c] += m
            err[r, c] += ev @ B.abs().t() + U.sum_error(2 * A.shape[0]) * m
    err = err + 4 * 2.0 ** -23 * mag
    return y, U.rounded(y, err, F32)


@pytest.mark.parametrize("scale", [2.0 ** -40, 2.0 ** -20, 2.0 ** -12, 2.0 ** -4, 2.0 ** 9, 2.0 ** 17, 2.0 ** 40])
@pytest.mark.parametrize("T,K", ODD_SHAPES)
def test_lora_linear_float16_keeps_projections_of_any_size(T, K, scale):
    """float16 weights, float32 results, nothing but the adapters: the values v lie far below and far
    above float16's own range and keep 22 bits."""
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(T + K)
    H, N, L = 72, 4096 if T > 1000 else 152, 3
    x, w = normal(gen, T, H, dtype=F16), torch.zeros(N, H, dtype=F16, device="cuda")
    slices = [(normal(gen, L, K, H, sigma=H ** -0.5, dtype=F16), normal(gen, L, N, K, dtype=F16), 0)]
    start, lens, idx = [0, T // 3], [T // 3, T - T // 3], [0, 1]
    o = torch.zeros(T, N, dtype=F32, device="cuda")
    sg.sgmv_lora_linear(x, w, slices, o, i64(start), i64(lens), i64(idx), 2, T, scaling=scale)
    want, bound = scaled_bound(x, w, slices, start, lens, idx, scale, 2.0 ** -22)
    U.assert_within(o, want, bound)


@pytest.mark.parametrize("T,K", ODD_SHAPES)
def test_lora_linear_float16_projections_of_unlike_sizes(T, K):
    """Slices, adapters and parts of the rank whose values differ by powers of two, beside a shared
    projection that has to stay as it is, in rows without an adapter too."""
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(T + K)
    H, L = 72, 4
    widths, offs, N = [40, 24, 32], [0, 40, 80], 4096 if T > 1000 else 152
    x, w = normal(gen, T, H, dtype=F16), normal(gen, N, H, sigma=H ** -0.5, dtype=F16)
    slices = [(normal(gen, L, K, H, sigma=H ** -0.5, dtype=F16), normal(gen, L, n, K, dtype=F16), off)
              for n, off in zip(widths, offs)]
    for s, p in enumerate((2.0 ** 10, 2.0 ** -8, 1.0)):
        slices[s][0].mul_(p)
    for a in range(L):
        slices[a % 3][0][a].mul_(2.0 ** -(2 * a))
    slices[2][0][:, K // 2:].mul_(2.0 ** -6)
    cut = sorted(np.random.default_rng(T).integers(0, T + 1, 4).tolist())
    start, lens = [0] + cut, [b - a for a, b in zip([0] + cut, cut + [T])]
    idx = [2, 0, -1, 3, 1]
    for scale in (2.0 ** 11, 2.0 ** -9):
        o = torch.zeros(T, N, dtype=F32, device="cuda")
        sg.sgmv_lora_linear(x, w, slices, o, i64(start), i64(lens), i64(idx), 5, T, scaling=scale)
        want, bound = scaled_bound(x, w, slices, start, lens, idx, scale, 2.0 ** -22)
        U.assert_within(o, want, bound)


@pytest.mark.parametrize("dtype,scale", [(BF16, 1.0), (BF16, 2.0 ** -60), (BF16, 2.0 ** 127), (F16, 1.0), (F16, 2.0 ** -30), (F16, 2.0 ** 40)])
@pytest.mark.parametrize("T,K", ODD_SHAPES)
def test_lora_linear_float32_results_hold_all_bits_of_the_projections(T, K, dtype, scale):
    """lora_B picks one value v a column, so that a float32 result is v itself: 24 bits of it with
    bfloat16 weights (values up to float32's largest), 22 with float16 weights."""
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(T + K)
    H, N, L = 72, 4096 if T > 1000 else 152, 3
    bits, parts = (8, 3) if dtype == BF16 else (11, 2)
    x = torch.zeros(T, H, dtype=dtype)
    la = torch.zeros(L, K, H, dtype=dtype)
    for i, h in enumerate((3, 40, 71)[:parts]):
        x[:, h] = 2.0 ** (-bits * i)
        la[:, :, h] = (torch.randint(2 ** (bits - 1), 2 ** bits, (L, K), generator=gen) * 2.0 ** (1 - bits)).to(dtype)
    la[1, :, 3] = 2 - 2.0 ** (1 - bits)  # the largest: rounding it to the parts' type goes up to 2
    sign = torch.where(torch.rand(T, generator=gen) < 0.5, -1.0, 1.0)
    x = (x * sign[:, None]).to(dtype).cuda()
    lb = torch.zeros(L, N, K, dtype=dtype)
    lb[:, torch.arange(N), torch.arange(N) % K] = 1.0
    w = torch.zeros(N, H, dtype=dtype, device="cuda")
    o = torch.full((T, N), 7.0, dtype=F32, device="cuda")
    start, lens, idx = [0, T // 3], [T // 3, T - T // 3], [0, 1]
    sg.sgmv_lora_linear(x, w, [(la.cuda(), lb.cuda(), 0)], o, i64(start), i64(lens), i64(idx), 2, T, scaling=scale)
    for st, n, a in zip(start, lens, idx):
        v = scale * (x[st:st + n].double().cpu() @ la[a].double().t())
        assert torch.equal(v, v.float().double())
        assert torch.equal(o[st:st + n].double().cpu(), v[:, torch.arange(N) % K])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,H", [(60, 64), (700, 64), (700, 67)])
def test_grouped_overlapping_segments_stay_in_their_rows(T, H, gated):
    """Overlapping segments break a precondition and their values are unspecified; rows outside all of
    them stay as they are."""
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(T)
    N, B = 96, 500
    x, w = normal(gen, T, H), normal(gen, 3, 2 * N if gated else N, H)
    full, o = guarded(T, N, BF16, 5, gen)
    o0 = o.clone()
    start, lens = [T // 4] * B, [T // 2] * B
    sg.sgmv_grouped_gemm(x, w, o, i64(start), i64(lens), i64([b % 3 for b in range(B)]), B, T, gated=gated)
    outside = list(range(T // 4)) + list(range(T // 4 + T // 2, T))
    assert torch.equal(o[outside], o0[outside]) and bool((full[:, N:] == 7.0).all())
