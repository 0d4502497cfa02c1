"""Microscaled 4-bit rows on the GPU: quantised, read back, and multiplied,
against their definitions in 64 bits (mx_util)."""
import numpy as np
import pytest
import torch

import matmul_util as U
import mx_util as M

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
INT = {BF16: torch.int16, F16: torch.int16, F32: torch.int32}


def i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


def quantize(x, pad_c=0, pad_s=0):
    """sgmv_mx_quantize into rows inside wider ones, whose other bytes have to stay."""
    import segmented_gather_gemm_amd as sg
    T, H = x.shape
    cb, sb = sg.mx_row_bytes(H)
    full_c = torch.full((T + 1, cb + pad_c), 0xA5, dtype=torch.uint8, device="cuda")
    full_s = torch.full((T + 1, sb + pad_s), 0xA5, dtype=torch.uint8, device="cuda")
    c, s = full_c[:T, :cb], full_s[:T, :sb]
    print(f"quantize {tuple(x.shape)} {x.dtype} stride {x.stride(0)}", flush=True)
    sg.sgmv_mx_quantize(x, c, s)
    torch.cuda.synchronize()
    assert bool((full_c[:, cb:] == 0xA5).all()) and bool((full_s[:, sb:] == 0xA5).all())
    assert bool((full_c[T] == 0xA5).all()) and bool((full_s[T] == 0xA5).all())
    return c, s


def same_codes(x, c, s):
    want_c, want_s = M.quantize(x)
    got_c, got_s = c.cpu().numpy(), s.cpu().numpy()
    assert np.array_equal(got_s, want_s), np.argwhere(got_s != want_s)[:4]
    assert np.array_equal(got_c, want_c), np.argwhere(got_c != want_c)[:4]


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_quantize_every_16_bit_value(dtype):
    """Every bit pattern, next to a block's largest value of each of several exponents (patterns
    larger than that set the scale themselves; blocks with an infinity or NaN are 255)."""
    every = torch.cat([torch.arange(65536, dtype=torch.int32), torch.zeros(31 * 2115 - 65536, dtype=torch.int32)])
    v = every.to(torch.int16).view(dtype).view(-1, 31)
    for top in (0.0, 2.0 ** -24, 2.0 ** -14, 0.75, 1.0, 3.0, 1000.0, 60000.0) + ((2.0 ** 100, 3e38, 2.0 ** -130) if dtype == BF16 else ()):
        rows = torch.cat([v, torch.full((v.shape[0], 1), top, dtype=dtype)], dim=1).cuda()
        same_codes(rows, *quantize(rows))


def test_quantize_every_float32_exponent():
    gen = torch.Generator().manual_seed(0)
    bits = torch.randint(-2 ** 31, 2 ** 31, (4096, 32), generator=gen).to(torch.int32)
    near = (bits & 0x807FFFFF) | ((torch.arange(4096, dtype=torch.int32) % 255)[:, None] << 23)  # one exponent a block
    ties = torch.tensor([7, 6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, 0.0]).repeat(4)[:32]
    tied = torch.ldexp(ties[None], torch.arange(-145, 125)[:, None])
    tied = torch.cat([tied, -tied, torch.nextafter(tied, tied * 2), torch.nextafter(tied, tied * 0)])
    for rows in (bits.view(F32), near.view(F32), tied):
        same_codes(rows, *quantize(rows.contiguous().cuda()))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,H,pad", [(1, 1, 0), (3, 31, 0), (2, 32, 0), (5, 33, 1), (1, 127, 0), (7, 128, 8), (2, 129, 3), (65, 200, 0),
                                     (300, 520, 24), (17, 1031, 0), (1, 4096, 0), (129, 4104, 8)])
def test_quantize_sizes_and_strides(dtype, T, H, pad):
    gen = torch.Generator().manual_seed(T * H)
    x = torch.randn(T, H + pad, generator=gen) * torch.exp(3 * torch.randn(T, H + pad, generator=gen))
    x[T // 2] = 0
    x = x.to(dtype).cuda()[:, :H]
    same_codes(x, *quantize(x, pad_c=16 * (pad % 3), pad_s=4 * (pad % 2)))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_quantize_values_that_are_not_finite(dtype):
    x = torch.randn(8, 160, generator=torch.Generator().manual_seed(1)).to(dtype)
    for r, v in enumerate((float("inf"), float("-inf"), float("nan"))):
        x[r, 5 + 32 * r] = v
        x[r + 4, 159] = v
    x = x.cuda()
    c, s = quantize(x)
    same_codes(x, c, s)
    assert int((s == 255).sum()) == 6


@pytest.mark.parametrize("out", [BF16, F16, F32])
def test_dequantize_every_code_and_scale(out):
    """Each of 256 bytes under each of 256 scales: exact, or rounded to nearest even where the dtype
    cannot hold the value."""
    import segmented_gather_gemm_amd as sg
    codes = torch.arange(256, dtype=torch.uint8).view(1, 4, 64).expand(256, 4, 64).reshape(256, 256).contiguous().cuda()
    scales = torch.arange(256, dtype=torch.uint8)[:, None].expand(256, 16).contiguous().cuda()
    o = torch.empty(256, 512, dtype=out, device="cuda")
    sg.sgmv_mx_dequantize(codes, scales, o)
    want = M.values(codes.cpu().numpy(), scales.cpu().numpy(), 512).to(out)
    got = o.cpu()
    assert bool(got[255].isnan().all())
    assert torch.equal(got[:255].view(INT[out]), want[:255].view(INT[out]))  # signs of zeros too


@pytest.mark.parametrize("out", [BF16, F16, F32])
@pytest.mark.parametrize("T,R,H,pad", [(1, 1, 1, 0), (5, 3, 33, 0), (70, 9, 128, 8), (4, 20, 257, 3), (300, 64, 1031, 1), (9, 9, 4096, 0)])
def test_dequantize_gathered_rows(out, T, R, H, pad):
    """Rows chosen by index, some twice, some outside the table (zeros)."""
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(T + H)
    cb, sb = sg.mx_row_bytes(H)
    codes = torch.randint(0, 256, (R, cb + 16), dtype=torch.uint8, generator=gen).cuda()[:, :cb]
    scales = torch.randint(100, 150, (R, sb + 4), dtype=torch.uint8, generator=gen).cuda()[:, :sb]
    rows = torch.randint(-1, R + 1, (T,), generator=gen)
    rows[0] = R - 1
    full = torch.full((T, H + pad), 7.0, dtype=out, device="cuda")
    o = full[:, :H]
    sg.sgmv_mx_dequantize(codes, scales, o, row_indices_tensor=rows.cuda())
    table = M.values(codes.cpu().numpy(), scales.cpu().numpy(), H)
    want = torch.zeros(T, H, dtype=torch.float64)
    ok = (rows >= 0) & (rows < R)
    want[ok] = table[rows[ok]]
    assert torch.equal(o.cpu(), want.to(out))
    assert bool((full[:, H:] == 7.0).all())


def test_round_trip_is_stable():
    """Quantising the values read back gives the same codes and scales: a block's largest value lies
    in [4, 6] scales after the first."""
    import segmented_gather_gemm_amd as sg
    x = torch.randn(50, 1000, generator=torch.Generator().manual_seed(2)).cuda()
    c, s = quantize(x)
    back = torch.empty_like(x)
    sg.sgmv_mx_dequantize(c, s, back)
    c2, s2 = quantize(back)
    assert torch.equal(c2, c) and torch.equal(s2, s)


# --------------------------------------------------------------------------
# Products.
# --------------------------------------------------------------------------

def normal(gen, *shape, sigma=1.0, dtype=BF16):
    return (torch.randn(*shape, generator=gen) * sigma).to(dtype)


def starts(lens):
    return np.concatenate([[0], np.cumsum(lens)[:-1]]).astype(int).tolist() if lens else []


def lora_case(T, H, widths, K, L, lens, idx, dtype=BF16, out=None, bias=False, add=False, scale=0.5, start=None, seed=0, pad_x=0,
              pad_out=0, pad_w=0, gaps=(), change=None):
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(seed)
    N = sum(widths) + sum(gaps)
    out = out or dtype
    x = normal(gen, T, H + pad_x, dtype=dtype).cuda()[:, :H]
    codes, scales = M.packed(normal(gen, N, H, sigma=H ** -0.5))
    if pad_w:
        codes = torch.nn.functional.pad(codes, (0, 16 * pad_w), value=0x77)[:, :codes.shape[1]]
        scales = torch.nn.functional.pad(scales, (0, 4 * pad_w), value=0xFF)[:, :scales.shape[1]]
    b = normal(gen, N, dtype=dtype).cuda() if bias else None
    slices, at = [], 0
    for i, n in enumerate(widths if K else []):
        slices.append((normal(gen, L, K, H, sigma=H ** -0.5, dtype=dtype).cuda(), normal(gen, L, n, K, sigma=0.3, dtype=dtype).cuda(), at))
        at += n + (gaps[i] if i < len(gaps) else 0)
    start = starts(lens) if start is None else start
    full = torch.full((T + 1, N + pad_out), 7.0, dtype=out, device="cuda")
    o = full[:T, :N]
    o.copy_(torch.randn(T, N, generator=gen).to(out))
    o0 = o.clone()
    if change:
        change(x, codes, scales)
    print(f"mx_lora_linear T={T} H={H} N={N} K={K} L={L} segments={len(lens)} {dtype}->{out}", flush=True)
    sg.sgmv_mx_lora_linear(x, codes, scales, slices, o, i64(start), i64(lens), i64(idx), len(lens), max(lens, default=0), scaling=scale,
                           bias=b, add_inputs=add)
    torch.cuda.synchronize()
    wv = M.values(codes.cpu().numpy(), scales.cpu().numpy(), H)
    want, bound = M.lora_linear(x, wv, b, slices, start, lens, idx, scale, o0, add, out)
    if change is None:
        U.assert_within(o, want, bound)
    assert bool((full[:T, N:] == 7.0).all()) and bool((full[T] == 7.0).all())
    return o, want, bound


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 32, 33, 64, 65, 127, 130, 257, 520])
def test_lora_linear_rows(T):
    half = max(1, T // 2)
    lens = [half, T - half] if T > 1 else [1]
    lora_case(T, 256, [320], 16, 3, lens, [2, -1][:len(lens)] if T % 2 else [1, 2][:len(lens)], seed=T)


@pytest.mark.parametrize("H", [1, 7, 8, 32, 40, 127, 128, 136, 255, 264, 384, 512, 520, 640, 1032, 2056, 4224])
@pytest.mark.parametrize("T", [5, 40, 300])
def test_lora_linear_hidden(T, H):
    lora_case(T, H, [136], 8, 2, [T], [1], dtype=F16, seed=H)


@pytest.mark.parametrize("widths", [[1], [8], [16], [24], [72], [128, 64, 64], [264], [520], [40, 8, 136], [67]])
@pytest.mark.parametrize("T", [3, 20, 140, 300])
def test_lora_linear_widths(T, widths):
    lora_case(T, 192, widths, 16, 4, [T - 2, 2], [3, 0], bias=True, seed=sum(widths))


@pytest.mark.parametrize("K", [0, 1, 8, 13, 16, 24, 32, 64, 100, 128, 256])
@pytest.mark.parametrize("T", [4, 30, 200])
def test_lora_linear_ranks(T, K):
    lora_case(T, 320, [192], K, 3, [T // 2, T // 2], [0, 2], seed=K)


@pytest.mark.parametrize("T,K,widths,idx", [(1, 16, [200], [2]), (1, 16, [40, 8, 600], [0]), (1, 8, [16, 16], [-1]), (2, 24, [72], [1, 1]),
                                            (2, 8, [1040, 520, 24], [2, 0]), (3, 16, [136], [1, -1, 0]), (6, 8, [5000], [0, 1, 2, 0, 1, 2])])
@pytest.mark.parametrize("H", [8, 520, 4096, 4104, 5000])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F32)])
def test_lora_linear_projects_in_the_product(T, K, widths, idx, H, dtype, out):
    """At most 48 rows of lora_A over the tokens: each workgroup of the product projects onto them itself."""
    lora_case(T, H, widths, K, 3, [1] * T, idx, dtype=dtype, out=out, bias=H == 520, add=T == 2, seed=H + T, pad_x=8, gaps=[8])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("out", [BF16, F16, F32])
@pytest.mark.parametrize("T,add", [(7, False), (7, True), (50, True), (190, False), (190, True), (400, True)])
def test_lora_linear_types(dtype, out, T, add):
    lora_case(T, 264, [136, 200], 24, 3, [T - 3, 3], [1, 2], dtype=dtype, out=out, bias=True, add=add)


@pytest.mark.parametrize("T,H,N,pad_x,pad_out,pad_w", [(9, 130, 67, 3, 5, 1), (150, 130, 67, 3, 5, 1), (9, 128, 66, 0, 1, 3), (300, 66, 131, 8, 0, 0),
                                                       (70, 7, 1, 1, 0, 2), (1, 1, 1, 0, 0, 0), (33, 1000, 200, 8, 8, 1)])
def test_lora_linear_odd_sizes_and_strides(T, H, N, pad_x, pad_out, pad_w):
    lora_case(T, H, [N], 5, 2, [T], [1], pad_x=pad_x, pad_out=pad_out, pad_w=pad_w, bias=True)


@pytest.mark.parametrize("T", [12, 40, 64, 300, 513])
def test_lora_linear_many_adapters(T):
    rng = np.random.default_rng(T)
    lora_case(T, 256, [256, 64], 16, 24, [1] * T, rng.integers(-1, 24, T).tolist(), seed=T)


@pytest.mark.parametrize("T", [10, 50, 300])
def test_lora_linear_segment_layouts(T):
    """Unsorted starts, gaps, empty segments, and segments that break a precondition: those get the
    shared projection alone."""
    start = [T - 5, 5, 20, 0, 4, T - 1, -1, 30, 30]
    lens = [5, 0, 0, 3, 1, 2, 3, 0, -2]
    idx = [1, 0, 1, 2, -1, 1, 1, 7, 1]
    lora_case(T, 128, [192], 16, 3, lens, idx, start=start)


@pytest.mark.parametrize("T", [9, 100])
def test_lora_linear_without_adapters(T):
    lora_case(T, 320, [200], 0, 0, [], [], bias=True, add=True)
    lora_case(T, 320, [200], 16, 0, [T], [0])             # an empty stack of adapters


@pytest.mark.parametrize("T", [4, 24, 64, 200, 300])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_lora_linear_values_that_are_not_finite(T, dtype):
    """An input block with an infinity or NaN makes its row NaN, a weight block of scale 255 its column;
    nothing else changes."""
    def spoil(x, codes, scales):
        x[1, 300], x[2, 0] = float("inf"), float("nan")
        scales[7, 2] = 255
    o, want, bound = lora_case(T, 330, [96], 0, 0, [], [], dtype=dtype, change=spoil)
    odd = torch.zeros(T, 96, dtype=torch.bool)
    odd[1], odd[2], odd[:, 7] = True, True, True
    assert torch.equal(o.cpu().isnan(), odd)
    assert bool((((o.cpu().double() - want).abs() <= bound) | odd).all())


@pytest.mark.parametrize("T", [3, 20, 300])
def test_lora_linear_scales_of_every_size(T):
    """Rows and weights whose scales span the whole range, so that their products do, too: sums that
    are finite in float32."""
    def spread(x, codes, scales):
        x.copy_((x.float() * torch.exp2(torch.linspace(-30, 10, x.shape[0], device=x.device))[:, None]).to(x.dtype))
        scales.copy_((scales.int() + torch.linspace(-60, 30, scales.shape[0], device=x.device).int()[:, None]).to(torch.uint8))
    o, want, bound = lora_case(T, 512, [160], 0, 0, [], [], out=F32, change=spread)
    U.assert_within(o, want, bound)


def grouped_case(T, H, N, E, lens, k=1, gated=False, gather=True, dtype=BF16, out=None, idx=None, start=None, rows=None, seed=0, pad_out=0,
                 pad_x=0):
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(seed)
    out = out or dtype
    start = starts(lens) if start is None else start
    R = max([s + n for s, n in zip(start, lens)] + [1]) + 2        # two rows behind the last segment
    if rows is None and gather:
        rows = torch.randint(0, T, (R,), generator=gen).tolist()
    if not gather:
        T = R
    x = normal(gen, T, H + pad_x, dtype=dtype).cuda()[:, :H]
    wide = 2 * N if gated else N
    codes, scales = M.packed(normal(gen, E, wide, H, sigma=2 * H ** -0.5))
    full = torch.full((R, N + pad_out), 7.0, dtype=out, device="cuda")
    o = full[:, :N]
    print(f"mx_grouped T={T} H={H} N={N} E={E} rows={R} gated={gated} gather={gather} {dtype}->{out}", flush=True)
    sg.sgmv_mx_grouped_gemm(x, codes, scales, o, i64(start), i64(lens), None if idx is None else i64(idx), len(lens), max(lens, default=0),
                            row_indices_tensor=i64(rows) if gather else None, gated=gated)
    torch.cuda.synchronize()
    wv = M.values(codes.cpu().numpy(), scales.cpu().numpy(), H)
    o0 = torch.full((R, N), 7.0, dtype=out)
    want, bound, written = M.grouped(x, wv, start, lens, idx, rows if gather else None, gated, o0)
    U.assert_within(o, want, bound)
    assert bool((o.cpu()[~written] == 7.0).all()) and bool((full[:, N:] == 7.0).all())


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("lens", [[1], [1, 0, 2, 1], [16, 17, 3], [0, 0, 0], [130, 1, 64, 0, 257], [5] * 40])
def test_grouped_segments(lens, gated):
    grouped_case(50, 384, 96, len(lens), lens, gated=gated, seed=sum(lens))


@pytest.mark.parametrize("H", [1, 40, 128, 200, 256, 384, 512, 1408, 2056])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("lens", [[3, 1], [70, 150]])
def test_grouped_hidden(H, gated, lens):
    grouped_case(40, H, 72, 2, lens, gated=gated, gather=False, dtype=F16, seed=H)


@pytest.mark.parametrize("N", [1, 8, 24, 67, 128, 136, 264])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("lens", [[2, 4, 1], [140, 20, 33]])
def test_grouped_widths(N, gated, lens):
    grouped_case(64, 256, N, 3, lens, gated=gated, seed=N, pad_out=N % 3)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("out", [BF16, F16, F32])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("lens", [[4, 4], [200, 90]])
def test_grouped_types(dtype, out, gather, lens):
    grouped_case(30, 320, 80, 2, lens, gated=True, gather=gather, dtype=dtype, out=out, pad_x=8)


@pytest.mark.parametrize("lens", [[2, 3, 1], [150, 30, 270]])
def test_grouped_indices(lens):
    """Experts by index (one twice, one -1, one past the stack), rows gathered from outside (zeros),
    segments out of order."""
    total = sum(lens)
    rows = [(i * 7) % 20 - 1 for i in range(total + 2)]            # -1 now and then
    rows[0] = 10 ** 12
    start = [lens[1] + lens[2], 0, lens[1]]
    grouped_case(18, 256, 80, 4, lens, idx=[3, 3, 0], start=start, rows=rows)
    grouped_case(18, 256, 80, 4, lens, idx=[-1, 4, 2], start=start, rows=rows, gated=True)


def test_grouped_without_inputs():
    """No input row at all: every row is the product of zeros."""
    import segmented_gather_gemm_amd as sg
    x = torch.zeros(0, 256, dtype=BF16, device="cuda")
    codes, scales = M.packed(torch.ones(1, 16, 256))
    o = torch.full((5, 16), 7.0, dtype=BF16, device="cuda")
    sg.sgmv_mx_grouped_gemm(x, codes, scales, o, i64([0]), i64([5]), None, 1, 5, row_indices_tensor=i64([0] * 5))
    assert bool((o == 0).all())
