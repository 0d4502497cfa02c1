"""The operators on microscaled 4-bit weights together (the example block with
4-bit weights): each step against its definition in 64 bits on the step before's
results, under graph capture, on streams of their own, from run to run, and
past 32-bit offsets."""
import importlib.util
import os

import pytest
import torch

import matmul_util as U
import mx_util as M

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def example():
    path = os.path.join(ROOT, "segmented_gather_gemm_amd", "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


def inputs(lens, hidden, adapters, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens_t = torch.tensor(lens, device="cuda")
    start = torch.cumsum(lens_t, 0) - lens_t
    adapter = torch.randint(-1, adapters, (len(lens),), generator=g, device="cuda")
    attn = torch.randn(sum(lens), hidden, generator=g, device="cuda").to(BF16)
    residual = torch.randn(sum(lens), hidden, generator=g, device="cuda").to(BF16)
    return start, lens_t, adapter, attn, residual


def values(pair, hidden):
    return M.values(pair[0].cpu().numpy(), pair[1].cpu().numpy(), hidden)


@pytest.mark.parametrize("lens", [[1], [1] * 20, [1] * 70, [130, 1, 77, 0, 300]])
def test_block_step_by_step(lens):
    B = example()
    w = B.random_weights(256, 192, 8, 3, 16)
    q = B.four_bit(w)
    start, lens_t, adapter, attn, residual = inputs(lens, 256, 3, len(lens))
    before, seen = residual.clone(), {}
    B.block(q, attn, residual, start, lens_t, adapter, 2, seen=seen)
    want, bound = M.lora_linear(attn, values(q.proj, 256), None, [(w.lora_a, w.lora_b, 0)], start.tolist(), lens, adapter.tolist(), 2.0,
                                before, True, BF16)
    U.assert_within(seen["projected"], want, bound, "projection")
    e_start, e_lens, rows = seen["start"].tolist(), seen["lens"].tolist(), seen["rows"].tolist()
    want, bound, _ = M.grouped(seen["x"], values(q.gate_up, 256), e_start, e_lens, None, rows, True, seen["hidden"])
    U.assert_within(seen["hidden"], want, bound, "gate and up")
    want, bound, _ = M.grouped(seen["hidden"], values(q.down, 192), e_start, e_lens, None, None, False, seen["out"])
    U.assert_within(seen["out"], want, bound, "down")
    want, bound = U.combine(seen["out"], seen["weights"], seen["slots"], seen["projected"], True)
    U.assert_within(residual, want, bound, "sum")


def test_weights_read_back_are_the_values_of_their_codes():
    B = example()
    w = B.random_weights(200, 192, 3, 2, 8)
    for t in (w.proj, w.gate_up, w.down):
        pair = B.packed(t)
        assert torch.equal(B.unpacked(pair, t).cpu().double(), values(pair, t.shape[-1]))


@pytest.mark.parametrize("lens", [[1] * 12, [1] * 50, [200, 61, 300]])
def test_graph_replays_match_eager(lens):
    B = example()
    w = B.four_bit(B.random_weights(256, 192, 8, 3, 16))
    start, lens_t, adapter, attn, first = inputs(lens, 256, 3, 7)
    eager = first.clone()
    B.block(w, attn, eager, start, lens_t, adapter, 2)
    residual = first.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.block(w, attn, residual, start, lens_t, adapter, 2)
    for replay in range(4):
        residual.copy_(first)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(residual, eager), f"replay {replay}"
        other = first.clone()
        B.block(w, attn, other, start, lens_t, adapter, 2)
        torch.cuda.synchronize()
        assert torch.equal(other, eager)


def test_quantising_in_a_graph_follows_its_inputs():
    import segmented_gather_gemm_amd as sg
    x = torch.randn(37, 300, device="cuda")
    c, s = (torch.empty(37, n, dtype=torch.uint8, device="cuda") for n in sg.mx_row_bytes(300))
    o = torch.empty(37, 300, device="cuda")
    sg.sgmv_mx_quantize(x, c, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sg.sgmv_mx_quantize(x, c, s)
        sg.sgmv_mx_dequantize(c, s, o)
    for seed in range(3):
        x.copy_(torch.randn(37, 300, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.cpu().double(), M.rounded(x))


def test_calls_on_other_streams_at_the_same_time():
    B = example()
    w = B.four_bit(B.random_weights(256, 192, 8, 3, 16))
    cases = [inputs(lens, 256, 3, s) for s, lens in enumerate(([40, 1, 90], [1] * 30, [3]))]
    want = []
    for start, lens_t, adapter, attn, residual in cases:
        r = residual.clone()
        B.block(w, attn, r, start, lens_t, adapter, 2)
        want.append(r)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = []
        for s, (start, lens_t, adapter, attn, residual) in zip(streams, cases):
            with torch.cuda.stream(s):
                r = residual.clone()
                B.block(w, attn, r, start, lens_t, adapter, 2)
                got.append(r)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,segments", [(1, 1), (16, 16), (31, 31), (64, 64), (200, 200), (513, 7)])
def test_results_do_not_depend_on_the_run(T, segments):
    """Adapters spread over a table of 1000 segments, most of them empty: the same float32 bits every time."""
    import segmented_gather_gemm_amd as sg
    g = torch.Generator(device="cuda").manual_seed(T)
    H, N, K, L, S = 520, 128, 16, 40, 1000
    x = torch.randn(T, H, generator=g, device="cuda").to(BF16)
    codes, scales = M.packed(torch.randn(N, H, generator=torch.Generator().manual_seed(T)))
    la, lb = torch.randn(L, K, H, generator=g, device="cuda").to(BF16), torch.randn(L, N, K, generator=g, device="cuda").to(BF16)
    lens, start = torch.zeros(S, dtype=torch.int64, device="cuda"), torch.zeros(S, dtype=torch.int64, device="cuda")
    at = torch.randperm(S, generator=g, device="cuda")[:segments]
    edges = torch.linspace(0, T, segments + 1, device="cuda").long()
    lens[at], start[at] = edges[1:] - edges[:-1], edges[:-1]
    idx = torch.randint(-1, L, (S,), generator=g, device="cuda")
    first = None
    for run in range(60):
        o = torch.zeros(T, N, dtype=F32, device="cuda")
        sg.sgmv_mx_lora_linear(x, codes, scales, [(la, lb, 0)], o, start, lens, idx, S, T)
        first = o if first is None else first
        assert torch.equal(o, first), f"run {run}"
    want, bound = M.lora_linear(x, M.values(codes.cpu().numpy(), scales.cpu().numpy(), H), None, [(la, lb, 0)], start.tolist(),
                                lens.tolist(), idx.tolist(), 1.0, first, False, F32)
    U.assert_within(first, want, bound)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T", [3, 30, 60, 100, 300])
def test_adapters_that_are_not_finite_stay_with_their_rows(T, dtype):
    """An infinity in one adapter's weights and a NaN in another's reach the rows of their own requests
    in their own slice; all else is as without them."""
    import segmented_gather_gemm_amd as sg
    g = torch.Generator().manual_seed(T)
    H, K, N = 256, 16, [48, 80]
    x = torch.randn(T, H, generator=g).to(dtype).cuda()
    codes, scales = M.packed(torch.randn(sum(N), H, generator=g))
    third = max(1, T // 3)
    lens, idx = [third, third, T - 2 * third], [0, 2, 1]
    start = [0, third, 2 * third]
    slices, at = [], 0
    for n in N:
        slices.append([torch.randn(3, K, H, generator=g).to(dtype).cuda(), torch.randn(3, n, K, generator=g).to(dtype).cuda(), at])
        at += n
    o = torch.empty(T, sum(N), dtype=F32, device="cuda")
    sg.sgmv_mx_lora_linear(x, codes, scales, [tuple(s) for s in slices], o, i64(start), i64(lens), i64(idx), 3, max(lens))
    clean = o.clone()
    slices[0][1][2, 5, 3] = float("inf")                          # adapter 2: the second request's rows, column 5
    slices[1][0][1, 0, 7] = float("nan")                          # adapter 1: the third's rows, the second slice's columns
    sg.sgmv_mx_lora_linear(x, codes, scales, [tuple(s) for s in slices], o, i64(start), i64(lens), i64(idx), 3, max(lens))
    odd = torch.zeros(T, sum(N), dtype=torch.bool, device="cuda")
    odd[third:2 * third, 5] = True
    odd[2 * third:, N[0]:] = True
    assert torch.equal(o[~odd], clean[~odd])
    assert bool((~o[odd].isfinite()).all())
    assert bool(o[2 * third:, N[0]:].isnan().all())


def test_past_32_bit_offsets():
    """Outputs, gathered inputs, weights and quantised rows of more than 2^32 bytes, at both ends."""
    import segmented_gather_gemm_amd as sg
    g = torch.Generator(device="cuda").manual_seed(0)
    T, H, N, K = 140000, 64, 16384, 8
    x = torch.randn(T, H, generator=g, device="cuda").to(BF16)
    codes, scales = M.packed(torch.randn(N, H, generator=torch.Generator().manual_seed(0)) / 8)
    la, lb = torch.randn(2, K, H, generator=g, device="cuda").to(BF16), torch.randn(2, N, K, generator=g, device="cuda").to(BF16)
    out = torch.empty(T, N, dtype=BF16, device="cuda")
    start, lens, idx = [0, 1000], [1000, T - 1000], [1, 0]
    wv = M.values(codes.cpu().numpy(), scales.cpu().numpy(), H)
    print("mx_lora_linear of 4.6 GB", flush=True)
    sg.sgmv_mx_lora_linear(x, codes, scales, [(la, lb, 0)], out, i64(start), i64(lens), i64(idx), 2, T)
    for rows, a in (([0, 999], 1), ([1000, 70000, 131072, T - 1], 0)):
        want, bound = M.lora_linear(x[rows], wv, None, [(la, lb, 0)], [0], [len(rows)], [a], 1.0, None, False, BF16)
        U.assert_within(out[rows], want, bound)
    wide = out                                                    # (140000, 16384): 4.6 GB of inputs
    we = M.packed(torch.randn(2, 24, N, generator=torch.Generator().manual_seed(1)) / 128)
    pick = [T - 1, 0, 131072, 65536, T - 2]
    y = torch.zeros(5, 24, dtype=F32, device="cuda")
    print("mx_grouped_gemm gathering from 4.6 GB", flush=True)
    sg.sgmv_mx_grouped_gemm(wide, *we, y, i64([0, 2]), i64([2, 3]), None, 2, 3, row_indices_tensor=i64(pick))
    want, bound, _ = M.grouped(wide[pick], values(we, N), [0, 2], [2, 3], None, None, False, y)
    U.assert_within(y, want, bound)
    c, s = (torch.empty(T, n, dtype=torch.uint8, device="cuda") for n in sg.mx_row_bytes(N))
    print("quantising 4.6 GB", flush=True)
    sg.sgmv_mx_quantize(wide, c, s)
    rows = [0, 1, 65536, 131072, T - 1]
    want_c, want_s = M.quantize(wide[rows])
    assert torch.equal(c[rows].cpu(), torch.from_numpy(want_c)) and torch.equal(s[rows].cpu(), torch.from_numpy(want_s))
    back = torch.empty(T, N, dtype=BF16, device="cuda")
    sg.sgmv_mx_dequantize(c, s, back)
    assert torch.equal(back[rows].cpu().double(), M.values(want_c, want_s, N))
    del back, out, wide
    # experts of 4.8 GB of codes, the last one among them
    E, n, h = 72, 4096, 32768
    codes = torch.randint(0, 256, (E, n, h // 2), dtype=torch.uint8, generator=g, device="cuda")
    scales = torch.randint(118, 122, (E, n, h // 32), dtype=torch.uint8, generator=g, device="cuda")
    x = torch.randn(40, h, generator=g, device="cuda").to(BF16)
    for rows in (2, 20):
        y = torch.zeros(2 * rows, n, dtype=F32, device="cuda")
        print("mx_grouped_gemm with 4.8 GB of weights", flush=True)
        sg.sgmv_mx_grouped_gemm(x[:2 * rows], codes, scales, y, i64([0, rows]), i64([rows, rows]), i64([E - 1, 1]), 2, rows)
        cols = [0, 1, 2047, n - 1]
        for seg, e in ((0, E - 1), (1, 1)):
            r = slice(seg * rows, (seg + 1) * rows)
            wv = M.values(codes[e, cols].cpu().numpy(), scales[e, cols].cpu().numpy(), h)
            xr = M.rounded(x[r])
            want, mag = xr @ wv.t(), xr.abs() @ wv.abs().t()
            U.assert_within(y[r][:, cols], want, U.rounded(want, U.sum_error(h) * mag, F32))


def test_workspaces_of_the_caller():
    import segmented_gather_gemm_amd as sg
    x = torch.randn(70, 200, device="cuda").to(BF16)
    codes, scales = M.packed(torch.randn(64, 200))
    la, lb = torch.randn(2, 8, 200, device="cuda").to(BF16), torch.randn(2, 64, 8, device="cuda").to(BF16)
    args = (i64([0]), i64([70]), i64([1]), 1, 70)
    want = sg.sgmv_mx_lora_linear(x, codes, scales, [(la, lb, 0)], torch.empty(70, 64, dtype=BF16, device="cuda"), *args)
    need = sg.mx_lora_linear_workspace_bytes(70, 200, 1, 8)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    got = sg.sgmv_mx_lora_linear(x, codes, scales, [(la, lb, 0)], torch.empty(70, 64, dtype=BF16, device="cuda"), *args, workspace=ws[:need])
    assert torch.equal(got, want) and bool((ws[need:] == 0xFF).all())
    with pytest.raises(ValueError, match="workspace"):
        sg.sgmv_mx_lora_linear(x, codes, scales, [(la, lb, 0)], got, *args, workspace=ws[:need - 256])
    e = (codes[None], scales[None])
    need = sg.mx_grouped_gemm_workspace_bytes(70, 200)
    want = sg.sgmv_mx_grouped_gemm(x, *e, torch.empty(70, 64, dtype=BF16, device="cuda"), i64([0]), i64([70]), None, 1, 70)
    ws.fill_(0xFF)
    got = sg.sgmv_mx_grouped_gemm(x, *e, torch.empty(70, 64, dtype=BF16, device="cuda"), i64([0]), i64([70]), None, 1, 70, workspace=ws[:need])
    assert torch.equal(got, want) and bool((ws[need:] == 0xFF).all())
    with pytest.raises(ValueError, match="workspace"):
        sg.sgmv_mx_grouped_gemm(x, *e, got, i64([0]), i64([70]), None, 1, 70, workspace=ws[:need - 1])


def test_wrappers_check_their_tensors():
    import segmented_gather_gemm_amd as sg
    x = torch.zeros(4, 128, dtype=BF16, device="cuda")
    o = torch.zeros(4, 4, dtype=BF16, device="cuda")
    c, s = torch.zeros(4, 64, dtype=torch.uint8, device="cuda"), torch.zeros(4, 4, dtype=torch.uint8, device="cuda")
    i = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="codes"):
        sg.sgmv_mx_quantize(x, c[:, :32], s)
    with pytest.raises(ValueError, match="scales"):
        sg.sgmv_mx_quantize(x, c, s.cpu())
    with pytest.raises(ValueError, match="rows"):
        sg.sgmv_mx_quantize(x, c[:3], s[:3])
    with pytest.raises(ValueError, match="row_indices"):
        sg.sgmv_mx_dequantize(c, s, x, row_indices_tensor=i[:2])
    with pytest.raises(ValueError, match="row_indices"):
        sg.sgmv_mx_dequantize(c[:3], s[:3], x)
    with pytest.raises(ValueError, match="bias"):
        sg.sgmv_mx_lora_linear(x, c, s, [], o, i, i, i, 0, 0, bias=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError, match="shorter"):
        sg.sgmv_mx_lora_linear(x, c, s, [], o, i, i, i, 5, 1)
    with pytest.raises(ValueError, match="inputs"):
        sg.sgmv_mx_lora_linear(x.cpu(), c, s, [], o, i, i, i, 0, 0)
    with pytest.raises(NotImplementedError):
        sg.sgmv_mx_lora_linear(x.float(), c, s, [], o, i, i, i, 0, 0)
    with pytest.raises(ValueError, match="3-D"):
        sg.sgmv_mx_grouped_gemm(x, c, s, o, i, i, None, 1, 1)
    with pytest.raises(ValueError, match="shorter"):
        sg.sgmv_mx_grouped_gemm(x, c[None], s[None], o, i, i, None, 5, 1)
    with pytest.raises(TypeError):
        sg.sgmv_mx_quantize(x.double(), c, s)
