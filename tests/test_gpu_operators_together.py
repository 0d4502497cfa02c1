"""The projection, expert and routing operators together (the example block),
under graph capture, on streams of their own, and past 32-bit offsets."""
import importlib.util
import os

import pytest
import torch

import matmul_util as U

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    path = os.path.join(ROOT, "segmented_gather_gemm_amd", "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def inputs(lens, hidden, adapters, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens_t = torch.tensor(lens, device="cuda")
    start = torch.cumsum(lens_t, 0) - lens_t
    adapter = torch.randint(-1, adapters, (len(lens),), generator=g, device="cuda")
    attn = torch.randn(sum(lens), hidden, generator=g, device="cuda").to(torch.bfloat16)
    residual = torch.randn(sum(lens), hidden, generator=g, device="cuda").to(torch.bfloat16)
    return start, lens_t, adapter, attn, residual


@pytest.mark.parametrize("lens", [[1], [1] * 20, [130, 1, 77, 0, 300]])
def test_block_matches_64_bits(lens):
    """The last rounding (2^-9 relative) on top of a normalised row's, a hidden row's and an expert
    row's, each of which may fall to the other side of a tie: 4 * 2^-9 in the 2-norm."""
    M = example()
    w = M.random_weights(256, 192, 8, 3, 16)
    start, lens_t, adapter, attn, residual = inputs(lens, 256, 3, len(lens))
    before = residual.clone()
    chosen = M.block(w, attn, residual, start, lens_t, adapter, 2)
    want = M.block_in_64_bits(w, attn, before, start, lens_t, adapter, chosen)
    assert float((residual.double() - want).norm() / want.norm()) < 4 * 2.0 ** -9


@pytest.mark.parametrize("lens", [[1] * 12, [200, 61, 300]])
def test_graph_replays_match_eager(lens):
    M = example()
    w = M.random_weights(256, 192, 8, 3, 16)
    start, lens_t, adapter, attn, first = inputs(lens, 256, 3, 7)
    eager = first.clone()
    M.block(w, attn, eager, start, lens_t, adapter, 2)
    residual = first.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.block(w, attn, residual, start, lens_t, adapter, 2)
    for replay in range(4):
        residual.copy_(first)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(residual, eager), f"replay {replay}"
        other = first.clone()
        M.block(w, attn, other, start, lens_t, adapter, 2)
        torch.cuda.synchronize()
        assert torch.equal(other, eager)


def test_calls_on_another_stream():
    """Enqueued on the current stream: work on two streams, each after its own inputs."""
    M = example()
    w = M.random_weights(256, 192, 8, 3, 16)
    cases = [inputs([40, 1, 90], 256, 3, s) for s in (1, 2)]
    want = []
    for start, lens_t, adapter, attn, residual in cases:
        r = residual.clone()
        M.block(w, attn, r, start, lens_t, adapter, 2)
        want.append(r)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for s, (start, lens_t, adapter, attn, residual) in zip(streams, cases):
        with torch.cuda.stream(s):
            r = residual.clone()
            M.block(w, attn, r, start, lens_t, adapter, 2)
            got.append(r)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_results_do_not_depend_on_the_run():
    M = example()
    w = M.random_weights(256, 192, 8, 3, 16)
    start, lens_t, adapter, attn, first = inputs([300, 2, 77], 256, 3, 3)
    runs = []
    for _ in range(3):
        r = first.clone()
        M.block(w, attn, r, start, lens_t, adapter, 2)
        runs.append(r)
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])


@pytest.mark.parametrize("T", [16, 31, 64, 200])
def test_results_do_not_depend_on_the_run_with_many_segments(T):
    """Several adapters in a tile, their segments spread over a table of 1000 (most empty), so that
    several waves find them: float32 results, the same bits every time."""
    import segmented_gather_gemm_amd as sg
    g = torch.Generator(device="cuda").manual_seed(T)
    H, N, K, L, B = 520, 128, 16, 40, 1000
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(N, H, generator=g, device="cuda").to(torch.bfloat16)
    la, lb = torch.randn(L, K, H, generator=g, device="cuda").to(torch.bfloat16), torch.randn(L, N, K, generator=g, device="cuda").to(torch.bfloat16)
    lens, start = torch.zeros(B, dtype=torch.int64, device="cuda"), torch.zeros(B, dtype=torch.int64, device="cuda")
    at = torch.randperm(B, generator=g, device="cuda")[:T]
    lens[at], start[at] = 1, torch.arange(T, device="cuda")
    idx = torch.randint(-1, L, (B,), generator=g, device="cuda")
    first = None
    for run in range(200):
        o = torch.zeros(T, N, dtype=torch.float32, device="cuda")
        sg.sgmv_lora_linear(x, w, [(la, lb, 0)], o, start, lens, idx, B, 1)
        first = o if first is None else first
        assert torch.equal(o, first), f"run {run}"


def test_outputs_past_32_bit_offsets():
    """An output of more than 2^32 bytes, and gathered inputs of more than 2^31: rows from both ends."""
    import segmented_gather_gemm_amd as sg
    T, H, N, K = 140000, 64, 16384, 8
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(N, H, generator=g, device="cuda") / 8).to(torch.bfloat16)
    la, lb = torch.randn(2, K, H, generator=g, device="cuda").to(torch.bfloat16), torch.randn(2, N, K, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    start, lens, idx = [0, 1000], [1000, T - 1000], [1, 0]
    i64 = lambda v: torch.tensor(v, dtype=torch.int64, device="cuda")  # noqa: E731
    print("lora_linear of 4.6 GB", flush=True)
    sg.sgmv_lora_linear(x, w, [(la, lb, 0)], out, i64(start), i64(lens), i64(idx), 2, T)
    for rows, a in (([0, 999], 1), ([1000, 70000, 131072, T - 1], 0)):
        want, bound = U.lora_linear(x[rows], w, None, [(la, lb, 0)], [0], [len(rows)], [a], 1.0, None, False, torch.bfloat16)
        U.assert_within(out[rows], want, bound)
    wide = out                                                     # (140000, 16384): 4.6 GB of inputs
    we = (torch.randn(2, 24, N, generator=g, device="cuda") / 128).to(torch.bfloat16)
    pick = [T - 1, 0, 131072, 65536, T - 2]
    y = torch.zeros(5, 24, dtype=torch.float32, device="cuda")
    print("grouped_gemm gathering from 4.6 GB", flush=True)
    sg.sgmv_grouped_gemm(wide, we, y, i64([0, 2]), i64([2, 3]), None, 2, 3, row_indices_tensor=i64(pick))
    want, bound, _ = U.grouped(wide[pick], we, [0, 2], [2, 3], None, None, False, y)
    U.assert_within(y, want, bound)


def test_wrappers_check_their_tensors():
    import segmented_gather_gemm_amd as sg
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="bias"):
        sg.sgmv_lora_linear(x, x, [], torch.zeros(4, 4, dtype=torch.bfloat16, device="cuda"), i, i, i, 0, 0,
                            bias=torch.zeros(3, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="shorter"):
        sg.sgmv_grouped_gemm(x, x[None], torch.zeros(4, 4, dtype=torch.bfloat16, device="cuda"), i, i, None, 5, 1)
    with pytest.raises(ValueError, match="row_indices"):
        sg.sgmv_grouped_gemm(x, x[None], torch.zeros(4, 4, dtype=torch.bfloat16, device="cuda"), i, i, None, 1, 1,
                             row_indices_tensor=i[:2])
    with pytest.raises(ValueError, match="experts"):
        sg.sgmv_route(x, torch.zeros(4, 2, device="cuda"), i, i, i, i, i)
    with pytest.raises(ValueError, match="workspace"):
        sg.sgmv_lora_linear(x, x, [(x[None], x[None], 0)], torch.zeros(4, 4, dtype=torch.bfloat16, device="cuda"),
                            i, i, i, 1, 1, workspace=torch.zeros(8, device="cuda"))
    with pytest.raises(NotImplementedError):
        sg.sgmv_lora_linear(x.float(), x.float(), [], torch.zeros(4, 4, device="cuda"), i, i, i, 0, 0)
