"""The expert routing and the weighted row sum on the GPU, against their plain
64-bit forms (matmul_util): whole numbers equal, weights within the error of
a float32 exponential and a sum of up to 1024 of them."""
import numpy as np
import pytest
import torch

import matmul_util as U

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def run_route(logits, k, renormalize):
    import segmented_gather_gemm_amd as sg
    T, E = logits.shape
    mk = dict(dtype=torch.int64, device="cuda")
    w = torch.full((T, k), -5.0, device="cuda")
    e, s = torch.full((T, k), -7, **mk), torch.full((T, k), -7, **mk)
    rows, start, lens = torch.full((T * k,), -7, **mk), torch.full((E,), -7, **mk), torch.full((E,), -7, **mk)
    print(f"route T={T} E={E} k={k} {logits.dtype}", flush=True)
    sg.sgmv_route(logits, w, e, s, rows, start, lens, renormalize=renormalize)
    return w, e, s, rows, start, lens


def check(logits, k, renormalize):
    got = run_route(logits, k, renormalize)
    want = U.route(logits, k, renormalize)
    for g, r, name in zip(got[1:], want[1:], ("experts", "slots", "rows", "start", "lens")):
        assert np.array_equal(g.cpu().numpy(), r), name
    # the exponential's argument is off by 2^-24 of the logits' size, the exponential by a few units
    E = logits.shape[1]
    x = logits.double().cpu().numpy()
    size = np.max(np.abs(np.where(np.isfinite(x), x, 0)), initial=1.0)
    tol = (8 + 4 * size + E / 16) * 2.0 ** -23
    err = np.abs(got[0].double().cpu().numpy() - want[0])
    assert np.all(err <= tol * want[0] + 1e-37), err.max()


@pytest.mark.parametrize("T", [1, 2, 31, 64, 65, 200, 1000, 4100])
@pytest.mark.parametrize("E,k,renormalize", [(8, 2, False), (64, 6, True), (128, 8, False)])
def test_route_tokens(T, E, k, renormalize):
    gen = torch.Generator().manual_seed(T)
    check((torch.randn(T, E, generator=gen) * 2).cuda(), k, renormalize)


@pytest.mark.parametrize("E", [1, 2, 7, 16, 17, 33, 63, 129, 256, 257, 500, 513, 1024])
@pytest.mark.parametrize("k", [1, 3, 16, 20, 32])
def test_route_experts(E, k):
    if k <= E:
        gen = torch.Generator().manual_seed(E)
        check((torch.randn(150, E, generator=gen) * 2).cuda(), k, k == 3)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_ties_go_to_the_lowest_expert(dtype, renormalize):
    gen = torch.Generator().manual_seed(5)
    logits = torch.randint(-2, 3, (300, 60), generator=gen).to(dtype).cuda()
    check(logits, 8, renormalize)
    check(torch.zeros(130, 40, dtype=dtype, device="cuda"), 5, renormalize)


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("T", [40, 700])
def test_route_closed_experts(T, renormalize):
    """-inf and NaN close an expert; rows with fewer open experts than choices, and with none."""
    gen = torch.Generator().manual_seed(T)
    logits = torch.randn(T, 48, generator=gen)
    logits[torch.rand(T, 48, generator=gen) < 0.9] = -float("inf")
    logits[torch.rand(T, 48, generator=gen) < 0.02] = float("nan")
    logits[3], logits[T - 1] = -float("inf"), float("nan")
    check(logits.cuda(), 6, renormalize)


@pytest.mark.parametrize("renormalize", [False, True])
def test_route_extreme_logits(renormalize):
    big = torch.finfo(F32).max
    logits = torch.tensor([[big, -big, 0.0, big], [-big, -big, -big, -big], [float("inf"), 1.0, float("inf"), 2.0],
                           [-1e30, 1e30, 0.0, 5.0], [1e-40, 0.0, -1e-40, 2e-40]]).cuda()
    check(logits, 3, renormalize)


def test_route_strided_logits_and_own_workspace():
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(9)
    wide = torch.randn(900, 75, generator=gen).cuda()
    check(wide[:, 3:70], 4, True)
    logits = wide[:, :64].contiguous()
    mk = dict(dtype=torch.int64, device="cuda")
    outs = [torch.empty(900, 4, device="cuda"), torch.empty(900, 4, **mk), torch.empty(900, 4, **mk),
            torch.empty(3600, **mk), torch.empty(64, **mk), torch.empty(64, **mk)]
    ws = torch.full((sg.route_workspace_bytes(900, 64, 4),), 255, dtype=torch.uint8, device="cuda")
    sg.sgmv_route(logits, *outs, workspace=ws)
    for a, b in zip(outs, run_route(logits, 4, False)):
        assert torch.equal(a, b)


def test_route_no_tokens():
    got = run_route(torch.empty(0, 9, device="cuda"), 2, False)
    assert got[4].tolist() == [0] * 9 and got[5].tolist() == [0] * 9


@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (5, 2, 64), (33, 6, 200), (130, 8, 1032), (9, 3, 13), (70, 4, 1)])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F32), (F32, F32), (F32, BF16), (BF16, F16)])
@pytest.mark.parametrize("add", [False, True])
def test_combine(T, k, H, dtype, out, add):
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(H)
    rows = torch.randn(T * k, H, generator=gen).to(dtype).cuda()
    w = torch.rand(T, k, generator=gen).cuda()
    slots = torch.randperm(T * k, generator=gen).reshape(T, k)
    slots[torch.rand(T, k, generator=gen) < 0.1] = -1
    slots[0, 0] = T * k  # past the rows: adds nothing
    o = torch.randn(T, H, generator=gen).to(out).cuda()
    o0 = o.clone()
    print(f"combine T={T} k={k} H={H} {dtype}->{out}", flush=True)
    sg.sgmv_combine(rows, w, slots.cuda(), o, add_inputs=add)
    want, bound = U.combine(rows, w, slots, o0, add)
    U.assert_within(o, want, bound)


def test_combine_strided_and_no_choices():
    import segmented_gather_gemm_amd as sg
    gen = torch.Generator().manual_seed(2)
    rows = torch.randn(40, 75, generator=gen).cuda()[:, 2:66]
    full = torch.full((20, 70), 7.0, dtype=BF16, device="cuda")
    o = full[:, 1:65]
    w, slots = torch.rand(20, 2, generator=gen).cuda(), torch.arange(40).reshape(20, 2)
    sg.sgmv_combine(rows, w, slots.cuda(), o)
    want, bound = U.combine(rows, w, slots, o, False)
    U.assert_within(o, want, bound)
    assert bool((full[:, 0] == 7.0).all()) and bool((full[:, 65:] == 7.0).all())
    none = torch.empty(20, 0, device="cuda")
    sg.sgmv_combine(rows, none, torch.empty(20, 0, dtype=torch.int64, device="cuda"), o)
    assert bool((o == 0).all())
