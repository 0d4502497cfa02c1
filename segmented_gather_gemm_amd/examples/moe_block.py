"""The projection, expert and routing operators together, as a serving step
runs them: the output projection of an attention block with each request's
adapter beside it, added to the residual stream, then a block of routed
experts on the normalised result.

    python segmented_gather_gemm_amd/examples/moe_block.py

Random weights; the result is compared with the same block in plain torch
operations in 64 bits.
"""
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.dirname(os.path.abspath(__file__)))))
import segmented_gather_gemm_amd as sg  # noqa: E402


@dataclass
class Weights:
    proj: torch.Tensor      # (hidden, hidden)
    lora_a: torch.Tensor    # (adapters, rank, hidden)
    lora_b: torch.Tensor    # (adapters, hidden, rank)
    router: torch.Tensor    # (experts, hidden)
    gate_up: torch.Tensor   # (experts, 2 * width, hidden)
    down: torch.Tensor      # (experts, hidden, width)


def random_weights(hidden, width, experts, adapters, rank, seed=0, device="cuda", dtype=torch.bfloat16):
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, sigma):
        return (torch.randn(*shape, generator=g, device=device) * sigma).to(dtype)

    return Weights(normal(hidden, hidden, sigma=hidden ** -0.5), normal(adapters, rank, hidden, sigma=hidden ** -0.5),
                   normal(adapters, hidden, rank, sigma=0.1), normal(experts, hidden, sigma=hidden ** -0.5),
                   normal(experts, 2 * width, hidden, sigma=hidden ** -0.5), normal(experts, hidden, width, sigma=width ** -0.5))


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(dim=1, keepdim=True) + 1e-6)).to(x.dtype)


def block(w, attn, residual, start, lens, adapter, top_k, scale=2.0):
    """residual (tokens, hidden) is updated in place; attn holds the tokens' attention outputs, packed
    by request (start, lens), adapter the requests' adapters (-1: none)."""
    T, H = residual.shape
    E, k, dev = w.router.shape[0], top_k, residual.device
    requests, longest = lens.shape[0], T
    # x = residual + proj attn + the requests' adapters, in one rounding
    sg.sgmv_lora_linear(attn, w.proj, [(w.lora_a, w.lora_b, 0)], residual, start, lens, adapter, requests,
                        longest, scaling=scale, add_inputs=True)
    x = norm(residual)
    # choices of experts, and the choices' rows in the order of the experts
    logits = torch.empty(T, E, dtype=torch.float32, device=dev)
    sg.sgmv_lora_linear(x, w.router, [], logits, start, lens, adapter, 0, 0)
    i64 = dict(dtype=torch.int64, device=dev)
    weights, chosen, slots = torch.empty(T, k, device=dev), torch.empty(T, k, **i64), torch.empty(T, k, **i64)
    rows, e_start, e_lens = torch.empty(T * k, **i64), torch.empty(E, **i64), torch.empty(E, **i64)
    sg.sgmv_route(logits, weights, chosen, slots, rows, e_start, e_lens, renormalize=True)
    # the experts on their rows; nothing of the routing comes back to the host
    hidden = torch.empty(T * k, w.down.shape[2], dtype=x.dtype, device=dev)
    sg.sgmv_grouped_gemm(x, w.gate_up, hidden, e_start, e_lens, None, E, T, row_indices_tensor=rows, gated=True)
    out = torch.empty(T * k, H, dtype=x.dtype, device=dev)
    sg.sgmv_grouped_gemm(hidden, w.down, out, e_start, e_lens, None, E, T)
    sg.sgmv_combine(out, weights, slots, residual, add_inputs=True)
    return chosen


def block_in_64_bits(w, attn, residual, start, lens, adapter, chosen, scale=2.0):
    """The same block from its formulas, with the choices of experts given and the roundings of the
    stored tensors (residual, normalised rows, hidden rows, expert rows) where block() has them."""
    dt = residual.dtype
    x = residual.double() + attn.double() @ w.proj.double().t()
    for st, n, a in zip(start.tolist(), lens.tolist(), adapter.tolist()):
        if a >= 0:
            r = attn[st:st + n].double()
            x[st:st + n] += scale * (r @ w.lora_a[a].double().t()) @ w.lora_b[a].double().t()
    x = x.to(dt)
    y = norm(x).double()
    logits = y @ w.router.double().t()
    p = torch.softmax(torch.gather(logits, 1, chosen), dim=1)
    res = x.double().clone()
    F = w.down.shape[2]
    for e in range(w.router.shape[0]):
        t, j = (chosen == e).nonzero(as_tuple=True)
        if len(t):
            z = y[t] @ w.gate_up[e].double().t()
            h = (torch.nn.functional.silu(z[:, :F]) * z[:, F:]).to(dt).double()
            o = (h @ w.down[e].double().t()).to(dt).double()
            res.index_add_(0, t, p[t, j][:, None] * o)
    return res


def main():
    hidden, width, experts, adapters, rank, top_k = 1024, 512, 16, 6, 16, 4
    w = random_weights(hidden, width, experts, adapters, rank)
    g = torch.Generator(device="cuda").manual_seed(1)
    for name, lens in (("decode, 24 requests", [1] * 24), ("prefill, 5 prompts", [130, 1, 77, 300, 64])):
        T = sum(lens)
        lens_t = torch.tensor(lens, device="cuda")
        start = torch.cumsum(lens_t, 0) - lens_t
        adapter = torch.randint(-1, adapters, (len(lens),), generator=g, device="cuda")
        attn = torch.randn(T, hidden, generator=g, device="cuda").to(torch.bfloat16)
        residual = torch.randn(T, hidden, generator=g, device="cuda").to(torch.bfloat16)
        before = residual.clone()
        chosen = block(w, attn, residual, start, lens_t, adapter, top_k)
        want = block_in_64_bits(w, attn, before, start, lens_t, adapter, chosen)
        off = float((residual.double() - want).norm() / want.norm())
        print(f"{name}: {T} tokens, {top_k} of {experts} experts each, relative difference from 64 bits {off:.2e}")


if __name__ == "__main__":
    main()
