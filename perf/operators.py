"""The projection, expert and routing operators as they are measured.

Each case is one pass through one of four operators of a serving step:

* ``lora_linear``   a shared projection with the low-rank adapters of many requests beside it;
* ``grouped_gemm``  matrix products grouped by expert over ragged row counts, plain or gated (SiLU);
* ``route``         the top-k choice of experts for every token and the expert-ordered row layout;
* ``combine``       the weighted sum of a token's expert rows.

``run`` computes them in plain torch operations in 32 bits, or through this
repository's package where ``own`` is true.  ``exact`` computes the same
outputs in 64 bits.
"""
import math

import numpy as np
import torch
import torch.nn.functional as F

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    """Sizes follow the repository's workloads (hidden 4096; widths 4096, 6144 = 4096 + 1024 + 1024
    and 28672 = 2 * 14336; segments U[64, 512] and U[1, 512]; ranks 16 and 64) or are generic."""
    return [
        # One request, one new token: a 4096-wide projection with its adapter.  Latency; 34 MB of weights.
        dict(name="lora_token", op="lora_linear", tokens=1, batches=1, shortest=1, longest=1, hidden=4096, widths="4096",
             rank=16, adapters=4, dtype="bf16", out="bf16", bias=False),
        # A decode step of 64 requests through the fused QKV projection, 32 adapters.
        dict(name="lora_decode_qkv", op="lora_linear", tokens=64, batches=64, shortest=1, longest=1, hidden=4096, widths="4096,1024,1024",
             rank=16, adapters=32, dtype="bf16", out="bf16", bias=False),
        # A prefill of 11 prompts at odd sizes: hidden and width that are no multiple of a tile, rank 24, a bias, float32 results.
        dict(name="lora_prefill_odd", op="lora_linear", tokens=2501, batches=11, shortest=1, longest=512, hidden=2056, widths="5000",
             rank=24, adapters=5, dtype="f16", out="f32", bias=True),
        # A large prefill batch through the fused gate/up projection: 64 prompts of 1 to 512 tokens, 64 adapters of rank 64.
        dict(name="lora_prefill_gate_up", op="lora_linear", tokens=16384, batches=64, shortest=1, longest=512, hidden=4096, widths="14336,14336",
             rank=64, adapters=64, dtype="bf16", out="bf16", bias=False),
        # A decode step of 8 requests through many small experts' gated products: most experts get no row, the others one or two.
        dict(name="experts_decode_up", op="grouped_gemm", tokens=8, choices=2, experts=32, skew=0.0, hidden=2048, width=1408, gated=True,
             gather=True, dtype="bf16", out="bf16"),
        # A prefill through 64 small experts with uneven loads, 6 choices a token.
        dict(name="experts_ragged_up", op="grouped_gemm", tokens=1000, choices=6, experts=64, skew=0.5, hidden=2048, width=1408, gated=True,
             gather=True, dtype="f16", out="f16"),
        # A large prefill through 8 wide experts: gate and up with their gate applied, rows gathered from the tokens.
        dict(name="experts_prefill_up", op="grouped_gemm", tokens=4096, choices=2, experts=8, skew=0.0, hidden=4096, width=14336, gated=True,
             gather=True, dtype="bf16", out="bf16"),
        # The same prefill's down products, on rows already in the experts' order.
        dict(name="experts_prefill_down", op="grouped_gemm", tokens=4096, choices=2, experts=8, skew=0.0, hidden=14336, width=4096, gated=False,
             gather=False, dtype="bf16", out="bf16"),
        # Routing of a decode step of 32 requests over 64 experts.
        dict(name="route_decode", op="route", tokens=32, experts=64, choices=6, renormalize=False, masked=0.0, dtype="f32"),
        # Routing of a large prefill over 128 experts, a tenth of them closed to each token and some rows of padding without any.
        dict(name="route_prefill", op="route", tokens=16384, experts=128, choices=8, renormalize=True, masked=0.1, dtype="bf16"),
        # The experts' rows of a decode step of 32 requests, summed for each token.
        dict(name="combine_decode", op="combine", tokens=32, choices=6, hidden=2048, dropped=0.0, dtype="bf16", out="bf16"),
        # The same for a large prefill, some choices without an expert.
        dict(name="combine_prefill", op="combine", tokens=16384, choices=8, hidden=2048, dropped=0.02, dtype="bf16", out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: token counts from one to 16384, sizes log-uniform, odd multiples of eight among them."""
    op = rng.choice(["lora_linear", "lora_linear", "grouped_gemm", "grouped_gemm", "route", "combine"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    while True:
        tokens = _log(rng, 1, 16384)
        if op == "lora_linear":
            batches = max(1, min(_log(rng, 1, 256), tokens))
            widths = [8 * _log(rng, 64, 1792) for _ in range(rng.randint(1, 3))]
            case = dict(op=op, tokens=tokens, batches=batches, shortest=1, longest=max(1, 2 * tokens // batches), hidden=8 * _log(rng, 64, 1024),
                        widths=",".join(map(str, widths)), rank=rng.choice([8, 16, 24, 32, 64, 128]), adapters=_log(rng, 1, 64), dtype=dtype,
                        out=rng.choice([dtype, dtype, "f32"]), bias=rng.random() < 0.3)
        elif op == "grouped_gemm":
            experts = _log(rng, 2, 128)
            gated = rng.random() < 0.5
            case = dict(op=op, tokens=tokens, choices=rng.randint(1, min(8, experts)), experts=experts, skew=rng.choice([0.0, 0.0, 0.5]),
                        hidden=8 * _log(rng, 64, 1024), width=8 * _log(rng, 64, 1792), gated=gated, gather=rng.random() < 0.7, dtype=dtype,
                        out=rng.choice([dtype, dtype, "f32"]))
        elif op == "route":
            experts = _log(rng, 4, 256)
            case = dict(op=op, tokens=tokens, experts=experts, choices=rng.randint(1, min(8, experts)), renormalize=rng.random() < 0.5,
                        masked=rng.choice([0.0, 0.1, 0.5]), dtype=rng.choice(["f32", "f32", "bf16", "f16"]))
        else:
            case = dict(op=op, tokens=tokens, choices=rng.randint(1, 8), hidden=8 * _log(rng, 64, 512), dropped=rng.choice([0.0, 0.02, 0.3]),
                        dtype=dtype, out=rng.choice([dtype, dtype, "f32"]))
        w = work(case)
        sizes = [case["tokens"], case.get("hidden", 0), case.get("width", 0)] + (widths if op == "lora_linear" else [])
        if w["flops"] <= 2e12 and w["bytes"] <= 1.2e9 and 3072 not in sizes:  # below the largest listed ones
            return case


# --------------------------------------------------------------------------
# Inputs.
# --------------------------------------------------------------------------

def _lengths(case, rng):
    """Segment lengths in [shortest, longest] that sum to the tokens."""
    B, T = case["batches"], case["tokens"]
    lens = rng.integers(case["shortest"], case["longest"] + 1, size=B).astype(np.int64)
    lens = np.maximum(1, lens * T // max(1, int(lens.sum())))
    while int(lens.sum()) != T:  # the rest goes to (or comes from) one segment after another
        rest = T - int(lens.sum())
        step = np.zeros(B, dtype=np.int64)
        able = np.flatnonzero(lens > 1) if rest < 0 else np.arange(B)
        step[able[:abs(rest)]] = 1 if rest > 0 else -1
        lens += step
    return rng.permutation(lens)


def _choices(case, rng):
    """(tokens, choices) distinct experts of every token, the first experts more loaded where `skew` says so."""
    T, E, k = case["tokens"], case["experts"], case["choices"]
    logp = -case["skew"] * np.log(np.arange(1, E + 1))
    keys = logp[None, :] + rng.gumbel(size=(T, E))
    return np.argsort(-keys, axis=1, kind="stable")[:, :k].astype(np.int64)


def _starts(lens):
    return np.concatenate([[0], np.cumsum(lens)[:-1]]).astype(np.int64)


def _device(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEVICE)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEVICE).manual_seed(seed)

    def normal(*shape, sigma=1.0, dtype=None):
        return torch.randn(*shape, generator=gen, device=DEVICE, dtype=dtype or DTYPES[case["dtype"]]).mul_(sigma)

    s = dict(case)
    op, T = case["op"], case["tokens"]
    if op == "lora_linear":
        H, K, L = case["hidden"], case["rank"], case["adapters"]
        widths = [int(v) for v in case["widths"].split(",")]
        lens = _lengths(case, rng)
        s["max_len"] = int(lens.max())
        s["start"], s["lens"] = _device(_starts(lens)), _device(lens)
        # one request in L + 1 runs on the shared projection alone
        s["idx"] = _device(rng.integers(-1, L, size=len(lens)).astype(np.int64))
        s["x"] = normal(T, H)
        s["w"] = normal(sum(widths), H, sigma=H ** -0.5)
        s["bias_v"] = normal(sum(widths), sigma=0.1) if case["bias"] else None
        s["slices"], at = [], 0
        for n in widths:
            s["slices"].append((normal(L, K, H, sigma=H ** -0.5), normal(L, n, K, sigma=0.02), at))
            at += n
        s["scale"] = 2.0
        s["out_t"] = torch.empty(T, sum(widths), dtype=DTYPES[case["out"]], device=DEVICE)
    elif op == "grouped_gemm":
        E, H, N = case["experts"], case["hidden"], case["width"]
        chosen = _choices(case, rng).reshape(-1)
        order = np.argsort(chosen, kind="stable")
        lens = np.bincount(chosen, minlength=E).astype(np.int64)
        s["max_len"] = int(lens.max())
        s["start"], s["lens"] = _device(_starts(lens)), _device(lens)
        s["rows"] = _device(order // case["choices"]) if case["gather"] else None
        s["x"] = normal(T if case["gather"] else len(order), H)
        s["w"] = normal(E, 2 * N if case["gated"] else N, H, sigma=H ** -0.5)
        s["out_t"] = torch.empty(len(order), N, dtype=DTYPES[case["out"]], device=DEVICE)
    elif op == "route":
        E, k = case["experts"], case["choices"]
        logits = normal(T, E, sigma=2.0, dtype=torch.float32).to(DTYPES[case["dtype"]])
        if case["masked"]:
            shut = torch.rand(T, E, generator=gen, device=DEVICE) < case["masked"]
            shut |= torch.rand(T, 1, generator=gen, device=DEVICE) < 0.02  # padding: no expert at all
            logits.masked_fill_(shut, -math.inf)
        s["logits"] = logits
        i64 = dict(dtype=torch.int64, device=DEVICE)
        s["weights"] = torch.empty(T, k, dtype=torch.float32, device=DEVICE)
        s["chosen"], s["slots"] = torch.empty(T, k, **i64), torch.empty(T, k, **i64)
        s["rows"], s["start"], s["lens"] = torch.empty(T * k, **i64), torch.empty(E, **i64), torch.empty(E, **i64)
    else:
        k, H = case["choices"], case["hidden"]
        slots = rng.permutation(T * k).reshape(T, k).astype(np.int64)
        gone = rng.random((T, k)) < case["dropped"]
        s["slots"] = _device(np.where(gone, -1, slots))
        weights = torch.rand(T, k, generator=gen, device=DEVICE) + 0.05
        s["weights"] = weights / weights.sum(dim=1, keepdim=True)
        s["rows"] = normal(T * k, H)
        s["out_t"] = torch.empty(T, H, dtype=DTYPES[case["out"]], device=DEVICE)
    return s


# --------------------------------------------------------------------------
# One pass.
# --------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import segmented_gather_gemm_amd as sg
    op = s["op"]
    if op == "lora_linear":
        return sg.sgmv_lora_linear(s["x"], s["w"], s["slices"], s["out_t"], s["start"], s["lens"], s["idx"], s["batches"], s["max_len"],
                                   scaling=s["scale"], bias=s["bias_v"])
    if op == "grouped_gemm":
        return sg.sgmv_grouped_gemm(s["x"], s["w"], s["out_t"], s["start"], s["lens"], None, s["experts"], s["max_len"],
                                    row_indices_tensor=s["rows"], gated=s["gated"])
    if op == "route":
        sg.sgmv_route(s["logits"], s["weights"], s["chosen"], s["slots"], s["rows"], s["start"], s["lens"], renormalize=s["renormalize"])
        return {"weights": s["weights"], "chosen": s["chosen"], "slots": s["slots"], "rows": s["rows"], "start": s["start"], "lens": s["lens"]}
    return sg.sgmv_combine(s["rows"], s["weights"], s["slots"], s["out_t"])


def _plain(s):
    return {"lora_linear": _plain_lora_linear, "grouped_gemm": _plain_grouped_gemm, "route": _plain_route, "combine": _plain_combine}[s["op"]](s)


def _padded(s, rows):
    """(segments, longest) row numbers of every segment, clamped to `rows`, and which of them are real."""
    at = torch.arange(s["max_len"], device=DEVICE)[None, :]
    real = at < s["lens"][:, None]
    return (s["start"][:, None] + at).clamp(0, rows - 1), real


def _plain_lora_linear(s):
    x = s["x"].float()
    out = x @ s["w"].float().t()
    if s["bias_v"] is not None:
        out = out + s["bias_v"].float()
    at, real = _padded(s, s["tokens"])
    real = real & (s["idx"] >= 0)[:, None]
    own_a = s["idx"].clamp(min=0)
    xs = x[at]                                                       # (segments, longest, hidden)
    for a, b, off in s["slices"]:
        v = torch.bmm(xs, a[own_a].float().transpose(1, 2).contiguous())
        d = torch.bmm(v, b[own_a].float().transpose(1, 2).contiguous()) * s["scale"]
        out[:, off:off + b.shape[1]].index_put_((at[real],), d[real], accumulate=True)
    return out.to(s["out_t"].dtype)


def _plain_grouped_gemm(s):
    x, N = s["x"].float(), s["width"]
    rows = s["out_t"].shape[0]
    at, real = _padded(s, rows)
    src = at if s["rows"] is None else s["rows"][at]
    y = torch.bmm(x[src], s["w"].float().transpose(1, 2).contiguous())  # (experts, longest, width)
    if s["gated"]:
        g, u = y[..., :N], y[..., N:]
        y = g / (1 + torch.exp(-g)) * u
    out = torch.empty(rows, N, device=DEVICE)
    out[at[real]] = y[real]
    return out.to(s["out_t"].dtype)


def _plain_route(s):
    T, E, k = s["tokens"], s["experts"], s["choices"]
    x = s["logits"].float()
    best, chosen = torch.sort(x, dim=1, descending=True, stable=True)   # ties: lowest expert first
    best, chosen = best[:, :k], chosen[:, :k]
    there = best > -math.inf
    top = best[:, :1].clamp(min=-3e38)                                  # finite where every expert is closed
    over = torch.exp(best - top).sum(dim=1, keepdim=True) if s["renormalize"] else torch.exp(x - top).sum(dim=1, keepdim=True)
    weights = torch.where(there, torch.exp(best - top) / over, torch.zeros_like(best))
    chosen = torch.where(there, chosen, torch.full_like(chosen, -1))
    flat = torch.where(there, chosen, torch.full_like(chosen, E)).reshape(-1)
    order = torch.sort(flat, stable=True)[1]                            # choices in order of expert, then token
    n = torch.arange(T * k, device=DEVICE)
    slots = torch.empty_like(n)
    slots[order] = n
    slots = torch.where(there.reshape(-1), slots, torch.full_like(slots, -1)).reshape(T, k)
    lens = torch.bincount(flat, minlength=E + 1)[:E]
    start = torch.cumsum(lens, 0) - lens
    rows = torch.where(n < lens.sum(), order // k, torch.full_like(n, -1))
    return {"weights": weights, "chosen": chosen, "slots": slots, "rows": rows, "start": start, "lens": lens}


def _plain_combine(s):
    there = s["slots"] >= 0
    rows = s["rows"].float()[s["slots"].clamp(min=0)]                   # (tokens, choices, hidden)
    w = torch.where(there, s["weights"], torch.zeros_like(s["weights"]))
    return (rows * w[..., None]).sum(dim=1).to(s["out_t"].dtype)


# --------------------------------------------------------------------------
# The definitions in 64 bits, segment by segment and choice by choice.
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "lora_linear":
        x = s["x"].double()
        out = F.linear(x, s["w"].double(), None if s["bias_v"] is None else s["bias_v"].double())
        for st, n, a in zip(s["start"].tolist(), s["lens"].tolist(), s["idx"].tolist()):
            if a >= 0:
                for la, lb, off in s["slices"]:
                    out[st:st + n, off:off + lb.shape[1]] += s["scale"] * F.linear(F.linear(x[st:st + n], la[a].double()), lb[a].double())
        return out
    if op == "grouped_gemm":
        out = torch.empty(s["out_t"].shape, dtype=torch.float64, device=DEVICE)
        for e, (st, n) in enumerate(zip(s["start"].tolist(), s["lens"].tolist())):
            if n:
                x = s["x"][st:st + n] if s["rows"] is None else s["x"][s["rows"][st:st + n]]
                w = s["w"][e].double()
                y = F.linear(x.double(), w[:case["width"]])
                out[st:st + n] = F.silu(y) * F.linear(x.double(), w[case["width"]:]) if case["gated"] else y
        return out
    if op == "route":
        x = s["logits"].double().cpu().numpy()
        picked = np.argsort(-x, axis=1, kind="stable")[:, :case["choices"]]
        best = np.take_along_axis(x, picked, axis=1)
        with np.errstate(invalid="ignore"):
            total = np.logaddexp.reduce(best if case["renormalize"] else x, axis=1)[:, None]
            weights = np.where(np.isfinite(best), np.exp(best - np.where(np.isfinite(total), total, 0)), 0.0)
        return {"weights": weights, "chosen": None, "slots": None, "rows": None, "start": None, "lens": None}
    out = torch.zeros(s["out_t"].shape, dtype=torch.float64, device=DEVICE)
    for j in range(case["choices"]):
        there = (s["slots"][:, j] >= 0).nonzero()[:, 0]
        out[there] += s["weights"][there, j].double()[:, None] * s["rows"][s["slots"][there, j]].double()
    return out


def work(case):
    """What one pass cannot do without: inputs read once, outputs written once, the products' operations."""
    op, T = case["op"], case["tokens"]
    i = BYTES[case["dtype"]]
    o = BYTES[case.get("out", "f32")]
    if op == "lora_linear":
        H, K, B = case["hidden"], case["rank"], case["batches"]
        widths = [int(v) for v in case["widths"].split(",")]
        N, S, L = sum(widths), len(widths), case["adapters"]
        seen = L * (1 - (1 - 1 / (L + 1)) ** B)                       # adapters that some segment has, on average
        return {"bytes": i * (T * H + N * H + seen * K * (S * H + N)) + o * T * N,
                "flops": 2.0 * T * H * N + 2.0 * T * L / (L + 1) * K * (S * H + N)}
    if op == "grouped_gemm":
        E, H, N = case["experts"], case["hidden"], case["width"]
        wide, R = (2 * N if case["gated"] else N), T * case["choices"]
        used = E * (1 - (1 - case["choices"] / E) ** T)                # experts with a row, on average (even loads)
        return {"bytes": i * ((T if case["gather"] else R) * H + used * wide * H) + o * R * N, "flops": 2.0 * R * H * wide}
    if op == "route":
        E, k = case["experts"], case["choices"]
        return {"bytes": i * T * E + T * k * (4 + 3 * 8) + 16 * E, "flops": 5.0 * T * E}
    k, H = case["choices"], case["hidden"]
    return {"bytes": T * k * (1 - case["dropped"]) * H * i + T * k * 12 + T * H * o, "flops": 2.0 * T * k * H}
