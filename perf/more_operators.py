"""The microscaled 4-bit operators as they are measured.

Each case is one pass through one of four operators:

* ``round_trip``  rows quantised to 4-bit codes with a scale for every 32 values, and read back;
* ``read``        rows of a 4-bit matrix read back, chosen by index or all of them;
* ``linear``      a shared projection with 4-bit weights and the low-rank adapters of many requests beside it;
* ``experts``     matrix products grouped by expert with 4-bit weights, plain or gated (SiLU).

``run`` computes them in plain torch operations in 32 bits, or through this
repository's package where ``own`` is true.  ``exact`` computes the same
outputs in 64 bits.

The format: 32 consecutive values of a row share a scale 2^e, e the exponent
of their largest magnitude less 2 (byte e + 127), and each is the nearest of
0, .5, 1, 1.5, 2, 3, 4 and 6 times it, ties to the even code, with a sign; two codes
a byte, the first in the low half.  Rows are filled up with zeros to groups of
128 values: 64 bytes of codes and 4 of scales each.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    """Sizes follow the repository's workloads (hidden 4096; widths 4096, 6144 = 4096 + 1024 + 1024
    and 28672 = 2 * 14336; segments U[1, 512]; ranks 16 and 64) or are generic."""
    return [
        # The activations of one new token: latency.
        dict(name="round_trip_token", op="round_trip", tokens=1, hidden=4096, dtype="bf16", out="bf16"),
        # A prefill's activations at an odd length, hidden size and type.
        dict(name="round_trip_odd", op="round_trip", tokens=2501, hidden=2056, dtype="f16", out="f32"),
        # A weight matrix as a checkpoint holds it, quantised at load and read back as 16 bits.
        dict(name="round_trip_weights", op="round_trip", tokens=28672, hidden=4096, dtype="f32", out="bf16"),
        # The embedding rows of a decode step of 64 requests out of a 4-bit table.
        dict(name="read_embedding", op="read", tokens=64, table=32768, hidden=4096, gather=True, out="bf16"),
        # A whole 4-bit gate/up matrix read back for a 16-bit path.
        dict(name="read_weights", op="read", tokens=28672, table=28672, hidden=4096, gather=False, out="bf16"),
        # One request, one new token: a 4096-wide projection with its adapter.  Latency; 9 MB of weights.
        dict(name="linear_token", op="linear", tokens=1, batches=1, hidden=4096, widths="4096", rank=16, adapters=4, dtype="bf16",
             out="bf16", bias=False),
        # A decode step of 64 requests through the fused QKV projection, 32 adapters.
        dict(name="linear_decode_qkv", op="linear", tokens=64, batches=64, hidden=4096, widths="4096,1024,1024", rank=16, adapters=32,
             dtype="bf16", out="bf16", bias=False),
        # A prefill of 11 prompts at odd sizes: a hidden size that is no whole number of blocks, rank 24, a bias, float32 results.
        dict(name="linear_prefill_odd", op="linear", tokens=2501, batches=11, hidden=2056, widths="5000", rank=24, adapters=5, dtype="f16",
             out="f32", bias=True),
        # A large prefill batch through the fused gate/up projection: 64 prompts, 64 adapters of rank 64.
        dict(name="linear_prefill_gate_up", op="linear", tokens=16384, batches=64, hidden=4096, widths="14336,14336", rank=64, adapters=64,
             dtype="bf16", out="bf16", bias=False),
        # A decode step of 8 requests through many small experts' gated products: most experts get no row, the others one or two.
        dict(name="experts_decode", op="experts", tokens=8, choices=2, experts=32, skew=0.0, hidden=2048, width=1408, gated=True,
             gather=True, dtype="bf16", out="bf16"),
        # A prefill through 64 small experts with uneven loads, 6 choices a token.
        dict(name="experts_ragged", op="experts", tokens=1000, choices=6, experts=64, skew=0.5, hidden=2048, width=1408, gated=True,
             gather=True, dtype="f16", out="f16"),
        # A large prefill's down products through 8 wide experts, on rows already in the experts' order.
        dict(name="experts_prefill_down", op="experts", tokens=4096, choices=2, experts=8, skew=0.0, hidden=14336, width=4096, gated=False,
             gather=False, dtype="bf16", out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _hidden(rng, hi):
    """A contraction length: whole groups of 128, multiples of eight, or any."""
    step = rng.choice([128, 8, 8, 1])
    return step * _log(rng, max(1, 64 // step), hi // step)


def draw(rng):
    """One more case: row counts from one to 16384 (28672 for whole matrices), sizes log-uniform, any hidden size."""
    op = rng.choice(["round_trip", "read", "linear", "linear", "experts", "experts"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    while True:
        tokens = _log(rng, 1, 16384)
        if op == "round_trip":
            case = dict(op=op, tokens=_log(rng, 1, 28672), hidden=_hidden(rng, 16384), dtype=rng.choice(["bf16", "f16", "f32"]),
                        out=rng.choice(["bf16", "f32"]))
        elif op == "read":
            gather = rng.random() < 0.6
            tokens = _log(rng, 1, 28672)
            case = dict(op=op, tokens=tokens, table=_log(rng, 64, 65536) if gather else tokens, hidden=_hidden(rng, 8192), gather=gather,
                        out=rng.choice(["bf16", "f16", "f32"]))
        elif op == "linear":
            batches = max(1, min(_log(rng, 1, 256), tokens))
            widths = [8 * _log(rng, 64, 1792) for _ in range(rng.randint(1, 3))]
            case = dict(op=op, tokens=tokens, batches=batches, hidden=_hidden(rng, 8192), widths=",".join(map(str, widths)),
                        rank=rng.choice([8, 16, 24, 32, 64, 128]), adapters=_log(rng, 1, 64), dtype=dtype,
                        out=rng.choice([dtype, dtype, "f32"]), bias=rng.random() < 0.3)
        else:
            experts = _log(rng, 2, 128)
            case = dict(op=op, tokens=tokens, choices=rng.randint(1, min(8, experts)), experts=experts, skew=rng.choice([0.0, 0.0, 0.5]),
                        hidden=_hidden(rng, 8192), width=8 * _log(rng, 64, 1792), gated=rng.random() < 0.5, gather=rng.random() < 0.7,
                        dtype=dtype, out=rng.choice([dtype, dtype, "f32"]))
        w = work(case)
        wide = case["experts"] * case["width"] * (2 if case["gated"] else 1) if op == "experts" else case.get("table", 0)
        # below the largest listed ones, and a table or a stack of experts that is made quickly
        if w["flops"] <= 2e12 and w["bytes"] <= 7e8 and wide * case["hidden"] <= 1.5e9:
            return case


# --------------------------------------------------------------------------
# Inputs.
# --------------------------------------------------------------------------

def _groups(hidden):
    return (hidden + 127) // 128


def _lengths(case, rng):
    """Segment lengths of at least one that sum to the tokens."""
    B, T = case["batches"], case["tokens"]
    lens = rng.integers(1, max(2, 2 * T // B), size=B).astype(np.int64)
    lens = np.maximum(1, lens * T // int(lens.sum()))
    while int(lens.sum()) != T:  # the rest goes to (or comes from) one segment after another
        rest = T - int(lens.sum())
        able = np.flatnonzero(lens > 1) if rest < 0 else np.arange(B)
        lens[able[:abs(rest)]] += 1 if rest > 0 else -1
    return rng.permutation(lens)


def _choices(case, rng):
    """(tokens, choices) distinct experts of every token, the first experts more loaded where `skew` says so."""
    T, E, k = case["tokens"], case["experts"], case["choices"]
    keys = rng.gumbel(size=(T, E)) - case["skew"] * np.log(np.arange(1, E + 1))[None, :]
    return np.argsort(-keys, axis=1, kind="stable")[:, :k].astype(np.int64)


def _starts(lens):
    return np.concatenate([[0], np.cumsum(lens)[:-1]]).astype(np.int64)


def _device(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEVICE)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEVICE).manual_seed(seed)

    def normal(*shape, sigma=1.0, dtype=None):
        return torch.randn(*shape, generator=gen, device=DEVICE, dtype=DTYPES[dtype or case["dtype"]]).mul_(sigma)

    def packed(rows, hidden, sigma):
        """4-bit weights as a checkpoint brings them: codes and scales of normal values."""
        G = _groups(hidden)
        codes = torch.empty(rows, 64 * G, dtype=torch.uint8, device=DEVICE)
        scales = torch.empty(rows, 4 * G, dtype=torch.uint8, device=DEVICE)
        step = max(1, (1 << 26) // hidden)
        for r in range(0, rows, step):
            n = min(step, rows - r)
            codes[r:r + n], scales[r:r + n] = _quantize(normal(n, hidden, sigma=sigma, dtype="bf16"))
        return codes, scales

    s = dict(case)
    op, T, H = case["op"], case["tokens"], case["hidden"]
    if op == "round_trip":
        # activations: a few channels are much larger than the others, and some rows are padding
        channels = torch.exp(torch.randn(H, generator=gen, device=DEVICE))
        x = torch.randn(T, H, generator=gen, device=DEVICE).mul_(channels)
        x.mul_((torch.rand(T, 1, generator=gen, device=DEVICE) >= 0.02) if T > 1 else 1.0)
        s["x"] = x.to(DTYPES[case["dtype"]])
        s["codes"] = torch.empty(T, 64 * _groups(H), dtype=torch.uint8, device=DEVICE)
        s["scales"] = torch.empty(T, 4 * _groups(H), dtype=torch.uint8, device=DEVICE)
        s["out_t"] = torch.empty(T, H, dtype=DTYPES[case["out"]], device=DEVICE)
    elif op == "read":
        s["codes"], s["scales"] = packed(case["table"], H, 0.02)
        s["rows"] = _device(rng.integers(0, case["table"], size=T).astype(np.int64)) if case["gather"] else None
        s["out_t"] = torch.empty(T, H, dtype=DTYPES[case["out"]], device=DEVICE)
    elif op == "linear":
        K, L = case["rank"], case["adapters"]
        widths = [int(v) for v in case["widths"].split(",")]
        lens = _lengths(case, rng)
        s["max_len"] = int(lens.max())
        s["start"], s["lens"] = _device(_starts(lens)), _device(lens)
        # one request in L + 1 runs on the shared projection alone
        s["idx"] = _device(rng.integers(-1, L, size=len(lens)).astype(np.int64))
        s["x"] = normal(T, H)
        s["codes"], s["scales"] = packed(sum(widths), H, H ** -0.5)
        s["bias_v"] = normal(sum(widths), sigma=0.1) if case["bias"] else None
        s["slices"], at = [], 0
        for n in widths:
            s["slices"].append((normal(L, K, H, sigma=H ** -0.5), normal(L, n, K, sigma=0.02), at))
            at += n
        s["scale"] = 2.0
        s["out_t"] = torch.empty(T, sum(widths), dtype=DTYPES[case["out"]], device=DEVICE)
    else:
        E, N = case["experts"], case["width"]
        chosen = _choices(case, rng).reshape(-1)
        order = np.argsort(chosen, kind="stable")
        lens = np.bincount(chosen, minlength=E).astype(np.int64)
        s["max_len"] = int(lens.max())
        s["start"], s["lens"] = _device(_starts(lens)), _device(lens)
        s["rows"] = _device(order // case["choices"]) if case["gather"] else None
        s["x"] = normal(T if case["gather"] else len(order), H)
        wide = 2 * N if case["gated"] else N
        codes, scales = packed(E * wide, H, H ** -0.5)
        s["codes"], s["scales"] = codes.view(E, wide, -1), scales.view(E, wide, -1)
        s["out_t"] = torch.empty(len(order), N, dtype=DTYPES[case["out"]], device=DEVICE)
    return s


# --------------------------------------------------------------------------
# One pass.
# --------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import segmented_gather_gemm_amd as sg
    op = s["op"]
    if op == "round_trip":
        sg.sgmv_mx_quantize(s["x"], s["codes"], s["scales"])
        return sg.sgmv_mx_dequantize(s["codes"], s["scales"], s["out_t"])
    if op == "read":
        return sg.sgmv_mx_dequantize(s["codes"], s["scales"], s["out_t"], row_indices_tensor=s["rows"])
    if op == "linear":
        return sg.sgmv_mx_lora_linear(s["x"], s["codes"], s["scales"], s["slices"], s["out_t"], s["start"], s["lens"], s["idx"],
                                      s["batches"], s["max_len"], scaling=s["scale"], bias=s["bias_v"])
    return sg.sgmv_mx_grouped_gemm(s["x"], s["codes"], s["scales"], s["out_t"], s["start"], s["lens"], None, s["experts"], s["max_len"],
                                   row_indices_tensor=s["rows"], gated=s["gated"])


def _plain(s):
    return {"round_trip": _plain_round_trip, "read": _plain_read, "linear": _plain_linear, "experts": _plain_experts}[s["op"]](s)


def _quantize(x):
    """Codes and scales of rows x; powers of two and the roundings to the grid are exact in 32 bits."""
    T, H = x.shape
    G = _groups(H)
    v = torch.zeros(T, 128 * G, device=x.device)
    v[:, :H] = x
    v = v.view(T, 4 * G, 32)
    e = torch.frexp(v.abs().amax(dim=2))[1].to(torch.int32) - 3
    e = torch.where(v.abs().amax(dim=2) > 0, e, torch.full_like(e, -127)).clamp(min=-127)
    y = torch.ldexp(v.abs(), -e[..., None])
    # spacing 1/2 below 2, 1 below 4, 2 above; torch rounds halves to even, which is the even code
    q = torch.where(y < 2, torch.round(y * 2) / 2, torch.where(y < 4, torch.round(y), torch.round(y / 2) * 2)).clamp(max=6)
    code = torch.where(q < 2, q * 2, torch.where(q < 4, q + 2, q / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).view(T, 64 * G, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8)


def _values(codes, scales, hidden):
    """The float32 values that codes and scales stand for, (..., hidden)."""
    c = torch.stack((codes & 15, codes >> 4), dim=-1).to(torch.int32).view(*scales.shape, 32)
    m = c & 7
    v = torch.where(m < 4, m.float() / 2, torch.where(m < 6, m.float() - 2, 2 * m.float() - 8))
    v = torch.where(c >= 8, -v, v)
    return torch.ldexp(v, (scales.to(torch.int32) - 127)[..., None]).flatten(-2)[..., :hidden]


def _plain_round_trip(s):
    return _values(*_quantize(s["x"]), s["hidden"]).to(s["out_t"].dtype)


def _plain_read(s):
    codes, scales = (s["codes"], s["scales"]) if s["rows"] is None else (s["codes"][s["rows"]], s["scales"][s["rows"]])
    return _values(codes, scales, s["hidden"]).to(s["out_t"].dtype)


def _padded(s, rows):
    """(segments, longest) row numbers of every segment, clamped to `rows`, and which of them are real."""
    at = torch.arange(s["max_len"], device=DEVICE)[None, :]
    real = at < s["lens"][:, None]
    return (s["start"][:, None] + at).clamp(0, rows - 1), real


def _plain_linear(s):
    H = s["hidden"]
    out = _values(*_quantize(s["x"]), H) @ _values(s["codes"], s["scales"], H).t()
    if s["bias_v"] is not None:
        out = out + s["bias_v"].float()
    at, real = _padded(s, s["tokens"])
    real = real & (s["idx"] >= 0)[:, None]
    own_a = s["idx"].clamp(min=0)
    xs = s["x"].float()[at]                                          # (segments, longest, hidden)
    for a, b, off in s["slices"]:
        v = torch.bmm(xs, a[own_a].float().transpose(1, 2).contiguous())
        d = torch.bmm(v, b[own_a].float().transpose(1, 2).contiguous()) * s["scale"]
        out[:, off:off + b.shape[1]].index_put_((at[real],), d[real], accumulate=True)
    return out.to(s["out_t"].dtype)


def _plain_experts(s):
    x, N = _values(*_quantize(s["x"]), s["hidden"]), s["width"]
    rows = s["out_t"].shape[0]
    at, real = _padded(s, rows)
    src = at if s["rows"] is None else s["rows"][at]
    y = torch.bmm(x[src], _values(s["codes"], s["scales"], s["hidden"]).transpose(1, 2).contiguous())  # (experts, longest, width)
    if s["gated"]:
        g, u = y[..., :N], y[..., N:]
        y = g / (1 + torch.exp(-g)) * u
    out = torch.empty(rows, N, device=DEVICE)
    out[at[real]] = y[real]
    return out.to(s["out_t"].dtype)


# --------------------------------------------------------------------------
# The definitions in 64 bits, segment by segment.
# --------------------------------------------------------------------------

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_rounded(x):
    """Rows x with each block of 32 rounded to its 4-bit values, in float64: each magnitude by where it lies
    between the grid's midpoints (one that is a midpoint goes to the even code)."""
    T, H = x.shape
    out = torch.empty(T, H, dtype=torch.float64, device=x.device)
    grid = torch.tensor(_GRID, dtype=torch.float64, device=x.device)
    for at in range(0, H, 32):
        v = x[:, at:at + 32].double()
        top = v.abs().amax(dim=1, keepdim=True)
        unit = torch.exp2(torch.floor(torch.log2(top)) - 2)
        unit = torch.where(unit * 8 <= top, unit * 2, torch.where(unit * 4 > top, unit / 2, unit))  # log2's own rounding
        unit = torch.where(top > 0, unit, torch.ones_like(unit)).clamp(min=2.0 ** -127)
        y = v.abs() / unit
        code = ((y > 0.25).long() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
        out[:, at:at + 32] = torch.copysign(grid[code] * unit, v)
    return out


def _exact_values(codes, scales, hidden):
    table = torch.tensor(_GRID + tuple(-v for v in _GRID), dtype=torch.float64, device=codes.device)
    out = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    out[:, 0::2] = table[(codes % 16).long()]
    out[:, 1::2] = table[(codes // 16).long()]
    return (out * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=1))[:, :hidden]


def exact(case, seed):
    s = prepare(case, seed)
    op, H = case["op"], case["hidden"]
    if op == "round_trip":
        return _exact_rounded(s["x"])
    if op == "read":
        rows = slice(None) if s["rows"] is None else s["rows"]
        return _exact_values(s["codes"][rows], s["scales"][rows], H)
    x = _exact_rounded(s["x"])
    if op == "linear":
        out = x @ _exact_values(s["codes"], s["scales"], H).t()
        if s["bias_v"] is not None:
            out += s["bias_v"].double()
        for st, n, a in zip(s["start"].tolist(), s["lens"].tolist(), s["idx"].tolist()):
            if a >= 0:
                r = s["x"][st:st + n].double()
                for la, lb, off in s["slices"]:
                    out[st:st + n, off:off + lb.shape[1]] += s["scale"] * ((r @ la[a].double().t()) @ lb[a].double().t())
        return out
    out = torch.empty(s["out_t"].shape, dtype=torch.float64, device=DEVICE)
    for e, (st, n) in enumerate(zip(s["start"].tolist(), s["lens"].tolist())):
        if n:
            r = x[st:st + n] if s["rows"] is None else x[s["rows"][st:st + n]]
            y = r @ _exact_values(s["codes"][e], s["scales"][e], H).t()
            if case["gated"]:
                g, u = y[:, :case["width"]], y[:, case["width"]:]
                y = g * torch.sigmoid(g) * u
            out[st:st + n] = y
    return out


def work(case):
    """What one pass cannot do without: inputs read once, outputs written once, the products' operations."""
    op, T, H = case["op"], case["tokens"], case["hidden"]
    i, o = BYTES[case.get("dtype", "f32")], BYTES[case["out"]]
    row = 68 * _groups(H)                                             # bytes of a row in 4 bits
    if op == "round_trip":
        return {"bytes": T * (H * i + row + H * o), "flops": 4.0 * T * H}
    if op == "read":
        return {"bytes": T * (row + H * o) + (8 * T if case["gather"] else 0), "flops": 1.0 * T * H}
    if op == "linear":
        K, B = case["rank"], case["batches"]
        widths = [int(v) for v in case["widths"].split(",")]
        N, S, L = sum(widths), len(widths), case["adapters"]
        seen = L * (1 - (1 - 1 / (L + 1)) ** B)                       # adapters that some segment has, on average
        return {"bytes": i * (T * H + seen * K * (S * H + N)) + N * row + o * T * N,
                "flops": 2.0 * T * H * N + 2.0 * T * L / (L + 1) * K * (S * H + N)}
    E, N = case["experts"], case["width"]
    wide, R = (2 * N if case["gated"] else N), T * case["choices"]
    used = E * (1 - (1 - case["choices"] / E) ** T)                    # experts with a row, on average (even loads)
    return {"bytes": i * (T if case["gather"] else R) * H + used * wide * row + o * R * N, "flops": 2.0 * R * H * wide}
