"""Plain 64-bit forms of the shared projection with adapters, the grouped
products, the routing and the weighted row sum, with the error each may have:
every float32 sum of n products is off by at most depth * 2^-23 times the sum
of the products' magnitudes (2^-23 covers adds that truncate), with a depth of
n / 32 + 64 matrix-instruction and wave partial sums, and each result is
rounded once to its type."""
import numpy as np
import torch

UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
SMALLEST = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
# what is left of a projected value kept as two 16-bit parts
SPLIT = {torch.float16: 2.0 ** -21, torch.bfloat16: 2.0 ** -16}


def sum_error(n):
    return (n / 32 + 64) * 2.0 ** -23


def rounded(y, err, dtype):
    """Error bound of a result y (its own error err) rounded to dtype."""
    return err + (y.abs() + err) * UNIT[dtype] + SMALLEST[dtype]


def lora_linear(x, w, bias, slices, start, lens, idx, scale, out0, add, dtype):
    """(exact result, error bound) in float64 on the CPU."""
    x, w = x.double().cpu(), w.double().cpu()
    H = x.shape[1]
    y = x @ w.t()
    mag = x.abs() @ w.abs().t()
    err = sum_error(H) * mag
    if bias is not None:
        y = y + bias.double().cpu()
        mag = mag + bias.double().cpu().abs()
    for st, n, a in zip(start, lens, idx):
        for la, lb, off in slices:
            L, K = la.shape[0], la.shape[1]
            if a < 0 or a >= L or n <= 0 or st < 0 or st + n > x.shape[0]:
                continue
            A, B = la[a].double().cpu(), lb[a].double().cpu()
            r, c = slice(st, st + n), slice(off, off + lb.shape[1])
            v = scale * (x[r] @ A.t())
            ev = abs(scale) * (sum_error(H) * (x[r].abs() @ A.abs().t()))
            ev = ev + v.abs() * (SPLIT[la.dtype] + 2.0 ** -22) + 2.0 ** -25
            y[r, c] += v @ B.t()
            m = (v.abs() + ev) @ B.abs().t()
            mag[r, c] += m
            err[r, c] += ev @ B.abs().t() + sum_error(2 * K) * m
    if add:
        o = out0.double().cpu()
        y = y + o
        mag = mag + o.abs()
    err = err + 4 * 2.0 ** -23 * mag
    return y, rounded(y, err, dtype)


def grouped(x, w, start, lens, idx, rows, gated, out0):
    """(exact result, error bound, written rows); untouched rows keep out0."""
    x = x.double().cpu()
    N = out0.shape[1]
    y = out0.double().cpu().clone()
    bound = torch.zeros_like(y)
    written = torch.zeros(y.shape[0], dtype=torch.bool)
    for b, (st, n) in enumerate(zip(start, lens)):
        e = b if idx is None else idx[b]
        if e < 0 or e >= w.shape[0] or n <= 0 or st < 0 or st + n > y.shape[0]:
            continue
        src = torch.arange(st, st + n) if rows is None else torch.as_tensor(rows[st:st + n])
        ok = (src >= 0) & (src < x.shape[0])
        xs = torch.zeros(n, x.shape[1], dtype=torch.float64)
        xs[ok] = x[src[ok]]
        we = w[e].double().cpu()
        z = xs @ we.t()
        ez = sum_error(x.shape[1]) * (xs.abs() @ we.abs().t())
        if gated:
            g, u, eg, eu = z[:, :N], z[:, N:], ez[:, :N], ez[:, N:]
            s = g / (1 + torch.exp(-g))
            y[st:st + n] = s * u
            es = 1.1 * eg + s.abs() * (2.0 ** -20 + g.abs() * 2.0 ** -23)  # |silu'| < 1.1; exp's own error
            z, ez = y[st:st + n], es * (u.abs() + eu) + s.abs() * eu
        y[st:st + n] = z
        bound[st:st + n] = rounded(z, ez, out0.dtype)
        written[st:st + n] = True
    return y, bound, written


def route(logits, k, renormalize):
    """The routing in float64: a loop over tokens and choices."""
    x = logits.double().cpu().numpy()
    T, E = x.shape
    x = np.where(np.isnan(x), -np.inf, x)
    weights, chosen = np.zeros((T, k)), -np.ones((T, k), dtype=np.int64)
    for t in range(T):
        order = sorted((e for e in range(E) if x[t, e] > -np.inf), key=lambda e: (-x[t, e], e))
        if not order:
            continue
        top = x[t, order[0]]
        share = {e: 1.0 if x[t, e] == top else float(np.exp(x[t, e] - top)) for e in order}
        picked = order[:k]
        total = sum(share[e] for e in (picked if renormalize else order))
        for j, e in enumerate(picked):
            chosen[t, j] = e
            weights[t, j] = share[e] / total
    slots = -np.ones((T, k), dtype=np.int64)
    rows = -np.ones(T * k, dtype=np.int64)
    start, lens = np.zeros(E, dtype=np.int64), np.zeros(E, dtype=np.int64)
    n = 0
    for e in range(E):
        start[e] = n
        for t, j in zip(*np.nonzero(chosen == e)):
            slots[t, j] = n
            rows[n] = t
            n += 1
        lens[e] = n - start[e]
    return weights, chosen, slots, rows, start, lens


def combine(rows, weights, slots, out0, add):
    r, w = rows.double().cpu(), weights.double().cpu()
    y = out0.double().cpu().clone() if add else torch.zeros(out0.shape, dtype=torch.float64)
    mag = y.abs()
    for t in range(slots.shape[0]):
        for j in range(slots.shape[1]):
            s = int(slots[t, j])
            if 0 <= s < r.shape[0]:
                y[t] += w[t, j] * r[s]
                mag[t] += (w[t, j] * r[s]).abs()
    err = (slots.shape[1] + 2) * 2.0 ** -23 * mag
    return y, rounded(y, err, out0.dtype)


def assert_within(got, want, bound, what=""):
    got = got.double().cpu()
    assert got.shape == want.shape
    bad = ~((got - want).abs() <= bound)
    if bad.any():
        i = int(bad.reshape(-1).nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {i}: "
                             f"{got.reshape(-1)[i]} for {want.reshape(-1)[i]} "
                             f"(bound {bound.reshape(-1)[i]:.3g})")
