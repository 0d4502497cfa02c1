"""Microscaled 4-bit values by their definition, in 64 bits, and the products
of them with the error each may have: products of 4-bit values are exact, so
the sums have the errors of matmul_util's."""
import numpy as np
import torch

import matmul_util as U

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def groups(hidden):
    return -(-hidden // 128)


def quantize(x):
    """(codes (T, 64 G), scales (T, 4 G)) of rows x as uint8 arrays.  A magnitude's code is the
    nearest of the grid; at the same distance from two, the even one."""
    v = x.detach().cpu().double().numpy()
    T, H = v.shape
    G = groups(H)
    blocks = np.zeros((T, 4 * G * 32))
    blocks[:, :H] = v
    blocks = blocks.reshape(T, 4 * G, 32)
    finite = np.isfinite(blocks).all(axis=2)
    blocks = np.where(finite[..., None], blocks, 0.0)
    top = np.abs(blocks).max(axis=2)
    with np.errstate(divide="ignore"):
        e = np.where(top > 0, np.frexp(top)[1] - 1 - 2, -127)     # frexp: top = m 2^k, m in [.5, 1)
    e = np.maximum(e, -127)
    y = np.ldexp(np.abs(blocks), -e[..., None])
    d = np.abs(y[..., None] - GRID)
    even_first = np.where(np.arange(8) % 2 == 0, 0.0, 1e-9)       # below any difference of distances here
    exact_tie = d == d.min(axis=-1, keepdims=True)
    code = np.argmin(np.where(exact_tie, even_first, 1.0), axis=-1)
    code = np.where(y >= 6, 7, code)
    code = (code + 8 * np.signbit(blocks)).astype(np.uint8)
    code = np.where(finite[..., None], code, 0).reshape(T, 64 * G, 2).astype(np.uint8)
    scales = np.where(finite, e + 127, 255).astype(np.uint8)
    return code[..., 0] | (code[..., 1] << 4), scales


def values(codes, scales, hidden):
    """float64 tensor (..., hidden) of what codes and scales stand for."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    c = np.stack((codes & 15, codes >> 4), axis=-1).reshape(*scales.shape, 32)
    v = GRID[c & 7] * np.where(c >= 8, -1.0, 1.0)
    v = np.ldexp(v, scales.astype(np.int64)[..., None] - 127)
    v = np.where(scales[..., None] == 255, np.nan, v)
    return torch.from_numpy(v.reshape(*scales.shape[:-1], -1)[..., :hidden].copy())


def rounded(x):
    """Rows x with their 4-bit values in the place of their own."""
    return values(*quantize(x), x.shape[1])


def packed(w, device="cuda"):
    """A weight (rows, hidden), or a stack of them, as codes and scales on the device."""
    lead, H = w.shape[:-1], w.shape[-1]
    c, s = quantize(w.reshape(-1, H))
    return (torch.from_numpy(c).view(*lead, -1).to(device), torch.from_numpy(s).view(*lead, -1).to(device))


def lora_linear(x, wv, bias, slices, start, lens, idx, scale, out0, add, dtype):
    """(exact result, error bound): the shared projection of rounded rows x with the values wv, and
    the adapters' part, which is matmul_util's with a weight of zeros."""
    xr = rounded(x)
    y, mag = xr @ wv.t(), xr.abs() @ wv.abs().t()
    err = U.sum_error(x.shape[1]) * mag
    zero = torch.zeros(wv.shape[0], x.shape[1], dtype=torch.float64)
    ya, ea = U.lora_linear(x, zero, bias, slices, start, lens, idx, scale, out0, add, torch.float32)
    err = err + ea + 4 * 2.0 ** -23 * mag
    return y + ya, U.rounded(y + ya, err, dtype)


def grouped(x, wv, start, lens, idx, rows, gated, out0):
    return U.grouped(rounded(x), wv, start, lens, idx, rows, gated, out0)
