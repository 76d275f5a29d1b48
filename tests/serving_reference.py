"""64-bit references of the MX4 and mixture-of-experts operators, and the tolerances of their tests (test infrastructure).

Tolerances count roundings, as in fused_reference.  fp16 activations of an MX4 product are off by at most 2^-19 of
their block's largest value; the errors have independent signs, so over a row they add up to at most 6 * 2^-19 *
sqrt(sum_b max_b^2 sum_{i in b} w_i^2) (more than ten standard deviations).  A matrix instruction adds at most 2^-23
of the running sum (it may cut instead of round), which stays below 4 r, r = sqrt(sum (w x)^2), for sums of independent
signs: 2^-21 r a step, one step of 128 inputs taking four pieces, then 16 partial sums.
"""
import math

import numpy as np
import torch

from fused_reference import H, SUB, TEN_SIGMA, act

MAGNITUDES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def mx4_values(codes, scales):
    """float64 values of MX4 codes [...][n / 2] and scales [...][n / 32] (NaN where the scale is 255)."""
    codes, scales = codes.cpu().long(), scales.cpu().long()
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    v = torch.where(q >= 8, -MAGNITUDES[q & 7], MAGNITUDES[q & 7])
    unit = torch.pow(torch.tensor(2.0, dtype=torch.float64), (scales - 127).double())
    unit = torch.where(scales == 255, torch.full_like(unit, math.nan), unit)
    return (v.unflatten(-1, (-1, 32)) * unit.unsqueeze(-1)).flatten(-2)


def mx4_quantize(v):
    """(codes, scales) as numpy computes them, one value at a time in exact arithmetic, from fp16 rows."""
    b = v.cpu().numpy().astype(np.float64).reshape(*v.shape[:-1], -1, 32)
    top = np.abs(b).max(-1)
    fine = np.isfinite(top)
    safe = np.where(fine & (top > 0), top, 1.0)
    e = np.frexp(safe)[1] - 3
    a = np.abs(np.where(fine[..., None], b, 0.0)) / np.exp2(e.astype(np.float64))[..., None]
    grid = MAGNITUDES.numpy()
    # nearest, the even code (mantissa bit 0) on a tie
    d = np.abs(a[..., None] - grid)
    near = d.min(-1, keepdims=True)
    cand = d == near
    even = cand & (np.arange(8) % 2 == 0)
    code = np.where(cand.sum(-1) > 1, even.argmax(-1), cand.argmax(-1))
    code = np.where(np.signbit(np.where(fine[..., None], b, 0.0)), code | 8, code)
    scales = np.where(~fine, 255, np.where(top > 0, e + 127, 0)).astype(np.uint8)
    code = code.reshape(*v.shape[:-1], -1).astype(np.uint8)
    return torch.from_numpy(code[..., 0::2] | (code[..., 1::2] << 4)), torch.from_numpy(scales)


def mx4_product(w, x, fp16_x):
    """z = x w^T in float64 and its error bound."""
    n = w.shape[-1]
    r = torch.sqrt((x * x) @ (w * w).t())
    e = (n / 32 + 16) * 2.0 ** -21 * r
    if fp16_x:
        top = x.unflatten(-1, (-1, 32)).abs().amax(-1)                       # [T][blocks]
        e = e + TEN_SIGMA * 2.0 ** -19 * torch.sqrt((top * top) @ (w * w).unflatten(-1, (-1, 32)).sum(-1).t())
    return x @ w.t(), e


def linear(z, ez, name, bias, residual):
    """(y, tolerance) of act(z + bias) + residual rounded to fp16."""
    if bias is not None:
        z = z + bias
    v, _ = act(name, z)
    e = 1.13 * ez + 2.0 ** -20 * (v.abs() + z.abs())
    y = v if residual is None else v + residual
    return y, e + 2.0 ** -23 * y.abs() + H * (y.abs() + e) + SUB


def gated(zg, eg, zu, eu, name):
    """(h, error bound before it is stored) of act(zg) zu."""
    v, _ = act(name, zg)
    h = v * zu
    return h, 1.13 * eg * (zu.abs() + eu) + v.abs() * eu + 2.0 ** -20 * (h.abs() + (zg * zu).abs())


def moe(layers, product, stored, x, ids, weights, name, residual):
    """(y, tolerance).  layers: three lists of float64 weights per expert; product(w, x): (z, error); stored(h): the error
    of storing h."""
    y = torch.zeros_like(x)
    e = torch.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            i = int(ids[t, j])
            if not 0 <= i < len(layers[0]):
                continue
            xt = x[t:t + 1]
            h, eh = gated(*product(layers[0][i], xt), *product(layers[1][i], xt), name)
            eh = eh + stored(h)
            z, ez = product(layers[2][i], h)
            ez = ez + eh @ layers[2][i].abs().t()
            wt = float(weights[t, j])
            y[t] += wt * z[0]
            e[t] += abs(wt) * (ez[0] + 2.0 ** -22 * z[0].abs())
    if residual is not None:
        y = y + residual
    return y, e + ids.shape[1] * 2.0 ** -23 * y.abs() + H * (y.abs() + e) + SUB
