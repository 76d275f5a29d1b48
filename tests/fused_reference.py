"""64-bit reference of the fused products and their gradients, and the tolerances of the tests (test infrastructure).

Tolerances count roundings.  A rounding to fp16 is off by at most H = 2^-11 of the value.  Where n fp16 weights
w_k are each rounded, their product with x is off by sum_k d_k w_k x_k with |d_k| <= H: the errors have independent
signs, so the sum has a standard deviation of at most H / sqrt(3) * r, r = sqrt(sum_k (w_k x_k)^2); 6 H r is ten of
them.  The same holds for a rounded operand dz.  fp32 accumulation adds at most 2^-24 of the running sum per step,
below 2^-24 * 4 sqrt(n) r for sums of independent signs.  Errors of the pre-activations reach y through the slopes of
y, evaluated at the reference.  The final rounding adds H |y| (and half the smallest subnormal, 2^-25).
"""
import math

import numpy as np
import torch

from oracle import aqlm_oracle as O

H = torch.finfo(torch.float16).eps / 2       # 2^-11
SUB = 2.0 ** -25
TEN_SIGMA = 6.0


def weights(L):
    """The layer's weights in float64 (the fp32 sum of fp16 codewords times the scale, each exact far below 2^-20)."""
    return torch.from_numpy(O.decode_fp32(L.codes, L.codebooks, L.scales).astype(np.float64))


def act(name, z):
    """Value and slope in float64."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "silu":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    if name == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def product(w, x, rounded):
    """x w^T and its error bound; rounded: the weights are rounded to fp16 once (M > 1), else they are exact."""
    z = x @ w.t()
    r = torch.sqrt((x * x) @ (w * w).t())
    return z, TEN_SIGMA * ((H if rounded else 0.0) + 2.0 ** -24 * 4 * math.sqrt(w.shape[1])) * r


def linear(w, x, name, bias, residual, rounded):
    """(y, y's tolerance, z, z's tolerance)."""
    z, ez = product(w, x, rounded)
    if bias is not None:
        z = z + bias
    v, s = act(name, z)
    # slopes of every activation here stay below 1.13; fp32 evaluation is within 2^-20 of the value
    y, e = v, 1.13 * ez + 2.0 ** -20 * (v.abs() + z.abs())
    if residual is not None:
        y = y + residual
    return y, e + H * (y.abs() + e) + SUB, z, ez + H * (z.abs() + ez) + SUB


def gated(wg, wu, x, name, bg, bu, rounded):
    """(y, tolerance, [(zg, tolerance), (zu, tolerance)])."""
    zs = []
    for w, b in ((wg, bg), (wu, bu)):
        z, e = product(w, x, rounded)
        zs.append((z if b is None else z + b, e))
    (zg, eg), (zu, eu) = zs
    v, _ = act(name, zg)
    ev = 1.13 * eg + 2.0 ** -20 * (v.abs() + zg.abs())
    y = v * zu
    e = ev * zu.abs() + v.abs() * eu + ev * eu
    return y, e + H * (y.abs() + e) + SUB, [(z, ez + H * (z.abs() + ez) + SUB) for z, ez in zs]


def linear_grads(dy, z, name):
    return [dy if name == "none" else dy * act(name, z)[1]]


def gated_grads(dy, zg, zu, name):
    v, s = act(name, zg)
    return [dy * zu * s, dy * v]


def back(dzs, ws, dz_rounded):
    """dx and its tolerance, the bias sums and theirs.  One rounding of every weight or of dz for M = 1, and one
    of each otherwise; both are counted always."""
    dx, r2, n = 0.0, 0.0, 0
    for dz, w in zip(dzs, ws):
        dx = dx + dz @ w
        r2 = r2 + (dz * dz) @ (w * w)
        n += w.shape[0]
    k = H * (math.sqrt(2.0) if dz_rounded else 1.0) + 2.0 ** -24 * 4 * math.sqrt(n) + 2.0 ** -20
    e = TEN_SIGMA * k * torch.sqrt(r2)
    # dz below fp16's normal range is off by up to half its smallest subnormal, 2^-25, whatever its size
    e = e + 2.0 ** -25 * TEN_SIGMA * sum(torch.sqrt((w * w).sum(0)) for w in ws)
    sums = []
    for dz in dzs:
        s = dz.sum(0)
        es = 2.0 ** -20 * dz.abs().sum(0)
        sums.append((s, es + H * (s.abs() + es) + SUB))
    return dx, e + H * (dx.abs() + e) + SUB, sums


def assert_within(got, want, tol, what):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - tol
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {over.numel()} outside, worst by {float(over.max()):.3g}"
