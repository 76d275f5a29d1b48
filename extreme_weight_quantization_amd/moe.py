"""Mixture-of-experts layers for serving (ctypes, declared in include/aqlm.h).

    aqlm_moe_route  the k experts of every token, and their weights, from the router's logits
    aqlm_moe        y_t = residual_t + sum_j w_tj Wd_e (act(Wg_e x_t) * (Wu_e x_t)), e = ids_tj, experts in an AQLM scheme
    aqlm_moe_mx4    the same with experts in MX4

As in ``fused``: tensors are checked for device, dtype, shape and contiguity, then handed to the C ABI with torch's
current HIP stream of their device; every step of the computation runs in the library's kernels, and no call records
an autograd graph.  A layer holds all experts: (codes [E][rows][in/g][M], codebooks [E][M][2^B][g], scales [E][rows]), or in
MX4 (codes [E][rows][in / 2], scales [E][rows][in / 32]).
"""
from __future__ import annotations

import ctypes

import torch

from .fused import _F16, _I16, _U8, _act, _bytes, _call, _optional, _output, _rows, _tensor, _workspace

SCORES = {"softmax": 0, "sigmoid": 1}   # aqlm_score
_I32, _F32 = torch.int32, torch.float32


def moe_route_workspace_bytes(experts: int, n_in: int, k: int, tokens: int) -> int:
    """Bytes of workspace aqlm_moe_route needs for the shape and any smaller number of tokens."""
    return _bytes("aqlm_moe_route_workspace_bytes", experts, n_in, k, tokens)


def moe_workspace_bytes(M: int, B: int, g: int, experts: int, n_in: int, inner: int, tokens: int, k: int) -> int:
    """Bytes of workspace aqlm_moe needs for the shape and any smaller number of tokens."""
    return _bytes("aqlm_moe_workspace_bytes", M, B, g, experts, n_in, inner, k, tokens)


def moe_mx4_workspace_bytes(experts: int, n_in: int, inner: int, tokens: int, k: int) -> int:
    """Bytes of workspace aqlm_moe_mx4 needs for the shape and any smaller number of tokens."""
    return _bytes("aqlm_moe_mx4_workspace_bytes", experts, n_in, inner, k, tokens)


def aqlm_moe_route(x, router, k, score="softmax", bias=None, renorm=True, scale=1.0, workspace=None):
    """(ids int32 [tokens][k], weights fp32 [tokens][k]) of fp16 x [tokens][in] and router [experts][in] (see aqlm.h).

    bias: fp32 [experts], added to the scores for the choice only."""
    try:
        how = SCORES[score]
    except (KeyError, TypeError):
        raise ValueError(f"score must be one of {', '.join(SCORES)}") from None
    dev, tokens = _rows("x", x)
    if router.dim() != 2:
        raise ValueError("router must be [experts][in]")
    experts, n_in = router.shape
    k = int(k)
    px, pr = _tensor("x", x, dev, (tokens, n_in)), _tensor("router", router, dev, (experts, n_in))
    pb = None if bias is None else _tensor("bias", bias, dev, (experts,), _F32)
    if not 1 <= k <= experts:
        raise ValueError("k must be between 1 and the number of experts")
    keep, ws, nws = _workspace(workspace, lambda: moe_route_workspace_bytes(experts, n_in, k, tokens), dev)
    ids, weights = x.new_empty((tokens, k), dtype=_I32), x.new_empty((tokens, k), dtype=_F32)
    _call("aqlm_moe_route", dev, px, pr, pb, ids.data_ptr(), weights.data_ptr(), ws, nws, how, int(bool(renorm)),
          float(scale), experts, n_in, k, tokens)
    return ids, weights


def _three(values):
    return (ctypes.c_void_p * 3)(*values)


def _experts(name, codes, codebooks, scales, dev):
    """(M, B, g), experts, rows, in and the three addresses of one stacked AQLM layer."""
    if codes.dim() != 4 or codebooks.dim() != 4:
        raise ValueError(f"{name}: codes must be [experts][rows][in/g][M] and codebooks [experts][M][2^B][g]")
    E, M, K, g = codebooks.shape
    rows, G = codes.shape[1], codes.shape[2]
    B = K.bit_length() - 1
    if K != 1 << B:
        raise ValueError("the codebook size must be a power of two")
    return ((M, B, g), E, rows, G * g,
            (_tensor(f"{name} codes", codes, dev, (E, rows, G, M), _U8 if B <= 8 else _I16),
             _tensor(f"{name} codebooks", codebooks, dev, (E, M, K, g)), _tensor(f"{name} scales", scales, dev, (E, rows))))


def _experts_mx4(name, codes, scales, dev):
    if codes.dim() != 3 or codes.shape[2] % 16:
        raise ValueError(f"{name}: codes must be [experts][rows][in / 2] with in a multiple of 32")
    E, rows, half = codes.shape
    return ((), E, rows, 2 * half, (_tensor(f"{name} codes", codes, dev, (E, rows, half), _U8),
                                    _tensor(f"{name} scales", scales, dev, (E, rows, half // 16), _U8)))


def _layers(make, gate, up, down, dev):
    """Scheme, experts, in, inner, and the host arrays of gate, up and down."""
    sch, E, inner, n_in, g = make("gate", *gate, dev)
    *like_gate, u = make("up", *up, dev)
    if like_gate != [sch, E, inner, n_in]:
        raise ValueError("gate and up must have the same scheme, experts, rows and in")
    *turned, d = make("down", *down, dev)
    if turned != [sch, E, n_in, inner]:
        raise ValueError("down must have gate's scheme and experts, and its rows and in exchanged")
    return sch, E, n_in, inner, [_three(a) for a in zip(g, u, d)]


def _moe(name, make, need, gate, up, down, x, ids, weights, act, residual, y, workspace):
    a = _act(act)
    dev, tokens = _rows("x", x)
    sch, E, n_in, inner, arrays = _layers(make, gate, up, down, dev)
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens][k]")
    k = ids.shape[1]
    px = _tensor("x", x, dev, (tokens, n_in))
    pi, pw = _tensor("ids", ids, dev, (tokens, k), _I32), _tensor("weights", weights, dev, (tokens, k), _F32)
    pr = _optional("residual", residual, dev, (tokens, n_in))
    y, py = _output("y", y, x, dev, (tokens, n_in))
    keep, ws, nws = _workspace(workspace, lambda: need(*sch, E, n_in, inner, tokens, k), dev)
    _call(name, dev, *arrays, px, pi, pw, pr, py, ws, nws, a, *sch, E, n_in, inner, k, tokens)
    return y


def aqlm_moe(gate, up, down, x, ids, weights, act="silu", residual=None, y=None, workspace=None):
    """A mixture-of-experts layer for few tokens, experts in one AQLM scheme (see aqlm.h).

    gate, up, down: (codes, codebooks, scales) stacked over the experts; ids, weights as aqlm_moe_route gives them;
    residual may be y itself."""
    return _moe("aqlm_moe", _experts, moe_workspace_bytes, gate, up, down, x, ids, weights, act, residual, y, workspace)


def aqlm_moe_mx4(gate, up, down, x, ids, weights, act="silu", residual=None, y=None, workspace=None):
    """aqlm_moe for experts in MX4: gate, up, down are (codes, scales) stacked over the experts."""
    return _moe("aqlm_moe_mx4", _experts_mx4, moe_mx4_workspace_bytes, gate, up, down, x, ids, weights, act, residual, y,
                workspace)
