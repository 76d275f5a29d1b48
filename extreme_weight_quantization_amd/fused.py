"""Fused products over AQLM layers and their backward passes (ctypes, declared in include/aqlm.h).

    aqlm_linear_act           z = W x + bias;  y = act(z) + residual
    aqlm_gated                zg = Wg x + bg;  zu = Wu x + bu;  y = act(zg) * zu
    aqlm_linear_act_backward  dz = dy * act'(z);  dx = dz W;  dbias = sum over tokens of dz
    aqlm_gated_backward       dzg = dy * zu * act'(zg);  dzu = dy * act(zg);  dx = dzg Wg + dzu Wu

As in ``binding``: tensors are checked for device, dtype, shape and contiguity, then handed to the C ABI with
torch's current HIP stream of their device; every step of the computation runs in the library's kernels.  The
quantized weights are frozen.  No call records an autograd graph: an input that requires a gradient gives a result
without one, and the backward calls are what a ``torch.autograd.Function`` around a layer runs.  A layer is (codes, codebooks, scales), or (SliceLists, codebooks, scales) for the
batch-1 calls over slice lists.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import SliceLists, _check, lists_fused_workspace_bytes, load_library

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}   # aqlm_act
_F16, _U8, _I16 = torch.float16, torch.uint8, torch.int16


def _act(act):
    try:
        return ACTIVATIONS[act]
    except (KeyError, TypeError):
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}") from None


def _tensor(name, t, dev, shape, dtype=_F16):
    """t is a contiguous `dtype` tensor of `shape` on dev; its address."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)}")
    if t.device != dev:
        raise ValueError(f"tensors are on different devices: {name} on {t.device}, not {dev}")
    return t.data_ptr()


def _optional(name, t, dev, shape):
    return None if t is None else _tensor(name, t, dev, shape)


def _layer(codes, codebooks, scales, dev):
    """(M, B, g), out, in and the three addresses of one layer."""
    if codebooks.dim() != 3 or codes.dim() != 3:
        raise ValueError("codes must be [out][in/g][M] and codebooks [M][2^B][g]")
    M, K, g = codebooks.shape
    out, G, m = codes.shape
    B = K.bit_length() - 1
    if K != 1 << B:
        raise ValueError("the codebook size must be a power of two")
    if m != M:
        raise ValueError(f"codes hold {m} codes per group but there are {M} codebooks")
    # one test for the usual case: these calls are made thousands of times a second
    if (codes.dtype is not (_U8 if B <= 8 else _I16) or codebooks.dtype is not _F16 or scales.dtype is not _F16
            or scales.shape != (out,) or codes.device != dev or codebooks.device != dev or scales.device != dev
            or not codes.is_contiguous() or not codebooks.is_contiguous() or not scales.is_contiguous()):
        _tensor("codes", codes, dev, (out, G, M), _U8 if B <= 8 else _I16)
        _tensor("codebooks", codebooks, dev, (M, K, g))
        _tensor("scales", scales, dev, (out,))
    return (M, B, g), out, G * g, (codes.data_ptr(), codebooks.data_ptr(), scales.data_ptr())


def _rows(name, x):
    """x is a GPU tensor [batch][...]; its device and batch."""
    if not x.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if x.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    return x.device, x.shape[0]


def _output(name, y, like, dev, shape):
    if y is None:
        y = like.new_empty(shape)   # like: the fp16 input (0.2 us less than torch.empty)
        return y, y.data_ptr()
    return y, _tensor(name, y, dev, shape)


def _workspace(workspace, need, dev):
    """Address and bytes of the workspace; one of `need()` bytes when none is given."""
    if workspace is None:
        n = need()
        if n == 0:
            return None, None, 0
        workspace = torch.empty((n,), dtype=_U8, device=dev)
    elif workspace.dtype != _U8 or not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {dev}")
    return workspace, workspace.data_ptr(), workspace.numel()


# torch.cuda.current_stream builds a Stream object (1.9 us); the raw getter is what it asks
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(name, dev, *args):
    """The library's `name`(..., stream) with `dev` current: kernels launch on the device of their tensors."""
    fn = getattr(binding._lib or load_library(), name)
    index = dev.index
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(index))
    if status:
        _check(status)


def _bytes(name, *shape) -> int:
    n = ctypes.c_int64(0)
    _check(getattr(load_library(), name)(*shape, ctypes.byref(n)))
    return n.value


def linear_act_workspace_bytes(M: int, B: int, g: int, out: int, n_in: int, batch: int) -> int:
    """Bytes of workspace aqlm_linear_act needs for the shape and any smaller batch of it."""
    return _bytes("aqlm_linear_act_workspace_bytes", M, B, g, out, n_in, batch)


def gated_workspace_bytes(M: int, B: int, g: int, out: int, n_in: int, batch: int) -> int:
    """Bytes of workspace aqlm_gated needs for the shape and any smaller batch of it (out: rows of either layer)."""
    return _bytes("aqlm_gated_workspace_bytes", M, B, g, out, n_in, batch)


def linear_act_backward_workspace_bytes(M: int, B: int, g: int, out: int, n_in: int, batch: int) -> int:
    """Bytes of workspace aqlm_linear_act_backward needs for the shape and any smaller batch of it."""
    return _bytes("aqlm_linear_act_backward_workspace_bytes", M, B, g, out, n_in, batch)


def gated_backward_workspace_bytes(M: int, B: int, g: int, out: int, n_in: int, batch: int) -> int:
    """Bytes of workspace aqlm_gated_backward needs for the shape and any smaller batch of it."""
    return _bytes("aqlm_gated_backward_workspace_bytes", M, B, g, out, n_in, batch)


def _pair(a, b):
    return (ctypes.c_void_p * 2)(a, b)


def _gated_layers(gate, up, dev):
    sch, out, n_in, g = _layer(*gate, dev)
    sch_u, out_u, n_in_u, u = _layer(*up, dev)
    if sch_u != sch or out_u != out or n_in_u != n_in:
        raise ValueError("gate and up must have the same (M, B, g), out and in")
    return sch, out, n_in, [_pair(a, b) for a, b in zip(g, u)]


def aqlm_linear_act(codes, codebooks, scales, x, act="none", bias=None, residual=None, z=None, y=None,
                    workspace=None):
    """y = act(W x + bias) + residual for any batch of rows of x (see aqlm.h).

    z ([batch][out]), when given, receives W x + bias for the backward pass; residual may be y itself."""
    a = _act(act)
    dev, batch = _rows("x", x)
    sch, out, n_in, layer = _layer(codes, codebooks, scales, dev)
    px = _tensor("x", x, dev, (batch, n_in))
    pb = _optional("bias", bias, dev, (out,))
    pr = _optional("residual", residual, dev, (batch, out))
    pz = _optional("z", z, dev, (batch, out))
    y, py = _output("y", y, x, dev, (batch, out))
    keep, ws, nws = _workspace(workspace, lambda: linear_act_workspace_bytes(*sch, out, n_in, batch), dev)
    _call("aqlm_linear_act", dev, *layer, px, pb, pr, pz, py, ws, nws, a, *sch, out, n_in, batch)
    return y


def aqlm_gated(gate, up, x, act="silu", gate_bias=None, up_bias=None, zg=None, zu=None, y=None, workspace=None):
    """y = act(Wg x + bg) * (Wu x + bu) for layers gate and up = (codes, codebooks, scales) (see aqlm.h).

    zg and zu ([batch][out]), when given, receive the two pre-activations for the backward pass."""
    a = _act(act)
    dev, batch = _rows("x", x)
    sch, out, n_in, (codes, codebooks, scales) = _gated_layers(gate, up, dev)
    px = _tensor("x", x, dev, (batch, n_in))
    bias = _pair(_optional("gate_bias", gate_bias, dev, (out,)), _optional("up_bias", up_bias, dev, (out,)))
    z = _pair(_optional("zg", zg, dev, (batch, out)), _optional("zu", zu, dev, (batch, out)))
    y, py = _output("y", y, x, dev, (batch, out))
    keep, ws, nws = _workspace(workspace, lambda: gated_workspace_bytes(*sch, out, n_in, batch), dev)
    _call("aqlm_gated", dev, codes, codebooks, scales, px, bias, z, py, ws, nws, a, *sch, out, n_in, batch)
    return y


def aqlm_linear_act_backward(codes, codebooks, scales, dy, act="none", z=None, need_dbias=False, dx=None,
                             workspace=None):
    """(dx, dbias) of aqlm_linear_act for the gradient dy of its result; the residual's gradient is dy itself.

    z: the pre-activations that aqlm_linear_act kept (None for act "none").  dbias is None unless need_dbias."""
    a = _act(act)
    dev, batch = _rows("dy", dy)
    sch, out, n_in, layer = _layer(codes, codebooks, scales, dev)
    pd = _tensor("dy", dy, dev, (batch, out))
    pz = _optional("z", z, dev, (batch, out))
    dbias = torch.empty((out,), dtype=_F16, device=dev) if need_dbias else None
    dx, px = _output("dx", dx, dy, dev, (batch, n_in))
    keep, ws, nws = _workspace(workspace, lambda: linear_act_backward_workspace_bytes(*sch, out, n_in, batch), dev)
    _call("aqlm_linear_act_backward", dev, *layer, pd, pz, px, dbias.data_ptr() if need_dbias else None,
          ws, nws, a, *sch, out, n_in, batch)
    return dx, dbias


def aqlm_gated_backward(gate, up, dy, zg, zu, act="silu", need_dbias=False, dx=None, workspace=None):
    """(dx, gate's dbias, up's dbias) of aqlm_gated for the gradient dy of its result.

    zg, zu: the pre-activations that aqlm_gated kept.  The bias gradients are None unless need_dbias."""
    a = _act(act)
    dev, batch = _rows("dy", dy)
    sch, out, n_in, (codes, codebooks, scales) = _gated_layers(gate, up, dev)
    pd = _tensor("dy", dy, dev, (batch, out))
    z = _pair(_tensor("zg", zg, dev, (batch, out)), _tensor("zu", zu, dev, (batch, out)))
    dbg = dbu = db = None
    if need_dbias:
        dbg, dbu = torch.empty((2, out), dtype=_F16, device=dev).unbind(0)
        db = _pair(dbg.data_ptr(), dbu.data_ptr())
    dx, px = _output("dx", dx, dy, dev, (batch, n_in))
    keep, ws, nws = _workspace(workspace, lambda: gated_backward_workspace_bytes(*sch, out, n_in, batch), dev)
    _call("aqlm_gated_backward", dev, codes, codebooks, scales, pd, z, px, db, ws, nws, a, *sch, out, n_in,
          batch)
    return dx, dbg, dbu


def _lists_shape(lists):
    if not isinstance(lists, SliceLists):
        raise ValueError("a layer over slice lists is (SliceLists, codebooks, scales)")
    return lists.out, lists.n_in


def _lists_layer(lists, codebooks, scales, dev):
    for name, t in (("table", lists.table), ("entries", lists.entries)):
        if t.device != dev:
            raise ValueError(f"tensors are on different devices: {name} on {t.device}, not {dev}")
    return (lists.table.data_ptr(), lists.entries.data_ptr(), lists.entries.numel(),
            _tensor("codebooks", codebooks, dev, (1, 1 << 16, 8)), _tensor("scales", scales, dev, (lists.out,)))


def _lists_x(x, n_in):
    dev, batch = _rows("x", x)
    if batch > 1:
        raise ValueError(f"x must be [1][{n_in}]")
    return dev, batch, _tensor("x", x, dev, (batch, n_in))


def aqlm_linear_act_lists(lists, codebooks, scales, x, act="none", bias=None, residual=None, z=None, y=None,
                          workspace=None):
    """aqlm_linear_act at batch 1 over slice lists (see aqlm.h); x is [1][in] (or [0][in])."""
    a = _act(act)
    out, n_in = _lists_shape(lists)
    dev, batch, px = _lists_x(x, n_in)
    table, entries, n_entries, cb, s = _lists_layer(lists, codebooks, scales, dev)
    pb = _optional("bias", bias, dev, (out,))
    pr = _optional("residual", residual, dev, (batch, out))
    pz = _optional("z", z, dev, (batch, out))
    y, py = _output("y", y, x, dev, (batch, out))
    keep, ws, nws = _workspace(workspace, lambda: lists_fused_workspace_bytes([out], n_in), dev)
    _call("aqlm_linear_act_lists", dev, table, entries, n_entries, cb, s, px, pb, pr, pz, py, ws, nws, a,
          1, 16, 8, out, n_in, batch)
    return y


def aqlm_gated_lists(gate, up, x, act="silu", gate_bias=None, up_bias=None, zg=None, zu=None, y=None,
                     workspace=None):
    """aqlm_gated at batch 1 for layers gate and up = (SliceLists, codebooks, scales) (see aqlm.h)."""
    a = _act(act)
    out, n_in = _lists_shape(gate[0])
    if _lists_shape(up[0]) != (out, n_in):
        raise ValueError("gate and up must have the same out and in")
    dev, batch, px = _lists_x(x, n_in)
    g, u = _lists_layer(*gate, dev), _lists_layer(*up, dev)
    bias = _pair(_optional("gate_bias", gate_bias, dev, (out,)), _optional("up_bias", up_bias, dev, (out,)))
    z = _pair(_optional("zg", zg, dev, (batch, out)), _optional("zu", zu, dev, (batch, out)))
    y, py = _output("y", y, x, dev, (batch, out))
    keep, ws, nws = _workspace(workspace, lambda: lists_fused_workspace_bytes([out, out], n_in), dev)
    _call("aqlm_gated_lists", dev, _pair(g[0], u[0]), _pair(g[1], u[1]),
          (ctypes.c_int64 * 2)(g[2], u[2]), _pair(g[3], u[3]), _pair(g[4], u[4]), px, bias, z, py, ws, nws, a, 1, 16, 8,
          out, n_in, batch)
    return y
