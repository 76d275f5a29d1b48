"""Layers in microscaled 4-bit floating point, MX4 (ctypes, declared in include/aqlm.h).

    aqlm_mx4_quantize  fp16 rows to (codes, scales)
    aqlm_mx4_decode    (codes, scales) to fp16 rows
    aqlm_mx4_linear    y = act(W x + bias) + residual, x in fp16 or itself a pair (codes, scales)

As in ``fused``: tensors are checked for device, dtype, shape and contiguity, then handed to the C ABI with torch's
current HIP stream of their device; every step of the computation runs in the library's kernels, and no call records
an autograd graph.  codes are uint8 [rows][in / 2], scales uint8 [rows][in / 32].
"""
from __future__ import annotations

from .fused import _F16, _U8, _act, _bytes, _call, _optional, _output, _rows, _tensor, _workspace

_BLOCK = 32


def mx4_linear_workspace_bytes(out: int, n_in: int, batch: int, x_mx4: bool = False) -> int:
    """Bytes of workspace aqlm_mx4_linear needs for the shape and any smaller batch of it."""
    return _bytes("aqlm_mx4_linear_workspace_bytes", int(bool(x_mx4)), out, n_in, batch)


def _pair(name, codes, scales, dev):
    """rows, in and the two addresses of an MX4 matrix."""
    if codes.dim() != 2 or codes.shape[1] % (_BLOCK // 2):
        raise ValueError(f"{name} codes must be [rows][in / 2] with in a multiple of {_BLOCK}")
    rows, n_in = codes.shape[0], 2 * codes.shape[1]
    return (rows, n_in, _tensor(f"{name} codes", codes, dev, (rows, n_in // 2), _U8),
            _tensor(f"{name} scales", scales, dev, (rows, n_in // _BLOCK), _U8))


def _bytes_of(name, t, like, dev, shape):
    """A uint8 result, a new one if none is given, and its address."""
    if t is None:
        t = like.new_empty(shape, dtype=_U8)
        return t, t.data_ptr()
    return t, _tensor(name, t, dev, shape, _U8)


def aqlm_mx4_quantize(w, codes=None, scales=None):
    """(codes, scales) of fp16 rows w [rows][in] (see aqlm.h)."""
    dev, rows = _rows("w", w)
    n_in = w.shape[1]
    pw = _tensor("w", w, dev, (rows, n_in))
    codes, pc = _bytes_of("codes", codes, w, dev, (rows, n_in // 2))
    scales, ps = _bytes_of("scales", scales, w, dev, (rows, n_in // _BLOCK))
    _call("aqlm_mx4_quantize", dev, pw, pc, ps, rows, n_in)
    return codes, scales


def aqlm_mx4_decode(codes, scales, w=None):
    """The fp16 values [rows][in] that MX4 codes stand for."""
    dev, _ = _rows("codes", codes)
    rows, n_in, pc, ps = _pair("the", codes, scales, dev)
    if w is None:
        w = codes.new_empty((rows, n_in), dtype=_F16)
        pw = w.data_ptr()
    else:
        pw = _tensor("w", w, dev, (rows, n_in))
    _call("aqlm_mx4_decode", dev, pc, ps, pw, rows, n_in)
    return w


def aqlm_mx4_linear(codes, scales, x, act="none", bias=None, residual=None, y=None, workspace=None):
    """y = act(W x + bias) + residual for W in MX4 and any batch of rows of x (see aqlm.h).

    x is an fp16 tensor [batch][in], or (codes, scales) of MX4 rows; residual may be y itself."""
    a = _act(act)
    four = isinstance(x, (tuple, list))
    if four and len(x) != 2:
        raise ValueError("x must be a tensor or a pair (codes, scales)")
    dev, batch = _rows("x", x[0] if four else x)
    out, n_in, pc, ps = _pair("weight", codes, scales, dev)
    if four:
        _, x_in, px, pxs = _pair("x", *x, dev)
        if x_in != n_in:
            raise ValueError(f"x must have {n_in} inputs")
    else:
        px, pxs = _tensor("x", x, dev, (batch, n_in)), None
    pb = _optional("bias", bias, dev, (out,))
    pr = _optional("residual", residual, dev, (batch, out))
    if y is None and four:
        y = x[0].new_empty((batch, out), dtype=_F16)
    y, py = _output("y", y, x, dev, (batch, out))
    keep, ws, nws = _workspace(workspace, lambda: mx4_linear_workspace_bytes(out, n_in, batch, four), dev)
    _call("aqlm_mx4_linear", dev, pc, ps, px, pxs, pb, pr, py, ws, nws, a, out, n_in, batch)
    return y
