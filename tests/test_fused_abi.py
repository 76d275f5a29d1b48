"""Refusals of the fused products on the host, before any HIP call (no GPU needed)."""
import ctypes

import pytest
import torch

import extreme_weight_quantization_amd as E
from extreme_weight_quantization_amd import binding

A = 1 << 20   # a 16-byte aligned fake device address: validation never dereferences it
BIG = 1 << 40
NAMES = ("aqlm_linear_act", "aqlm_gated", "aqlm_linear_act_backward", "aqlm_gated_backward")
SHAPE = dict(act=2, M=2, B=8, g=8, out=16, n_in=64, batch=40)


@pytest.fixture(scope="module")
def lib():
    return E.load_library()


def pair(v):
    return None if v is None else (ctypes.c_void_p * 2)(*v) if isinstance(v, (tuple, list)) else (ctypes.c_void_p * 2)(v, v)


def call(name, **kw):
    a = dict(codes=A, codebooks=A, scales=A, x=A, bias=A, residual=A, z=A, y=A, dx=A, dbias=A, ws=A, ws_bytes=BIG, **SHAPE)
    a.update(kw)
    tail = (a["ws"], a["ws_bytes"], a["act"], a["M"], a["B"], a["g"], a["out"], a["n_in"], a["batch"], None)
    fn = getattr(E.load_library(), name)
    one, two = (a["codes"], a["codebooks"], a["scales"]), tuple(pair(a[k]) for k in ("codes", "codebooks", "scales"))
    if name == "aqlm_linear_act":
        return fn(*one, a["x"], a["bias"], a["residual"], a["z"], a["y"], *tail)
    if name == "aqlm_gated":
        return fn(*two, a["x"], pair(a["bias"]), pair(a["z"]), a["y"], *tail)
    if name == "aqlm_linear_act_backward":
        return fn(*one, a["x"], a["z"], a["dx"], a["dbias"], *tail)
    return fn(*two, a["x"], pair(a["z"]), a["dx"], pair(a["dbias"]), *tail)


def result(name):
    return "dx" if name.endswith("backward") else "y"


@pytest.mark.parametrize("name", NAMES)
def test_refusals(lib, name):
    for key in ("codes", "codebooks", "scales", "x", result(name), "ws"):
        assert call(name, **{key: 0}) == binding.AQLM_ERR_NULL, key
        if key != "scales":
            assert call(name, **{key: A + 8}) == binding.AQLM_ERR_ALIGN, key
    assert call(name, scales=A + 1) == binding.AQLM_ERR_ALIGN
    assert call(name, z=A + 8) == binding.AQLM_ERR_ALIGN
    assert call(name, **{"dbias" if name.endswith("backward") else "bias": A + 1}) == binding.AQLM_ERR_ALIGN
    for act in (-1, 5):
        assert call(name, act=act) == binding.AQLM_ERR_ACT
    for M, B, g in ((9, 8, 8), (0, 8, 8), (2, 17, 8), (1, 0, 8), (2, 8, 3), (1, 16, 64)):
        assert call(name, M=M, B=B, g=g) == binding.AQLM_ERR_SCHEME
    for kw in (dict(n_in=60), dict(n_in=0), dict(n_in=(1 << 20) + 8), dict(out=-1), dict(batch=-1),
               dict(out=(1 << 24) + 1), dict(batch=1 << 31), dict(ws_bytes=1 << 8),
               dict(out=1 << 24, n_in=1 << 20), dict(out=-(1 << 63)), dict(batch=-(1 << 63)), dict(n_in=-(1 << 63))):
        assert call(name, **kw) == binding.AQLM_ERR_SHAPE, kw
    assert call(name, M=1, B=8, g=32, n_in=48) == binding.AQLM_ERR_SHAPE


def test_refusals_of_single_calls(lib):
    assert call("aqlm_linear_act", residual=A + 8) == binding.AQLM_ERR_ALIGN
    # an activation's backward pass needs its pre-activations, the gated one always
    assert call("aqlm_linear_act_backward", z=0) == binding.AQLM_ERR_NULL
    for act in range(5):
        assert call("aqlm_gated_backward", act=act, z=(A, 0)) == binding.AQLM_ERR_NULL
    assert call("aqlm_gated_backward", z=None) == binding.AQLM_ERR_NULL
    assert call("aqlm_gated_backward", dbias=(A, 0)) == binding.AQLM_ERR_NULL   # both bias sums or none
    assert call("aqlm_gated_backward", dbias=(0, A)) == binding.AQLM_ERR_NULL
    for name in ("aqlm_gated", "aqlm_gated_backward"):
        for key in ("codes", "codebooks", "scales"):
            assert call(name, **{key: None}) == binding.AQLM_ERR_NULL
            assert call(name, **{key: (A, 0)}) == binding.AQLM_ERR_NULL


def test_empty_problems_use_no_pointers(lib):
    for name in ("aqlm_linear_act", "aqlm_gated"):
        for kw in (dict(out=0), dict(batch=0)):
            assert call(name, codes=0, codebooks=0, scales=0, x=0, y=0, ws=0, ws_bytes=0, **kw) == binding.AQLM_OK
    for name in ("aqlm_linear_act_backward", "aqlm_gated_backward"):
        assert call(name, batch=0, codes=0, x=0, dx=0, dbias=0, z=0, ws=0, ws_bytes=0) == binding.AQLM_OK
        assert call(name, out=0, dx=0) == binding.AQLM_ERR_NULL   # dx = 0 has to be written


def test_workspace_bytes(lib):
    fns = (E.linear_act_workspace_bytes, E.gated_workspace_bytes, E.linear_act_backward_workspace_bytes,
           E.gated_backward_workspace_bytes)
    for f in fns:
        assert f(2, 8, 8, 0, 64, 5) == 0 and f(2, 8, 8, 64, 64, 0) == 0
        assert f(2, 8, 8, 1000, 1000, 500) > 0
        for bad in ((9, 8, 8, 64, 64, 1), (2, 8, 8, -1, 64, 1), (2, 8, 8, 64, 60, 1), (2, 8, 8, 64, 64, -1)):
            with pytest.raises(ValueError):
                f(*bad)
    # exactly the workspace is enough, one byte less is not
    for name, f in zip(NAMES, fns):
        n = f(2, 8, 8, 16, 72, 40)
        assert call(name, n_in=72, ws_bytes=n - 1) == binding.AQLM_ERR_SHAPE
    for name in NAMES:
        assert getattr(lib, name + "_workspace_bytes")(2, 8, 8, 64, 64, 1, None) == binding.AQLM_ERR_NULL


def lists_call(two, **kw):
    a = dict(table=A, entries=A, eb=1 << 20, cb=A, scales=A, x=A, bias=A, residual=A, z=A, y=A, ws=A, ws_bytes=BIG,
             act=2, M=1, B=16, g=8, out=64, n_in=512, batch=1)
    a.update(kw)
    tail = (a["ws"], a["ws_bytes"], a["act"], a["M"], a["B"], a["g"], a["out"], a["n_in"], a["batch"], None)
    lib = E.load_library()
    if not two:
        return lib.aqlm_linear_act_lists(a["table"], a["entries"], a["eb"], a["cb"], a["scales"], a["x"], a["bias"],
                                         a["residual"], a["z"], a["y"], *tail)
    eb = None if a["eb"] is None else (ctypes.c_int64 * 2)(a["eb"], a["eb"])
    return lib.aqlm_gated_lists(pair(a["table"]), pair(a["entries"]), eb, pair(a["cb"]), pair(a["scales"]), a["x"],
                                pair(a["bias"]), pair(a["z"]), a["y"], *tail)


@pytest.mark.parametrize("two", [False, True])
def test_refusals_of_the_list_calls(lib, two):
    for key in ("table", "entries", "cb", "scales", "x", "y", "ws"):
        assert lists_call(two, **{key: 0}) == binding.AQLM_ERR_NULL, key
        if key != "scales":
            assert lists_call(two, **{key: A + 8}) == binding.AQLM_ERR_ALIGN, key
    for key in ("scales", "bias"):
        assert lists_call(two, **{key: A + 1}) == binding.AQLM_ERR_ALIGN
    assert lists_call(two, z=A + 8) == binding.AQLM_ERR_ALIGN
    assert lists_call(two, act=5) == binding.AQLM_ERR_ACT
    assert lists_call(two, M=2, B=8) == binding.AQLM_ERR_SCHEME
    for kw in (dict(batch=2), dict(batch=-1), dict(n_in=516), dict(eb=-1), dict(ws_bytes=100), dict(ws_bytes=-1)):
        assert lists_call(two, **kw) == binding.AQLM_ERR_SHAPE, kw
    for kw in (dict(batch=0), dict(out=0)):
        assert lists_call(two, table=0, entries=0, x=0, y=0, ws=0, **kw) == binding.AQLM_OK
    need = E.lists_fused_workspace_bytes([64] * (1 + two), 512)
    assert lists_call(two, ws_bytes=need - 256) == binding.AQLM_ERR_SHAPE
    if two:
        for key in ("table", "entries", "cb", "scales", "eb"):
            assert lists_call(two, **{key: None}) == binding.AQLM_ERR_NULL


def test_the_binding_refuses(lib):
    codes = torch.zeros((4, 8, 2), dtype=torch.uint8)
    cb = torch.zeros((2, 256, 8), dtype=torch.float16)
    s = torch.ones(4, dtype=torch.float16)
    x, dy = torch.zeros((1, 64), dtype=torch.float16), torch.zeros((1, 4), dtype=torch.float16)
    layer = (codes, cb, s)
    with pytest.raises(ValueError, match="GPU tensor"):
        E.aqlm_linear_act(*layer, x)
    with pytest.raises(ValueError, match="GPU tensor"):
        E.aqlm_gated(layer, layer, x)
    with pytest.raises(ValueError, match="GPU tensor"):
        E.aqlm_linear_act_backward(*layer, dy)
    with pytest.raises(ValueError, match="GPU tensor"):
        E.aqlm_gated_backward(layer, layer, dy, dy, dy)
    for bad in ("swish", None, 3, []):
        with pytest.raises(ValueError, match="act must be one of"):
            E.aqlm_linear_act(*layer, x, act=bad)


def test_the_binding_checks_layers():
    """The checks that come after the device's, on CPU tensors handed to them directly."""
    from extreme_weight_quantization_amd import fused
    dev = torch.device("cpu")
    codes = torch.zeros((4, 8, 2), dtype=torch.uint8)
    cb, s = torch.zeros((2, 256, 8), dtype=torch.float16), torch.ones(4, dtype=torch.float16)
    assert fused._layer(codes, cb, s, dev)[:3] == ((2, 8, 8), 4, 64)
    for bad in ((codes.to(torch.int16), cb, s), (codes[:, :, :1].contiguous(), cb, s), (codes, cb[:, :200], s),
                (codes, cb.float(), s), (codes, cb, s[:3]), (codes, cb, s.float()), (codes[0], cb, s),
                (codes.transpose(0, 1), cb, torch.ones(8, dtype=torch.float16)), (codes, cb[0], s)):
        with pytest.raises(ValueError):
            fused._layer(*bad, dev)
    with pytest.raises(ValueError):
        fused._gated_layers((codes, cb, s), (codes[:3], cb, s[:3]), dev)
    for bad in (s.float(), s[:3], torch.ones(8, dtype=torch.float16)[::2], s.to("meta")):
        with pytest.raises(ValueError):
            fused._tensor("t", bad, dev, (4,))
    for bad in (torch.zeros(8), torch.zeros(16, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            fused._workspace(bad, lambda: 0, dev)
