"""Refusals of the MX4 and mixture-of-experts operators on the host, before any HIP call (no GPU needed)."""
import ctypes

import pytest
import torch

import extreme_weight_quantization_amd as E
from extreme_weight_quantization_amd import binding, moe, mx4

A = 1 << 20   # a 16-byte aligned fake device address: validation never dereferences it
BIG = 1 << 40
OK, NULL, SHAPE, SCHEME, ALIGN = (binding.AQLM_OK, binding.AQLM_ERR_NULL, binding.AQLM_ERR_SHAPE, binding.AQLM_ERR_SCHEME,
                                  binding.AQLM_ERR_ALIGN)
LOW = -(1 << 63)


@pytest.fixture(scope="module")
def lib():
    return E.load_library()


def convert(name, a=A, b=A, c=A, rows=4, n_in=64):
    return getattr(E.load_library(), name)(a, b, c, rows, n_in, None)


def test_conversions(lib):
    for name in ("aqlm_mx4_quantize", "aqlm_mx4_decode"):
        for key in "abc":
            assert convert(name, **{key: 0}) == NULL
            # the scales (third of quantize, second of decode) may lie anywhere
            anywhere = "c" if name.endswith("quantize") else "b"
            if key != anywhere:
                assert convert(name, **{key: A + 8}) == ALIGN
        for kw in (dict(rows=-1), dict(rows=LOW), dict(rows=(1 << 40) + 1), dict(n_in=0), dict(n_in=33), dict(n_in=48),
                   dict(n_in=(1 << 20) + 32), dict(n_in=-32)):
            assert convert(name, **kw) == SHAPE, kw
        assert convert(name, a=0, b=0, c=0, rows=0) == OK


def linear(**kw):
    a = dict(codes=A, scales=A, x=A, xs=0, bias=A, residual=A, y=A, ws=A, ws_bytes=BIG, act=2, out=16, n_in=4096, batch=40)
    a.update(kw)
    return E.load_library().aqlm_mx4_linear(*a.values(), None)


def test_linear(lib):
    for key in ("codes", "scales", "x", "y", "ws"):
        assert linear(**{key: 0}) == NULL, key
    for key in ("codes", "x", "residual", "y", "ws"):
        assert linear(**{key: A + 8}) == ALIGN, key
    assert linear(bias=A + 1) == ALIGN
    for a in (-1, 5):
        assert linear(act=a) == binding.AQLM_ERR_ACT
    for kw in (dict(n_in=0), dict(n_in=40), dict(n_in=(1 << 20) + 32), dict(out=-1), dict(out=(1 << 24) + 1), dict(batch=-1),
               dict(batch=(1 << 30) + 1), dict(batch=LOW), dict(out=LOW), dict(n_in=LOW), dict(ws_bytes=100), dict(ws_bytes=-1)):
        assert linear(**kw) == SHAPE, kw
    for kw in (dict(out=0), dict(batch=0)):
        assert linear(codes=0, scales=0, x=0, y=0, ws=0, ws_bytes=0, **kw) == OK


def test_linear_workspace(lib):
    f = E.mx4_linear_workspace_bytes
    assert f(0, 4096, 40) == 0 and f(64, 4096, 0) == 0
    assert linear(ws_bytes=f(16, 4096, 40) - 1) == SHAPE
    for n_in in (32, 1056, 4096, 28672):
        for four in (False, True):
            sizes = [f(1000, n_in, t, x_mx4=four) for t in list(range(1, 300)) + [1000, 2048, 5000, 1 << 20]]
            assert sizes == sorted(sizes)
    for bad in ((-1, 64, 1), (64, 60, 1), (64, 64, -1)):
        with pytest.raises(ValueError):
            f(*bad)
    assert lib.aqlm_mx4_linear_workspace_bytes(0, 64, 64, 1, None) == NULL


def route(**kw):
    a = dict(x=A, router=A, bias=0, ids=A, weights=A, ws=A, ws_bytes=BIG, score=0, renorm=1, scale=1.0, experts=8, n_in=64, k=2,
             tokens=3)
    a.update(kw)
    return E.load_library().aqlm_moe_route(*a.values(), None)


def test_route(lib):
    for key in ("x", "router", "ids", "weights", "ws"):
        assert route(**{key: 0}) == NULL, key
    for key, off in (("x", 8), ("router", 8), ("ids", 2), ("weights", 2), ("bias", 2), ("ws", 8)):
        assert route(**{key: A + off}) == ALIGN, key
    for s in (-1, 2):
        assert route(score=s) == binding.AQLM_ERR_ACT
    for kw in (dict(k=0), dict(k=9), dict(k=17, experts=64), dict(experts=0), dict(experts=513), dict(n_in=0), dict(n_in=4),
               dict(n_in=(1 << 20) + 8), dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(ws_bytes=8), dict(k=LOW),
               dict(experts=LOW), dict(tokens=LOW)):
        assert route(**kw) == SHAPE, kw
    assert route(tokens=0, x=0, router=0, ids=0, weights=0, ws=0, ws_bytes=0) == OK
    n = E.moe_route_workspace_bytes(8, 64, 2, 3)
    assert route(ws_bytes=n - 1) == SHAPE
    for e in (1, 8, 64, 511):
        for n_in in (8, 1000, 4096):
            sizes = [E.moe_route_workspace_bytes(e, n_in, 1, t) for t in list(range(1, 700)) + [5000, 1 << 20]]
            assert sizes == sorted(sizes)


def three(v):
    return None if v is None else (ctypes.c_void_p * 3)(*(v if isinstance(v, tuple) else (v, v, v)))


def layer(four, **kw):
    a = dict(codes=A, codebooks=A, scales=A, x=A, ids=A, weights=A, residual=A, y=A, ws=A, ws_bytes=BIG, act=2, M=2, B=8, g=8,
             experts=4, n_in=64, inner=96, k=2, tokens=5)
    a.update(kw)
    for key in ("codes", "codebooks", "scales"):
        a[key] = three(a[key])
    if four:
        for key in ("codebooks", "M", "B", "g"):
            del a[key]
        return E.load_library().aqlm_moe_mx4(*a.values(), None)
    return E.load_library().aqlm_moe(*a.values(), None)


@pytest.mark.parametrize("four", [False, True])
def test_layer(lib, four):
    arrays = ("codes", "scales") if four else ("codes", "codebooks", "scales")
    for key in arrays:
        assert layer(four, **{key: None}) == NULL
        for i in range(3):
            assert layer(four, **{key: tuple(0 if j == i else A for j in range(3))}) == NULL
    for key in ("x", "ids", "weights", "y", "ws"):
        assert layer(four, **{key: 0}) == NULL, key
    for key, off in (("x", 8), ("ids", 2), ("weights", 2), ("residual", 8), ("y", 8), ("ws", 8), ("codes", 8)):
        assert layer(four, **{key: A + off}) == ALIGN, key
    if not four:
        assert layer(four, codebooks=A + 8) == ALIGN and layer(four, scales=A + 1) == ALIGN
        for M, B, g in ((9, 8, 8), (0, 8, 8), (2, 17, 8), (2, 8, 3)):
            assert layer(four, M=M, B=B, g=g) == SCHEME
    for a in (-1, 5):
        assert layer(four, act=a) == binding.AQLM_ERR_ACT
    for kw in (dict(experts=0), dict(experts=513), dict(k=0), dict(k=17), dict(n_in=0), dict(n_in=(1 << 20) + 32), dict(inner=0),
               dict(inner=100), dict(n_in=100), dict(tokens=-1), dict(tokens=513), dict(tokens=1025, k=1), dict(ws_bytes=100),
               dict(tokens=LOW), dict(inner=LOW), dict(k=LOW), dict(experts=LOW)):
        assert layer(four, **kw) == SHAPE, kw
    assert layer(four, tokens=0, x=0, ids=0, weights=0, y=0, ws=0, ws_bytes=0) == OK
    f = (lambda t: E.moe_mx4_workspace_bytes(4, 64, 96, t, 2)) if four else (lambda t: E.moe_workspace_bytes(2, 8, 8, 4, 64, 96, t, 2))
    assert layer(four, ws_bytes=f(5) - 1) == SHAPE and f(0) == 0
    sizes = [f(t) for t in range(1, 513)]
    assert sizes == sorted(sizes)
    with pytest.raises(ValueError):
        f(513)


def test_the_binding_refuses(lib):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)   # noqa: E731
    f16 = lambda *s: torch.zeros(s, dtype=torch.float16)   # noqa: E731
    for call in (lambda: E.aqlm_mx4_quantize(f16(2, 64)), lambda: E.aqlm_mx4_decode(u8(2, 32), u8(2, 2)),
                 lambda: E.aqlm_mx4_linear(u8(2, 32), u8(2, 2), f16(1, 64)),
                 lambda: E.aqlm_mx4_linear(u8(2, 32), u8(2, 2), (u8(1, 32), u8(1, 2))),
                 lambda: E.aqlm_moe_route(f16(1, 64), f16(4, 64), 2),
                 lambda: E.aqlm_moe_mx4(*[(u8(2, 64, 32), u8(2, 64, 2))] * 3, f16(1, 64), None, None)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(ValueError, match="score must be"):
        E.aqlm_moe_route(f16(1, 64), f16(4, 64), 2, score="top")
    with pytest.raises(ValueError, match="score must be"):
        E.aqlm_moe_route(f16(1, 64), f16(4, 64), 2, score=["softmax"])
    with pytest.raises(ValueError, match="act must be one of"):
        E.aqlm_mx4_linear(u8(2, 32), u8(2, 2), f16(1, 64), act="swish")
    with pytest.raises(ValueError, match="pair"):
        E.aqlm_mx4_linear(u8(2, 32), u8(2, 2), (u8(1, 32),))


def test_the_binding_checks_layers():
    """The checks that come after the device's, on CPU tensors handed to them directly."""
    dev = torch.device("cpu")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)   # noqa: E731
    assert mx4._pair("w", u8(3, 32), u8(3, 2), dev)[:2] == (3, 64)
    for codes, scales in ((u8(3, 24), u8(3, 1)), (u8(3, 32), u8(3, 3)), (u8(3, 32).short(), u8(3, 2)), (u8(32, 3).t(), u8(3, 2)),
                          (u8(3, 32), u8(3, 2).to("meta")), (u8(1, 3, 32), u8(3, 2))):
        with pytest.raises(ValueError):
            mx4._pair("w", codes, scales, dev)
    cb = torch.zeros((4, 2, 256, 8), dtype=torch.float16)
    f16 = lambda *s: torch.zeros(s, dtype=torch.float16)   # noqa: E731
    gate, down = (u8(4, 96, 8, 2), cb, f16(4, 96)), (u8(4, 64, 12, 2), cb, f16(4, 64))
    assert moe._layers(moe._experts, gate, gate, down, dev)[:4] == ((2, 8, 8), 4, 64, 96)
    for bad in ((gate, gate, gate), (gate, down, down), (gate, gate, (u8(4, 64, 12, 2), cb[:, :1].contiguous(), f16(4, 64))),
                ((u8(3, 96, 8, 2), cb, f16(4, 96)), gate, down), ((u8(4, 96, 8, 2).short(), cb, f16(4, 96)), gate, down),
                ((u8(96, 8, 2), cb, f16(4, 96)), gate, down), ((u8(4, 96, 8, 2), cb[:, :, :200], f16(4, 96)), gate, down)):
        with pytest.raises(ValueError):
            moe._layers(moe._experts, *bad, dev)
    g4, d4 = (u8(4, 96, 32), u8(4, 96, 2)), (u8(4, 64, 48), u8(4, 64, 3))
    assert moe._layers(moe._experts_mx4, g4, g4, d4, dev)[:4] == ((), 4, 64, 96)
    for bad in ((g4, g4, g4), (g4, d4, d4), ((u8(4, 96, 24), u8(4, 96, 2)), g4, d4), ((u8(4, 96, 32), u8(4, 96, 3)), g4, d4)):
        with pytest.raises(ValueError):
            moe._layers(moe._experts_mx4, *bad, dev)
