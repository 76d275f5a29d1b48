"""Where the library says that no weight is rounded, none is: products whose large codewords cancel exactly, so that a
weight or a sum of codewords rounded to fp16 would be many times the tolerance (reference: tests/fused_reference.py).

Neighbouring groups (backward: rows) hold the same codes in all codebooks but the last and meet opposite factors.  The
last codebook is 2^-8 of the others, so the result is of the size of its differences, while a rounded weight is off by
up to 2^-11 of the large codewords: some 4e-3 rms over 512 inputs, against a tolerance below 1e-3 for fp32 sums."""
import numpy as np
import pytest
import torch

import extreme_weight_quantization_amd as E
import fused_reference as R
from extreme_weight_quantization_amd import synth

pytestmark = pytest.mark.gpu

SCHEMES = {"2x8": (2, 8, 8), "4x8g16": (4, 8, 16), "8x8g32": (8, 8, 32), "3x5g2": (3, 5, 2), "2x10g4": (2, 10, 4)}
SMALL = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need an MI355X")
    E.load_library()


def layer(scheme, out, n_in, seed, rows):
    """Neighbouring groups, or rows, share all codes but the last codebook's; (GPU tensors, float64 weights)."""
    M, B, g = SCHEMES[scheme]
    L = synth.make_layer_mbg(M, B, g, out, n_in, 1, seed, 1.0)
    L.codebooks[M - 1] = (L.codebooks[M - 1].astype(np.float64) * SMALL).astype(np.float16)
    if rows:
        L.codes[1::2, :, :-1] = L.codes[0:out // 2 * 2:2, :, :-1]
        L.scales[1::2] = L.scales[0:out // 2 * 2:2]
    else:
        G = n_in // g
        L.codes[:, 1::2, :-1] = L.codes[:, 0:G // 2 * 2:2, :-1]
    return tuple(torch.from_numpy(a).cuda() for a in (L.codes, L.codebooks, L.scales)), R.weights(L)


def plain_layer(scheme, out, n_in, seed):
    """Independent codes and like codebooks; a product with x has about unit variance."""
    M, B, g = SCHEMES[scheme]
    L = synth.make_layer_mbg(M, B, g, out, n_in, 1, seed, 0.05)
    L.scales = (L.scales.astype(np.float64) / (0.05 * np.sqrt(M * n_in))).astype(np.float16)
    return tuple(torch.from_numpy(a).cuda() for a in (L.codes, L.codebooks, L.scales)), R.weights(L)


def inputs(rng, T, n, step):
    """Normal fp16 numbers, each run of `step` the negative of the one before it."""
    v = rng.normal(0, 1, (T, n // (2 * step), 1, step))
    return torch.from_numpy(np.concatenate((v, -v), 2).reshape(T, n).astype(np.float16))


FORWARD = [*[("2x8", out, n, T) for out, n in ((272, 512), (131, 528)) for T in (1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 64)],
           *[("2x8", 4112, 8192, T) for T in (1, 2, 3, 4)], ("2x8", 1040, 2048, 40),
           *[("2x8", out, n, T) for out, n in ((272, 512), (131, 528)) for T in (65, 80, 97, 128, 130, 257, 320, 384)],
           *[("4x8g16", out, n, T) for out, n in ((272, 512), (131, 544)) for T in (17, 33, 64, 65, 80, 97, 130, 256)],
           *[(s, 72, 512, T) for s in ("4x8g16", "8x8g32", "3x5g2", "2x10g4") for T in (1, 2, 5, 8, 9, 16)]]


@pytest.mark.parametrize("scheme,out,n_in,T", FORWARD)
def test_forward(scheme, out, n_in, T):
    rng = np.random.default_rng(T)
    gate, wg = layer(scheme, out, n_in, 1, False)
    up, wu = layer(scheme, out, n_in, 2, False)
    x = inputs(rng, T, n_in, SCHEMES[scheme][2])
    z = torch.empty((T, out), dtype=torch.float16, device="cuda")
    y = E.aqlm_linear_act(*gate, x.cuda(), z=z)
    want, tol, wz, tz = R.linear(wg, x.double(), "none", None, None, False)
    R.assert_within(y, want, tol, "y")
    R.assert_within(z, wz, tz, "z")
    y = E.aqlm_gated(gate, up, x.cuda(), act="none")
    want, tol, _ = R.gated(wg, wu, x.double(), "none", None, None, False)
    R.assert_within(y, want, tol, "gated y")


# beyond the batches of the gated product
LINEAR = [*[("2x8", out, n, T) for out, n in ((272, 512), (131, 528)) for T in (385, 500, 512)],
          *[("4x8g16", out, n, T) for out, n in ((272, 512), (131, 544)) for T in (257, 300, 320)]]


@pytest.mark.parametrize("scheme,out,n_in,T", LINEAR)
def test_linear(scheme, out, n_in, T):
    rng = np.random.default_rng(T)
    gpu, w = layer(scheme, out, n_in, 1, False)
    x = inputs(rng, T, n_in, SCHEMES[scheme][2])
    y = E.aqlm_linear_act(*gpu, x.cuda())
    want, tol, _, _ = R.linear(w, x.double(), "none", None, None, False)
    R.assert_within(y, want, tol, "y")


# both sides of the gated product's last batch straight from the codes
@pytest.mark.parametrize("scheme,T", [("2x8", 384), ("2x8", 385), ("4x8g16", 256), ("4x8g16", 257)])
def test_gated_limits(scheme, T):
    rng = np.random.default_rng(T)
    for out, n_in in ((272, 512), (131, 544)):
        (gate, wg), (up, wu) = (plain_layer(scheme, out, n_in, seed) for seed in (1, 2))
        x = torch.from_numpy(rng.normal(0, 1, (T, n_in)).astype(np.float16))
        zg, zu = (torch.empty((T, out), dtype=torch.float16, device="cuda") for _ in range(2))
        y = E.aqlm_gated(gate, up, x.cuda(), zg=zg, zu=zu)
        want, tol, zs = R.gated(wg, wu, x.double(), "silu", None, None, T in (385, 257))
        R.assert_within(y, want, tol, "y")
        for got, (z, tz) in zip((zg, zu), zs):
            R.assert_within(got, z, tz, "z")


BACKWARD = [*[("2x8", out, T) for out in (512, 520, 1036) for T in (1, 8, 16, 17, 33, 64, 65, 200, 256)],
            *[("4x8g16", out, T) for out in (512, 520, 1036) for T in (1, 16, 17, 64, 128)]]


@pytest.mark.parametrize("scheme,out,T", BACKWARD)
def test_backward(scheme, out, T):
    """The factors of a pair are equal but for their sign, and so are their roundings: what is left of them is H of the
    pair's difference."""
    rng = np.random.default_rng(T)
    n_in = 272
    gpu, w = layer(scheme, out, n_in, 3, True)
    dy = inputs(rng, T, out, 1)
    dx, _ = E.aqlm_linear_act_backward(*gpu, dy.cuda())
    d = dy.double()
    want = d @ w
    pairs = (d[:, ::2] ** 2) @ ((w[::2] - w[1::2]) ** 2)
    e = R.TEN_SIGMA * (R.H * pairs.sqrt() + 2.0 ** -24 * 4 * out ** 0.5 * ((d * d) @ (w * w)).sqrt())
    R.assert_within(dx, want, e + R.H * (want.abs() + e) + R.SUB, "dx")
