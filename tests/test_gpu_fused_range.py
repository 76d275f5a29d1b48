"""Gradients whose products leave fp16's range on the way to a dx inside it: dz and the row scales reach the matrix
cores without overflow and without a loss of small values (reference: tests/fused_reference.py).

The operand of dx is d = dz times, where the codewords are multiplied as they are, the row's scale.  It is rounded to
fp16 once after an exact power of two per token and block of rows, which leaves a block's largest |d| at 2^-5 or more;
an element is off by H of itself or, where that power makes it subnormal, by 2^-25 of the scaled unit, which is below
2^-20 of the block's largest (2^-19 of the token's, with the second rounding of a block that joins a larger one)."""
import itertools

import numpy as np
import pytest
import torch

import extreme_weight_quantization_amd as E
import fused_reference as R
from extreme_weight_quantization_amd import synth

pytestmark = pytest.mark.gpu

SCHEMES = {"2x8": (2, 8, 8), "1x16": (1, 16, 8), "4x8g16": (4, 8, 16), "1x8g4": (1, 8, 4), "2x10g4": (2, 10, 4)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need an MI355X")
    E.load_library()


def layer(scheme, out, n_in, seed, sigma=0.05, size=1.0):
    """Weights of about `size` / sqrt(in); codebooks of standard deviation sigma.  (GPU tensors, float64 weights, scales)"""
    M, B, g = SCHEMES[scheme]
    L = synth.make_layer_mbg(M, B, g, out, n_in, 1, seed, sigma)
    L.scales = (L.scales.astype(np.float64) * (size / (sigma * np.sqrt(M * n_in)))).astype(np.float16)
    gpu = tuple(torch.from_numpy(a).cuda() for a in (L.codes, L.codebooks, L.scales))
    return gpu, R.weights(L), torch.from_numpy(L.scales.astype(np.float64))


def normal(rng, *shape, scale=1.0):
    """fp16 normal numbers; scale broadcasts."""
    return torch.from_numpy(np.clip(rng.normal(0, 1, shape) * np.asarray(scale), -65504, 65504).astype(np.float16))


def tolerance(dzs, ws, ss):
    """dx and its bound: one rounding of every weight and of every element of d, the latter at least 2^-19 of the
    token's largest |d|, with and without the scale in d; a weight below 2^-14 is off by up to 2^-25."""
    dx, r2, small2, sub2, n = 0.0, 0.0, 0.0, 0.0, 0
    plain, scaled = (torch.stack([d.abs().amax(1, keepdim=True) for d in ds]).amax(0)
                     for ds in (dzs, [dz * s for dz, s in zip(dzs, ss)]))
    for dz, w, s in zip(dzs, ws, ss):
        dx = dx + dz @ w
        r2 = r2 + (dz * dz) @ (w * w)
        small2 = small2 + torch.maximum(plain ** 2 * (w * w).sum(0), scaled ** 2 * ((w / s[:, None]) ** 2).sum(0))
        sub2 = sub2 + (dz * dz).sum(1, keepdim=True)
        n += w.shape[0]
    k = R.H * 2 ** 0.5 + 2.0 ** -24 * 4 * n ** 0.5 + 2.0 ** -20
    e = R.TEN_SIGMA * (k * r2.sqrt() + 2.0 ** -19 * small2.sqrt() + 2.0 ** -25 * sub2.sqrt())
    return dx, e + R.H * (dx.abs() + e) + R.SUB


def check_gated(scheme, out, n_in, T, dy, zg, zu, name="silu", size=1.0, sigma=0.05, seed=0):
    gate, wg, sg = layer(scheme, out, n_in, 2 * seed, sigma, size)
    up, wu, su = layer(scheme, out, n_in, 2 * seed + 1, sigma, size)
    dx, dbg, dbu = E.aqlm_gated_backward(gate, up, dy.cuda(), zg.cuda(), zu.cuda(), act=name, need_dbias=True)
    dzs = R.gated_grads(dy.double(), zg.double(), zu.double(), name)
    want, tol = tolerance(dzs, [wg, wu], [sg, su])
    assert want.abs().max() < 60000, "the expected dx is inside fp16's range"
    R.assert_within(dx, want, tol, "dx")
    return dzs


def check_linear(scheme, out, n_in, T, dy, z, name, size=1.0, sigma=0.05, seed=0):
    gpu, w, s = layer(scheme, out, n_in, seed, sigma, size)
    dx, _ = E.aqlm_linear_act_backward(*gpu, dy.cuda(), act=name, z=None if z is None else z.cuda())
    dzs = R.linear_grads(dy.double(), None if z is None else z.double(), name)
    want, tol = tolerance(dzs, [w], [s])
    assert want.abs().max() < 60000
    R.assert_within(dx, want, tol, "dx")
    return dzs


# the gradients inside the product, the codes direct, decoded first with and without split k steps
TOKENS = [5, 40, 100, 300, 1100]
CASES = list(itertools.product(SCHEMES, TOKENS))


@pytest.mark.parametrize("scheme,T", CASES)
def test_gated_gradients_beyond_the_range(scheme, T):
    """dy zu act' in the hundred thousands, dx in the hundreds."""
    rng = np.random.default_rng(1)
    for out, n_in in ((264, 272), (1100, 528)):
        dzs = check_gated(scheme, out, n_in, T, normal(rng, T, out, scale=200), normal(rng, T, out),
                          normal(rng, T, out, scale=500), size=2.0 ** -8)
        assert dzs[0].abs().max() > 70000


@pytest.mark.parametrize("scheme,T", CASES)
def test_linear_gradients_near_the_end_of_the_range(scheme, T):
    """|dy| up to 65504 times scales whose mantissa is up to 2."""
    rng = np.random.default_rng(2)
    for name in ("none", "gelu"):
        out, n_in = 264, 272
        dy = normal(rng, T, out, scale=30000)
        check_linear(scheme, out, n_in, T, dy, None if name == "none" else normal(rng, T, out), name, size=2.0 ** -7)


@pytest.mark.parametrize("scheme,T", CASES)
def test_small_gradients_keep_their_bits(scheme, T):
    """dy zu act' around 2^-20 in every element, weights large: dx is a normal number with all of its bits."""
    rng = np.random.default_rng(3)
    for out, n_in in ((264, 272), (1100, 528)):
        dzs = check_gated(scheme, out, n_in, T, normal(rng, T, out, scale=2.0 ** -12), normal(rng, T, out),
                          normal(rng, T, out, scale=2.0 ** -8), name="relu", size=2.0 ** 8)
        assert dzs[0].abs().max() < 2.0 ** -14
    check_linear(scheme, 264, 272, T, normal(rng, T, 264, scale=2.0 ** -13), normal(rng, T, 264, scale=0.125) - 4, "gelu",
                 size=2.0 ** 9)


@pytest.mark.parametrize("scheme,T", CASES)
def test_tokens_and_rows_of_very_different_size(scheme, T):
    """Tokens from 2^-12 to 2^8, and inside a token runs of rows 2^-16 to 2^4 of it: rising, falling and mixed."""
    rng = np.random.default_rng(4)
    out, n_in = 2200, 272
    tok = 2.0 ** rng.uniform(-12, 8, (T, 1))
    for k, blocks in enumerate(([-16, -8, 0, 2, 4], [4, 2, 0, -8, -16], [0, -14, 4, -16, 0], [-3, 3, -3, 3, -3])):
        rows = 2.0 ** np.repeat(np.array(blocks, dtype=np.float64), 512)[:out]
        check_gated(scheme, out, n_in, T, normal(rng, T, out, scale=tok * rows), normal(rng, T, out),
                    normal(rng, T, out, scale=16), size=2.0 ** -3, seed=k)
    zeros = normal(rng, T, out)
    zeros[:, :700] = 0
    zeros[::2, 1500:] = 0
    zeros[T // 2] = 0
    check_gated(scheme, out, n_in, T, zeros, normal(rng, T, out), normal(rng, T, out, scale=64), seed=5)


@pytest.mark.parametrize("scheme,T", [(s, t) for s, t in CASES if s in ("1x16", "1x8g4") or t <= 100 and s in ("2x8", "4x8g16")])
def test_codewords_and_scales_whose_product_is_no_fp16_number(scheme, T):
    """Where codewords are multiplied as they are, their product with the row's scale need not fit fp16."""
    rng = np.random.default_rng(6)
    out, n_in = 264, 272
    for sigma, size, dy_scale in ((2.0 ** -9, 2.0 ** -13, 2.0 ** 14), (2.0 ** 13, 2.0 ** 21, 2.0 ** -12)):
        gpu, w, s = layer(scheme, out, n_in, 6, sigma, size)
        dy, z = normal(rng, T, out, scale=dy_scale), normal(rng, T, out)
        dx, _ = E.aqlm_linear_act_backward(*gpu, dy.cuda(), act="relu", z=z.cuda())
        dz = R.linear_grads(dy.double(), z.double(), "relu")[0]
        want, r = dz @ w, ((dz * dz) @ (w * w)).sqrt()
        small = 2.0 ** -19 * (dz * s).abs().amax(1, keepdim=True) * ((w / s[:, None]) ** 2).sum(0).sqrt()
        e = R.TEN_SIGMA * ((R.H + 2.0 ** -24 * 4 * out ** 0.5 + 2.0 ** -20) * r + small)
        assert want.abs().max() < 60000
        R.assert_within(dx, want, e + R.H * (want.abs() + e) + R.SUB, f"dx {sigma}")


def test_an_infinite_gradient_next_to_large_and_small_ones():
    """Infinities and NaN do not take part in the choice of the power of two and stay in their token."""
    rng = np.random.default_rng(7)
    for scheme, T in itertools.product(("2x8", "1x16", "1x8g4"), (7, 40, 300)):
        out, n_in = 1100, 272
        gate, wg, sg = layer(scheme, out, n_in, 0, size=2.0 ** -8)
        up, wu, su = layer(scheme, out, n_in, 1, size=2.0 ** -8)
        dy, zg, zu = normal(rng, T, out, scale=200), normal(rng, T, out), normal(rng, T, out, scale=500)
        bad = dy.clone()
        bad[1, 3], bad[3, 1000] = float("inf"), float("nan")
        a = E.aqlm_gated_backward(gate, up, dy.cuda(), zg.cuda(), zu.cuda())[0]
        b = E.aqlm_gated_backward(gate, up, bad.cuda(), zg.cuda(), zu.cuda())[0]
        keep = [t for t in range(T) if t not in (1, 3)]
        assert torch.isfinite(a).all() and torch.equal(a[keep], b[keep]), (scheme, T)
        assert not torch.isfinite(b[1]).any() and torch.isnan(b[3]).all(), (scheme, T)


@pytest.mark.parametrize("scheme", list(SCHEMES))
@pytest.mark.parametrize("out,n_in,T", [(264, 272, 1100), (264, 272, 100), (264, 272, 7), (20000, 64, 300), (64, 64, 5003)])
def test_the_two_layers_of_a_token_at_different_levels(scheme, out, n_in, T):
    """dzg far above dzu in most tokens, below it in some: few and many blocks a token, more tokens than weights."""
    rng = np.random.default_rng(8)
    zu = normal(rng, T, out, scale=2.0 ** np.where(np.arange(T) % 5 == 2, -13.0, 14.0)[:, None])
    zg = normal(rng, T, out, scale=2.0 ** np.where(np.arange(T) % 5 == 2, 3.0, -8.0)[:, None])
    check_gated(scheme, out, n_in, T, normal(rng, T, out, scale=8), zg, zu, size=2.0 ** -9)


@pytest.mark.parametrize("T", [5, 40, 300])
def test_nan_pre_activations_give_nan(T):
    """For every activation that looks at them."""
    rng = np.random.default_rng(9)
    for name in ("relu", "silu", "gelu", "gelu_tanh"):
        gate, _, _ = layer("2x8", 264, 272, 0)
        up, _, _ = layer("2x8", 264, 272, 1)
        dy, zg, zu = normal(rng, T, 264) + 2, normal(rng, T, 264), normal(rng, T, 264)
        bad = zg.clone()
        bad[2, 100] = float("nan")
        a, b = (E.aqlm_linear_act_backward(*gate, dy.cuda(), act=name, z=z.cuda(), need_dbias=True) for z in (zg, bad))
        keep = [t for t in range(T) if t != 2]
        assert torch.equal(a[0][keep], b[0][keep]) and torch.isnan(b[0][2]).all(), (name, T)
        assert torch.isnan(b[1][100]) and int(torch.isnan(b[1]).sum()) == 1, (name, T)
        a, b = (E.aqlm_gated_backward(gate, up, dy.cuda(), z.cuda(), zu.cuda(), act=name)[0] for z in (zg, bad))
        assert torch.equal(a[keep], b[keep]) and torch.isnan(b[2]).all(), (name, T)
