"""The streaming 2x8 kernel with an epilogue (gemv_stream.hip): every batch that it serves, ragged slabs and row tails,
bias, residual and kept pre-activations, and sizes on both sides of each of its rules."""
import os
import re

import numpy as np
import pytest
import torch

import extreme_weight_quantization_amd as E
import fused_reference as R
from test_gpu_fused import half, layer

pytestmark = pytest.mark.gpu

SOURCE = os.path.join(os.path.dirname(os.path.abspath(E.__file__)), "csrc", "gemv_stream.hip")
CONSTANTS = {k: int(v) for k, v in re.findall(r"constexpr int (kS\w+) = (\d+);", open(SOURCE).read())}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need an MI355X")
    E.load_library()


def streams(out, n_in, T, two):
    """The kernel's rule: rows in whole 16 bytes of codes, enough slab steps a wave, and what its LDS holds."""
    c = CONSTANTS
    tile, cus = 8 if two else 16, torch.cuda.get_device_properties(0).multi_processor_count
    if T > c["kSMaxT"] or n_in % 64:
        return False
    n_rt = -(-out // tile)
    rmax, groups = -(-n_rt // min(n_rt, cus)), n_in // 8
    n_slab = -(-groups // c["kSSlab"])
    if rmax * n_slab < (c["kSMinSteps34"] if T > 2 else c["kSMinSteps"]) * c["kSWaves"]:
        return False
    x = -(-T * (-(-groups // 64) * 64 + 1) // 64) * 64 * 16
    sums = rmax * (min(c["kSWaves"], n_slab) + 1) * 16 * T * 4
    return 2 * 256 * c["kSRepl"] * 16 + x + sums <= 160 * 1024


# (out, in) and the batches that stream, on 256 compute units
LINEAR = [((4100, 8192), (1, 2, 3, 4)), ((8197, 8256), (1, 2, 3, 4)), ((257, 8256), (1, 2)), ((4112, 7936), (1, 2)),
          ((256, 8192), (1, 2)), ((256, 7936), ())]
GATED = [((2050, 8256), (1, 2, 3, 4)), ((2045, 8192), (1, 2)), ((2045, 7936), ()), ((3, 8256), (1, 2)), ((4104, 5440), (1, 2, 3, 4)),
         ((6144, 10240), (1, 2, 3, 4)), ((6152, 10240), (1, 2, 3))]


@pytest.mark.parametrize("size,served", LINEAR)
def test_linear(size, served):
    out, n_in = size
    rng = np.random.default_rng(out)
    gpu, w, _ = layer("2x8", out, n_in, out)
    for i, T in enumerate((1, 2, 3, 4, 5)):
        assert streams(out, n_in, T, False) == (T in served), (out, n_in, T)
        name = ("silu", "none", "gelu", "relu", "gelu_tanh")[i]
        x, b, r = half(rng, T, n_in), half(rng, out), half(rng, T, out)
        for keep, bias, residual in ((True, True, True), (False, i % 2 == 0, i % 2 == 1)):
            z = torch.full((T, out), float("nan"), dtype=torch.float16, device="cuda") if keep else None
            y = E.aqlm_linear_act(*gpu, x.cuda(), act=name, bias=b.cuda() if bias else None,
                                  residual=r.cuda() if residual else None, z=z)
            want, tol, wz, tz = R.linear(w, x.double(), name, b.double() if bias else None,
                                         r.double() if residual else None, False)
            R.assert_within(y, want, tol, f"y {T}")
            if keep:
                R.assert_within(z, wz, tz, f"z {T}")
        h = r.cuda()
        assert torch.equal(E.aqlm_linear_act(*gpu, x.cuda(), residual=h),
                           E.aqlm_linear_act(*gpu, x.cuda(), residual=h, y=h)), T


@pytest.mark.parametrize("size,served", GATED)
def test_gated(size, served):
    out, n_in = size
    rng = np.random.default_rng(out)
    gate, wg, _ = layer("2x8", out, n_in, out)
    up, wu, _ = layer("2x8", out, n_in, out + 1)
    for i, T in enumerate((1, 2, 3, 4, 5)):
        assert streams(out, n_in, T, True) == (T in served), (out, n_in, T)
        name = ("silu", "none", "gelu", "relu", "gelu_tanh")[i]
        x, bg, bu = half(rng, T, n_in), half(rng, out), half(rng, out)
        zg, zu = (torch.full((T, out), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
        y = E.aqlm_gated(gate, up, x.cuda(), act=name, gate_bias=bg.cuda(), up_bias=bu.cuda(), zg=zg, zu=zu)
        want, tol, zs = R.gated(wg, wu, x.double(), name, bg.double(), bu.double(), False)
        R.assert_within(y, want, tol, f"y {T}")
        for got, (z, tz), what in zip((zg, zu), zs, ("zg", "zu")):
            R.assert_within(got, z, tz, f"{what} {T}")
        # one of the two biases and one of the two pre-activations
        zu = torch.full((T, out), float("nan"), dtype=torch.float16, device="cuda")
        y = E.aqlm_gated(gate, up, x.cuda(), act=name, up_bias=bu.cuda(), zu=zu)
        want, tol, zs = R.gated(wg, wu, x.double(), name, None, bu.double(), False)
        R.assert_within(y, want, tol, f"y {T}")
        R.assert_within(zu, *zs[1], f"zu {T}")


def test_bad_rows_stay_alone():
    """NaN in one row of x and an infinite codeword, where the last slab and the last row tile are ragged."""
    rng = np.random.default_rng(1)
    for out, n_in in ((4101, 8256), (2051, 8256)):
        (codes, cb, s), _, _ = layer("2x8", out, n_in, 3)
        up, _, _ = layer("2x8", out, n_in, 4)
        codes[codes == 7] = 8
        codes[out - 1, -1, 0] = 7
        bad = cb.clone()
        bad[0, 7, 2] = float("inf")
        cb[0, 7] = 0.5
        for T in (1, 2, 3, 4):
            x = half(rng, T, n_in).cuda()
            x[x == 0] = 1
            for f in (lambda c, v: E.aqlm_linear_act(codes, c, s, v), lambda c, v: E.aqlm_gated((codes, c, s), up, v, act="none")):
                a, b = f(cb, x), f(bad, x)
                assert torch.equal(a[:, :-1], b[:, :-1]) and torch.isinf(b[:, -1]).all(), (out, T)
                if T > 1:
                    v = x.clone()
                    v[T - 1, -1] = float("nan")
                    b = f(cb, v)
                    assert torch.equal(a[:-1], b[:-1]) and torch.isnan(b[-1]).all(), (out, T)
