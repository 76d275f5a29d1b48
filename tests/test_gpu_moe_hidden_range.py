"""Hidden values of the experts in AQLM schemes far from 1: kept to 2^-22 of each or 2^-28, up to 2^8 * 65504.
(serving_reference.py: what tolerances count.)"""
import pytest
import torch

import extreme_weight_quantization_amd as E
from test_gpu_moe import Layer

pytestmark = pytest.mark.gpu
SCHEMES = [(2, 8, 8), (1, 16, 8), (1, 8, 4), (4, 8, 16), (3, 5, 2)]
NAMES = ["2x8", "1x16", "1x8g4", "4x8g16", "3x5g2"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need an MI355X")
    E.load_library()


def layer(scheme, tokens, seed):
    L = Layer(scheme, 3, 96, 64, seed=seed)
    # hi = nearest(h / 2^8) is off by 2^-11 of itself or 2^-25, lo = nearest(2^11 (h / 2^8 - hi)) again
    L.stored = lambda h: 2.0 ** -22 * h.abs() + 2.0 ** -28
    return L, *L.inputs(tokens, 2, seed=seed + 1)[:3]


@pytest.mark.parametrize("tokens", [1, 5, 20])
@pytest.mark.parametrize("scheme", SCHEMES, ids=NAMES)
def test_large_values(scheme, tokens):
    """Beyond fp16's range: hidden values of about 10^6, results of about 1."""
    L, x, ids, w = layer(scheme, tokens, seed=1)
    y = L.check(x * 1000, ids, w * 1e-6, "none")
    assert bool(y.isfinite().all()) and float(y.abs().max()) > 0.1


@pytest.mark.parametrize("tokens", [1, 5, 20])
@pytest.mark.parametrize("scheme", SCHEMES, ids=NAMES)
def test_small_values(scheme, tokens):
    """Hidden values of about 10^-5, results of about 1."""
    L, x, ids, w = layer(scheme, tokens, seed=2)
    y = L.check(x / 300, ids, w * 1e5, "none")
    assert float(y.abs().max()) > 0.1


@pytest.mark.parametrize("scheme", SCHEMES, ids=NAMES)
def test_beyond_the_range(scheme):
    """Larger than 2^8 * 65504 is infinite, with its sign: results are infinite or NaN, and only that token's."""
    L, x, ids, w = layer(scheme, 5, seed=3)
    x[2] = x[2].sign() * 60000
    clean = L.run(x, ids, w * 1e-6, "none").cpu()
    assert not bool(clean[2].isfinite().any())
    keep = torch.arange(5) != 2
    assert bool(clean[keep].isfinite().all())
