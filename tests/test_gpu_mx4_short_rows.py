"""MX4 activations of fewer than 16 blocks in all against large layers: their scales are an array shorter than the tile
kernel's 16-byte loads, so these calls go to the rows kernel.  (serving_reference.py: what tolerances count.)"""
import pytest
import torch

import extreme_weight_quantization_amd as E
import serving_reference as R
from test_gpu_mx4 import activations, check, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need an MI355X")
    E.load_library()


@pytest.mark.parametrize("n_in,out,t", [(32, 4300001, 1), (32, 4300001, 15), (32, 4300001, 16), (480, 285000, 1), (256, 530000, 2),
                                        (512, 270000, 1)])
def test_few_blocks_of_mx4_activations(n_in, out, t):
    """More than 2^27 weights, either side of 16 blocks.  The bytes around x's scales are NaN scales: none may count."""
    codes, scales = weights(out, n_in, t)
    x = activations(t, n_in, t + 1)
    xq, xs = E.aqlm_mx4_quantize(x.cuda())
    buffer = torch.full((64 + xs.numel() + 64,), 255, dtype=torch.uint8, device="cuda")
    place = buffer[64:64 + xs.numel()].view(t, -1)
    place.copy_(xs)
    y = E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), (xq, place))
    rows = torch.cat([torch.arange(0, 300), torch.arange(out // 2, out // 2 + 300), torch.arange(out - 300, out)])
    z, ez = R.mx4_product(R.mx4_values(codes[rows], scales[rows]), R.mx4_values(*R.mx4_quantize(x)), False)
    want, tol = R.linear(z, ez, "none", None, None)
    check(y.cpu()[:, rows], want, tol)
