"""The largest batches: more workgroups than one launch takes, which are launched in parts of the batch."""
import math

import pytest
import torch

import extreme_weight_quantization_amd as E
import serving_reference as R
from test_gpu_moe import gen, route_reference
from test_gpu_mx4 import activations, check, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need an MI355X")
    E.load_library()


@pytest.mark.parametrize("four", [False, True], ids=["fp16", "mx4"])
@pytest.mark.parametrize("n_in,out,t", [(32, 3, (1 << 22) + 1000), (96, 5, (1 << 22) + 65), (64, 1, (1 << 23) + 17)])
def test_linear_of_tiny_layers_and_many_tokens(n_in, out, t, four):
    codes, scales = weights(out, n_in, 1)
    some = activations(1000, n_in, 2)
    x = some.cuda().repeat(-(-t // 1000), 1)[:t].contiguous()
    bias = torch.randn(out, generator=gen(3)).half()
    residual = torch.randn((t, out), generator=gen(4)).half()
    y = residual.cuda()
    xin = E.aqlm_mx4_quantize(x) if four else x
    E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), xin, act="silu", bias=bias.cuda(), residual=y, y=y)
    # the tokens around every power of two from 2^21 on, and the last ones
    at = torch.cat([torch.arange(b - 70, b + 70) for b in (70, 1 << 21, 1 << 22, 1 << 23) if b + 70 < t] + [torch.arange(t - 200, t)])
    xv = R.mx4_values(*R.mx4_quantize(some)) if four else some.double()
    z, ez = R.mx4_product(R.mx4_values(codes, scales), xv[at % 1000], not four)
    want, tol = R.linear(z, ez, "silu", bias.double(), residual[at].double())
    check(y[at.cuda()], want, tol)
    # equal tokens have equal results but for the residual: all of them, on the GPU
    plain = E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), xin, act="silu", bias=bias.cuda())
    assert torch.equal(plain, plain[:1000].repeat(-(-t // 1000), 1)[:t])
