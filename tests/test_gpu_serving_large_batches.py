"""The largest batches: more workgroups than one launch takes, which are launched in parts of the batch."""
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


@pytest.mark.parametrize("score,biased", [("softmax", True), ("sigmoid", False)])
@pytest.mark.parametrize("tokens", [(1 << 22) + 1, (1 << 23) + 19])
def test_route_of_the_most_tokens(score, biased, tokens):
    """512 experts, in 64 bits (softmax with a bias) and with sums of 32: more than 2^32 threads in all."""
    experts, n_in, k = 512, 8, 3
    some = torch.randn((4096, n_in), generator=gen(5)).half()
    router = torch.randn((experts, n_in), generator=gen(6)).half()
    bias = torch.randn(experts, generator=gen(7)) * 0.1 if biased else None
    x = some.cuda().repeat(-(-tokens // 4096), 1)[:tokens].contiguous()
    ids, w = E.aqlm_moe_route(x, router.cuda(), k, score=score, bias=None if bias is None else bias.cuda())
    want_i, want_w = route_reference(some, router, k, score, bias, True, 1.0)
    assert torch.equal(ids[:4096].cpu(), want_i)
    # sums of 8 products in fp32: d = 8 2^-23 |x| |r| at most
    d = 2.0 ** -20 * some.double().norm(dim=1, keepdim=True) * router.double().norm(dim=1).max()
    assert bool(((w[:4096].cpu().double() - want_w).abs() <= (torch.expm1(2 * d) + 2.0 ** -23) * want_w).all())
    for got in (ids, w):   # equal tokens, equal results: all of them
        assert torch.equal(got, got[:4096].repeat(-(-tokens // 4096), 1)[:tokens])


def test_route_workspace_of_the_most_tokens():
    sizes = [E.moe_route_workspace_bytes(512, 8, 3, t) for t in (1, 1000, 1 << 21, 1 << 22, (1 << 22) + 1, 1 << 24)]
    assert sizes == sorted(sizes)
