"""Products of MX4 weights with fp16 activations lose nothing but what sums in 32 bits lose: what a large activation stands next
to, and what its weight is, does not matter.  (serving_reference.py: what tolerances count.)"""
import math

import numpy as np
import pytest
import torch

import extreme_weight_quantization_amd as E
import serving_reference as R
from test_gpu_moe import Layer, gen
from test_gpu_mx4 import activations, check, weights

pytestmark = pytest.mark.gpu
F16, U8 = torch.float16, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need an MI355X")
    E.load_library()


def diagonal(n, scales):
    """MX4 rows with a single weight 1 2^(scale - 127) on the diagonal, scales [n]; the other blocks of a row have scale 127."""
    codes = torch.zeros((n, n // 2), dtype=U8)
    i = torch.arange(n)
    codes[i, i // 2] = torch.where(i % 2 == 0, 0x02, 0x20).to(U8)
    s = torch.full((n, n // 32), 127, dtype=U8)
    s[i, i // 32] = scales.to(U8)
    return codes, s


TOKENS = [1, 5, 16, 17, 40, 64, 65, 300]


@pytest.mark.parametrize("t", TOKENS)
@pytest.mark.parametrize("n", [32, 160, 544, 4128])
def test_a_unit_matrix_returns_every_fp16_value(n, t):
    """Finite values of all sizes side by side, subnormal ones among them: y is x, to the bit but for the sign of 0."""
    bits = np.random.default_rng(n + t).integers(0, 65536, (t, n)).astype(np.uint16)
    bits[(bits & 0x7C00) == 0x7C00] &= 0xBFFF   # infinities and NaN to finite values
    x = torch.from_numpy(bits.view(np.float16))
    codes, scales = diagonal(n, torch.full((n,), 127))
    y = E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), x.cuda()).cpu()
    assert torch.equal(y, x)


@pytest.mark.parametrize("t", TOKENS)
def test_scales_on_both_sides_of_fp16s_range(t):
    """One weight 2^(s - 127) a row, s from 1 to 254 in turn: y is x 2^(s - 127), rounded once."""
    n = 1056
    s = torch.arange(n) % 254 + 1
    codes, scales = diagonal(n, s)
    x = (torch.randint(1, 2048, (t, n), generator=gen(t)).double() * torch.exp2((127 - s).clamp(-20, 4).double())).half()
    want = x.double() * torch.exp2((s - 127).double())
    with np.errstate(over="ignore"):
        want = torch.from_numpy(want.numpy().astype(np.float16))
    y = E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), x.cuda()).cpu()
    assert torch.equal(y, want)


@pytest.mark.parametrize("t", TOKENS)
@pytest.mark.parametrize("n_in,out", [(32, 40), (128, 300), (1056, 70), (4128, 150)])
def test_large_activations_next_to_others(n_in, out, t):
    """One channel of every block a thousand times the others, with weights of 0 there in half of the rows."""
    codes, scales = weights(out, n_in, n_in, low=120, high=124)
    spike = torch.arange(0, n_in, 32) + 5
    codes[::2, spike // 2] &= 0x0F   # value 5 of a block is in a high half
    x = torch.randn((t, n_in), generator=gen(t)).half()
    x[:, spike] *= 2048
    z, ez = R.mx4_product(R.mx4_values(codes, scales), x.double(), False)
    want, tol = R.linear(z, ez, "none", None, None)
    check(E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), x.cuda()), want, tol)


@pytest.mark.parametrize("t", TOKENS)
@pytest.mark.parametrize("low,high", [(100, 108), (136, 146), (60, 190), (1, 104)])
def test_odd_scales_of_all_kinds(low, high, t):
    n_in, out = 1056, 90
    codes, scales = weights(out, n_in, t, low=low, high=high)
    x = activations(t, n_in, t + 1) * 2.0 ** -8
    want_w = R.mx4_values(codes, scales)
    z, ez = R.mx4_product(want_w, x.double(), False)
    scale = torch.exp2(-torch.log2(z.abs().amax(1, keepdim=True)).round().clamp(-24, 24))   # results near 1, where fp16 can hold them
    x = (x.double() * scale).half()
    z, ez = R.mx4_product(want_w, x.double(), False)
    want, tol = R.linear(z, ez, "none", None, None)
    y = E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), x.cuda()).cpu().double()
    finite = want.abs() < 60000
    assert bool(((y - want).abs() <= tol)[finite].all())
    assert not bool((y[~finite].abs() < 59000).any())


@pytest.mark.parametrize("t", [1, 16, 40, 70])
def test_odd_blocks_in_captured_calls(t):
    """The same calls with and without odd blocks: a graph goes by the weights that it finds."""
    n_in, out = 1056, 60
    codes, scales = (v.cuda() for v in weights(out, n_in, 3))
    x = activations(t, n_in, 4).cuda()
    ws = torch.empty(max(16, E.mx4_linear_workspace_bytes(out, n_in, t)), dtype=U8, device="cuda")
    y = torch.empty((t, out), dtype=F16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        E.aqlm_mx4_linear(codes, scales, x, y=y, workspace=ws)
        with torch.cuda.graph(graph, stream=side):
            E.aqlm_mx4_linear(codes, scales, x, y=y, workspace=ws)
    torch.cuda.synchronize()
    for odd in (None, (7, 3, 40), (59, 32, 200), None, (0, 0, 255)):
        now = scales.clone()
        if odd is not None:
            scales[odd[0], odd[1]] = odd[2]
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got.nan_to_num(7.0), E.aqlm_mx4_linear(codes, scales, x).nan_to_num(7.0))
        w = R.mx4_values(codes.cpu(), scales.cpu())
        z, ez = R.mx4_product(w, x.cpu().double(), False)
        want, tol = R.linear(z, ez, "none", None, None)
        off = (got.cpu().double() - want).abs() <= tol
        assert bool((off | want.isnan() | (want.abs() > 60000)).all())
        assert odd is None or odd[2] != 255 or bool(got[:, odd[0]].isnan().all())
        scales.copy_(now)


@pytest.mark.parametrize("n_in,out,t", [(4096, 16384, 16), (8192, 14000, 8), (65536, 100, 1), (32768, 300, 2), (4128, 14000, 16), (65568, 40, 1),
                                        (5120, 12300, 12), (4096, 28000, 16), (8192, 9000, 16), (1024, 21000, 3)])
def test_the_most_rows_that_lds_holds(n_in, out, t):
    """Activations of 128 KB and a step more, for workgroups of one to eight tiles."""
    codes, scales = weights(out, n_in, t)
    x = activations(t, n_in, t + 1)
    y = E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), x.cuda())
    rows = torch.unique(torch.cat([torch.arange(0, min(out, 100)), torch.arange(out // 2, min(out, out // 2 + 100)), torch.arange(max(0, out - 300), out)]))
    z, ez = R.mx4_product(R.mx4_values(codes[rows], scales[rows]), x.double(), False)
    want, tol = R.linear(z, ez, "none", None, None)
    check(y.cpu()[:, rows], want, tol)


# ------------------------------------------------------------------------------------------------ experts


def spiky(tokens, k, n_in, inner, seed):
    """A layer whose hidden vectors have a value 2^12 times the others in every block of 32, with down weights of 0 there."""
    L = Layer("mx4", 4, n_in, inner, seed=seed)
    at = torch.arange(0, inner, 32) + 5
    (gc, gs), (uc, us), (dc, ds) = L.layers
    gs[:, at] += 6
    us[:, at] += 6
    dc[:, :, at // 2] &= 0x0F
    for (c, s), to in zip(L.layers, L.weights):
        w = R.mx4_values(c.cpu(), s.cpu())
        for e in range(4):
            to[e] = w[e]
    # a hidden value is off by 2^-22 of itself or 2^-28; fp16 activations and codes enter the products as they are
    L.stored = lambda h: 2.0 ** -22 * h.abs() + 2.0 ** -28
    L.product = lambda w, x: R.mx4_product(w, x, False)
    return L, *L.inputs(tokens, k, seed=seed + 1)


@pytest.mark.parametrize("tokens,k", [(1, 2), (3, 2), (9, 4), (20, 2), (70, 1)])
@pytest.mark.parametrize("n_in,inner", [(96, 64), (1056, 160), (160, 1056)])
def test_experts_with_large_hidden_values_next_to_others(n_in, inner, tokens, k):
    L, x, ids, w, residual = spiky(tokens, k, n_in, inner, seed=n_in)
    L.check(x / 8, ids, w, "none")
    L.check(x / 8, ids, w, "silu", residual)


@pytest.mark.parametrize("tokens", [1, 5, 20])
def test_hidden_values_far_from_one(tokens):
    L = Layer("mx4", 3, 96, 64, seed=1)
    L.stored = lambda h: 2.0 ** -22 * h.abs() + 2.0 ** -28
    L.product = lambda w, x: R.mx4_product(w, x, False)
    x, ids, w, _ = L.inputs(tokens, 2, seed=2)
    for factor, weight in ((1000, 1e-6), (1 / 300, 1e5)):
        y = L.check(x * factor, ids, w * weight, "none")
        assert bool(y.isfinite().all()) and float(y.abs().max()) > 0.01


@pytest.mark.parametrize("tokens,k", [(1, 2), (9, 4), (40, 2)])
def test_experts_with_odd_scales(tokens, k):
    """Blocks of scales that fp16 does not hold in all three layers of one expert; the others' results stay as they were."""
    L = Layer("mx4", 4, 160, 96, seed=7)
    x, ids, w, residual = L.inputs(tokens, k, seed=8)
    clean = L.run(x, ids, w, residual=residual).cpu()
    for (c, s), to in zip(L.layers, L.weights):
        s[2, 3, 1], s[2, 5, 0], s[2, 70, 2] = 30, 101, 103
        s[2, 8] = 0
        to[2] = R.mx4_values(c[2].cpu(), s[2].cpu())
    L.product = lambda w, x: R.mx4_product(w, x, False)
    L.stored = lambda h: 2.0 ** -22 * h.abs() + 2.0 ** -28
    y = L.check(x, ids, w, "silu", residual).cpu()
    others = ~(ids == 2).any(1)
    assert torch.equal(y[others], clean[others])
    L.layers[0][1][2, 4, 1] = 255
    got = L.run(x, ids, w, residual=residual).cpu()
    assert bool(got[~others].isnan().all()) and torch.equal(got[others], clean[others])
    assert math.isfinite(float(clean.abs().max()))
