"""The router and the mixture-of-experts layer on the GPU against 64 bits (serving_reference.py: what tolerances count)."""
import math

import numpy as np
import pytest
import torch

import extreme_weight_quantization_amd as E
import fused_reference as FR
import serving_reference as R
from oracle import aqlm_oracle as O

pytestmark = pytest.mark.gpu
F16, U8 = torch.float16, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need an MI355X")
    E.load_library()


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------------------------------------ router


def route_reference(x, router, k, score, bias, renorm, scale):
    logits = x.double() @ router.double().t()
    s = torch.softmax(logits, -1) if score == "softmax" else torch.sigmoid(logits)
    rank = logits if score == "softmax" and bias is None else s if bias is None else s + bias.double()
    ids = torch.sort(rank, dim=-1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, ids)
    return ids.int(), (w / w.sum(-1, keepdim=True) if renorm else w) * scale


@pytest.mark.parametrize("tokens", [1, 2, 16, 17, 100, 1000])
@pytest.mark.parametrize("experts,n_in,k", [(1, 8, 1), (2, 64, 2), (8, 1000, 2), (17, 4096, 4), (64, 2048, 8), (128, 520, 8),
                                            (200, 96, 16), (256, 1024, 8), (512, 264, 16)])
def test_route(experts, n_in, k, tokens):
    n = experts + n_in + tokens
    g = gen(n)
    x = torch.randn((tokens, n_in), generator=g).half()
    router = (torch.randn((experts, n_in), generator=g) / math.sqrt(n_in)).half()
    bias = torch.randn(experts, generator=g) * 0.1
    for score in ("softmax", "sigmoid"):
        for b, renorm, scale in ((None, True, 1.0), (bias, False, 2.5)):
            ids, w = E.aqlm_moe_route(x.cuda(), router.cuda(), k, score=score, bias=None if b is None else b.cuda(), renorm=renorm,
                                      scale=scale)
            want_i, want_w = route_reference(x, router, k, score, b, renorm, scale)
            assert torch.equal(ids.cpu(), want_i)
            # scores in 64 bits, one rounding to fp32
            assert bool(((w.cpu().double() - want_w).abs() <= 2.0 ** -23 * want_w.abs() + 1e-44).all())


def test_route_ties_take_the_lowest_index():
    g = gen(1)
    base = torch.randn((4, 256), generator=g).half()
    router = base[torch.tensor([2, 0, 1, 0, 3, 2, 1, 0, 3, 2] * 13)]   # 130 experts, four different rows
    x = torch.randn((50, 256), generator=g).half()
    ids, w = E.aqlm_moe_route(x.cuda(), router.cuda(), 16)
    want_i, _ = route_reference(x, router, 16, "softmax", None, True, 1.0)
    assert torch.equal(ids.cpu(), want_i)
    zero = E.aqlm_moe_route(torch.zeros((3, 256), dtype=F16, device="cuda"), router.cuda(), 5)[0].cpu()
    assert zero.tolist() == [[0, 1, 2, 3, 4]] * 3


def test_route_choices_do_not_depend_on_the_batch():
    """Logits that differ by one part in 2^30 keep their order however the sums are split."""
    n_in, tokens = 2048, 700
    x = torch.ones((tokens, n_in), dtype=F16)
    x[:, 1] = 2.0 ** -14
    router = torch.ones((40, n_in), dtype=F16)
    router[:, 1] = torch.arange(40).half() * 2.0 ** -8    # logits 2047 + i 2^-22
    for t in (1, 16, 100, tokens):
        ids = E.aqlm_moe_route(x[:t].cuda(), router.cuda(), 4)[0].cpu()
        assert ids.tolist() == [[39, 38, 37, 36]] * t


def test_route_non_finite_logits():
    g = gen(2)
    x = torch.randn((6, 64), generator=g).half()
    router = torch.randn((10, 64), generator=g).half()
    router[3, 5] = math.nan
    x[1, 7] = math.nan
    router[6] = 0
    x[2] = 0
    router[6, 0], x[2, 0] = math.inf, 1.0
    for score in ("softmax", "sigmoid"):
        ids, w = (v.cpu() for v in E.aqlm_moe_route(x.cuda(), router.cuda(), 10, score=score, renorm=False))
        for t in range(6):
            assert sorted(ids[t].tolist()) == list(range(10))   # every expert once
        assert ids[1].tolist() == list(range(10)) and bool(w[1].isnan().all())
        assert ids[0, 9] == 3 and ids[2, 0] == 6 and bool(w[0, 9].isnan())
        if score == "sigmoid":
            assert bool(w[0, :9].isfinite().all()) and w[2, 0] == 1.0
        else:
            assert bool(w[0].isnan().all())
    assert E.aqlm_moe_route(x[:0].cuda(), router.cuda(), 3)[0].shape == (0, 3)


def many_tokens(experts, n_in):
    """Tokens from which on logits are summed in 32 bits first."""
    return -(-2 ** 29 // (experts * n_in))


@pytest.mark.parametrize("score,biased,renorm", [("softmax", False, True), ("sigmoid", False, False), ("sigmoid", True, True),
                                                 ("softmax", True, False)])
@pytest.mark.parametrize("experts,n_in,k,more", [(1, 8192, 1, 1), (40, 1000, 3, 5), (64, 4096, 8, 0), (130, 264, 16, 63), (256, 4096, 8, 1),
                                                 (512, 2056, 16, 31)])
def test_route_of_many_tokens(experts, n_in, k, more, score, biased, renorm):
    tokens = many_tokens(experts, n_in) + more
    g = gen(experts + n_in)
    x = torch.randn((tokens, n_in), generator=g).half()
    router = (torch.randn((experts, n_in), generator=g) / math.sqrt(n_in)).half()
    bias = torch.randn(experts, generator=g) * 0.1 if biased else None
    ids, w = E.aqlm_moe_route(x.cuda(), router.cuda(), k, score=score, bias=None if bias is None else bias.cuda(), renorm=renorm)
    want_i, want_w = route_reference(x, router, k, score, bias, renorm, 1.0)
    assert torch.equal(ids.cpu(), want_i)
    # A logit is off by at most d = 2^-17 |x| |r|: a score by a factor e^d, against a sum of scores by e^2d.
    d = 2.0 ** -17 * (x.double().norm(dim=1, keepdim=True) * router.double().norm(dim=1).max())
    assert bool(((w.cpu().double() - want_w).abs() <= (torch.expm1(2 * d) + 2.0 ** -23) * want_w).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_of_many_tokens_with_exact_sums(score):
    """Small whole numbers: sums of 32 bits are exact, so that weights are as for few tokens; many logits tie."""
    experts, n_in, k = 96, 2048, 8
    g = gen(3)
    x = torch.randint(-2, 3, (many_tokens(experts, n_in) + 3, n_in), generator=g).half()
    router = (torch.randint(-2, 3, (experts, n_in), generator=g) / 64).half()
    ids, w = E.aqlm_moe_route(x.cuda(), router.cuda(), k, score=score)
    want_i, want_w = route_reference(x, router, k, score, None, True, 1.0)
    assert torch.equal(ids.cpu(), want_i)
    assert bool(((w.cpu().double() - want_w).abs() <= 2.0 ** -23 * want_w).all())
    few_i, few_w = E.aqlm_moe_route(x[:100].cuda(), router.cuda(), k, score=score)
    assert torch.equal(few_i, ids[:100]) and torch.equal(few_w, w[:100])


def test_route_of_many_tokens_close_and_equal_logits():
    n_in, experts = 2048, 40
    tokens = many_tokens(experts, n_in)
    x = torch.ones((tokens, n_in), dtype=F16)
    x[:, 1] = 2.0 ** -14
    router = torch.ones((experts, n_in), dtype=F16)
    router[:, 1] = torch.arange(experts).half() * 2.0 ** -8    # logits 2047 + i 2^-22
    assert E.aqlm_moe_route(x.cuda(), router.cuda(), 4)[0].cpu().tolist() == [[39, 38, 37, 36]] * tokens
    router[:, 1] = 1
    bias = torch.zeros(experts)
    bias[7] = -math.inf
    bias[0] = -1.0
    for score in ("softmax", "sigmoid"):
        assert E.aqlm_moe_route(x.cuda(), router.cuda(), 3, score=score)[0].cpu().tolist() == [[0, 1, 2]] * tokens
        got = E.aqlm_moe_route(x.cuda(), router.cuda(), experts // 8 + 3, score=score, bias=bias.cuda())[0].cpu()
        assert got.tolist() == [[1, 2, 3, 4, 5, 6, 8, 9]] * tokens
    zero = E.aqlm_moe_route(torch.zeros_like(x).cuda(), router.cuda(), 5)[0].cpu()
    assert zero.tolist() == [[0, 1, 2, 3, 4]] * tokens


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_of_many_tokens_non_finite_logits(score):
    g = gen(4)
    experts, n_in = 20, 4096
    tokens = many_tokens(experts, n_in)
    x = torch.randn((tokens, n_in), generator=g).half()
    router = (torch.randn((experts, n_in), generator=g) / 64).half()
    router[11, 4090] = math.nan
    x[1, 7] = math.nan
    router[6] = 0
    x[2] = 0
    router[6, 0], x[2, 0] = math.inf, 1.0
    x[:, 0] = x[:, 0].abs() + 1   # logit 6 is infinite
    x[5, 0] = -1.0                # minus infinity
    ids, w = (v.cpu() for v in E.aqlm_moe_route(x.cuda(), router.cuda(), 16, score=score, renorm=False))
    logits = x.double() @ router.double().t()
    logits[:, 11], logits[1] = math.nan, math.nan
    logits[:, 6] = torch.where(x[:, 0] > 0, math.inf, -math.inf)
    logits[1] = math.nan
    order = torch.sort(torch.nan_to_num(logits, nan=-1e300, posinf=1e300, neginf=-1e299), dim=1, descending=True, stable=True)
    assert torch.equal(ids, order.indices[:, :16].int())
    if score == "sigmoid":
        rows = torch.tensor([t for t in range(tokens) if t != 1])
        assert bool((w[rows][ids[rows] == 6] == torch.where(x[rows, 0] > 0, 1.0, 0.0)[(ids[rows] == 6).any(1)]).all())
    assert bool(w[1].isnan().all())



def test_captured_route_of_many_tokens_follows_its_input():
    experts, n_in, k = 64, 4096, 8
    tokens = many_tokens(experts, n_in)
    g = gen(5)
    router = (torch.randn((experts, n_in), generator=g) / 64).half().cuda()
    x = torch.randn((tokens, n_in), generator=g).half().cuda()
    ws = torch.empty(E.moe_route_workspace_bytes(experts, n_in, k, tokens), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        E.aqlm_moe_route(x, router, k, workspace=ws)
        with torch.cuda.graph(graph, stream=side):
            ids, w = E.aqlm_moe_route(x, router, k, workspace=ws)
    torch.cuda.synchronize()
    for seed in (6, 7, 8):
        x.copy_(torch.randn((tokens, n_in), generator=gen(seed)).half())
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        got = ids.clone(), w.clone()
        want = E.aqlm_moe_route(x, router, k)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(got[0].cpu(), route_reference(x.cpu(), router.cpu(), k, "softmax", None, True, 1.0)[0])


# ------------------------------------------------------------------------------------------------ layers


def aqlm_layer(M, B, g, experts, rows, n_in, seed):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 1 << B, (experts, rows, n_in // g, M))
    codes = codes.astype(np.uint8) if B <= 8 else codes.astype(np.uint16).view(np.int16)
    sigma = 0.05
    cb = (rng.standard_normal((experts, M, 1 << B, g)) * sigma).astype(np.float16)
    s = (rng.uniform(0.5, 1.5, (experts, rows)) / (sigma * math.sqrt(M * n_in))).astype(np.float16)
    w = [torch.from_numpy(O.decode_fp32(codes[e], cb[e], s[e]).astype(np.float64)) for e in range(experts)]
    return tuple(torch.from_numpy(v).cuda() for v in (codes, cb, s)), w


def mx4_layer(experts, rows, n_in, seed):
    g = gen(seed)
    v = (torch.randn((experts * rows, n_in), generator=g) / math.sqrt(n_in)).half()
    codes, scales = R.mx4_quantize(v)
    w = R.mx4_values(codes, scales).view(experts, rows, n_in)
    return (codes.view(experts, rows, -1).cuda(), scales.view(experts, rows, -1).cuda()), [w[e] for e in range(experts)]


class Layer:
    def __init__(self, scheme, experts, n_in, inner, seed):
        if scheme == "mx4":
            made = [mx4_layer(experts, r, n, seed + i) for i, (r, n) in enumerate(((inner, n_in), (inner, n_in), (n_in, inner)))]
            self.call = E.aqlm_moe_mx4
            self.bytes = lambda t, k: E.moe_mx4_workspace_bytes(experts, n_in, inner, t, k)
            self.product = lambda w, x: R.mx4_product(w, x, True)
            self.stored = lambda h: 2.0 ** -19 * h.unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True).expand(-1, -1, 32).flatten(-2)
        else:
            M, B, g = scheme
            made = [aqlm_layer(M, B, g, experts, r, n, seed + i) for i, (r, n) in enumerate(((inner, n_in), (inner, n_in), (n_in, inner)))]
            self.call = E.aqlm_moe
            self.bytes = lambda t, k: E.moe_workspace_bytes(M, B, g, experts, n_in, inner, t, k)
            self.product = lambda w, x: FR.product(w, x, False)
            self.stored = lambda h: 2.0 ** -22 * h.abs() + 2.0 ** -25
        self.layers, self.weights = [m[0] for m in made], [m[1] for m in made]
        self.experts, self.n_in = experts, n_in

    def inputs(self, tokens, k, seed, distinct=True):
        g = gen(seed)
        x = torch.randn((tokens, self.n_in), generator=g).half()
        logits = torch.randn((tokens, self.experts), generator=g) + torch.randn(self.experts, generator=g)
        if distinct:
            ids = torch.topk(logits, k).indices.int()
        else:
            ids = torch.randint(-1, self.experts, (tokens, k), generator=g, dtype=torch.int32)
        return x, ids, torch.rand((tokens, k), generator=g), torch.randn((tokens, self.n_in), generator=g).half()

    def run(self, x, ids, w, act="silu", residual=None, **kw):
        return self.call(*self.layers, x.cuda(), ids.cuda(), w.cuda(), act=act, residual=None if residual is None else residual.cuda(), **kw)

    def check(self, x, ids, w, act="silu", residual=None):
        y = self.run(x, ids, w, act, residual)
        want, tol = R.moe(self.weights, self.product, self.stored, x.double(), ids, w, act, None if residual is None else residual.double())
        off = (y.cpu().double() - want).abs() - tol
        assert bool((off <= 0).all()), f"worst {off.max():.3g} over, {int((off > 0).sum())} of {off.numel()}"
        return y


SCHEMES = [(2, 8, 8), (1, 16, 8), (1, 8, 4), (4, 8, 16), (8, 8, 32), (1, 12, 4), (3, 5, 2), "mx4"]
NAMES = ["2x8", "1x16", "1x8g4", "4x8g16", "8x8g32", "1x12g4", "3x5g2", "mx4"]


@pytest.mark.parametrize("scheme", SCHEMES, ids=NAMES)
@pytest.mark.parametrize("tokens,k", [(1, 1), (1, 4), (2, 3), (5, 2), (9, 2), (16, 3), (17, 1), (33, 4), (70, 2)])
def test_layer(scheme, tokens, k):
    n = tokens * 8 + k
    L = Layer(scheme, 6, 96 + 32 * (n % 3), 64 + 32 * (n % 2), seed=n)
    x, ids, w, residual = L.inputs(tokens, k, seed=n)
    L.check(x, ids, w, ("silu", "gelu", "relu", "gelu_tanh", "none")[n % 5], residual if n % 2 else None)


@pytest.mark.parametrize("scheme", [(2, 8, 8), (1, 16, 8), (4, 8, 16), "mx4"], ids=["2x8", "1x16", "4x8g16", "mx4"])
@pytest.mark.parametrize("n_in,inner,tokens", [(4096, 160, 3), (160, 4128, 2), (2080, 1056, 20), (1056, 2080, 1)])
def test_layer_sizes(scheme, n_in, inner, tokens):
    L = Layer(scheme, 3, n_in, inner, seed=5)
    x, ids, w, residual = L.inputs(tokens, 2, seed=6)
    L.check(x, ids, w, "silu", residual)


@pytest.mark.parametrize("n_in,inner", [(8, 8), (40, 24), (72, 200), (520, 264)])
def test_2x8_and_1x16_odd_rows(n_in, inner):
    """Code rows that do not start on 16 bytes, and an expert's first row neither."""
    for scheme in ((2, 8, 8), (1, 16, 8)):
        L = Layer(scheme, 5, n_in, inner, seed=7)
        for tokens in (1, 3, 12, 40):
            L.check(*L.inputs(tokens, 2, seed=tokens)[:3])


@pytest.mark.parametrize("scheme", [(2, 8, 8), (3, 5, 2), "mx4"], ids=["2x8", "3x5g2", "mx4"])
def test_missing_and_repeated_choices(scheme):
    L = Layer(scheme, 5, 96, 64, seed=3)
    x, ids, w, residual = L.inputs(30, 4, seed=4, distinct=False)
    ids[0] = -1                                       # a token without experts
    ids[1] = 2                                        # one expert four times
    ids[2] = torch.tensor([5, 1 << 30, -(1 << 31), 4])   # ids that are no experts
    ids[:, 3] = 1                                     # an expert that everybody asks for
    ids[0, 3] = -1
    y = L.check(x, ids, w, "silu", residual)
    assert torch.equal(y[0].cpu(), residual[0])
    none = torch.full((30, 4), -1, dtype=torch.int32)
    assert torch.equal(L.run(x, none, w, residual=residual).cpu(), residual)
    assert float(L.run(x, none, w).abs().max()) == 0
    bad = w.clone()
    bad[5, 0] = math.nan
    ids[5, 0] = 0
    got = L.run(x, ids, bad, residual=residual).cpu()
    assert bool(got[5].isnan().all())
    keep = torch.arange(30) != 5
    assert torch.equal(got[keep], L.run(x, ids, w, residual=residual).cpu()[keep])


@pytest.mark.parametrize("scheme", [(2, 8, 8), "mx4"], ids=["2x8", "mx4"])
def test_many_experts_and_the_most_pairs(scheme):
    L = Layer(scheme, 512, 32, 32, seed=8)
    x, ids, w, residual = L.inputs(64, 16, seed=9)
    L.check(x, ids, w, "silu", residual)
    x, ids, w, residual = L.inputs(1024, 1, seed=10)
    ids[:600] = 511
    L.check(x, ids, w, "silu", residual)


@pytest.mark.parametrize("scheme", [(2, 8, 8), "mx4"], ids=["2x8", "mx4"])
def test_non_finite_activations_stay_with_their_token(scheme):
    L = Layer(scheme, 4, 96, 64, seed=11)
    x, ids, w, residual = L.inputs(20, 2, seed=12)
    clean = L.run(x, ids, w, residual=residual).cpu()
    x[3, 5], x[8, 70] = math.nan, math.inf
    got = L.run(x, ids, w, residual=residual).cpu()
    keep = (torch.arange(20) != 3) & (torch.arange(20) != 8)
    assert torch.equal(got[keep], clean[keep]) and bool(got[3].isnan().all()) and not bool(got[8].isfinite().any())


@pytest.mark.parametrize("scheme", [(2, 8, 8), "mx4"], ids=["2x8", "mx4"])
def test_large_hidden_values(scheme):
    """Hidden values near the end of fp16's range keep their precision."""
    L = Layer(scheme, 2, 64, 64, seed=13)
    x, ids, w, _ = L.inputs(4, 1, seed=14)
    L.check(x * 80, ids, w * 1e-3, "none")
    L.check(x * 1e-2, ids, w, "none")


@pytest.mark.parametrize("scheme", [(2, 8, 8), (1, 16, 8), "mx4"], ids=["2x8", "1x16", "mx4"])
def test_graph_replays_in_place_and_streams(scheme):
    L = Layer(scheme, 8, 256, 160, seed=15)
    tokens, k = 12, 2
    cases = [L.inputs(tokens, k, seed=s) for s in range(3)]
    want = [L.run(x, i, w, residual=r) for x, i, w, r in cases]
    ws = torch.full((L.bytes(tokens, k),), 0xFF, dtype=U8, device="cuda")
    x, ids, w, y = (v.cuda().clone() for v in cases[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.call(*L.layers, x, ids, w, residual=y, y=y.clone(), workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            L.call(*L.layers, x, ids, w, residual=y, y=y, workspace=ws)
    for c in (1, 0, 2, 1):
        for dst, src in zip((x, ids, w, y), cases[c]):
            dst.copy_(src.cuda())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[c])
        assert torch.equal(L.run(*cases[0][:3], residual=cases[0][3]), want[0])
    got = [[], []]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for rep in range(10):
        for s, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[s].append(L.run(*cases[s][:3], residual=cases[s][3]))
    torch.cuda.synchronize()
    for s in range(2):
        assert all(torch.equal(v, want[s]) for v in got[s])


def test_a_block_of_them_together():
    """A projection in MX4, the router on its result, and the experts, for one token and for many."""
    g = gen(20)
    n_in, inner, experts, k = 256, 160, 16, 4
    proj = (torch.randn((n_in, n_in), generator=g) / 16).half()
    router = (torch.randn((experts, n_in), generator=g) / 4).half()
    L = Layer((2, 8, 8), experts, n_in, inner, seed=21)
    codes, scales = E.aqlm_mx4_quantize(proj.cuda())
    for tokens in (1, 7, 40):
        x = torch.randn((tokens, n_in), generator=g).half()
        h = E.aqlm_mx4_linear(codes, scales, x.cuda(), residual=x.cuda())
        ids, w = E.aqlm_moe_route(h, router.cuda(), k)
        y = L.call(*L.layers, h, ids, w, residual=h)
        z, ez = R.mx4_product(R.mx4_values(codes, scales), x.double(), True)
        want, tol = R.linear(z, ez, "none", None, x.double())
        assert bool(((h.cpu().double() - want).abs() <= tol).all())
        want_i, want_w = route_reference(h.cpu(), router, k, "softmax", None, True, 1.0)   # from the h that was computed
        assert torch.equal(ids.cpu(), want_i)
        want, tol = R.moe(L.weights, L.product, L.stored, h.cpu().double(), want_i, want_w, "silu", h.cpu().double())
        tol = tol + 2.0 ** -20 * want.abs()   # the weights' rounding to fp32
        assert bool(((y.cpu().double() - want).abs() <= tol).all())


def test_refusals():
    L = Layer((2, 8, 8), 4, 64, 64, seed=22)
    x, ids, w, r = (v.cuda() for v in L.inputs(3, 2, seed=23))
    for bad in (dict(x=x[:, :32]), dict(x=x.float()), dict(ids=ids.long()), dict(w=w.half()), dict(ids=ids[:2]), dict(w=w[:, :1]),
                dict(residual=r[:2]), dict(x=x.cpu())):
        a = {**dict(x=x, ids=ids, w=w, residual=r), **bad}
        with pytest.raises((ValueError, AttributeError)):
            L.call(*L.layers, a["x"], a["ids"], a["w"], residual=a["residual"])
    with pytest.raises(ValueError):
        E.aqlm_moe_route(x, x, 4)   # more choices than experts
    with pytest.raises(ValueError):
        E.aqlm_moe_route(x, r, 1, bias=torch.zeros(3, device="cuda").half())
    assert L.run(x[:0], ids[:0], w[:0]).shape == (0, 64)
