"""MX4 quantisation and products on the GPU against 64 bits (serving_reference.py says what the tolerances count)."""
import math

import numpy as np
import pytest
import torch

import extreme_weight_quantization_amd as E
import serving_reference as R

pytestmark = pytest.mark.gpu
F16, U8 = torch.float16, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need an MI355X")
    E.load_library()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def weights(out, n_in, seed, low=110, high=125):
    g = gen(seed)
    codes = torch.randint(0, 256, (out, n_in // 2), generator=g, dtype=torch.int32).to(U8)
    return codes, torch.randint(low, high, (out, n_in // 32), generator=g, dtype=torch.int32).to(U8)


def activations(t, n_in, seed, spread=0):
    g = gen(seed)
    x = torch.randn((t, n_in), generator=g)
    x[:, :: max(1, n_in // 7)] *= 8
    if spread:
        x = x * torch.exp2(torch.randint(-spread, 1, (t, n_in), generator=g).float())
    return x.half()


def check(got, want, tol):
    got = got.cpu().double()
    off = (got - want).abs() - tol
    assert bool((off <= 0).all()), f"worst {off.max():.3g} over, {int((off > 0).sum())} of {off.numel()}"


# ------------------------------------------------------------------------------------------------ conversions


def test_quantize_every_fp16_value():
    """Every finite fp16 pattern in blocks of its own neighbours, and shuffled among all others."""
    bits = np.arange(65536, dtype=np.uint16)
    finite = bits[np.isfinite(bits.view(np.float16))]
    rng = np.random.default_rng(0)
    rows = [finite[: len(finite) // 32 * 32], rng.permutation(finite)[: len(finite) // 32 * 32]]
    # one large value of each exponent with all others beside it
    for e in range(0, 31, 3):
        r = rows[1].reshape(-1, 32).copy()
        r[:, rng.integers(0, 32)] = np.uint16(e << 10 | 0x155)
        rows.append(r.reshape(-1))
    v = torch.from_numpy(np.stack(rows).view(np.float16)).view(-1, 32 * 62)
    codes, scales = E.aqlm_mx4_quantize(v.cuda())
    want_c, want_s = R.mx4_quantize(v)
    assert torch.equal(scales.cpu(), want_s)
    assert torch.equal(codes.cpu(), want_c)
    back = E.aqlm_mx4_decode(codes, scales)
    assert torch.equal(back.cpu().double(), R.mx4_values(want_c, want_s))   # without rounding


def test_quantize_special_blocks():
    v = torch.zeros((6, 64), dtype=F16)
    v[1] = -0.0
    v[2, 3], v[2, 40] = math.inf, 1.0
    v[3, 31], v[3, 32] = math.nan, -2.0
    v[4] = 2.0 ** -24
    v[5] = 65504.0
    codes, scales = (t.cpu() for t in E.aqlm_mx4_quantize(v.cuda()))
    assert scales[0].tolist() == [0, 0] and int(codes[0].max()) == 0
    assert scales[1].tolist() == [0, 0] and set(codes[1].tolist()) == {0x88}
    assert scales[2].tolist() == [255, 125] and int(codes[2, :16].max()) == 0
    assert scales[3].tolist() == [255, 126] and int(codes[3, :16].max()) == 0
    back = E.aqlm_mx4_decode(codes.cuda(), scales.cuda()).cpu()
    assert bool(back[2, :32].isnan().all()) and back[2, 40] == 1.0 and back[3, 32] == -2.0
    assert torch.equal(back[4], v[4]) and bool((back[5] == 6 * 2.0 ** 13).all())


@pytest.mark.parametrize("rows,n_in", [(1, 32), (3, 96), (257, 1056), (40, 8192)])
def test_quantize_and_decode_sizes(rows, n_in):
    v = activations(rows, n_in, seed=rows, spread=20)
    guard = torch.full((rows + 1, n_in // 2), 0xAB, dtype=U8, device="cuda")
    codes, scales = E.aqlm_mx4_quantize(v.cuda(), codes=guard[:rows])
    want_c, want_s = R.mx4_quantize(v)
    assert torch.equal(codes.cpu(), want_c) and torch.equal(scales.cpu(), want_s)
    assert bool((guard[rows] == 0xAB).all())
    out = torch.full((rows + 1, n_in), 7.0, dtype=F16, device="cuda")
    E.aqlm_mx4_decode(codes, scales, w=out[:rows])
    assert torch.equal(out[:rows].cpu().double(), R.mx4_values(want_c, want_s)) and bool((out[rows] == 7).all())


def test_decode_every_scale():
    """All 16 codes at all 256 scales: one rounding to fp16, 0 and infinity at its ends, NaN at 255."""
    codes = torch.arange(16, dtype=torch.int32)
    codes = (codes | (codes.flip(0) << 4)).to(U8).expand(256, 16).contiguous()
    scales = torch.arange(256, dtype=torch.int32).to(U8).view(256, 1)
    got = E.aqlm_mx4_decode(codes.cuda(), scales.cuda()).cpu()
    with np.errstate(over="ignore"):
        want = torch.from_numpy(R.mx4_values(codes, scales).numpy().astype(np.float16))
    assert torch.equal(got[:255], want[:255]) and bool(got[255].isnan().all())


# ------------------------------------------------------------------------------------------------ products

SHAPES = [   # in, out, tokens
    (32, 1, 1), (32, 17, 3), (96, 15, 1), (128, 16, 16), (160, 33, 17), (1056, 300, 1), (4096, 257, 2), (4096, 64, 8),
    (4128, 48, 9), (2048, 1000, 16), (8192, 100, 5), (11008, 130, 1), (11008, 40, 15), (1056, 65, 32), (512, 40, 33), (4096, 96, 48),
    (1024, 129, 64), (1056, 70, 65), (256, 300, 130), (4096, 256, 200), (544, 515, 300), (1024, 768, 1000), (64, 5, 2049)]


@pytest.mark.parametrize("four", [False, True], ids=["fp16", "mx4"])
@pytest.mark.parametrize("n_in,out,t", SHAPES)
def test_linear(n_in, out, t, four):
    n = n_in + out + t
    act = ("none", "silu", "gelu", "gelu_tanh", "relu")[n % 5]
    codes, scales = weights(out, n_in, n)
    x = activations(t, n_in, n + 1)
    g = gen(n + 2)
    bias = torch.randn(out, generator=g).half() if n % 2 else None
    residual = torch.randn((t, out), generator=g).half() if n % 3 else None
    dev = [None if v is None else v.cuda() for v in (codes, scales, x, bias, residual)]
    xin = E.aqlm_mx4_quantize(dev[2]) if four else dev[2]
    guard = torch.full((t + 1, out), 7.0, dtype=F16, device="cuda")
    y = E.aqlm_mx4_linear(dev[0], dev[1], xin, act=act, bias=dev[3], residual=dev[4], y=guard[:t])
    xv = R.mx4_values(*R.mx4_quantize(x)) if four else x.double()
    z, ez = R.mx4_product(R.mx4_values(codes, scales), xv, not four)
    want, tol = R.linear(z, ez, act, None if bias is None else bias.double(), None if residual is None else residual.double())
    check(y, want, tol)
    assert bool((guard[t] == 7).all())   # rows behind the last stay as they were
    again = E.aqlm_mx4_linear(dev[0], dev[1], xin, act=act, bias=dev[3], residual=dev[4])
    assert torch.equal(again, y)


@pytest.mark.parametrize("four", [False, True], ids=["fp16", "mx4"])
@pytest.mark.parametrize("n_in,out,t", [(4096, 5, 33), (4128, 300, 40), (8192, 129, 64), (11008, 64, 63), (4640, 1, 34)])
def test_linear_of_33_to_64_tokens_and_long_rows(n_in, out, t, four):
    test_linear(n_in, out, t, four)


@pytest.mark.parametrize("n_in,out,t", [(512, 4100, 1), (2080, 4096, 5), (4096, 4113, 8), (3104, 8192, 1), (12000, 4200, 2), (32768, 40, 1),
                                        (24576, 4100, 1), (512, 8193, 16)])
def test_linear_of_one_and_two_tiles_a_workgroup(n_in, out, t):
    test_linear(n_in, out, t, False)


@pytest.mark.parametrize("t", [1, 6, 20, 33, 65])
@pytest.mark.parametrize("four", [False, True], ids=["fp16", "mx4"])
@pytest.mark.parametrize("n_in,out", [(1024, 65800), (8192, 8320), (8192, 16500)])
def test_linear_of_large_layers(n_in, out, t, four):
    codes, scales = weights(out, n_in, t)
    x = activations(t, n_in, t + 1)
    xin = E.aqlm_mx4_quantize(x.cuda()) if four else x.cuda()
    y = E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), xin)
    xv = R.mx4_values(*R.mx4_quantize(x)) if four else x.double()
    rows = torch.cat([torch.arange(0, 300), torch.arange(out // 2, out // 2 + 300), torch.arange(out - 300, out)])
    z, ez = R.mx4_product(R.mx4_values(codes[rows], scales[rows]), xv, not four)
    want, tol = R.linear(z, ez, "none", None, None)
    check(y.cpu()[:, rows], want, tol)


@pytest.mark.parametrize("t", [1, 20, 300])
def test_activations_of_unlike_sizes_in_a_block(t):
    """Values 2^-8 of their block's largest and more are multiplied exactly, smaller ones to 2^-19 of it."""
    n_in, out = 1024, 48
    for seed, spread in ((1, 6), (2, 12), (3, 30)):
        codes, scales = weights(out, n_in, seed)
        x = activations(t, n_in, seed, spread=spread)
        z, ez = R.mx4_product(R.mx4_values(codes, scales), x.double(), True)
        want, tol = R.linear(z, ez, "none", None, None)
        check(E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), x.cuda()), want, tol)


@pytest.mark.parametrize("t", [1, 40, 300])
def test_single_activations_pass_exactly(t):
    """One value a token against weights of 1 in one row: the product is the fp16 value itself, at any size."""
    n_in = 128
    values = torch.tensor([65504.0, -65472.0, 63488.0, 61440.0, 32768.0, 2047.0, 1 + 2.0 ** -10, -1 / 3, 2.0 ** -14, 2.0 ** -24,
                           -1023 * 2.0 ** -24, 0.0], dtype=torch.float64).half()
    x = torch.zeros((t, n_in), dtype=F16)
    for i in range(t):
        x[i, (i * 37) % n_in] = values[i % len(values)]
    codes = torch.full((16, n_in // 2), 0x22, dtype=U8)
    scales = torch.full((16, n_in // 32), 127, dtype=U8)
    y = E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), x.cuda()).cpu()
    assert torch.equal(y, x.sum(1, keepdim=True).expand(t, 16))


@pytest.mark.parametrize("four", [False, True], ids=["fp16", "mx4"])
@pytest.mark.parametrize("t", [2, 40, 300])
def test_weights_of_extreme_scales(t, four):
    """Blocks of 2^-120 next to blocks of 2^3: nothing overflows, nothing is lost but what fp32 loses."""
    n_in, out = 512, 32
    codes, scales = weights(out, n_in, 9)
    scales[:, ::3], scales[:, 1::3] = 7, 130
    x = activations(t, n_in, 10)
    xin = E.aqlm_mx4_quantize(x.cuda()) if four else x.cuda()
    xv = R.mx4_values(*R.mx4_quantize(x)) if four else x.double()
    z, ez = R.mx4_product(R.mx4_values(codes, scales), xv, not four)
    want, tol = R.linear(z, ez, "none", None, None)
    check(E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), xin), want, tol)


@pytest.mark.parametrize("four", [False, True], ids=["fp16", "mx4"])
@pytest.mark.parametrize("t", [5, 40, 300])
def test_non_finite_values_stay_with_their_row_and_token(t, four):
    n_in, out = 288, 40
    codes, scales = weights(out, n_in, 3)
    scales[7, 2] = 255
    x = activations(t, n_in, 4)
    clean = E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), E.aqlm_mx4_quantize(x.cuda()) if four else x.cuda()).cpu()
    x[1, 5], x[3, 287] = math.inf, math.nan
    y = E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), E.aqlm_mx4_quantize(x.cuda()) if four else x.cuda()).cpu()
    assert bool(y[1].isnan().all()) and bool(y[3].isnan().all()) and bool(y[:, 7].isnan().all())
    keep = torch.ones(t, out, dtype=torch.bool)
    keep[1] = keep[3] = False
    keep[:, 7] = False
    assert torch.equal(y[keep], clean[keep]) and bool(clean[keep].isfinite().all())
    residual = torch.zeros((t, out), dtype=F16)
    residual[0, 3] = -math.inf
    y = E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), E.aqlm_mx4_quantize(x.cuda()) if four else x.cuda(), residual=residual.cuda()).cpu()
    assert y[0, 3] == -math.inf and bool(y[0, :3].isfinite().all())


@pytest.mark.parametrize("t", [1, 17, 100, 300])
def test_zero_activations_and_empty_calls(t):
    codes, scales = (v.cuda() for v in weights(24, 96, 5))
    x = torch.zeros((t, 96), dtype=F16, device="cuda")
    assert float(E.aqlm_mx4_linear(codes, scales, x).abs().max()) == 0
    assert float(E.aqlm_mx4_linear(codes, scales, E.aqlm_mx4_quantize(x)).abs().max()) == 0
    assert E.aqlm_mx4_linear(codes, scales, x[:0]).shape == (0, 24)
    assert E.aqlm_mx4_linear(codes[:0], scales[:0], x).shape == (t, 0)
    assert E.aqlm_mx4_quantize(x[:0])[0].shape == (0, 48)


@pytest.mark.parametrize("t", [1, 40, 300])
def test_scales_at_any_address_and_residual_in_place(t):
    n_in, out = 1056, 70
    codes, scales = weights(out, n_in, 6)
    x, res = activations(t, n_in, 7), activations(t, out, 8)
    want = E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), x.cuda(), residual=res.cuda())
    odd = torch.empty(scales.numel() + 3, dtype=U8, device="cuda")[3:].view(out, -1)
    odd.copy_(scales)
    assert odd.data_ptr() % 4 == 3
    y = res.cuda().clone()
    E.aqlm_mx4_linear(codes.cuda(), odd, x.cuda(), residual=y, y=y)
    assert torch.equal(y, want)
    xq, xs = E.aqlm_mx4_quantize(x.cuda())
    oddx = torch.empty(xs.numel() + 1, dtype=U8, device="cuda")[1:].view(t, -1)
    oddx.copy_(xs)
    assert torch.equal(E.aqlm_mx4_linear(codes.cuda(), odd, (xq, oddx)), E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), (xq, xs)))


def test_batches_do_not_change_a_token_by_more_than_rounding():
    """One workspace for the largest batch serves all smaller ones, whatever it held before."""
    n_in, out = 1056, 200
    codes, scales = weights(out, n_in, 11)
    x = activations(400, n_in, 12).cuda()
    z, ez = R.mx4_product(R.mx4_values(codes, scales), x.cpu().double(), True)
    want, tol = R.linear(z, ez, "none", None, None)
    ws = torch.full((E.mx4_linear_workspace_bytes(out, n_in, 400),), 0xFF, dtype=U8, device="cuda")
    for t in (400, 1, 64, 65, 16, 17, 300, 33, 129, 2):
        check(E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), x[:t], workspace=ws), want[:t], tol[:t])


@pytest.mark.parametrize("four", [False, True], ids=["fp16", "mx4"])
@pytest.mark.parametrize("t", [1, 40, 300])
def test_graph_replays_and_streams(t, four):
    n_in, out = 2048, 300
    codes, scales = (v.cuda() for v in weights(out, n_in, 13))
    xs = [activations(t, n_in, s).cuda() for s in range(4)]
    ws = torch.empty(max(16, E.mx4_linear_workspace_bytes(out, n_in, t)), dtype=U8, device="cuda")

    def run(x, y=None, workspace=None):
        return E.aqlm_mx4_linear(codes, scales, E.aqlm_mx4_quantize(x) if four else x, act="silu", y=y, workspace=workspace)

    want = [run(x) for x in xs]
    x, y = xs[0].clone(), torch.empty((t, out), dtype=F16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(x, y, ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            run(x, y, ws)
    for i in (1, 2, 0, 3):
        x.copy_(xs[i])
        y.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        assert torch.equal(run(xs[(i + 1) % 4]), want[(i + 1) % 4])   # eager work between replays
    # two streams at once, workspaces of their own
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    torch.cuda.synchronize()
    for rep in range(10):
        for s, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[s].append(run(xs[s + 1]))
    torch.cuda.synchronize()
    for s in range(2):
        assert all(torch.equal(v, want[s + 1]) for v in got[s])


def test_offsets_beyond_32_bits():
    """A layer of more than 2^32 weights: its last rows."""
    out, n_in = 270000, 16384
    codes = torch.zeros((out, n_in // 2), dtype=U8, device="cuda")
    scales = torch.full((out, n_in // 32), 127, dtype=U8, device="cuda")
    last, ls = weights(20, n_in, 14)
    codes[-20:], scales[-20:] = last.cuda(), ls.cuda()
    for t in (1, 70):
        x = activations(t, n_in, 15)
        y = E.aqlm_mx4_linear(codes, scales, x.cuda())
        z, ez = R.mx4_product(R.mx4_values(last, ls), x.double(), True)
        want, tol = R.linear(z, ez, "none", None, None)
        check(y[:, -20:], want, tol)
        assert float(y[:, :-20].abs().max()) == 0


def test_refusals():
    codes, scales = (v.cuda() for v in weights(8, 64, 1))
    x = torch.zeros((4, 64), dtype=F16, device="cuda")
    with pytest.raises(ValueError):
        E.aqlm_mx4_linear(codes, scales, x[:, ::2])
    with pytest.raises(ValueError):
        E.aqlm_mx4_linear(codes, scales, x.float())
    with pytest.raises(ValueError):
        E.aqlm_mx4_linear(codes, scales, x.cpu())
    with pytest.raises(ValueError):
        E.aqlm_mx4_linear(codes, scales.cpu(), x)
    with pytest.raises(ValueError):
        E.aqlm_mx4_linear(codes, scales, x, residual=torch.zeros((3, 8), dtype=F16, device="cuda"))
    with pytest.raises(ValueError):
        E.aqlm_mx4_linear(codes, scales, torch.zeros((4, 128), dtype=F16, device="cuda"))
    with pytest.raises(ValueError):
        E.aqlm_mx4_quantize(torch.zeros((4, 40), dtype=F16, device="cuda"))
    with pytest.raises(ValueError):   # one byte too few
        n = E.mx4_linear_workspace_bytes(8, 64, 300)
        E.aqlm_mx4_linear(codes, scales, torch.zeros((300, 64), dtype=F16, device="cuda"),
                          workspace=torch.empty(n - 1, dtype=U8, device="cuda"))


@pytest.mark.parametrize("four", [False, True], ids=["fp16", "mx4"])
@pytest.mark.parametrize("n_in,t", [(4128, 1), (4128, 40), (4128, 130), (8192, 64), (512, 3), (544, 7)])
def test_long_rows_with_odd_scales_and_non_finite_blocks(n_in, t, four):
    out = 150
    codes, scales = weights(out, n_in, n_in + t)
    scales[9, n_in // 32 - 1] = 255
    x = activations(t, n_in, t)
    if t > 2:
        x[2, n_in - 1] = math.inf
    odd = torch.empty(scales.numel() + 1, dtype=U8, device="cuda")[1:].view(out, -1)
    odd.copy_(scales)
    xin = E.aqlm_mx4_quantize(x.cuda()) if four else x.cuda()
    y = E.aqlm_mx4_linear(codes.cuda(), odd, xin).cpu()
    rows = [t0 for t0 in range(t) if t0 != 2]
    keep = [r for r in range(out) if r != 9]
    assert bool(y[:, 9].isnan().all()) and (t <= 2 or bool(y[2].isnan().all()))
    xv = (R.mx4_values(*R.mx4_quantize(x[rows])) if four else x[rows].double())
    z, ez = R.mx4_product(R.mx4_values(codes[keep], scales[keep]), xv, not four)
    want, tol = R.linear(z, ez, "none", None, None)
    check(y[rows][:, keep], want, tol)


@pytest.mark.parametrize("t", [1, 40, 70])
def test_longest_rows(t):
    n_in, out = 1 << 20, 18
    codes, scales = weights(out, n_in, t)
    x = activations(t, n_in, t)
    for four in (False, True):
        xin = E.aqlm_mx4_quantize(x.cuda()) if four else x.cuda()
        y = E.aqlm_mx4_linear(codes.cuda(), scales.cuda(), xin)
        xv = R.mx4_values(*R.mx4_quantize(x)) if four else x.double()
        z, ez = R.mx4_product(R.mx4_values(codes, scales), xv, not four)
        want, tol = R.linear(z, ez, "none", None, None)
        check(y, want, tol)


@pytest.mark.parametrize("four", [False, True], ids=["fp16", "mx4"])
def test_captured_products_of_40_tokens_follow_their_inputs(four):
    n_in, out, t = 4096, 200, 40
    codes, scales = (v.cuda() for v in weights(out, n_in, 31))
    x = activations(t, n_in, 32).cuda()
    ws = torch.empty(max(16, E.mx4_linear_workspace_bytes(out, n_in, t, x_mx4=four)), dtype=U8, device="cuda")
    y = torch.empty((t, out), dtype=F16, device="cuda")

    def call():
        return E.aqlm_mx4_linear(codes, scales, E.aqlm_mx4_quantize(x) if four else x, act="silu", y=y, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call()
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.synchronize()
    for seed in (33, 34, 35):
        x.copy_(activations(t, n_in, seed))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, call())
