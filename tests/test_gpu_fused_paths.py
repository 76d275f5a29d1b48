"""The fused products where their path changes: batch and layer sizes on both sides of every rule, arrays beyond 4 GB,
non-finite codewords, graphs and streams (reference and tolerances: tests/fused_reference.py)."""
import itertools

import numpy as np
import pytest
import torch

import extreme_weight_quantization_amd as E
import fused_reference as R
from extreme_weight_quantization_amd import synth
from test_gpu_fused import SCHEMES, half, layer, run_gated, run_gated_back, run_linear, run_linear_back

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need an MI355X")
    E.load_library()


# forward: 2x8 adds its codewords in fp16 above 64 tokens and is decoded first above 512; 1x16 needs 128 units of 256
# rows x 256 inputs (512 above 128 tokens) and is decoded first above 256 tokens, 4x8 g16 above 320
@pytest.mark.parametrize("scheme,out,n_in,T", [
    *[("2x8", 1100, 520, T) for T in (32, 33, 64, 65, 96, 97, 128, 130, 160, 161, 511, 512, 513)],
    *[("2x8", 700, 5000, T) for T in (66, 130)], *[("2x8", 300, 256, T) for T in (65, 90)], ("2x8", 5000, 696, 80),
    *[("2x8", 8, 8, T) for T in (17, 512, 513)],
    *[("1x16", 4096, 2048, T) for T in (17, 32, 33, 64, 65, 127, 128, 129)],   # 128 units
    ("1x16", 4096, 2040, 128), ("1x16", 4094, 1800, 128), ("1x16", 3840, 2048, 128),   # 128, 128, 120 units
    ("1x16", 8192, 4096, 129), ("1x16", 8188, 4080, 256), ("1x16", 8192, 4096, 257), ("1x16", 8192, 3840, 256),
    *[("4x8g16", 300, 528, T) for T in (17, 33, 64, 65, 96, 97, 128, 160, 320, 321, 1024, 1025)],
    ("4x8g16", 1100, 1024, 40), ("4x8g16", 1100, 1152, 200), ("4x8g16", 9, 16, 64),
])
def test_forward_paths(scheme, out, n_in, T):
    run_linear(scheme, out, n_in, T, "silu", True, True, True, seed=T)
    if out * n_in < 5e6 or T == 128:
        run_gated(scheme, out, n_in, T, "gelu_tanh", True, True, seed=T)


# backward: the gradients inside the product up to 16 tokens of few chunks and rows of whole 16 bytes; the codes direct
# up to 256 tokens (2x8) and 128 (1x16, 4x8 g16)
@pytest.mark.parametrize("scheme,out,n_in,T", [
    *[("2x8", 1100, 520, T) for T in (1, 16, 17, 32, 33, 64, 65, 128, 129, 255, 256, 257)],
    *[("1x16", 1100, 520, T) for T in (1, 16, 17, 32, 33, 64, 65, 127, 128, 129)],
    *[("2x8", out, 264, 16) for out in (8, 40, 96, 104, 100, 101)],
    *[("1x16", out, 264, 15) for out in (8, 40, 96, 104, 100, 101)],
    ("2x8", 4096, 4096, 16), ("2x8", 4104, 4224, 16), ("1x16", 4096, 8192, 3), ("1x16", 4224, 8192, 16),   # both sides of the chunks
    *[("4x8g16", 520, 272, T) for T in (1, 16, 17, 33, 64, 127, 128, 129, 1030)],
    *[("4x8g16", out, 272, 16) for out in (8, 40, 104, 101)],
    ("1x8g4", 136, 72, 5003),
])
def test_backward_paths(scheme, out, n_in, T):
    run_linear_back(scheme, out, n_in, T, "gelu", True, seed=T)
    if out * n_in < 5e6:
        run_gated_back(scheme, out, n_in, T, "silu", True, seed=T)


# few tiles of a dense product: its steps are split over workgroups, 128 or 256 tokens to a tile
@pytest.mark.parametrize("out,n_in", [(130, 8192), (64, 4112), (1000, 2000), (2064, 320)])
@pytest.mark.parametrize("T", [40, 128, 200, 256, 700])
@pytest.mark.parametrize("scheme", ["1x8g4", "4x8g16"])
def test_dense_splits(scheme, out, n_in, T):
    run_linear(scheme, out, n_in, T, "gelu", True, True, True)
    run_gated(scheme, out, n_in, T, "silu", False, True)
    run_linear_back(scheme, n_in, out - out % 16, T, "relu", True)   # the summed axis is the rows


def test_infinite_codewords():
    """An infinite weight reaches the outputs that it takes part in, and nothing beside them."""
    rng = np.random.default_rng(9)
    for scheme, (out, n_in), T in itertools.product(("2x8", "1x16", "4x8g16"), ((131, 208), (257, 528), (72, 1104)),
                                                    (1, 4, 16, 17, 40, 100, 130, 260, 600)):
        M, B, g = SCHEMES[scheme]
        (codes, cb, s), _, _ = layer(scheme, out, n_in, 21)
        codes[codes == 7] = 8
        rows, groups = (out - 1, 3), (n_in // g - 1, 0)
        for r, q in zip(rows, groups):
            codes[r, q, 0] = 7
        cb[0, 7] = 0.5
        bad = cb.clone()
        bad[0, 7, 2] = float("inf")
        ks = [q * g + 2 for q in groups]
        x, dy, z = half(rng, T, n_in).cuda(), half(rng, T, out).cuda(), half(rng, T, out).cuda()
        x[x == 0] = 1
        dy[dy.abs() < 0.01] = 1
        a, b = (E.aqlm_linear_act(codes, c, s, x) for c in (cb, bad))
        keep = [r for r in range(out) if r not in rows]
        assert torch.equal(a[:, keep], b[:, keep]), (scheme, out, n_in, T)
        for r, k in zip(rows, ks):
            assert torch.equal(b[:, r], torch.sign(x[:, k]) * torch.sign(s[r]) * float("inf")), (scheme, out, n_in, T)
        a, b = (E.aqlm_linear_act_backward(codes, c, s, dy)[0] for c in (cb, bad))
        keep = [k for k in range(n_in) if k not in ks]
        assert torch.equal(a[:, keep], b[:, keep]), (scheme, out, n_in, T)
        for r, k in zip(rows, ks):
            assert torch.equal(b[:, k], torch.sign(dy[:, r]) * torch.sign(s[r]) * float("inf")), (scheme, out, n_in, T)
        a, b = (E.aqlm_gated_backward((codes, c, s), (codes, cb, s), dy, z, z, act="relu")[0] for c in (cb, bad))
        assert torch.equal(a[:, keep], b[:, keep]), (scheme, out, n_in, T)


def test_infinite_gradients_stay_in_their_token():
    """Infinities and NaN in the last token's gradient, at batches that end inside every token tile."""
    rng = np.random.default_rng(10)
    for scheme, T in itertools.product(("2x8", "1x16", "4x8g16"), (2, 15, 16, 17, 33, 65, 127, 129, 257, 300)):
        gate, _, _ = layer(scheme, 264, 272, 22)
        up, _, _ = layer(scheme, 264, 272, 23)
        dy, zg, zu = (half(rng, T, 264).cuda() for _ in range(3))
        bad, zb = dy.clone(), zg.clone()
        bad[T - 1, ::3] = float("inf")
        zb[T - 1, 1::3] = float("nan")
        a = E.aqlm_gated_backward(gate, up, dy, zg, zu, need_dbias=True)
        b = E.aqlm_gated_backward(gate, up, bad, zb, zu, need_dbias=True)
        assert torch.equal(a[0][:-1], b[0][:-1]) and torch.isnan(b[0][-1]).all()
        for i in (1, 2):   # the bias sums of the rows that are finite in every token
            assert torch.equal(a[i][2::3], b[i][2::3]) and not torch.isfinite(b[i][1::3]).any()


def rows_of(codes, cb, s, rows):
    """float64 weights of some rows of a layer on the GPU."""
    M, B, g = cb.shape[0], cb.shape[1].bit_length() - 1, cb.shape[2]
    L = synth.Layer("rows", M, B, g, cb.cpu().numpy(), codes[rows].cpu().numpy(), s[rows].cpu().numpy(), None)
    return R.weights(L)


@pytest.mark.parametrize("scheme", ["2x8", "1x16", "4x8g16"])
def test_a_layer_beyond_4_gb(scheme):
    """Codes beyond 4 GB, and at 600 tokens a workspace and outputs beyond it, at rows on both sides of every power."""
    out, n_in, M, B, g = 2_200_003, 8192, *SCHEMES[scheme]
    gen = torch.Generator(device="cuda").manual_seed(5)
    (_, cb, _), _, rounded = layer(scheme, 16, n_in, 24)
    if B == 8:
        codes = torch.randint(0, 256, (out, n_in // g, M), dtype=torch.uint8, device="cuda", generator=gen)
    else:
        codes = torch.randint(-(1 << 15), 1 << 15, (out, n_in // g, M), dtype=torch.int16, device="cuda", generator=gen)
    s = torch.rand((out,), device="cuda", generator=gen).half() * 0.25 + 0.125
    rows = sorted({0, 1, 255, 256, out - 1, out - 2, out - 257, *(int(2 ** 31 // n_in) + k for k in (-1, 0, 1)),
                   *(int(2 ** 32 // (n_in // 4)) + k for k in (-1, 0, 1)), 1 << 20, (1 << 21) - 1, 1 << 21})
    w = rows_of(codes, cb, s, rows)
    rng = np.random.default_rng(11)
    for T in (1, 16, 40, 600):
        x = half(rng, T, n_in)
        y = E.aqlm_linear_act(codes, cb, s, x.cuda(), act="silu")[:, rows]
        want, tol, _, _ = R.linear(w, x.double(), "silu", None, None, rounded)
        R.assert_within(y, want, tol, f"y {T}")
        del y
    for T in (1, 40, 600):   # all other rows' gradients are zero
        dy = torch.zeros((T, out), dtype=torch.float16, device="cuda")
        some = half(rng, T, len(rows))
        dy[:, rows] = some.cuda()
        dx, db = E.aqlm_linear_act_backward(codes, cb, s, dy, need_dbias=True)
        want, tol, sums = R.back([some.double()], [w], True)
        R.assert_within(dx, want, tol, f"dx {T}")
        R.assert_within(db[rows], *sums[0], "dbias")
        del dy, dx, db
        torch.cuda.empty_cache()


def test_a_batch_beyond_4_gb():
    """x and dx of 4.4e9 elements: the first and last tokens, and those around each power of two."""
    T, out, n_in = 270_011, 16, 16384
    gpu, w, rounded = layer("2x8", out, n_in, 25)
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.empty((T, n_in), dtype=torch.float16, device="cuda").normal_(generator=gen)
    rows = [0, 1, (1 << 17) - 1, 1 << 17, (1 << 18) - 1, 1 << 18, T - 2, T - 1]
    z = torch.empty((T, out), dtype=torch.float16, device="cuda")
    y = E.aqlm_linear_act(*gpu, x, act="gelu", z=z)
    want, tol, wz, tz = R.linear(w, x[rows].double().cpu(), "gelu", None, None, rounded)
    R.assert_within(y[rows], want, tol, "y")
    R.assert_within(z[rows], wz, tz, "z")
    dy = torch.empty((T, out), dtype=torch.float16, device="cuda").normal_(0, 0.125, generator=gen)
    dx, db = E.aqlm_linear_act_backward(*gpu, dy, act="gelu", z=z, need_dbias=True, dx=x)
    dz = R.linear_grads(dy.double().cpu(), z.double().cpu(), "gelu")[0]
    want, tol, _ = R.back([dz[rows]], [w], True)
    R.assert_within(dx[rows], want, tol, "dx")
    # fp32 sums of T terms of either sign: (T / 16) / 4 + 8 steps of 2^-24 of a running sum below 4 sqrt(T) rms
    sums, rms = dz.sum(0), dz.square().mean(0).sqrt()
    tol = (T / 64 + 8) * 2.0 ** -24 * 4 * T ** 0.5 * rms
    R.assert_within(db, sums, tol + R.H * (sums.abs() + tol) + R.SUB, "dbias")


def block(scheme, seed):
    gate, _, _ = layer(scheme, 528, 272, seed)
    up, _, _ = layer(scheme, 528, 272, seed + 1)
    down, _, _ = layer(scheme, 272, 528, seed + 2)

    def step(x, zg, zu, zd):
        """A feed-forward block on the residual stream and its gradients."""
        h = E.aqlm_gated(gate, up, x, zg=zg, zu=zu)
        y = E.aqlm_linear_act(*down, h, act="gelu", residual=x, z=zd)
        dh, db = E.aqlm_linear_act_backward(*down, y, act="gelu", z=zd, need_dbias=True)
        dx, dbg, dbu = E.aqlm_gated_backward(gate, up, dh, zg, zu, need_dbias=True)
        return [y, dx, db, dbg, dbu]
    return step


def block_arrays(T):
    return [torch.empty((T, n), dtype=torch.float16, device="cuda") for n in (528, 528, 272)]


@pytest.mark.parametrize("scheme", ["2x8", "1x16", "4x8g16"])
@pytest.mark.parametrize("T", [7, 70, 200, 600])
def test_graph_replays(scheme, T):
    """Two captured blocks replayed in turn between eager calls: each replay gives the eager results."""
    rng = np.random.default_rng(12)
    step = block(scheme, 30)
    xs = [half(rng, T, 272).cuda() for _ in range(2)]
    arrays = [block_arrays(T) for _ in range(2)]
    for x, a in zip(xs, arrays):
        step(x, *a)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x, a in zip(xs, arrays):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(x, *a))
        graphs.append(g)
    for _ in range(4):
        for x in xs:
            x.copy_(half(rng, T, 272).cuda())
        for g in graphs:
            g.replay()
        got = [[t.clone() for t in o] for o in outs]
        want = [step(x, *block_arrays(T)) for x in xs]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w)), (scheme, T)


@pytest.mark.parametrize("T", [7, 70, 600])
def test_two_streams_at_once(T):
    """Calls in flight on two streams at the same time, each with its own workspaces."""
    rng = np.random.default_rng(13)
    for scheme in ("2x8", "1x16"):
        step = block(scheme, 40)
        xs = [half(rng, T, 272).cuda() for _ in range(2)]
        want = [step(x, *block_arrays(T)) for x in xs]
        arrays = [block_arrays(T) for _ in range(2)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        got = [[], []]
        for _ in range(8):
            for i, stream in enumerate(streams):
                with torch.cuda.stream(stream):
                    got[i].append(step(xs[i], *arrays[i]))
        torch.cuda.synchronize()
        for i in range(2):
            for g in got[i]:
                assert all(torch.equal(a, b) for a, b in zip(g, want[i])), (scheme, T)


@pytest.mark.parametrize("T", [17, 64, 65, 96, 97, 130, 160, 257, 300])
def test_the_workspace_is_enough(T):
    """With exactly the bytes asked for, the results are those of a larger one and nothing behind them changes."""
    rng = np.random.default_rng(14)
    for scheme, (out, n_in) in itertools.product(("2x8", "1x16", "4x8g16"), ((72, 272), (700, 1040), (3000, 256), (96, 4096))):
        M, B, g = SCHEMES[scheme]
        gate, _, _ = layer(scheme, out, n_in, 50)
        up, _, _ = layer(scheme, out, n_in, 51)
        x, dy, z = half(rng, T, n_in).cuda(), half(rng, T, out).cuda(), half(rng, T, out).cuda()
        for name, f in (("linear_act", lambda **k: [E.aqlm_linear_act(*gate, x, act="silu", **k)]),
                        ("gated", lambda **k: [E.aqlm_gated(gate, up, x, **k)]),
                        ("linear_act_backward", lambda **k: E.aqlm_linear_act_backward(*gate, dy, act="silu", z=z,
                                                                                       need_dbias=True, **k)),
                        ("gated_backward", lambda **k: E.aqlm_gated_backward(gate, up, dy, z, z, need_dbias=True, **k))):
            need = getattr(E, name + "_workspace_bytes")(M, B, g, out, n_in, T)
            buf = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")   # parts unwritten would be NaN
            got, want = f(workspace=buf[:need]), f(workspace=torch.zeros(2 * need + 4096, dtype=torch.uint8, device="cuda"))
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (name, scheme, out, n_in)
            assert bool((buf[need:] == 0xFF).all()), (name, scheme, out, n_in)
