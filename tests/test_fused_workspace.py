"""Workspace sizes of the fused products: a buffer for the largest batch serves every smaller one (no GPU needed)."""
import random

import pytest

import extreme_weight_quantization_amd as E

QUERIES = (E.linear_act_workspace_bytes, E.gated_workspace_bytes, E.linear_act_backward_workspace_bytes,
           E.gated_backward_workspace_bytes)
SCHEMES = ((2, 8, 8), (1, 16, 8), (4, 8, 16), (1, 8, 4), (8, 8, 32), (2, 10, 4))
LAYERS = ((4096, 4096), (4096, 11008), (11008, 4096), (28672, 8192), (8, 64), (100, 8192), (2733, 1000 // 32 * 32), (65536, 64),
          (64, 65536), (1 << 20, 256))


@pytest.mark.parametrize("query", QUERIES)
@pytest.mark.parametrize("scheme", SCHEMES)
def test_never_less_for_a_larger_batch(query, scheme):
    for out, n_in in LAYERS:
        most = 0
        for T in sorted({*range(0, 1400), *range(1400, 9000, 61), *(2 ** k + d for k in range(11, 20) for d in (-1, 0, 1))}):
            n = query(*scheme, out, n_in, T)
            assert n >= most, (scheme, out, n_in, T)
            most = n


@pytest.mark.parametrize("query", QUERIES)
def test_never_less_at_random_sizes(query):
    rng = random.Random(1)
    for _ in range(300):
        M, B, g = rng.choice(SCHEMES)
        out, n_in = int(2 ** rng.uniform(0, 16)), g * int(2 ** rng.uniform(0, 10))
        batches = sorted(int(2 ** rng.uniform(0, 17)) for _ in range(200))
        sizes = [query(M, B, g, out, n_in, T) for T in batches]
        assert sizes == sorted(sizes), (M, B, g, out, n_in)


def test_what_is_reserved_stays_near_what_the_weights_take():
    """Decoded weights, activations or gradients, and fp32 parts of the results: a bounded set, or the two that a
    product straight from the codes writes of each row block (backward: one of each layer's dx)."""
    pad = lambda v: (v + 63) // 64 * 64   # noqa: E731
    for scheme in SCHEMES:
        for out, n_in in LAYERS:
            for T in (17, 64, 300, 2048, 8192):
                for query, n, back in zip(QUERIES, (1, 2, 1, 2), (False, False, True, True)):
                    w = 2 * n * pad(out) * pad(n_in)
                    rows = 2 * T * (n * pad(out) if back else pad(n_in)) + (8 * T * n * pad(out) // 4 if back else 0)
                    parts = 4 * min(T, 512) * n * (pad(n_in) if back else 2 * pad(out))
                    assert query(*scheme, out, n_in, T) <= 2 * (w + rows) + parts + (256 << 20), (scheme, out, n_in, T)
