"""Experts that a token names more than once, in batches of fewer than 16 tokens: an expert then has more columns than
there are tokens.  Tokens differ, so that a column which takes another token's activations shows.  (serving_reference.py: what
tolerances count.)"""
import pytest
import torch

import extreme_weight_quantization_amd as E
from test_gpu_moe import Layer, gen

pytestmark = pytest.mark.gpu

AQLM = [(2, 8, 8), (1, 16, 8), (1, 8, 4), (4, 8, 16), (8, 8, 32), (3, 5, 2)]
AQLM_NAMES = ["2x8", "1x16", "1x8g4", "4x8g16", "8x8g32", "3x5g2"]
TOKENS_K = [(1, 2), (1, 4), (1, 16), (2, 2), (2, 8), (3, 4), (4, 2), (5, 2), (5, 8), (8, 2), (8, 4), (15, 2), (15, 8)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need an MI355X")
    E.load_library()


def repeated(tokens, k, experts, how, seed):
    if how == "all":          # one expert, as the padding rows of a captured batch name it
        return torch.full((tokens, k), 1, dtype=torch.int32)
    ids = torch.randint(0, experts, (tokens, k), generator=gen(seed), dtype=torch.int32)
    ids[:, 1] = ids[:, 0]     # every token one of its experts twice
    ids[-1] = 2               # the last one the same expert every time
    return ids


def run(scheme, n_in, inner, tokens, k, how):
    n = tokens * 32 + k
    L = Layer(scheme, 4, n_in, inner, seed=n)
    x, _, w, residual = L.inputs(tokens, k, seed=n + 1, distinct=False)
    L.check(x, repeated(tokens, k, 4, how, n + 2), w, "silu", residual if n % 2 else None)


@pytest.mark.parametrize("how", ["all", "partly"])
@pytest.mark.parametrize("tokens,k", TOKENS_K)
@pytest.mark.parametrize("scheme", AQLM, ids=AQLM_NAMES)
def test_aqlm_experts(scheme, tokens, k, how):
    run(scheme, 96, 64, tokens, k, how)


@pytest.mark.parametrize("tokens,k", [(1, 4), (3, 4), (5, 2), (8, 2)])
@pytest.mark.parametrize("scheme", AQLM[:4], ids=AQLM_NAMES[:4])
def test_aqlm_experts_with_long_rows(scheme, tokens, k):
    """Rows of more than 2048 inputs: 16 waves a tile instead of two teams."""
    run(scheme, 2080, 2112, tokens, k, "partly")


@pytest.mark.parametrize("how", ["all", "partly"])
@pytest.mark.parametrize("tokens,k", TOKENS_K)
def test_mx4_experts(tokens, k, how):
    run("mx4", 96, 64, tokens, k, how)


@pytest.mark.parametrize("n_in,inner,tokens,k", [(4096, 96, 1, 4), (4096, 96, 7, 2), (4096, 64, 8, 8), (2048, 1056, 15, 4),
                                                 (32768, 32, 1, 2), (16384, 32, 2, 8), (16384, 32, 3, 8), (1056, 4128, 5, 4)])
def test_mx4_experts_with_long_rows(n_in, inner, tokens, k):
    """Activations split in LDS, up to the most that fit, and split before."""
    run("mx4", n_in, inner, tokens, k, "partly")


@pytest.mark.parametrize("scheme", [(2, 8, 8), (1, 16, 8), "mx4"], ids=["2x8", "1x16", "mx4"])
def test_padding_rows_of_a_batch_leave_the_others_alone(scheme):
    """Rows behind the last token that all name expert 0, as a captured batch has them: the tokens' results are those of the
    batch without them."""
    L = Layer(scheme, 4, 160, 96, seed=5)
    x, ids, w, residual = L.inputs(8, 2, seed=6)
    x[5:], ids[5:], w[5:], residual[5:] = 0, 0, 0, 0
    y = L.check(x, ids, w, "silu", residual).cpu()
    assert float(y[5:].abs().max()) == 0
    assert torch.equal(y[:5], L.run(x[:5], ids[:5], w[:5], residual=residual[:5]).cpu())
