"""One workspace, sized for the largest batch, serves calls of every smaller batch with the results of a private one."""
import numpy as np
import pytest
import torch

import extreme_weight_quantization_amd as E
from test_gpu_fused import SCHEMES, half, layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need an MI355X")
    E.load_library()


@pytest.mark.parametrize("scheme,out,n_in", [("2x8", 1000, 2048), ("2x8", 72, 8192), ("1x16", 4096, 2048), ("1x16", 264, 272),
                                             ("4x8g16", 520, 1040), ("1x8g4", 136, 4096)])
def test_one_buffer_for_all_batches(scheme, out, n_in):
    rng = np.random.default_rng(1)
    M, B, g = SCHEMES[scheme]
    gate, _, _ = layer(scheme, out, n_in, 1)
    up, _, _ = layer(scheme, out, n_in, 2)
    largest = 1100
    x, dy, z = half(rng, largest, n_in).cuda(), half(rng, largest, out).cuda(), half(rng, largest, out).cuda()
    calls = {"linear_act": lambda T, **k: [E.aqlm_linear_act(*gate, x[:T], act="silu", **k)],
             "gated": lambda T, **k: [E.aqlm_gated(gate, up, x[:T], **k)],
             "linear_act_backward": lambda T, **k: E.aqlm_linear_act_backward(*gate, dy[:T], act="silu", z=z[:T],
                                                                              need_dbias=True, **k),
             "gated_backward": lambda T, **k: E.aqlm_gated_backward(gate, up, dy[:T], z[:T], z[:T], need_dbias=True, **k)}
    for name, f in calls.items():
        need = getattr(E, name + "_workspace_bytes")(M, B, g, out, n_in, largest)
        buf = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
        for T in (1, 16, 17, 40, 64, 65, 128, 129, 130, 256, 257, 320, 321, 512, 513, 640, 923, 1057, 1100):
            got, want = f(T, workspace=buf[:need]), f(T)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (name, T)
        assert bool((buf[need:] == 0xFF).all()), name
