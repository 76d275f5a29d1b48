"""The binding of the experts' layers checks each of them once a call (no GPU needed)."""
import torch

from extreme_weight_quantization_amd import moe


def test_every_layer_is_checked_once():
    dev = torch.device("cpu")
    gate = (torch.zeros((4, 96, 32), dtype=torch.uint8), torch.zeros((4, 96, 2), dtype=torch.uint8))
    down = (torch.zeros((4, 64, 48), dtype=torch.uint8), torch.zeros((4, 64, 3), dtype=torch.uint8))
    up = tuple(t.clone() for t in gate)
    seen = []

    def make(name, *args):
        seen.append(name)
        return moe._experts_mx4(name, *args)

    sch, E, n_in, inner, arrays = moe._layers(make, gate, up, down, dev)
    assert seen == ["gate", "up", "down"]
    assert (sch, E, n_in, inner) == ((), 4, 64, 96)
    assert [list(a) for a in arrays] == [[layer[i].data_ptr() for layer in (gate, up, down)] for i in range(2)]
