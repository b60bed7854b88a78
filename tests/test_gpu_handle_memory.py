"""What a parameter handle holds on the device."""
import pytest
import torch

import rotated_bit_kv_isoquant_b200 as iq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [128, 256])
def test_handles_of_many_layers_are_small(d):
    """A handle holds its rotation parameters and their blocks, tens of KB, whatever is done with
    it; 64 of them, as for the layers of a model, fit a few MB."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    first = iq.isoq_make_params(0, d, 8)
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    handles = [iq.isoq_make_params(i, d, 8) for i in range(64)]
    used = before - torch.cuda.mem_get_info()[0]
    assert used <= 8 << 20, f"64 handles take {used >> 20} MB"
    del first, handles
