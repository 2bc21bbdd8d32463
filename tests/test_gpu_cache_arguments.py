"""Arguments of the cache operators that are refused before anything is launched."""

import pytest
import torch

import speculative_decoding_verification_temp_gb300 as sv

pytestmark = pytest.mark.gpu


def setup(dtype=torch.bfloat16):
    k, v = (torch.zeros(4, 16, 2, 64, dtype=dtype, device="cuda") for _ in "kv")
    new = [torch.ones(1, 2, 2, 64, dtype=dtype, device="cuda") for _ in "kv"]
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    ctx = torch.zeros(1, dtype=torch.int32, device="cuda")
    return k, v, new, table, ctx, sv.rotary_frequency(64).frequency


def test_frequencies_that_require_gradients():
    k, v, new, table, ctx, f = setup()
    f.requires_grad_()
    position = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        sv.rotary(new[0], position, f)
    with pytest.raises(ValueError):
        sv.cache_append_rotary(*new, k, v, table, ctx, f)
    assert not k.any() and not v.any()
    with torch.no_grad():
        assert torch.equal(sv.rotary(new[0], position, f), new[0])


@pytest.mark.parametrize("position", [[0, 1], 0, torch.zeros(2, dtype=torch.int32)], ids=["list", "number", "cpu"])
def test_positions_that_are_no_tensors_of_the_device(position):
    k, v, new, table, ctx, f = setup()
    with pytest.raises(ValueError):
        sv.cache_append_rotary(*new, k, v, table, ctx, f, position=position)
    with pytest.raises(ValueError):
        sv.paged_attention(new[0], k, v, table, ctx, position=position)
    assert not k.any() and not v.any()
