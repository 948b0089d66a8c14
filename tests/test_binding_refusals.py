"""CPU: the binding names what is wrong with a layer's sizes and operands."""
import pytest
import torch

import gated_deltanet_decode_amd as gdn


@pytest.mark.parametrize("kw", [dict(batch=0), dict(num_heads=0, num_groups=0), dict(batch=-1)])
def test_prompt_of_an_empty_layer(kw):
    d = gdn.ssm_dims(**{**dict(batch=2, num_heads=4, num_groups=2, head_dim=64, state_dim=64), **kw})
    with pytest.raises(gdn.GdnError):
        gdn.ssm_prefill(d, None, None, None, torch.zeros(2, 8, 64), None, None, None, None)


@pytest.mark.parametrize("x", [None, torch.zeros(0), torch.zeros(2, 8, 63)])
def test_prompt_without_whole_rows(x):
    with pytest.raises(ValueError, match="x must be"):
        gdn.ssm_prefill(gdn.ssm_dims(2, 4, 2, 64, 64), None, None, None, x, None, None, None, None)
