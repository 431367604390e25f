"""The mixers' Python layer on the CPU: what a caller may rely on before a call reaches the
library (which needs a GPU)."""
import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv


@pytest.mark.parametrize("name", ["k", "v", "k_amax", "v_amax"])
def test_a_caches_tensors_cannot_be_replaced(name):
    """The descriptor holds their addresses, so another tensor in a tensor's place is refused."""
    cache = nv.PagedKVCache.__new__(nv.PagedKVCache)       # (its constructor wants cuda tensors)
    with pytest.raises(AttributeError):
        setattr(cache, name, torch.zeros(1))
