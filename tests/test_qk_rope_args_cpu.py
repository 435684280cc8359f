"""Arguments of the norm and rotation that the binding refuses before any call."""
import pytest
import torch

from gated_deltanet_chunked_gb300 import gdn


@pytest.mark.parametrize("shape", [(), (1, 1, 4), (2, 2, 4)])
@pytest.mark.parametrize("axis", [False, True])
def test_positions_of_other_dimensions(shape, axis):
    q, freq = torch.zeros(4, 2, 128), torch.zeros(64)
    pos = torch.zeros(shape, dtype=torch.int32)
    pair_axis = torch.zeros(64, dtype=torch.int32) if axis else None
    with pytest.raises(ValueError, match="positions"):
        gdn.gdn_qk_norm_rope(q, q, None, None, freq, pos, pair_axis=pair_axis)
    with pytest.raises(ValueError, match="positions"):
        gdn.gdn_qk_norm_rope_bwd(q, q, q, q, None, None, freq, pos, pair_axis=pair_axis)
