"""How long linear attention's segments are, from the workspaces' sizes: each way where it was measured to be the faster
one by a tenth at least."""
import ctypes

import pytest

from gated_deltanet_chunked_gb300 import gdn
from test_training_cpu import problem

STATE = 128 * 128 * 4


def segments(io_dtype, total, hv, num_seqs, back=False):
    """Segments that a call has at most, 0 where every sequence is one for sure (a state for each head, segment and role)."""
    p = problem(total_tokens=total, num_seqs=num_seqs, hq=hv, hv=hv, io_dtype=io_dtype)
    name = f"gdn_linear_attention{'_bwd' if back else ''}_workspace_size"
    return getattr(gdn.load(), name)(ctypes.byref(p)) // (hv * (3 if back else 1) * STATE)


BF16, F32 = gdn.GDN_DT_BF16, gdn.GDN_DT_F32


@pytest.mark.parametrize("back", [False, True])
def test_a_short_prompt_is_one_segment(back):
    """bf16: 16 us in one kernel, 25 in three."""
    assert segments(BF16, 200, 2, 1, back) == 0


def test_few_blocks_are_cut():
    """f32, 200 tokens: 27 us cut into blocks of 32, 79 whole."""
    assert segments(F32, 200, 2, 1) == 200 // 32 + 1


def test_whole_rounds_of_equal_sequences():
    """4 sequences of 1500 tokens x 40 heads, 160 CTAs of them on 152 SMs: f32 982 us whole and 792 to 833 cut; bf16 98
    whole and 116 cut."""
    assert segments(F32, 6000, 40, 4) > 6000 // 1500 + 4
    assert segments(BF16, 6000, 40, 4) <= 6000 // 1500 + 4


def test_a_round_of_whole_sequences():
    """The same backward, 480 CTAs: f32 1975 us whole and 2055 to 2862 cut, bf16 258 and 310."""
    for dtype in (F32, BF16):
        assert segments(dtype, 6000, 40, 4, True) <= 6000 // 1500 + 4
