"""Linear attention where its pipelines go round many times, walks of long sequences left whole and segments of many chunks
summed and chained: every token of a few heads, normwise, against the definition in 64 bits."""
import pytest
import torch

import linattn_long_ref as L
import test_gpu_linattn as la
from gated_deltanet_chunked_gb300 import gdn

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DTYPES = la.DTYPES


def segment_rows(d, back):
    """Rows that a segment has at least, from the workspace's size: a state for each head and segment (and role)."""
    T, hq, hv, N = len(d["q"]), d["q"].shape[1], d["v"].shape[1], len(d["cu"]) - 1
    need = gdn._linattn_layout(d["q"].shape, d["v"].shape, d["q"].dtype, d["cu"].shape)[3 if back else 2]
    if back and hq != hv:
        need -= 2 * T * hv * 512
    per_segment = (3 if back else 1) * hv * 65536
    return T // max(need // per_segment - N + 1, 1)


def inputs(seed, lens, hq, hv, dtype, init, dev):
    """As la.make, on the GPU."""
    gen = torch.Generator(device=dev).manual_seed(seed)
    normal = lambda *shape, to=F32: torch.randn(shape, generator=gen, device=dev).to(to)
    T, N = sum(lens), len(lens)
    d = {"q": normal(T, hq, 128, to=dtype), "k": normal(T, hq, 128, to=dtype), "v": normal(T, hv, 128, to=dtype),
         "dout": normal(T, hv, 128, to=dtype), "scale": la.SCALE, "s0": normal(N, hv, 128, 128) if init else None,
         "dfinal": normal(N, hv, 128, 128) if init else None}
    d["decay"] = -2.0 ** (-10.0 * (torch.arange(hv, device=dev) + 1) / hv)
    d["cu"] = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)
    return d


@DTYPES
@pytest.mark.parametrize("hq,hv", [(40, 40), (20, 40)], ids=["heads", "groups"])
def test_whole_sequences(cuda, dtype, hq, hv):
    """Walks of 12 chunks, in time and against it, with states in and out."""
    lens = [1500, 1536, 1400, 1531]
    d = inputs(50, lens, hq, hv, dtype, True, cuda)
    if dtype == BF16:  # left whole
        assert min(segment_rows(d, back) for back in (False, True)) >= max(lens)
    res = la.run(d)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    L.compare(res, d, lens, dtype, [0, hq - 1])


SLOW = [-1e-5, 0.0]  # heads that keep nearly everything, so that one segment's sum goes on into all later ones


def test_summed_segments(cuda):
    """Segments of 57 chunks, forward."""
    d = inputs(51, [65536], 16, 32, BF16, True, cuda)
    d["decay"][-2:] = torch.tensor(SLOW, device=cuda)
    assert 50 * 128 <= segment_rows(d, False) <= 65536 // 8
    out, final = gdn.gdn_linear_attention(d["q"], d["k"], d["v"], d["decay"], d["scale"], initial_state=d["s0"],
                                          cu_seqlens=d["cu"])
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    L.compare({"out": out, "final": final}, d, [65536], BF16, [0, 15])


@DTYPES
@pytest.mark.parametrize("hq,hv", [(8, 8), (4, 8)], ids=["heads", "groups"])
def test_summed_segments_backward(cuda, dtype, hq, hv):
    """Segments of 8 chunks forward and 26 backward, the last one ragged."""
    d = inputs(52, [20001], hq, hv, dtype, True, cuda)
    d["decay"][-2:] = torch.tensor(SLOW, device=cuda)
    if dtype == BF16:
        assert segment_rows(d, False) >= 8 * 128 and 20 * 128 <= segment_rows(d, True) <= 20001 // 5
    res = la.run(d)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    L.compare(res, d, [20001], dtype, [0, hq - 1])


@DTYPES
@pytest.mark.parametrize("hq,hv", [(1, 1), (1, 3)])
@pytest.mark.parametrize("init", [False, True], ids=["zero", "init"])
def test_few_chunks_normwise(cuda, dtype, hq, hv, init):
    lens = [1100, 129, 300, 256]
    d = inputs(53, lens, hq, hv, dtype, init, cuda)
    L.compare(la.run(d), d, lens, dtype, range(hq))


@DTYPES
@pytest.mark.parametrize("decay", [[0.0, -1e-4], [-0.7, -5.0], [-30.0, -0.34657]])
def test_decays_normwise(cuda, dtype, decay):
    lens = [700, 130, 1024]
    d = inputs(54, lens, 2, 2, dtype, True, cuda)
    d["decay"] = torch.tensor(decay, device=cuda)
    L.compare(la.run(d), d, lens, dtype, [0, 1])
