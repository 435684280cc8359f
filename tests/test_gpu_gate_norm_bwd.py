"""gdn_gated_rmsnorm_bwd against the definition in 64 bits, with bounds that
count the roundings (train_ref)."""
import pytest
import torch

import train_ref as R
from gated_deltanet_chunked_gb300 import gdn

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DTYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
EPS = 1e-6


def make(seed, T, hv, dtype):
    gen = torch.Generator().manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen)
    return {"dy": normal(T, hv, 128).to(dtype), "o": (normal(T, hv, 128) * 0.05).to(dtype),
            "z": normal(T, hv, 128).to(dtype), "w": normal(128) + 1}


def run(d, dev, **kw):
    c = {k: v.to(dev) for k, v in d.items()}
    do, dz, dw = gdn.gdn_gated_rmsnorm_bwd(c["dy"], c["o"], c["z"], c["w"], EPS, **kw)
    return {"do": do, "dz": dz, "dweight": dw}


def compare(res, d, dtype):
    flat = {k: R.f64(v).reshape(-1, 128) for k, v in d.items() if k != "w"}
    ref = R.gate_bwd(flat["dy"], flat["o"], flat["z"], R.f64(d["w"]), EPS, dtype)
    for name, t in res.items():
        R.assert_within(t if name == "dweight" else t.reshape(-1, 128), *ref[name], name)


@DTYPES
@pytest.mark.parametrize("T,hv", [(1, 1), (1, 3), (5, 1), (16, 1), (37, 3), (333, 2), (1000, 32), (4096, 8)])
def test_sizes(cuda, T, hv, dtype):
    d = make(T + hv, T, hv, dtype)
    compare(run(d, cuda), d, dtype)


@DTYPES
def test_zero_rows_and_saturated_gates(cuda, dtype):
    d = make(3, 50, 2, dtype)
    d["o"][7] = 0
    d["z"][9, :, :40] = 60.0
    d["z"][10, :, :40] = -60.0
    d["z"][11] = -200.0
    d["z"][12] = 200.0
    d["z"][13] = 0.0
    d["dy"][14] = 0
    compare(run(d, cuda), d, dtype)


@DTYPES
def test_in_place_and_without_the_weight(cuda, dtype):
    d = make(4, 77, 3, dtype)
    ref = run(d, cuda)
    for a, b in (("dy", "z"), ("o", "dy"), ("z", "o")):
        c = {k: v.to(cuda) for k, v in d.items()}
        do, dz, dw = gdn.gdn_gated_rmsnorm_bwd(c["dy"], c["o"], c["z"], c["w"], EPS, do=c[a], dz=c[b])
        assert torch.equal(do, ref["do"]) and torch.equal(dz, ref["dz"]) and torch.equal(dw, ref["dweight"])
    res = run(d, cuda, need_dweight=False)
    assert res["dweight"] is None and torch.equal(res["do"], ref["do"])


def test_a_row_with_nan_stays_one_row(cuda):
    d = make(5, 30, 2, BF16)
    clean = run(d, cuda)
    d["o"][11, 1, 5] = float("nan")
    res = run(d, cuda)
    keep = [r for r in range(60) if r != 23]
    for k in ("do", "dz"):
        assert torch.equal(res[k].reshape(60, 128)[keep], clean[k].reshape(60, 128)[keep]), k


def test_no_rows(cuda):
    d = {k: v.to(cuda) for k, v in make(6, 4, 2, F32).items()}
    do, dz, dw = gdn.gdn_gated_rmsnorm_bwd(d["dy"][:0], d["o"][:0], d["z"][:0], d["w"], EPS,
                                           dweight=torch.ones(128, device=cuda))
    torch.cuda.synchronize()
    assert do.shape == (0, 2, 128) and (dw == 0).all()


def test_same_bits_every_time_and_in_a_graph(cuda):
    d = {k: v.to(cuda) for k, v in make(7, 3000, 4, BF16).items()}
    ref, again = run(d, cuda), run(d, cuda)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run(d, cuda)
    graph.replay()
    torch.cuda.synchronize()
    for k in ref:
        assert torch.equal(ref[k], again[k]) and torch.equal(ref[k], captured[k]), k
