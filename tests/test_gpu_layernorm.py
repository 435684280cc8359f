"""gdn_layernorm and its backward pass against the definition in 64 bits, with
bounds that count the roundings (train_ref)."""
import pytest
import torch

import train_ref as R
from gated_deltanet_chunked_gb300 import gdn

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DTYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
EPS = 1e-5


def make(seed, rows, width, dtype, affine=True, offset=0.3):
    gen = torch.Generator().manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen)
    return {"x": (normal(rows, width) * 1.5 + offset).to(dtype), "dy": normal(rows, width).to(dtype),
            "w": normal(width) + 1 if affine else None, "b": normal(width) if affine else None}


def run(d, dev, eps=EPS):
    c = {k: None if v is None else v.to(dev) for k, v in d.items()}
    y, mean, rstd = gdn.gdn_layernorm(c["x"], c["w"], c["b"], eps, save_stats=True)
    dx, dw, db = gdn.gdn_layernorm_bwd(c["dy"], c["x"], mean, rstd, c["w"])
    return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dweight": dw, "dbias": db}


def compare(res, d, dtype, eps=EPS):
    x, w = R.f64(d["x"]), R.f64(d["w"])
    ref = R.layernorm(x, w, R.f64(d["b"]), eps, dtype)
    ref |= R.layernorm_bwd(R.f64(d["dy"]), x, R.f64(res["mean"]), R.f64(res["rstd"]), w, dtype)
    for name, t in res.items():
        R.assert_within(t, *ref[name], name)


@DTYPES
@pytest.mark.parametrize("width", [1, 2, 7, 8, 16, 63, 64, 65, 100, 128, 129, 136, 250, 256, 257, 264, 511, 512, 513,
                                   520, 1001, 1024, 2056, 4096, 4100, 8184, 8192, 8193, 8200, 16383, 16384])
def test_widths(cuda, width, dtype):
    for rows in (1, 37):
        d = make(width, rows, width, dtype)
        compare(run(d, cuda), d, dtype)


@DTYPES
@pytest.mark.parametrize("rows,width", [(2, 128), (31, 128), (3000, 128), (20011, 64), (2500, 1001), (2500, 600), (2501, 700),
                                        (2500, 720), (1300, 2048)])
def test_rows(cuda, rows, width, dtype):
    d = make(rows, rows, width, dtype)
    compare(run(d, cuda), d, dtype)


@DTYPES
def test_without_weight_and_bias(cuda, dtype):
    d = make(5, 70, 384, dtype, affine=False)
    compare(run(d, cuda), d, dtype)


@pytest.mark.parametrize("width", [96, 2000])
def test_large_offset_does_not_cancel(cuda, width):
    """A mean 10^3 times the deviation: the squares are taken about the mean."""
    d = make(6, 40, width, F32, offset=1500.0)
    compare(run(d, cuda), d, F32)


@DTYPES
def test_constant_rows(cuda, dtype):
    d = make(8, 9, 640, dtype)
    d["x"][3] = 0.75
    d["x"][4] = 0.0
    res = run(d, cuda)
    compare(res, d, dtype)
    R.assert_within(res["y"][4:5], *((R.f64(d["b"])[None], R.U[dtype] * abs(R.f64(d["b"])[None]))), "zero row")


@pytest.mark.parametrize("width", [128, 640])
def test_a_row_with_nan_stays_one_row(cuda, width):
    d = make(9, 20, width, BF16)
    clean = run(d, cuda)
    d["x"][7, 3] = float("nan")
    d["x"][12, 0] = float("inf")
    res = run(d, cuda)
    keep = [r for r in range(20) if r not in (7, 12)]
    for k in ("y", "dx", "mean", "rstd"):
        assert torch.equal(res[k][keep], clean[k][keep]), k
        assert torch.isnan(res[k][7]).all(), k


@DTYPES
@pytest.mark.parametrize("width", [100, 1001, 1024])
def test_in_place(cuda, width, dtype):
    d = make(10, 33, width, dtype)
    ref = run(d, cuda)
    x, w, b = d["x"].to(cuda), d["w"].to(cuda), d["b"].to(cuda)
    y = gdn.gdn_layernorm(x, w, b, EPS, out=x)
    assert y is x and torch.equal(x, ref["y"])
    for into in ("dy", "x"):
        c = {k: v.to(cuda) for k, v in d.items()}
        dx, dw, db = gdn.gdn_layernorm_bwd(c["dy"], c["x"], ref["mean"], ref["rstd"], c["w"], dx=c[into])
        assert torch.equal(dx, ref["dx"]) and torch.equal(dw, ref["dweight"]) and torch.equal(db, ref["dbias"])


def test_leading_dimensions_and_parts_of_the_answer(cuda):
    d = make(11, 24, 200, BF16)
    ref = run(d, cuda)
    c = {k: v.to(cuda) for k, v in d.items()}
    y, mean, rstd = gdn.gdn_layernorm(c["x"].reshape(2, 3, 4, 200), c["w"], c["b"], EPS, save_stats=True)
    assert mean.shape == (2, 3, 4) and torch.equal(y.reshape(24, 200), ref["y"])
    dx, dw, db = gdn.gdn_layernorm_bwd(c["dy"].reshape(2, 3, 4, 200), c["x"].reshape(2, 3, 4, 200), mean, rstd,
                                       c["w"], need_dbias=False)
    assert db is None and torch.equal(dw, ref["dweight"]) and torch.equal(dx.reshape(24, 200), ref["dx"])
    dx, dw, db = gdn.gdn_layernorm_bwd(c["dy"], c["x"], ref["mean"], ref["rstd"], c["w"], need_dweight=False)
    assert dw is None and torch.equal(db, ref["dbias"])
    dx, dw, db = gdn.gdn_layernorm_bwd(c["dy"], c["x"], ref["mean"], ref["rstd"], c["w"], need_dweight=False,
                                       need_dbias=False)
    assert dw is None and db is None and torch.equal(dx, ref["dx"])
    one = gdn.gdn_layernorm(c["x"][5], c["w"], c["b"], EPS)
    assert torch.equal(one, ref["y"][5])


@DTYPES
@pytest.mark.parametrize("width", [7, 128, 1001, 2048, 8192, 16383, 16384])
def test_one_of_the_two_sums(cuda, width, dtype):
    """Each sum alone has the bits that it has next to the other."""
    d = make(12, 41, width, dtype)
    ref = run(d, cuda)
    c = {k: v.to(cuda) for k, v in d.items()}
    for need_dw, need_db in ((True, False), (False, True)):
        dx, dw, db = gdn.gdn_layernorm_bwd(c["dy"], c["x"], ref["mean"], ref["rstd"], c["w"], need_dweight=need_dw,
                                           need_dbias=need_db)
        assert torch.equal(dx, ref["dx"])
        assert torch.equal(dw, ref["dweight"]) if need_dw else dw is None
        assert torch.equal(db, ref["dbias"]) if need_db else db is None


def test_no_rows(cuda):
    x = torch.empty(0, 300, device=cuda)
    y, mean, rstd = gdn.gdn_layernorm(x, save_stats=True)
    dw = torch.ones(300, device=cuda)
    dx, dw, db = gdn.gdn_layernorm_bwd(x, x, mean, rstd, dweight=dw)
    torch.cuda.synchronize()
    assert y.shape == (0, 300) and (dw == 0).all() and (db == 0).all()


def test_same_bits_every_time_and_in_a_graph(cuda):
    for rows, width in ((5000, 128), (700, 2048)):
        d = make(12, rows, width, BF16)
        c = {k: v.to(cuda) for k, v in d.items()}
        ref = run(c, cuda)
        again = run(c, cuda)
        graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = run(c, cuda)
        with torch.cuda.graph(graph2):
            captured2 = run(c, cuda)
        graph.replay()
        graph2.replay()
        graph.replay()
        torch.cuda.synchronize()
        for k in ref:
            assert torch.equal(ref[k], again[k]) and torch.equal(ref[k], captured[k]), k
            assert torch.equal(ref[k], captured2[k]), k


@DTYPES
@pytest.mark.parametrize("rows,width", [(701, 4097), (700, 5000), (650, 6408), (701, 8192), (613, 8193),
                                        (400, 12288), (701, 12345),
                                        (333, 16383), (701, 16384)])
def test_many_rows_over_several_ctas(cuda, rows, width, dtype):
    """Wide rows are on a cluster of CTAs: the sums that these exchange for a
    row are not another row's, and a row of NaN stays one row."""
    d = make(rows, rows, width, dtype)
    ref = run(d, cuda)
    compare(ref, d, dtype)
    again = run(d, cuda)
    d["x"][300, width // 2] = float("nan")
    res = run(d, cuda)
    for k in ("y", "dx", "mean", "rstd", "dweight", "dbias"):
        assert torch.equal(again[k], ref[k]), k
        if k in ("dweight", "dbias"):
            continue
        keep = [r for r in range(rows) if r != 300]
        assert torch.equal(res[k][keep], ref[k][keep]) and torch.isnan(res[k][300]).all(), k


@DTYPES
@pytest.mark.parametrize("width", [9001, 12288, 16383])
def test_in_place_over_several_ctas(cuda, width, dtype):
    d = make(13, 90, width, dtype)
    ref = run(d, cuda)
    c = {k: v.to(cuda) for k, v in d.items()}
    y = gdn.gdn_layernorm(c["x"], c["w"], c["b"], EPS, out=c["x"])
    assert y is c["x"] and torch.equal(y, ref["y"])
    for into in ("dy", "x"):
        c = {k: v.to(cuda) for k, v in d.items()}
        dx, dw, db = gdn.gdn_layernorm_bwd(c["dy"], c["x"], ref["mean"], ref["rstd"], c["w"], dx=c[into])
        assert torch.equal(dx, ref["dx"]) and torch.equal(dw, ref["dweight"]) and torch.equal(db, ref["dbias"])


@pytest.mark.parametrize("rows,width", [(300, 16384), (300, 16383), (3000, 1024)])
def test_two_calls_at_once_and_in_graphs(cuda, rows, width):
    """Calls on two streams, eager and replayed, do not see each other."""
    sets = [{k: v.to(cuda) for k, v in make(14 + i, rows, width, BF16).items()} for i in range(2)]
    refs = [run(c, cuda) for c in sets]
    streams = [torch.cuda.Stream(cuda) for _ in sets]
    torch.cuda.synchronize()
    graphs, captured = [], []
    for c in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured.append(run(c, cuda))
        graphs.append(graph)
    eager = [[], []]
    for _ in range(5):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                eager[i].append(run(sets[i], cuda))
                graphs[i].replay()
    torch.cuda.synchronize()
    for i, ref in enumerate(refs):
        for k in ref:
            assert torch.equal(captured[i][k], ref[k]) and all(torch.equal(e[k], ref[k]) for e in eager[i]), k


def test_on_a_stream_given_by_the_caller(cuda):
    d = {k: v.to(cuda) for k, v in make(15, 200, 1001, BF16).items()}
    ref = run(d, cuda)
    side = torch.cuda.Stream(cuda)
    torch.cuda.synchronize()
    y, mean, rstd = gdn.gdn_layernorm(d["x"], d["w"], d["b"], EPS, save_stats=True, stream=side)
    dx, dw, db = gdn.gdn_layernorm_bwd(d["dy"], d["x"], mean, rstd, d["w"], stream=side)
    side.synchronize()
    for k, t in zip(("y", "mean", "rstd", "dx", "dweight", "dbias"), (y, mean, rstd, dx, dw, db)):
        assert torch.equal(t, ref[k]), k


def test_offsets_past_32_bits(cuda):
    rows, width = (1 << 32) // 8192 + 3, 8192
    x = torch.randn(rows, width, device=cuda, dtype=BF16)
    y, mean, rstd = gdn.gdn_layernorm(x, save_stats=True)
    dx, _, _ = gdn.gdn_layernorm_bwd(x, x, mean, rstd, need_dweight=False, need_dbias=False)
    torch.cuda.synchronize()
    tail = R.f64(x[-2:])
    ref = R.layernorm(tail, None, None, EPS, BF16)
    R.assert_within(y[-2:], *ref["y"], "y")
    R.assert_within(dx[-2:], *R.layernorm_bwd(tail, tail, R.f64(mean[-2:]), R.f64(rstd[-2:]), None, BF16)["dx"], "dx")
