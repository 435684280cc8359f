"""gdn_linear_recurrence, its backward pass and its decode step against the
definition in 64 bits, with bounds that count the roundings (train_ref)."""
import numpy as np
import pytest
import torch

import train_ref as R
from gated_deltanet_chunked_gb300 import gdn

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DTYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
GATES = pytest.mark.parametrize("gate", ["head", "channel"])

LENS = {
    "one_token": [1],
    "below_tile": [63],
    "tile": [64],
    "above_tile": [65],
    "ragged": [1, 0, 63, 64, 65, 513, 1000, 7, 0, 129],
    "empty_ends": [0, 0, 5, 0],
    "nothing": [0, 0],
    "one_long": [2500],
    "tokens": [1] * 70,
    "empties_between_tokens": [1] + [0] * 40 + [2] + [0] * 40 + [600] + [0] * 40,
}


def make(seed, lens, hv, dtype, gate, init, mu=-1.0):
    gen = torch.Generator().manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen)
    T, N = sum(lens), len(lens)
    d = {"x": normal(T, hv, 128).to(dtype), "dout": normal(T, hv, 128).to(dtype),
         "h0": normal(N, hv, 128) if init else None, "dfinal": normal(N, hv, 128) if init else None}
    raw = normal(*((T, hv) if gate == "head" else (T, hv, 128))) + mu
    d["g"] = -torch.nn.functional.softplus(raw).to(F32 if gate == "head" else dtype)
    d["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    return d


def to(d, dev):
    return {k: (v.to(dev) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def run(c, cu="cu"):
    cu = c[cu] if cu else None
    out, final, states = gdn.gdn_linear_recurrence(c["x"], c["g"], initial_state=c["h0"], cu_seqlens=cu,
                                                   save_states=True)
    dx, dg, dh0 = gdn.gdn_linear_recurrence_bwd(c["dout"], c["x"], c["g"], states, initial_state=c["h0"],
                                                cu_seqlens=cu, dfinal_state=c["dfinal"])
    return {"out": out, "final": final, "dx": dx, "dg": dg, "dh0": dh0}


def compare(res, d, lens, dtype):
    ref = R.recurrence(R.f64(d["x"]), R.f64(d["g"]), R.f64(d["h0"]), lens, R.f64(d["dout"]), R.f64(d["dfinal"]), dtype)
    for name, x in res.items():
        if x is not None:
            R.assert_within(x, *ref[name], name)


@DTYPES
@GATES
@pytest.mark.parametrize("lens", list(LENS.values()), ids=list(LENS))
@pytest.mark.parametrize("init", [False, True], ids=["zero", "init"])
def test_forward_backward(cuda, lens, dtype, gate, init):
    d = make(7, lens, 3, dtype, gate, init)
    res = run(to(d, cuda))
    torch.cuda.synchronize()
    assert gdn.gdn_read_device_status() == gdn.GDN_OK
    compare(res, d, lens, dtype)


@GATES
@pytest.mark.parametrize("hv", [1, 2, 8, 33])
def test_head_counts(cuda, hv, gate):
    lens = [700, 1, 1500]
    d = make(hv, lens, hv, BF16, gate, True)
    compare(run(to(d, cuda)), d, lens, BF16)


@DTYPES
@GATES
def test_dense_batch_is_the_packed_one(cuda, dtype, gate):
    d = to(make(11, [150] * 3, 2, dtype, gate, True), cuda)
    packed = run(d)
    for k in ("x", "dout", "g"):
        d[k] = d[k].reshape(3, 150, *d[k].shape[1:])
    dense = run(d, cu=None)
    for k, v in packed.items():
        assert torch.equal(v, dense[k].reshape(v.shape)), k


@pytest.mark.parametrize("batch,seqlen", [(3, 0), (1, 1), (5, 7), (2, 128), (1, 3000), (40, 3)])
def test_dense_batches(cuda, batch, seqlen):
    lens = [seqlen] * batch
    d = make(12, lens, 2, BF16, "channel", True)
    c = to(d, cuda)
    for k in ("x", "dout", "g"):
        c[k] = c[k].reshape(batch, seqlen, 2, 128)
    res = run(c, cu=None)
    compare({k: v.reshape(sum(lens), 2, 128) if k in ("out", "dx", "dg") else v for k, v in res.items()}, d, lens, BF16)


@GATES
@pytest.mark.parametrize("hv", [1, 160])
@pytest.mark.parametrize("lens", [[5120, 1, 127, 128, 3000, 0, 64, 64, 4000, 2], [128] * 30 + [0, 0] + [64] * 9,
                                  [1] * 700 + [1500] + [1] * 70, [4096, 4096]], ids=["long", "tiles", "ones", "two"])
def test_boundaries_that_rounds_skip_and_meet(cuda, lens, hv, gate):
    """Sequences longer than a round, ending at tiles' ends, and more than 32 in a tile, with clusters of one CTA and
    of many."""
    if hv > 1:  # more clusters than fit at once with more than one CTA each
        lens = [min(v, 300) for v in lens[:5] + lens[-5:]]
    d = make(60, lens, hv, BF16, gate, True)
    compare(run(to(d, cuda)), d, lens, BF16)


@DTYPES
@GATES
@pytest.mark.parametrize("mu", [-8.0, 4.0], ids=["slow_decay", "fast_decay"])
def test_decays(cuda, dtype, gate, mu):
    lens = [900, 1100]
    d = make(13, lens, 2, dtype, gate, True, mu=mu)
    d["g"][5:9] = 0.0  # nothing forgotten
    d["g"][70:75] = -200.0  # exp underflows
    d["g"][76, :1] = -float("inf")  # the state is dropped
    d["g"][950] = -float("inf")
    compare(run(to(d, cuda)), d, lens, dtype)


@DTYPES
@GATES
def test_no_gradient_of_the_final_state_given(cuda, dtype, gate):
    lens = [300, 0, 77]
    d = make(17, lens, 2, dtype, gate, True)
    d["dfinal"] = None
    compare(run(to(d, cuda)), d, lens, dtype)


@GATES
def test_sequences_do_not_touch_each_other(cuda, gate):
    """Infinities and NaN of one sequence stay in it, forward and backward."""
    lens = [100, 30, 64, 10, 500]
    d = make(19, lens, 2, BF16, gate, True)
    clean = run(to(d, cuda))
    bad = {k: (v.clone() if v is not None else None) for k, v in d.items()}
    for seq, value in ((1, float("nan")), (3, float("inf"))):
        a, b = sum(lens[:seq]), sum(lens[:seq + 1])
        bad["x"][a + 2:b] = value
        bad["dout"][a:b - 2] = value
        bad["h0"][seq] = value
        bad["dfinal"][seq] = value
    res = run(to(bad, cuda))
    for seq in (0, 2, 4):
        a, b = sum(lens[:seq]), sum(lens[:seq + 1])
        for k in ("out", "dx", "dg"):
            assert torch.equal(res[k][a:b], clean[k][a:b]), (k, seq)
        for k in ("final", "dh0"):
            assert torch.equal(res[k][seq], clean[k][seq]), (k, seq)
    assert torch.isnan(res["out"][sum(lens[:2]) - 1]).all()


@DTYPES
def test_continuing_a_sequence_from_its_final_state(cuda, dtype):
    d = to(make(23, [1000], 2, dtype, "channel", False), cuda)
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device=cuda)
    whole, final = gdn.gdn_linear_recurrence(d["x"], d["g"], cu_seqlens=cu(1000))
    a, mid = gdn.gdn_linear_recurrence(d["x"][:333], d["g"][:333], cu_seqlens=cu(333))
    b, last = gdn.gdn_linear_recurrence(d["x"][333:].contiguous(), d["g"][333:].contiguous(), initial_state=mid,
                                        cu_seqlens=cu(667))
    h = d["x"].cpu()
    ref = R.recurrence(R.f64(h), R.f64(d["g"]), None, [1000], dtype=dtype)
    R.assert_within(torch.cat([a, b]), *ref["out"], "in two calls")
    R.assert_within(whole, *ref["out"], "in one call")
    R.assert_within(last, *ref["final"], "final state of the second call")


@DTYPES
@GATES
def test_step(cuda, dtype, gate):
    N, hv, slots = 37, 3, 50
    d = make(29, [1] * N, hv, dtype, gate, False)
    gen = torch.Generator().manual_seed(1)
    state = torch.randn(slots, hv, 128, generator=gen)
    idx = torch.randperm(slots, generator=gen)[:N].to(torch.int32)
    idx[4], idx[36] = -1, -7
    st = state.to(cuda)
    out = torch.full((N, hv, 128), 3.0, dtype=dtype, device=cuda)
    gdn.gdn_linear_recurrence_step(d["x"].to(cuda), d["g"].to(cuda), st, state_indices=idx.to(cuda), out=out)
    torch.cuda.synchronize()
    assert gdn.gdn_read_device_status() == gdn.GDN_OK
    live = (idx >= 0).nonzero()[:, 0]
    li = idx[live].long()
    ref = R.recurrence(R.f64(d["x"][live]), R.f64(d["g"][live]), R.f64(state[li]), [1] * len(live), dtype=dtype)
    R.assert_within(out[live.to(cuda)], *ref["out"], "out")
    R.assert_within(st[li.to(cuda)], *ref["final"], "state")
    assert (out[4] == 3).all() and (out[36] == 3).all()
    rest = torch.ones(slots, dtype=torch.bool)
    rest[li] = False
    assert torch.equal(st.cpu()[rest], state[rest])


def test_step_by_step_is_the_sequence(cuda):
    d = to(make(31, [1] * 40, 2, F32, "channel", False), cuda)
    state = torch.zeros(1, 2, 128, device=cuda)
    outs = [gdn.gdn_linear_recurrence_step(d["x"][t:t + 1], d["g"][t:t + 1], state) for t in range(40)]
    ref = R.recurrence(R.f64(d["x"]), R.f64(d["g"]), None, [40], dtype=F32)
    R.assert_within(torch.cat(outs), *ref["out"], "out")
    R.assert_within(state, *ref["final"], "state")


def test_step_index_out_of_range_is_recorded(cuda):
    d = to(make(37, [1] * 3, 2, F32, "head", False), cuda)
    state = torch.ones(4, 2, 128, device=cuda)
    out = torch.full((3, 2, 128), 5.0, device=cuda)
    idx = torch.tensor([0, 4, 2], dtype=torch.int32, device=cuda)
    gdn.gdn_linear_recurrence_step(d["x"], d["g"], state, state_indices=idx, out=out)
    assert gdn.gdn_get_device_status() == gdn.GDN_EDEVICE_INPUT
    assert (out[1] == 5).all() and (state[1] == 1).all() and (state[3] == 1).all()


@pytest.mark.parametrize("cu", [[1, 10, 30], [0, 20, 10, 30], [0, 10, 29], [0, 40, 30], [0, -5, 30]])
def test_bad_offsets_are_recorded_and_nothing_is_written(cuda, cu):
    d = to(make(41, [30], 2, BF16, "channel", False), cuda)
    bad = torch.tensor(cu, dtype=torch.int32, device=cuda)
    n = len(cu) - 1
    out = torch.full((30, 2, 128), 2.0, dtype=BF16, device=cuda)
    final = torch.full((n, 2, 128), 2.0, device=cuda)
    states = torch.full((1, 2, 128), 2.0, device=cuda)
    gdn.gdn_linear_recurrence(d["x"], d["g"], cu_seqlens=bad, out=out, final_state=final, states=states)
    assert gdn.gdn_get_device_status() == gdn.GDN_EDEVICE_INPUT
    dx, dg = torch.full_like(out, 2.0), torch.full_like(out, 2.0)
    dh0 = torch.full((n, 2, 128), 2.0, device=cuda)
    gdn.gdn_linear_recurrence_bwd(d["dout"], d["x"], d["g"], states, cu_seqlens=bad, dx=dx, dg=dg, dinitial_state=dh0)
    assert gdn.gdn_get_device_status() == gdn.GDN_EDEVICE_INPUT
    for t in (out, final, states, dx, dg, dh0):
        assert (t == 2).all()
    assert gdn.gdn_get_device_status() == gdn.GDN_OK


@GATES
def test_same_bits_every_time_and_in_a_graph(cuda, gate):
    lens = [700, 0, 3, 1800]
    d = to(make(43, lens, 4, BF16, gate, True), cuda)
    first = run(d)
    again = run(d)
    for k in first:
        assert torch.equal(first[k], again[k]), k
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(d)
    torch.cuda.current_stream().wait_stream(side)
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run(d)
    with torch.cuda.graph(graph2):
        captured2 = run(d)
    d["x"].mul_(0.5)
    d["dout"].mul_(0.25)
    fresh = run(d)
    graph.replay()
    graph2.replay()
    graph.replay()
    torch.cuda.synchronize()
    for k in fresh:
        assert torch.equal(captured[k], fresh[k]) and torch.equal(captured2[k], fresh[k]), k


def test_two_calls_at_once(cuda):
    """Two streams, no state in common: each gives what it gives alone."""
    sets = [to(make(50 + i, lens, 4, BF16, gate, True), cuda)
            for i, (lens, gate) in enumerate([([3000], "channel"), ([900, 0, 1200], "head")])]
    alone = [run(d) for d in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for d, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(run(d))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            for k in a:
                assert torch.equal(a[k], b[k]), k
    assert gdn.gdn_read_device_status() == gdn.GDN_OK


def test_nan_gate_stays_in_its_channel(cuda):
    lens = [200, 100]
    d = make(53, lens, 2, BF16, "channel", True)
    clean = run(to(d, cuda))
    d["g"][50, 1, 7] = float("nan")
    res = run(to(d, cuda))
    keep = torch.ones(2, 128, dtype=torch.bool, device=cuda)
    keep[1, 7] = False
    for k in ("out", "dx", "dg"):
        assert torch.equal(res[k][:, keep], clean[k][:, keep]), k
        assert torch.equal(res[k][200:], clean[k][200:]), k
    assert torch.isnan(res["out"][50:200, 1, 7]).all()


def test_on_a_stream_given_by_the_caller(cuda):
    lens = [400, 90]
    d = to(make(47, lens, 2, BF16, "channel", True), cuda)
    ref = run(d)
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        out, final, states = gdn.gdn_linear_recurrence(d["x"], d["g"], initial_state=d["h0"], cu_seqlens=d["cu"],
                                                       save_states=True, stream=stream)
        res = gdn.gdn_linear_recurrence_bwd(d["dout"], d["x"], d["g"], states, initial_state=d["h0"],
                                            cu_seqlens=d["cu"], dfinal_state=d["dfinal"], stream=handle)
        torch.cuda.synchronize()
        for got, k in zip((out, final, *res), ("out", "final", "dx", "dg", "dh0")):
            assert torch.equal(got, ref[k]), k


def test_offsets_past_32_bits(cuda):
    """More than 2^32 elements: the last sequence, whose rows lie past that, against the definition."""
    hv, tail = 32, 300
    T = (1 << 32) // (hv * 128) + 1000
    gen = torch.Generator(device=cuda).manual_seed(3)
    x = torch.randn(T, hv, 128, generator=gen, device=cuda, dtype=BF16)
    g = -torch.rand(T, hv, generator=gen, device=cuda)
    cu = torch.tensor([0, T - tail, T], dtype=torch.int32, device=cuda)
    out, final, states = gdn.gdn_linear_recurrence(x, g, cu_seqlens=cu, save_states=True)
    dx, dg, _ = gdn.gdn_linear_recurrence_bwd(x, x, g, states, cu_seqlens=cu)
    torch.cuda.synchronize()
    sel = [0, 31]
    xt, gt = R.f64(x[-tail:, sel]), R.f64(g[-tail:, sel])
    ref = R.recurrence(xt, gt, None, [tail], xt, None, BF16)
    R.assert_within(out[-tail:, sel], *ref["out"], "out")
    R.assert_within(dx[-tail:, sel], *ref["dx"], "dx")
    R.assert_within(dg[-tail:, sel], *ref["dg"], "dg")
    R.assert_within(final[1:, sel], *ref["final"], "final")
