"""gdn_linear_attention, its backward pass and its decode step against the
definition in 64 bits, with bounds that count the roundings (linattn_ref)."""
import numpy as np
import pytest
import torch

import linattn_ref as R
from gated_deltanet_chunked_gb300 import gdn

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DTYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
SCALE = 128 ** -0.5
LENS = {
    "one_token": [1],
    "below_chunk": [127],
    "chunk": [128],
    "above_chunk": [129],
    "two_chunks": [256],
    "ragged": [1, 0, 31, 32, 33, 129, 300, 7, 0, 127],
    "empty_ends": [0, 0, 5, 0],
    "one_long": [1100],
}


def make(seed, lens, hq, hv, dtype, init, decay=None):
    gen = torch.Generator().manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen)
    T, N = sum(lens), len(lens)
    d = {"q": normal(T, hq, 128).to(dtype), "k": normal(T, hq, 128).to(dtype), "v": normal(T, hv, 128).to(dtype),
         "dout": normal(T, hv, 128).to(dtype), "scale": SCALE,
         "s0": normal(N, hv, 128, 128) if init else None, "dfinal": normal(N, hv, 128, 128) if init else None}
    if decay is None:
        decay = -2.0 ** (-8.0 * (torch.arange(hv) + 1) / hv) * (0.5 + torch.rand(hv, generator=gen))
    d["decay"] = decay
    d["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    return d


def to(d, dev):
    return {k: (v.to(dev) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def run(c, cu="cu", **kw):
    cu = c[cu] if cu else None
    out, final = gdn.gdn_linear_attention(c["q"], c["k"], c["v"], c["decay"], c["scale"], initial_state=c["s0"],
                                          cu_seqlens=cu, **kw)
    dq, dk, dv, ds0 = gdn.gdn_linear_attention_bwd(c["dout"], c["q"], c["k"], c["v"], c["decay"], c["scale"],
                                                   initial_state=c["s0"], cu_seqlens=cu, dfinal_state=c["dfinal"], **kw)
    return {"out": out, "final": final, "dq": dq, "dk": dk, "dv": dv, "ds0": ds0}


def compare(res, d, lens, dtype):
    ref = R.attention(d, lens, dtype)
    for name, x in res.items():
        if x is not None:
            R.assert_within(x, *ref[name], name)


def same(a, b):
    for k in a:
        assert (a[k] is None) == (b[k] is None) and (a[k] is None or torch.equal(a[k], b[k])), k


@DTYPES
@pytest.mark.parametrize("hq,hv", [(1, 1), (1, 3), (2, 2)])
@pytest.mark.parametrize("lens", list(LENS.values()), ids=list(LENS))
@pytest.mark.parametrize("init", [False, True], ids=["zero", "init"])
def test_forward_backward(cuda, lens, dtype, hq, hv, init):
    d = make(7, lens, hq, hv, dtype, init)
    res = run(to(d, cuda))
    torch.cuda.synchronize()
    assert gdn.gdn_read_device_status() == gdn.GDN_OK
    compare(res, d, lens, dtype)


@DTYPES
@pytest.mark.parametrize("decay", [[0.0, -1e-4], [-0.7, -5.0], [-30.0, float("-inf")], [-0.34657, -1e-7]])
def test_decays(cuda, dtype, decay):
    """From a state that keeps all to one that keeps nothing."""
    lens = [700, 0, 130, 1]
    d = make(8, lens, 1, 2, dtype, True, torch.tensor(decay))
    compare(run(to(d, cuda)), d, lens, dtype)


@DTYPES
def test_many_heads(cuda, dtype):
    lens = [150, 3]
    d = make(9, lens, 11, 33, dtype, True)
    compare(run(to(d, cuda)), d, lens, dtype)


@DTYPES
@pytest.mark.parametrize("batch,seqlen", [(3, 0), (1, 1), (5, 7), (2, 128), (3, 150)])
def test_dense_batch_is_the_packed_one(cuda, dtype, batch, seqlen):
    d = to(make(11, [seqlen] * batch, 1, 2, dtype, True), cuda)
    packed = run(d)
    for k in ("q", "k", "v", "dout"):
        d[k] = d[k].reshape(batch, seqlen, *d[k].shape[1:])
    dense = run(d, cu=None)
    same(packed, {k: v.reshape(packed[k].shape) for k, v in dense.items()})


@DTYPES
def test_same_bits_whatever_the_workspace_held(cuda, dtype):
    d = to(make(12, [900, 77, 300], 2, 4, dtype, True), cuda)
    ref = run(d)
    for fill in (0, 255):
        ws = torch.full((64 << 20,), fill, dtype=torch.uint8, device=cuda)
        same(run(d, workspace=ws), ref)


@DTYPES
def test_many_tokens(cuda, dtype):
    """Segments chained over a long axis, against the recurrence token by token on the GPU in 64 bits (one head)."""
    T, hv = 9000, 3
    d = make(13, [T], 1, hv, dtype, True)
    c = to(d, cuda)
    out, final = gdn.gdn_linear_attention(c["q"], c["k"], c["v"], c["decay"], SCALE, initial_state=c["s0"],
                                          cu_seqlens=c["cu"])
    h = 2
    S = c["s0"][0, h].double()
    M = S.abs()
    keep = c["decay"][h].double().exp()
    q, k, v = c["q"][:, 0].double(), c["k"][:, 0].double(), c["v"][:, h].double()
    ref, maj = torch.empty(T, 128, dtype=torch.float64, device=cuda), torch.empty(T, 128, dtype=torch.float64, device=cuda)
    for t in range(T):
        S = keep * S + k[t][:, None] * v[t]
        M = keep * M + k[t].abs()[:, None] * v[t].abs()
        ref[t], maj[t] = q[t] @ S, q[t].abs() @ M
    ref, maj = ref.cpu().numpy() * SCALE, maj.cpu().numpy() * SCALE
    half = R.H[dtype]
    f32 = 1024 + 7 * (T // 32)  # roundings of an age of T / 32 blocks (linattn_ref)
    err = (f32 * R.u if dtype == F32 else half * (1 + half) + 4 * 2048 * R.u) * maj
    R.assert_within(out[:, h], ref, err + half * (np.abs(ref) + err), "out")
    R.assert_within(final[0, h], S.cpu().numpy(), max(f32, 4 * 2048) * R.u * M.cpu().numpy(), "final")


@DTYPES
def test_two_calls_in_turn_are_one(cuda, dtype):
    """A sequence cut in two, the state passed on, then a decode step."""
    d = make(14, [400], 2, 4, dtype, True)
    c = to(d, cuda)
    ref = R.attention(d, [400], dtype)
    args = lambda a, b: (c["q"][a:b].contiguous(), c["k"][a:b].contiguous(), c["v"][a:b].contiguous(), c["decay"], SCALE)
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device=cuda)
    o1, s1 = gdn.gdn_linear_attention(*args(0, 157), initial_state=c["s0"], cu_seqlens=cu(157))
    o2, s2 = gdn.gdn_linear_attention(*args(157, 399), initial_state=s1, cu_seqlens=cu(242))
    o3 = gdn.gdn_linear_attention_step(*args(399, 400), s2)
    R.assert_within(torch.cat([o1, o2, o3]), *ref["out"], "out")
    R.assert_within(s2, *ref["final"], "final")


@DTYPES
@pytest.mark.parametrize("bad", [[1, 100, 200], [0, 150, 100], [0, 100, 199], [0, 100, 201], [0, -5, 200], [0, 300, 200]])
def test_bad_offsets_write_nothing(cuda, dtype, bad):
    d = to(make(15, [100, 100], 1, 2, dtype, True), cuda)
    d["cu"] = torch.tensor(bad, dtype=torch.int32, device=cuda)
    out, fin = torch.full_like(d["v"], 3.0), torch.full_like(d["s0"], 3.0)
    gdn.gdn_linear_attention(d["q"], d["k"], d["v"], d["decay"], SCALE, cu_seqlens=d["cu"], out=out, final_state=fin)
    assert gdn.gdn_get_device_status() == gdn.GDN_EDEVICE_INPUT
    assert (out == 3).all() and (fin == 3).all()
    grads = [torch.full_like(d[k], 3.0) for k in ("q", "k", "v")]
    gdn.gdn_linear_attention_bwd(d["dout"], d["q"], d["k"], d["v"], d["decay"], SCALE, cu_seqlens=d["cu"], dq=grads[0],
                                 dk=grads[1], dv=grads[2])
    assert gdn.gdn_get_device_status() == gdn.GDN_EDEVICE_INPUT
    assert all((x == 3).all() for x in grads)


@DTYPES
@pytest.mark.parametrize("hq,hv", [(2, 2), (1, 2), (2, 6)])
@pytest.mark.parametrize("bad", [[0, 150, 100], [0, 100, 199]])
def test_bad_offsets_leave_gradients(cuda, dtype, hq, hv, bad):
    """With and without sums over a group's heads, whatever the workspace holds."""
    d = to(make(23, [100, 100], hq, hv, dtype, True), cuda)
    d["cu"] = torch.tensor(bad, dtype=torch.int32, device=cuda)
    grads = [torch.full_like(d[k], 3.0) for k in ("q", "k", "v", "s0")]
    workspace = torch.zeros(1 << 24, dtype=torch.uint8, device=cuda)
    gdn.gdn_linear_attention_bwd(d["dout"], d["q"], d["k"], d["v"], d["decay"], SCALE, initial_state=d["s0"],
                                 cu_seqlens=d["cu"], dfinal_state=d["dfinal"], dq=grads[0], dk=grads[1], dv=grads[2],
                                 dinitial_state=grads[3], workspace=workspace)
    assert gdn.gdn_get_device_status() == gdn.GDN_EDEVICE_INPUT
    for name, x in zip(("dq", "dk", "dv", "dinitial_state"), grads):
        assert (x == 3).all(), name


@DTYPES
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_infinities_stay_in_their_sequence_and_head(cuda, dtype, value):
    lens, hv = [100, 200, 60], 2
    d = make(16, lens, 2, hv, dtype, True)
    clean = run(to(d, cuda))
    for name in ("q", "k", "v", "dout"):
        c = to({**d, name: d[name].clone()}, cuda)
        c[name][100:300, 0] = value  # the second sequence, head 0
        res = run(c)
        for k in ("out", "dq", "dk", "dv"):
            assert torch.equal(res[k][:, 1], clean[k][:, 1]), (name, k)
            assert torch.equal(res[k][:100], clean[k][:100]) and torch.equal(res[k][300:], clean[k][300:]), (name, k)
        for k in ("final", "ds0"):
            assert torch.equal(res[k][:, 1], clean[k][:, 1]), (name, k)
            assert torch.equal(res[k][0], clean[k][0]) and torch.equal(res[k][2], clean[k][2]), (name, k)


@DTYPES
def test_outputs_16_bytes_off_a_sector(cuda, dtype):
    lens = [300, 9]
    d = to(make(17, lens, 1, 2, dtype, False), cuda)
    ref = run(d)
    step = 16 // d["v"].element_size()
    shifted = lambda x: torch.full((x.numel() + 2 * step,), 5.0, dtype=dtype, device=cuda)
    raw = shifted(d["v"])
    out = raw[step:-step].view(d["v"].shape)
    gdn.gdn_linear_attention(d["q"], d["k"], d["v"], d["decay"], SCALE, cu_seqlens=d["cu"], out=out)
    assert torch.equal(out, ref["out"]) and (raw[:step] == 5).all() and (raw[-step:] == 5).all()
    raws = [shifted(d[k]) for k in ("q", "k", "v")]
    dq, dk, dv = (r[step:-step].view(d[k].shape) for r, k in zip(raws, ("q", "k", "v")))
    gdn.gdn_linear_attention_bwd(d["dout"], d["q"], d["k"], d["v"], d["decay"], SCALE, cu_seqlens=d["cu"], dq=dq, dk=dk,
                                 dv=dv)
    for r, g, k in zip(raws, (dq, dk, dv), ("dq", "dk", "dv")):
        assert torch.equal(g, ref[k]) and (r[:step] == 5).all() and (r[-step:] == 5).all(), k


@DTYPES
def test_streams_and_graphs(cuda, dtype):
    """Two calls at once, on streams of their own, and two captured graphs replayed one after the other."""
    sets = [to(make(18 + i, [500, 40 * i, 300], 2, 4, dtype, True), cuda) for i in range(2)]
    ref = [run(s) for s in sets]
    streams = [torch.cuda.Stream(cuda) for _ in sets]
    torch.cuda.synchronize()
    got = []
    for s, st in zip(sets, streams):
        out, fin = gdn.gdn_linear_attention(s["q"], s["k"], s["v"], s["decay"], SCALE, initial_state=s["s0"],
                                            cu_seqlens=s["cu"], stream=st)
        got.append((out, fin))
    torch.cuda.synchronize()
    for (out, fin), r in zip(got, ref):
        assert torch.equal(out, r["out"]) and torch.equal(fin, r["final"])
    graphs, held = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(run(s))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for h, r in zip(held, ref):
        same(h, r)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK


def test_elements_beyond_32_bits(cuda):
    """The last sequence of a batch whose tensors have more than 2^31 elements."""
    hv, lens = 160, [105000, 300]
    T = sum(lens)
    assert T * hv * 128 > 1 << 31
    gen = torch.Generator(device=cuda).manual_seed(3)
    c = {k: torch.randn(T, hv, 128, generator=gen, device=cuda, dtype=BF16) for k in ("q", "k", "v")}
    decay = torch.linspace(-0.5, -0.01, hv, device=cuda)
    cu = torch.tensor([0, lens[0], T], dtype=torch.int32, device=cuda)
    out, final = gdn.gdn_linear_attention(c["q"], c["k"], c["v"], decay, SCALE, cu_seqlens=cu)
    heads = [0, hv - 1]
    part = lambda x: x[lens[0]:, heads].cpu()
    d = {"q": part(c["q"]), "k": part(c["k"]), "v": part(c["v"]), "dout": part(c["v"]), "decay": decay[heads].cpu(),
         "scale": SCALE, "s0": None, "dfinal": None}
    ref = R.attention(d, [300], BF16)
    R.assert_within(out[lens[0]:, heads], *ref["out"], "out")
    R.assert_within(final[1:, heads], *ref["final"], "final")


# ---- decode step ----


@DTYPES
@pytest.mark.parametrize("state_dtype", [F32, BF16], ids=["state_f32", "state_bf16"])
@pytest.mark.parametrize("n,hq,hv", [(1, 1, 1), (5, 2, 6), (70, 3, 3)])
def test_step(cuda, dtype, state_dtype, n, hq, hv):
    gen = torch.Generator().manual_seed(n)
    normal = lambda *shape: torch.randn(shape, generator=gen)
    slots = n + 4
    d = {"q": normal(n, hq, 128).to(dtype), "k": normal(n, hq, 128).to(dtype), "v": normal(n, hv, 128).to(dtype),
         "decay": -torch.rand(hv, generator=gen), "scale": SCALE}
    cache = normal(slots, hv, 128, 128).to(state_dtype)
    idx = torch.randperm(slots, generator=gen)[:n].to(torch.int32)
    d["state"] = cache[idx.long()]
    (out, bo), (new, bs) = R.step(d, dtype, state_dtype)
    c, got = to(d, cuda), cache.to(cuda)
    y = gdn.gdn_linear_attention_step(c["q"], c["k"], c["v"], c["decay"], SCALE, got, state_indices=idx.to(cuda))
    R.assert_within(y, out, bo, "out")
    R.assert_within(got[idx.long().to(cuda)], new, bs, "state")
    rest = torch.ones(slots, dtype=torch.bool)
    rest[idx.long()] = False
    assert torch.equal(got.cpu()[rest], cache[rest])  # the other slots


def test_step_padding_and_bad_slots(cuda):
    d = to(make(21, [4], 1, 2, BF16, False), cuda)
    state = torch.randn(3, 2, 128, 128, device=cuda)
    before, out = state.clone(), torch.full_like(d["v"], 7.0)
    idx = torch.tensor([2, -1, 3, 0], dtype=torch.int32, device=cuda)
    gdn.gdn_linear_attention_step(d["q"], d["k"], d["v"], d["decay"], SCALE, state, state_indices=idx, out=out)
    assert gdn.gdn_get_device_status() == gdn.GDN_EDEVICE_INPUT
    assert (out[1] == 7).all() and (out[2] == 7).all() and (out[0] != 7).any() and (out[3] != 7).any()
    assert torch.equal(state[1], before[1]) and not torch.equal(state[0], before[0])


def test_steps_in_a_graph_advance_the_state(cuda):
    d = to(make(22, [6], 2, 4, F32, False), cuda)
    state = torch.randn(6, 4, 128, 128, device=cuda)
    ref, outs = state.clone(), []
    for _ in range(3):
        outs.append(gdn.gdn_linear_attention_step(d["q"], d["k"], d["v"], d["decay"], SCALE, ref))
    g, got = torch.cuda.CUDAGraph(), state.clone()
    with torch.cuda.graph(g):
        out = gdn.gdn_linear_attention_step(d["q"], d["k"], d["v"], d["decay"], SCALE, got)
    for i in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, outs[i])
    assert torch.equal(got, ref)
