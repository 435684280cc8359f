"""gdn_qk_norm_rope and its backward pass against the definition in 64 bits,
with bounds that count the roundings (linattn_ref)."""
import pytest
import torch

import linattn_ref as R
from gated_deltanet_chunked_gb300 import gdn

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DTYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
EPS = 1e-6


def make(seed, T, hq, hk, dtype, rotary, axes=1, weights=True, packed=False, far=1 << 20):
    gen = torch.Generator().manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen)
    half = rotary // 2
    d = {"dq": normal(T, hq, 128).to(dtype), "dk": normal(T, hk, 128).to(dtype)}
    d["rows"] = normal(T, (hq + hk) * 128 + 128).to(dtype)
    if not packed:
        d["q"], d["k"] = d["rows"][:, :hq * 128].reshape(T, hq, 128), d["rows"][:, hq * 128:-128].reshape(T, hk, 128)
    d["qw"] = torch.rand(128, generator=gen) + 0.5 if weights else None
    d["kw"] = normal(128) if weights else None
    d["inv_freq"] = (1e6 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float()
    d["pos"] = torch.randint(0, far, (axes, T) if axes > 1 else (T,), generator=gen, dtype=torch.int64).to(torch.int32)
    d["axis"] = torch.randint(0, axes, (half,), generator=gen).to(torch.int32) if axes > 1 else None
    return d


def to(d, dev, hq):
    c = {k: (v.to(dev) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    if "q" not in c:
        c["q"], c["k"] = (x.unflatten(1, (-1, 128)) for x in (c["rows"][:, :hq * 128], c["rows"][:, hq * 128:-128]))
    return c


def args(c):
    return c["q"], c["k"], c["qw"], c["kw"], c["inv_freq"], c["pos"]


def run(c, interleaved, **kw):
    y = gdn.gdn_qk_norm_rope(*args(c), pair_axis=c["axis"], interleaved=interleaved, eps=EPS)
    g = gdn.gdn_qk_norm_rope_bwd(c["dq"], c["dk"], *args(c), pair_axis=c["axis"], interleaved=interleaved, eps=EPS, **kw)
    return dict(zip(("q", "k", "dq", "dk", "dqw", "dkw"), (*y, *g)))


def compare(res, c, interleaved, dtype):
    for n in ("q", "k"):
        ref = R.rope(c[n], c[n + "w"], c["d" + n], c["inv_freq"], c["pos"], c["axis"], interleaved, EPS, dtype)
        R.assert_within(res[n], *ref["y"], n)
        R.assert_within(res["d" + n], *ref["dx"], "d" + n)
        R.assert_within(res["d" + n + "w"], *ref["dw"], "d" + n + " weight")


@DTYPES
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("rotary", [0, 2, 8, 16, 30, 32, 64, 74, 126, 128])
def test_rotations(cuda, dtype, interleaved, rotary):
    c = to(make(rotary, 21, 3, 2, dtype, rotary), cuda, 3)
    compare(run(c, interleaved), c, interleaved, dtype)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK


@DTYPES
@pytest.mark.parametrize("T,hq,hk", [(1, 1, 1), (1, 40, 3), (700, 1, 1), (333, 16, 16), (5000, 5, 2), (3, 200, 100)])
@pytest.mark.parametrize("packed", [False, True], ids=["apart", "packed"])
def test_shapes(cuda, dtype, T, hq, hk, packed):
    c = to(make(T + hq, T, hq, hk, dtype, 128, packed=packed), cuda, hq)
    compare(run(c, False), c, False, dtype)


@DTYPES
@pytest.mark.parametrize("axes", [2, 3, 8])
def test_axes(cuda, dtype, axes):
    c = to(make(axes, 130, 4, 1, dtype, 64, axes=axes, packed=True), cuda, 4)
    compare(run(c, False), c, False, dtype)


@DTYPES
def test_far_and_negative_positions(cuda, dtype):
    c = to(make(5, 64, 2, 2, dtype, 128, far=(1 << 31) - 1), cuda, 2)
    c["pos"][::2] *= -1
    c["pos"][0], c["pos"][1], c["pos"][2] = -(1 << 31), (1 << 31) - 1, 0
    compare(run(c, False), c, False, dtype)


@DTYPES
def test_no_weights_and_no_tokens(cuda, dtype):
    c = to(make(6, 50, 2, 3, dtype, 128, weights=False), cuda, 2)
    compare(run(c, True), c, True, dtype)
    e = to(make(6, 0, 2, 3, dtype, 128), cuda, 2)
    res = run(e, False)
    assert res["q"].shape == (0, 2, 128) and (res["dqw"] == 0).all() and (res["dkw"] == 0).all()


@DTYPES
@pytest.mark.parametrize("rotary", [128, 30])
def test_in_place(cuda, dtype, rotary):
    """Over q and k in a projection's rows (v's channels stay), and gradients over the outputs' gradients."""
    d = make(7, 100, 4, 2, dtype, rotary, packed=True)
    ref = run(to(d, cuda, 4), False)
    c = to(d, cuda, 4)
    c["rows"] = c["rows"].clone()
    c["q"], c["k"] = (x.unflatten(1, (-1, 128)) for x in (c["rows"][:, :512], c["rows"][:, 512:-128]))
    g = gdn.gdn_qk_norm_rope_bwd(c["dq"], c["dk"], *args(c), eps=EPS, dq=c["dq"], dk=c["dk"])
    assert g[0] is c["dq"] and torch.equal(g[0], ref["dq"]) and torch.equal(g[1], ref["dk"])
    gdn.gdn_qk_norm_rope(*args(c), eps=EPS, out_q=c["q"], out_k=c["k"])
    assert torch.equal(c["q"], ref["q"]) and torch.equal(c["k"], ref["k"])
    assert torch.equal(c["rows"][:, -128:].cpu(), d["rows"][:, -128:])


def test_same_bits_and_streams(cuda):
    c = to(make(8, 3000, 8, 8, BF16, 128), cuda, 8)
    ref = run(c, False)
    st = torch.cuda.Stream(cuda)
    torch.cuda.synchronize()
    res = run(c, False, stream=st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = run(c, False)
    g.replay()
    torch.cuda.synchronize()
    for k in ref:
        assert torch.equal(ref[k], res[k]) and torch.equal(ref[k], held[k]), k


def test_bad_axis_writes_nothing(cuda):
    c = to(make(9, 70, 2, 2, BF16, 128, axes=3), cuda, 2)
    for bad in (-1, 3):
        axis = c["axis"].clone()
        axis[40] = bad
        out = [torch.full_like(c[k], 2.0) for k in ("q", "k")]
        gdn.gdn_qk_norm_rope(*args(c), pair_axis=axis, out_q=out[0], out_k=out[1])
        assert gdn.gdn_get_device_status() == gdn.GDN_EDEVICE_INPUT
        assert all((x == 2).all() for x in out)


def test_bad_axis_backward(cuda):
    """dq and dk stay as they were, and the weights' gradients are zeros whatever the workspace holds."""
    c = to(make(9, 70, 2, 2, BF16, 128, axes=3), cuda, 2)
    axis = c["axis"].clone()
    axis[40] = 3
    out = [torch.full_like(c[k], 2.0) for k in ("dq", "dk")]
    ws = torch.full((1 << 20,), 63, dtype=torch.uint8, device=cuda)
    g = gdn.gdn_qk_norm_rope_bwd(c["dq"], c["dk"], *args(c), pair_axis=axis, dq=out[0], dk=out[1], workspace=ws)
    assert gdn.gdn_get_device_status() == gdn.GDN_EDEVICE_INPUT
    assert all((x == 2).all() for x in out) and (g[2] == 0).all() and (g[3] == 0).all()


def test_one_weight_gradient(cuda):
    """Either weight's gradient without the other is the one of both."""
    c = to(make(11, 300, 3, 2, BF16, 128), cuda, 2)
    both = gdn.gdn_qk_norm_rope_bwd(c["dq"], c["dk"], *args(c), eps=EPS)
    for i, name in ((2, "dq_weight"), (3, "dk_weight")):
        w = torch.full((128,), 5.0, device=cuda)
        g = gdn.gdn_qk_norm_rope_bwd(c["dq"], c["dk"], *args(c), eps=EPS, need_dweight=False, **{name: w})
        assert torch.equal(w, both[i]) and torch.equal(g[0], both[0]) and torch.equal(g[1], both[1])
        assert g[5 - i] is None
    g = gdn.gdn_qk_norm_rope_bwd(c["dq"], c["dk"], *args(c), eps=EPS, need_dweight=False)
    assert torch.equal(g[0], both[0]) and torch.equal(g[1], both[1]) and g[2] is None and g[3] is None


def test_infinities_stay_in_their_row(cuda):
    c = to(make(10, 40, 3, 2, BF16, 128), cuda, 3)
    ref = run(c, False)
    c["q"] = c["q"].clone()
    c["q"][7, 1] = float("nan")
    c["q"][8, 2, 5] = float("inf")
    res = run(c, False)
    keep = torch.ones(40, 3, dtype=torch.bool, device=cuda)
    keep[7, 1] = keep[8, 2] = False
    for k in ("q", "dq"):
        assert torch.equal(res[k][keep], ref[k][keep])
    assert torch.equal(res["k"], ref["k"]) and torch.equal(res["dk"], ref["dk"]) and torch.equal(res["dkw"], ref["dkw"])
