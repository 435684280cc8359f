"""A layer of the operators together, as it is used: norm and rotation of q and k
in a projection's rows, linear attention, the output gate; its training step
against torch's differentiation of the formulas in 64 bits, and a decode that
goes on from a prompt's state."""
import pytest
import torch

import linattn_ref as R
from gated_deltanet_chunked_gb300 import gdn

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
HQ, HV, EPS, SCALE = 2, 4, 1e-6, 128 ** -0.5


def inputs(dtype, T, dev):
    gen = torch.Generator().manual_seed(4)
    normal = lambda *shape: torch.randn(shape, generator=gen)
    d = {"rows": normal(T, (2 * HQ + HV) * 128), "z": normal(T, HV, 128), "dy": normal(T, HV, 128)}
    d = {k: v.to(dtype).to(dev) for k, v in d.items()}
    d["qw"], d["kw"], d["gw"] = ((torch.rand(128, generator=gen) + 0.5).to(dev) for _ in range(3))
    d["decay"] = torch.tensor([-0.6, -0.2, -0.05, -0.01], device=dev)
    d["inv_freq"] = (1e4 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().to(dev)
    d["pos"] = torch.arange(T, dtype=torch.int32, device=dev)
    return d


def split(rows):
    return (rows[:, :HQ * 128].unflatten(1, (HQ, 128)), rows[:, HQ * 128:2 * HQ * 128].unflatten(1, (HQ, 128)),
            rows[:, 2 * HQ * 128:].unflatten(1, (HV, 128)))


def reference(d):
    """Everything in 64 bits, the attention as a masked product."""
    leaf = {k: d[k].double().requires_grad_() for k in ("rows", "z", "qw", "kw", "gw")}
    q, k, v = split(leaf["rows"])
    angle = (d["pos"].double()[:, None] * d["inv_freq"].double())[:, None]

    def turned(x, w):
        n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        a, b = n[..., :64], n[..., 64:]
        return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1)

    q, k = (turned(x, leaf[w]).repeat_interleave(HV // HQ, 1) for x, w in ((q, "qw"), (k, "kw")))
    t = torch.arange(len(v), device=v.device)
    age = (t[:, None] - t).double()
    mask = torch.where(age >= 0, (d["decay"].double()[:, None, None] * age.clamp(min=0)).exp(), 0.0)
    o = torch.einsum("hij,jhd->ihd", torch.einsum("ihd,jhd->hij", q, k) * mask * SCALE, v)
    y = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS) * leaf["gw"] * leaf["z"] * torch.sigmoid(leaf["z"])
    grads = torch.autograd.grad(y, list(leaf.values()), d["dy"].double())
    return y.detach(), dict(zip(leaf, grads))


@pytest.mark.parametrize("dtype,tol", [(F32, 1e-5), (BF16, 2e-2)], ids=["f32", "bf16"])
def test_training_step(cuda, dtype, tol):
    """Normwise. bf16: each of the five kernels rounds what it hands on (2^-8 at most, 2^-9 on average), and the
    attention twice inside: 2e-2 is above the sum of all. f32: 1024 u of the majorant, which these sums exceed by a
    factor below 3 normwise, is an upper bound of the attention's error; errors of random signs stay far below."""
    T = 333
    d = inputs(dtype, T, cuda)
    ref, grads = reference(d)
    cu = torch.tensor([0, T], dtype=torch.int32, device=cuda)
    q, k, v = split(d["rows"])
    v = v.contiguous()
    norm = (d["qw"], d["kw"], d["inv_freq"], d["pos"])
    qr, kr = gdn.gdn_qk_norm_rope(q, k, *norm, eps=EPS)
    o, _ = gdn.gdn_linear_attention(qr, kr, v, d["decay"], SCALE, cu_seqlens=cu)
    y = gdn.gdn_gated_rmsnorm(o, d["z"], d["gw"], EPS)
    do, dz, dgw = gdn.gdn_gated_rmsnorm_bwd(d["dy"], o, d["z"], d["gw"], EPS)
    dqr, dkr, dv, _ = gdn.gdn_linear_attention_bwd(do, qr, kr, v, d["decay"], SCALE, cu_seqlens=cu)
    drows = torch.empty_like(d["rows"])
    gq, gk, gv = split(drows)
    _, _, dqw, dkw = gdn.gdn_qk_norm_rope_bwd(dqr, dkr, q, k, *norm, eps=EPS, dq=gq, dk=gk)
    gv.copy_(dv)
    got = {"rows": drows, "z": dz, "qw": dqw, "kw": dkw, "gw": dgw}
    off = lambda a, b: ((a.double() - b).norm() / b.norm()).item()
    assert off(y, ref) <= tol
    for name, g in grads.items():
        assert off(got[name], g) <= tol, (name, off(got[name], g))
    assert gdn.gdn_get_device_status() == gdn.GDN_OK


def test_gradient_against_differences(cuda):
    """The directional derivative of the f32 layer's attention by central differences. With step h the quotient is off
    by the operator's own rounding, 1e-6 of the sum, over 2 h: below 1e-3 of it at h = 1e-2 (in q the output is linear,
    so that there is no other error)."""
    T = 150
    d = inputs(F32, T, cuda)
    q, k, v = (x.contiguous() for x in split(d["rows"]))
    cu = torch.tensor([0, T], dtype=torch.int32, device=cuda)
    gen = torch.Generator(device=cuda).manual_seed(5)
    f = lambda q, k, v: (gdn.gdn_linear_attention(q, k, v, d["decay"], SCALE, cu_seqlens=cu)[0].double()
                         * d["dy"].double()).sum().item()
    grads = gdn.gdn_linear_attention_bwd(d["dy"], q, k, v, d["decay"], SCALE, cu_seqlens=cu)[:3]
    for i, g in enumerate(grads):
        x = [q, k, v]
        way = torch.randn(x[i].shape, generator=gen, device=cuda)
        way = way + g / g.norm() * way.norm()  # not at right angles to the gradient
        h, ends = 1e-2, []
        for sign in (1, -1):
            x = [q, k, v]
            x[i] = x[i] + sign * h * way
            ends.append(f(*x))
        want = (g.double() * way.double()).sum().item()
        assert abs((ends[0] - ends[1]) / (2 * h) - want) <= 2e-3 * abs(want), i


@pytest.mark.parametrize("dtype,tol", [(F32, 1e-5), (BF16, 1e-2)], ids=["f32", "bf16"])
def test_decode_goes_on_from_a_prompt(cuda, dtype, tol):
    """Ten tokens one by one behind a prompt give what the whole sequence gives at once (normwise; each side's error is
    below half of tol)."""
    T, new = 210, 10
    d = inputs(dtype, T, cuda)
    q, k, v = split(d["rows"])
    qr, kr = gdn.gdn_qk_norm_rope(q, k, d["qw"], d["kw"], d["inv_freq"], d["pos"], eps=EPS)
    v = v.contiguous()
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device=cuda)
    whole, last = gdn.gdn_linear_attention(qr, kr, v, d["decay"], SCALE, cu_seqlens=cu(T))
    P = T - new
    _, state = gdn.gdn_linear_attention(qr[:P], kr[:P], v[:P], d["decay"], SCALE, cu_seqlens=cu(P))
    for t in range(P, T):
        one = slice(t, t + 1)
        q1, k1 = gdn.gdn_qk_norm_rope(q[one], k[one], d["qw"], d["kw"], d["inv_freq"], d["pos"][one], eps=EPS)
        assert torch.equal(q1, qr[one]) and torch.equal(k1, kr[one])
        o = gdn.gdn_linear_attention_step(q1, k1, v[one], d["decay"], SCALE, state)
        assert (o - whole[one]).double().norm() <= tol * whole[one].double().norm()
    assert (state - last).double().norm() <= 1e-5 * last.double().norm()
