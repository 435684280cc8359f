"""A run of the training operators as a recurrent block uses them: layer norm,
gates from raw projections, the gated linear recurrence over packed sequences,
the output gate, and the way back; and prefill followed by decode steps.

The block's gradients are compared with autograd through the same block in 64
bits, in the f32 form; there each operator is within a few f32 roundings and
the chain's 7 operators pass them on with factors of order one, so a relative
2-norm of 1e-5 (about 80 roundings' half steps) bounds it with room. In bf16
every stage's output is rounded (2^-8 at most, 2^-9.6 in the mean square), and
8 such roundings meet in a gradient at most: 8 x 2^-8 / sqrt(3) = 1.8e-2."""
import pytest
import torch

from gated_deltanet_chunked_gb300 import gdn

pytestmark = pytest.mark.gpu

EPS_LN, EPS_GATE = 1e-5, 1e-6


def block(p, gdn):
    """Forward and backward pass through the library's operators."""
    T, hv = p["x"].shape[0], p["a"].shape[1]
    y, mean, rstd = gdn.gdn_layernorm(p["x"], p["ln_w"], p["ln_b"], EPS_LN, save_stats=True)
    g, _ = gdn.gdn_gating(p["a"], p["a"], p["A_log"], p["dt_bias"])
    o, final, states = gdn.gdn_linear_recurrence(y.view(T, hv, 128), g, initial_state=p["h0"], cu_seqlens=p["cu"],
                                                 save_states=True)
    out = gdn.gdn_gated_rmsnorm(o, p["z"], p["gate_w"], EPS_GATE)
    do, dz, dgw = gdn.gdn_gated_rmsnorm_bwd(p["dout"], o, p["z"], p["gate_w"], EPS_GATE)
    dy, dg, dh0 = gdn.gdn_linear_recurrence_bwd(do, y.view(T, hv, 128), g, states, initial_state=p["h0"],
                                                cu_seqlens=p["cu"], dfinal_state=p["dfinal"])
    dx, dw, db = gdn.gdn_layernorm_bwd(dy.view(T, hv * 128), p["x"], mean, rstd, p["ln_w"])
    return {"out": out, "final": final, "x": dx, "ln_w": dw, "ln_b": db, "g": dg, "z": dz, "gate_w": dgw, "h0": dh0}


def block64(p, lens):
    q = {k: v.detach().cpu().double() for k, v in p.items() if k != "cu"}
    T, hv = q["x"].shape[0], q["a"].shape[1]
    leaves = {k: q[k].requires_grad_() for k in ("x", "ln_w", "ln_b", "z", "gate_w", "h0")}
    x = q["x"]
    c = x - x.mean(1, keepdim=True)
    y = c / torch.sqrt((c * c).mean(1, keepdim=True) + EPS_LN) * q["ln_w"] + q["ln_b"]
    g = (-torch.exp(q["A_log"]) * torch.nn.functional.softplus(q["a"] + q["dt_bias"])).requires_grad_()
    leaves["g"] = g
    rows, finals, t = [], [], 0
    for n, length in enumerate(lens):
        h = q["h0"][n]
        for i in range(t, t + length):
            h = torch.exp(g[i])[:, None] * h + y[i].view(hv, 128)
            rows.append(h)
        t += length
        finals.append(h)
    o, final = torch.stack(rows), torch.stack(finals)
    out = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS_GATE) * q["gate_w"] * torch.nn.functional.silu(q["z"])
    ((out * q["dout"]).sum() + (final * q["dfinal"]).sum()).backward()
    return {"out": out.detach(), "final": final.detach(), **{k: v.grad for k, v in leaves.items()}}


def params(dev, lens, hv, dtype):
    gen = torch.Generator().manual_seed(5)
    normal = lambda *shape: torch.randn(shape, generator=gen)
    T, N = sum(lens), len(lens)
    p = {"x": normal(T, hv * 128).to(dtype), "ln_w": normal(hv * 128) * 0.1 + 1, "ln_b": normal(hv * 128) * 0.1,
         "a": normal(T, hv), "A_log": torch.rand(hv, generator=gen) * 2.7,
         "dt_bias": torch.rand(hv, generator=gen) * 4 - 6, "h0": normal(N, hv, 128),
         "z": normal(T, hv, 128).to(dtype), "gate_w": torch.rand(128, generator=gen) + 0.5,
         "dout": normal(T, hv, 128).to(dtype), "dfinal": normal(N, hv, 128)}
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    p["cu"] = torch.tensor(cu, dtype=torch.int32)
    return {k: v.to(dev) for k, v in p.items()}


@pytest.mark.parametrize("dtype,bar", [(torch.float32, 1e-5), (torch.bfloat16, 1.8e-2)], ids=["f32", "bf16"])
def test_block_forward_and_backward(cuda, dtype, bar):
    lens, hv = [70, 1, 0, 130, 33], 3
    p = params(cuda, lens, hv, dtype)
    res = block(p, gdn)
    torch.cuda.synchronize()
    assert gdn.gdn_read_device_status() == gdn.GDN_OK
    ref = block64(p, lens)
    for k, v in res.items():
        r = ref[k].double()
        err = (v.detach().cpu().double() - r).norm() / r.norm()
        assert err <= bar, f"{k}: {err:.2e}"


def test_block_captured_into_a_graph(cuda):
    p = params(cuda, [70, 1, 0, 130, 33], 3, torch.bfloat16)
    ref = block(p, gdn)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = block(p, gdn)
    for v in captured.values():
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for k, v in ref.items():
        assert torch.equal(v, captured[k]), k


FIRST_CALL_IN_A_GRAPH = """
import sys
sys.path[:0] = [{tests!r}, {root!r}]
import torch
from test_gpu_training_block import block, params
from gated_deltanet_chunked_gb300 import gdn
gdn.load()
dev = torch.device("cuda:0")
p = params(dev, [300, 0, 65], 3, torch.bfloat16)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    captured = block(p, gdn)
g.replay()
torch.cuda.synchronize()
ref = block(p, gdn)
torch.cuda.synchronize()
assert all(torch.equal(v, captured[k]) for k, v in ref.items())
print("same")
"""


def test_first_call_of_a_process_is_captured(cuda):
    """Nothing has to be called before the capture (in a process of its own)."""
    import os
    import subprocess
    import sys

    here = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALL_IN_A_GRAPH.format(tests=here, root=os.path.dirname(here))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


def test_prefill_then_decode(cuda):
    """Two prompts of one packed prefill go on with decode steps on a slot
    cache; both parts together are the whole sequences."""
    lens, steps, hv = [100, 37], 5, 2
    gen = torch.Generator().manual_seed(9)
    xs = [torch.randn(n + steps, hv, 128, generator=gen).to(cuda) for n in lens]
    gs = [(-torch.rand(n + steps, hv, generator=gen)).to(cuda) for n in lens]
    cu = torch.tensor([0, 100, 137], dtype=torch.int32, device=cuda)
    _, final = gdn.gdn_linear_recurrence(torch.cat([x[:n] for x, n in zip(xs, lens)]),
                                         torch.cat([g[:n] for g, n in zip(gs, lens)]), cu_seqlens=cu)
    cache = torch.zeros(6, hv, 128, device=cuda)
    slots = torch.tensor([4, 1], dtype=torch.int32, device=cuda)
    cache[slots.long()] = final
    for i in range(steps):
        gdn.gdn_linear_recurrence_step(torch.stack([x[n + i] for x, n in zip(xs, lens)]),
                                       torch.stack([g[n + i] for g, n in zip(gs, lens)]), cache, state_indices=slots)
    whole = torch.cat(xs), torch.cat(gs)
    _, ref = gdn.gdn_linear_recurrence(*whole, cu_seqlens=torch.tensor([0, 105, 147], dtype=torch.int32, device=cuda))
    # the same products in another grouping: a few f32 roundings of a state of order 1
    assert torch.allclose(cache[slots.long()], ref, rtol=1e-5, atol=1e-5)
    assert (cache[[0, 2, 3, 5]] == 0).all()
