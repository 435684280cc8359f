"""The recurrent block's training and long-sequence operators as measured work.

Three operators, each in a plain form (elementary torch operations in 32 bits, rounded once) and,
with ``own`` set, through the library's entry points:

* recurrence: the gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t per channel of [hv, 128],
  over packed sequences, with its backward pass, and its decode step on a state cache;
* layernorm: the layer norm over the last dimension and its backward pass with the weight's and
  the bias's gradient;
* gate_bwd: the backward pass of the output gate y = o / sqrt(mean(o^2) + eps) * w * silu(z).

A case is a dict of plain values. ``lens`` holds the packed sequences' lengths as text.
"""
import math

import torch

own = False

HEAD = 128
EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _rec(name, dtype, hv, lens, gate, train, init, mu):
    return {"name": name, "op": "recurrence", "dtype": dtype, "hv": hv, "lens": lens, "gate": gate, "train": train,
            "init": init, "mu": mu}


def _ln(name, dtype, rows, width, train):
    return {"name": name, "op": "layernorm", "dtype": dtype, "rows": rows, "width": width, "train": train}


def listed():
    return [
        # the tiny f32 configuration: a 200-token prompt from a saved state; latency counts
        _rec("rec_tiny_f32_T200", "f32", 2, "200", "head", False, True, 0.0),
        # prefill of one 4096-token prompt, a gate for every channel
        _rec("rec_prefill_T4096", "bf16", 32, "4096", "channel", False, False, 0.0),
        # a training step on eight packed sequences (38429 tokens) with gates per head, as gdn_gating makes them
        _rec("rec_train_packed8", "bf16", 32, "4878,3108,6236,2922,7168,6006,4934,3177", "head", True, True, -2.0),
        # a training step on one long sequence: the largest case
        _rec("rec_train_T65536", "bf16", 32, "65536", "channel", True, False, -2.0),
        # fine-tuning in f32 on a ragged batch with empty and one-token sequences
        _rec("rec_train_ragged_f32", "f32", 3, "1,0,63,64,65,513,1000,7,0,129", "channel", True, True, -1.0),
        # one decode token for each of 256 sequences, states in a slot cache
        {"name": "rec_step_N256", "op": "step", "dtype": "bf16", "hv": 32, "n": 256, "gate": "channel", "mu": 0.0},
        # the norm before a block, one decode token
        _ln("ln_row_D4096", "bf16", 1, 4096, False),
        # the norm before a block in a training step of 4096 tokens
        _ln("ln_train_R4096_D4096", "bf16", 4096, 4096, True),
        # rows whose width is odd: no row but the first is aligned
        _ln("ln_train_R1237_D1001", "f32", 1237, 1001, True),
        # a norm of every 128-channel head of 4096 tokens
        _ln("ln_train_heads", "bf16", 4096 * 32, HEAD, True),
        # the output gate's backward pass at the prefill workload's size
        {"name": "gate_bwd_T4096", "op": "gate_bwd", "dtype": "bf16", "hv": 32, "rows": 4096},
        # the same for a short f32 sequence with an odd head count
        {"name": "gate_bwd_f32_T333", "op": "gate_bwd", "dtype": "f32", "hv": 3, "rows": 333},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["recurrence", "recurrence", "recurrence", "step", "layernorm", "layernorm", "gate_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "recurrence":
        hv = _log_int(rng, 1, 32)
        total = _log_int(rng, 1, 65536 if dtype == "bf16" else 32768)
        n = min(_log_int(rng, 1, 64), total)
        cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        return {"op": kind, "dtype": dtype, "hv": hv, "lens": ",".join(map(str, lens)),
                "gate": rng.choice(["channel", "head"]), "train": rng.random() < 0.6, "init": rng.random() < 0.6,
                "mu": rng.choice([0.0, -1.0, -2.0, -4.0])}
    if kind == "step":
        return {"op": kind, "dtype": dtype, "hv": _log_int(rng, 1, 32), "n": _log_int(rng, 1, 1024),
                "gate": rng.choice(["channel", "head"]), "mu": rng.choice([0.0, -2.0])}
    if kind == "layernorm":
        width = _log_int(rng, 8, 16384)
        if rng.random() < 0.6:  # widths that a model has
            width = max(8, width // 8 * 8)
        return {"op": kind, "dtype": dtype, "rows": _log_int(rng, 1, min(65536, 100_000_000 // width)), "width": width,
                "train": rng.random() < 0.7}
    return {"op": kind, "dtype": dtype, "hv": _log_int(rng, 1, 32), "rows": _log_int(rng, 1, 32768)}


def _lens(case):
    return [int(v) for v in case["lens"].split(",")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, sigma=1.0, mu=0.0, to=torch.float32):
        return (torch.randn(shape, generator=gen, device="cuda") * sigma + mu).to(to)

    def gates(tokens):
        """Log-decays -softplus(N(mu, 1)): one per head (f32) or one per channel (io type)."""
        head = case["gate"] == "head"
        raw = normal(*((tokens, case["hv"]) if head else (tokens, case["hv"], HEAD)), mu=case["mu"])
        return -torch.logaddexp(raw, torch.zeros_like(raw)).to(torch.float32 if head else dtype)

    s = {"case": case}
    if case["op"] == "recurrence":
        lens, hv = _lens(case), case["hv"]
        total = sum(lens)
        s["x"] = normal(total, hv, HEAD, to=dtype)
        s["g"] = gates(total)
        s["h0"] = normal(len(lens), hv, HEAD, sigma=0.5) if case["init"] else None
        bounds = [0]
        for n in lens:
            bounds.append(bounds[-1] + n)
        s["cu"] = torch.tensor(bounds, dtype=torch.int32, device="cuda")
        if case["train"]:
            s["dout"] = normal(total, hv, HEAD, to=dtype)
            s["dfinal"] = normal(len(lens), hv, HEAD) if case["init"] else None
    elif case["op"] == "step":
        n, hv = case["n"], case["hv"]
        s["x"] = normal(n, hv, HEAD, to=dtype)
        s["g"] = gates(n)
        s["state"] = normal(n + 3, hv, HEAD, sigma=0.5)
        s["slots"] = torch.randperm(n + 3, generator=gen, device="cuda")[:n].to(torch.int32)
    elif case["op"] == "layernorm":
        rows, width = case["rows"], case["width"]
        s["x"] = normal(rows, width, sigma=1.5, mu=0.3, to=dtype)
        s["weight"] = torch.rand(width, generator=gen, device="cuda") + 0.5
        s["bias"] = normal(width, sigma=0.1)
        if case["train"]:
            s["dy"] = normal(rows, width, to=dtype)
    else:
        shape = (case["rows"], case["hv"], HEAD)
        s["o"] = normal(*shape, sigma=0.05, to=dtype)
        s["z"] = normal(*shape, to=dtype)
        s["dy"] = normal(*shape, to=dtype)
        s["weight"] = torch.rand(HEAD, generator=gen, device="cuda") + 0.5
    return s


# ---- plain forms -------------------------------------------------------------


def _scan(a, b, longest):
    """y[t] = a[t] y[t-1] + b[t] by doubling; a is zero where a sequence starts, none is longer than `longest`."""
    d = 1
    while d < longest:
        b = torch.cat([b[:d], b[d:] + a[d:] * b[:-d]])
        if 2 * d < longest:
            a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return b


def _plain_recurrence(s):
    case, x = s["case"], s["x"].float()
    decay = torch.exp(s["g"].float())
    if decay.dim() == 2:
        decay = decay[:, :, None]
    lens = _lens(case)
    longest = max(lens)
    cu = s["cu"].long()
    held = cu[1:] > cu[:-1]  # sequences with tokens
    first, last = cu[:-1][held], cu[1:][held] - 1
    n, hv = len(lens), case["hv"]
    h0 = s["h0"] if s["h0"] is not None else torch.zeros(n, hv, HEAD, device=x.device)

    cut = decay.clone()
    cut[first] = 0.0
    b = x.clone()
    b[first] += decay[first] * h0[held]
    h = _scan(cut, b, longest)
    final = h0.clone()
    final[held] = h[last]
    out = {"out": h.to(s["x"].dtype), "final": final}
    if not case["train"]:
        return out
    b = s["dout"].to(torch.float32, copy=True)  # the state's own tensor stays as it is
    if s["dfinal"] is not None:
        b[last] += s["dfinal"][held]
    nxt = torch.cat([decay[1:], decay[:1]])
    nxt[last] = 0.0
    dh = _scan(nxt.flip(0), b.flip(0), longest).flip(0)
    before = torch.cat([h[:1], h[:-1]])
    before[first] = h0[held]
    dg = decay * before * dh
    out["dx"] = dh.to(s["x"].dtype)
    out["dg"] = dg.sum(-1) if case["gate"] == "head" else dg.to(s["g"].dtype)
    if s["h0"] is not None:
        dh0 = s["dfinal"].clone()
        dh0[held] = decay[first] * dh[first]
        out["dh0"] = dh0
    return out


def _plain_step(s):
    decay = torch.exp(s["g"].float())
    if decay.dim() == 2:
        decay = decay[:, :, None]
    slots = s["slots"].long()
    h = decay * s["state"][slots] + s["x"].float()
    s["state"][slots] = h
    return {"out": h.to(s["x"].dtype), "state": s["state"]}


def _plain_layernorm(s):
    x = s["x"].float()
    centred = x - x.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt((centred * centred).mean(-1, keepdim=True) + EPS)
    xhat = centred * rstd
    out = {"y": (xhat * s["weight"] + s["bias"]).to(s["x"].dtype)}
    if s["case"]["train"]:
        dy = s["dy"].float()
        wdy = dy * s["weight"]
        dx = rstd * (wdy - wdy.mean(-1, keepdim=True) - xhat * (wdy * xhat).mean(-1, keepdim=True))
        out |= {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}
    return out


def _plain_gate_bwd(s):
    o, z, dy, w = s["o"].float(), s["z"].float(), s["dy"].float(), s["weight"]
    rms = 1.0 / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS)
    n = o * rms
    sig = 1.0 / (1.0 + torch.exp(-z))
    silu = z * sig
    u = dy * w * silu
    do = rms * (u - n * (u * n).mean(-1, keepdim=True))
    dz = dy * n * w * sig * (1.0 + z * (1.0 - sig))
    dt = s["o"].dtype
    return {"do": do.to(dt), "dz": dz.to(dt), "dweight": (dy * n * silu).sum((0, 1))}


# ---- the library's calls -----------------------------------------------------


def _own_recurrence(gdn, s):
    if not s["case"]["train"]:
        out, final = gdn.gdn_linear_recurrence(s["x"], s["g"], initial_state=s["h0"], cu_seqlens=s["cu"])
        return {"out": out, "final": final}
    out, final, states = gdn.gdn_linear_recurrence(s["x"], s["g"], initial_state=s["h0"], cu_seqlens=s["cu"],
                                                   save_states=True)
    dx, dg, dh0 = gdn.gdn_linear_recurrence_bwd(s["dout"], s["x"], s["g"], states, initial_state=s["h0"],
                                                cu_seqlens=s["cu"], dfinal_state=s["dfinal"])
    res = {"out": out, "final": final, "dx": dx, "dg": dg}
    if s["h0"] is not None:
        res["dh0"] = dh0
    return res


def _own_step(gdn, s):
    out = gdn.gdn_linear_recurrence_step(s["x"], s["g"], s["state"], state_indices=s["slots"])
    return {"out": out, "state": s["state"]}


def _own_layernorm(gdn, s):
    if not s["case"]["train"]:
        return {"y": gdn.gdn_layernorm(s["x"], s["weight"], s["bias"], EPS)}
    y, mean, rstd = gdn.gdn_layernorm(s["x"], s["weight"], s["bias"], EPS, save_stats=True)
    dx, dweight, dbias = gdn.gdn_layernorm_bwd(s["dy"], s["x"], mean, rstd, s["weight"])
    return {"y": y, "dx": dx, "dweight": dweight, "dbias": dbias}


def _own_gate_bwd(gdn, s):
    do, dz, dweight = gdn.gdn_gated_rmsnorm_bwd(s["dy"], s["o"], s["z"], s["weight"], EPS)
    return {"do": do, "dz": dz, "dweight": dweight}


def run(state):
    op = state["case"]["op"]
    if own:
        from gated_deltanet_chunked_gb300 import gdn

        return {"recurrence": _own_recurrence, "step": _own_step, "layernorm": _own_layernorm,
                "gate_bwd": _own_gate_bwd}[op](gdn, state)
    return {"recurrence": _plain_recurrence, "step": _plain_step, "layernorm": _plain_layernorm,
            "gate_bwd": _plain_gate_bwd}[op](state)


# ---- what a pass cannot do without -------------------------------------------


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "recurrence":
        lens = _lens(case)
        rows = sum(lens) * case["hv"]
        el, seqs = rows * HEAD, len(lens) * case["hv"] * HEAD
        gate = rows * 4 if case["gate"] == "head" else el * e
        # x, g in, out and the final state out; a training step also takes dout (and the final state's gradient)
        # and gives dx, dg (and the initial state's gradient)
        bytes_ = el * e * 2 + gate + seqs * 4 * (2 if case["init"] else 1)
        flops = 3 * el
        if case["train"]:
            bytes_ += el * e * 2 + gate + (seqs * 8 if case["init"] else 0)
            flops += 6 * el
        return {"bytes": bytes_, "flops": flops}
    if case["op"] == "step":
        rows = case["n"] * case["hv"]
        el = rows * HEAD
        gate = rows * 4 if case["gate"] == "head" else el * e
        return {"bytes": el * (2 * e + 8) + gate + 4 * case["n"], "flops": 3 * el}
    if case["op"] == "layernorm":
        el = case["rows"] * case["width"]
        bytes_, flops = el * e * 2 + case["width"] * 8, 8 * el
        if case["train"]:
            bytes_ += el * e * 2 + case["width"] * 8
            flops += 14 * el
        return {"bytes": bytes_, "flops": flops}
    el = case["rows"] * case["hv"] * HEAD
    return {"bytes": el * e * 5 + HEAD * 8, "flops": 24 * el}


# ---- definitions in 64 bits --------------------------------------------------


def _exact_recurrence(case, s):
    x, decay = s["x"].double(), s["g"].double().exp()
    lens, hv = _lens(case), case["hv"]
    if decay.dim() == 2:
        decay = decay.unsqueeze(-1).expand(-1, hv, HEAD).contiguous()
    out = torch.empty_like(x)
    final = torch.zeros(len(lens), hv, HEAD, dtype=torch.float64, device=x.device)
    if s["h0"] is not None:
        final.copy_(s["h0"])
    t = 0
    for n, length in enumerate(lens):
        h = final[n].clone()
        for i in range(t, t + length):
            torch.addcmul(x[i], decay[i], h, out=out[i])
            h = out[i]
        final[n] = h
        t += length
    res = {"out": out, "final": final}
    if not case["train"]:
        return res
    dout = s["dout"].double()
    dx = torch.empty_like(x)
    prior = torch.empty_like(x)
    dh0 = torch.zeros_like(final)
    t = 0
    for n, length in enumerate(lens):
        e = torch.zeros(hv, HEAD, dtype=torch.float64, device=x.device)
        if s["dfinal"] is not None:
            e = s["dfinal"][n].double()
        for i in range(t + length - 1, t - 1, -1):
            torch.add(dout[i], e, out=dx[i])
            e = decay[i] * dx[i]
        dh0[n] = e
        if length:
            prior[t] = s["h0"][n] if s["h0"] is not None else 0.0
            prior[t + 1:t + length] = out[t:t + length - 1]
        t += length
    prior.mul_(decay).mul_(dx)
    res |= {"dx": dx, "dg": prior.sum(-1) if case["gate"] == "head" else prior}
    if s["h0"] is not None:
        res["dh0"] = dh0
    return res


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "recurrence":
        return _exact_recurrence(case, s)
    if case["op"] == "step":
        g, state = s["g"].double(), s["state"].double()
        if g.dim() == 2:
            g = g.unsqueeze(-1)
        idx = s["slots"].long()
        h = torch.addcmul(s["x"].double(), g.exp(), state.index_select(0, idx))
        return {"out": h, "state": state.index_copy(0, idx, h)}
    if case["op"] == "layernorm":
        x, w = s["x"].double(), s["weight"].double()
        var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
        xhat = (x - mean) / (var + EPS).sqrt()
        res = {"y": torch.addcmul(s["bias"].double(), xhat, w)}
        if case["train"]:
            dy = s["dy"].double()
            # through the Jacobian (I - 1 1^T / D - xhat xhat^T / D) / sqrt(var + eps)
            gx = dy * w
            gx = gx - gx.sum(1, keepdim=True) / case["width"] - xhat * ((gx * xhat).sum(1, keepdim=True) / case["width"])
            res |= {"dx": gx / (var + EPS).sqrt(), "dweight": torch.einsum("rd,rd->d", dy, xhat), "dbias": dy.sum(0)}
        return res
    o, z, dy, w = s["o"].double(), s["z"].double(), s["dy"].double(), s["weight"].double()
    den = (o.square().sum(-1, keepdim=True) / HEAD + EPS).sqrt()
    sig = torch.sigmoid(z)
    up = dy * w * z * sig
    do = up / den - o * (up * o).sum(-1, keepdim=True) / (HEAD * den ** 3)
    dz = dy * w * o / den * (sig + z * sig * (1.0 - sig))
    return {"do": do, "dz": dz, "dweight": (dy * z * sig * o / den).reshape(-1, HEAD).sum(0)}
