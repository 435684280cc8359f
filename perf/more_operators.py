"""Linear attention with a decay for each head, and its front end, as measured work.

Three operators, each in a plain form (elementary torch operations in 32 bits, rounded once) and,
with ``own`` set, through the library's entry points:

* attention: S_t = exp(decay_h) S_{t-1} + k_t^T v_t, o_t = scale q_t S_t over packed sequences, heads of
  128 channels, hv / hq value heads to a query and key head, with initial and final states; a training
  case also takes its backward pass;
* step: the same for one token of each sequence, on a cache of states;
* rope: the RMS norm of every query and key head and the rotation by position in one pass, over all or
  the first channels of a head, the pairs half a rotation apart or next to each other, with one position
  a token or one for each of several axes; a training case also takes its backward pass.

A case is a dict of plain values. ``lens`` holds the packed sequences' lengths as text.
"""
import math

import torch

own = False

HEAD = 128
CHUNK = 128  # the plain form's chunk
EPS = 1e-6
BASE = 1e6  # of the rotation's frequencies
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _attn(name, dtype, hq, hv, lens, train, init):
    return {"name": name, "op": "attention", "dtype": dtype, "hq": hq, "hv": hv, "lens": lens, "train": train,
            "init": init}


def _rope(name, dtype, hq, hk, rows, rotary, pairs, axes, packed, train):
    return {"name": name, "op": "rope", "dtype": dtype, "hq": hq, "hk": hk, "rows": rows, "rotary": rotary,
            "pairs": pairs, "axes": axes, "packed": packed, "train": train}


def listed():
    return [
        # the tiny f32 configuration: a 200-token prompt from a saved state; latency counts
        _attn("attn_tiny_f32_T200", "f32", 2, 2, "200", False, True),
        # prefill of one 4096-token prompt
        _attn("attn_prefill_T4096", "bf16", 16, 32, "4096", False, False),
        # prefill of eight packed prompts (38429 tokens), each from a saved state
        _attn("attn_prefill_packed8", "bf16", 16, 32, "4878,3108,6236,2922,7168,6006,4934,3177", False, True),
        # prefill of one long prompt: the largest case
        _attn("attn_prefill_T65536", "bf16", 16, 32, "65536", False, False),
        # a training step on 4096 tokens
        _attn("attn_train_T4096", "bf16", 16, 32, "4096", True, False),
        # fine-tuning in f32 on a ragged batch with empty and one-token sequences
        _attn("attn_train_ragged_f32", "f32", 3, 3, "1,0,63,64,65,513,1000,7,0,129", True, True),
        # one decode token for each of 256 sequences, f32 states in a slot cache
        {"name": "step_N256", "op": "step", "dtype": "bf16", "state": "f32", "hq": 16, "hv": 32, "n": 256},
        # one decode token for each of five sequences, on a bf16 cache
        {"name": "step_N5_bf16_state", "op": "step", "dtype": "bf16", "state": "bf16", "hq": 16, "hv": 32, "n": 5},
        # the front end of a decode step
        _rope("rope_decode_N256", "bf16", 16, 16, 256, HEAD, "halves", 1, False, False),
        # the front end in a training step of 4096 tokens, q and k in one projection's rows
        _rope("rope_train_T4096", "bf16", 16, 16, 4096, HEAD, "halves", 1, True, True),
        # a long prompt of text and images: three axes, a quarter of each head rotated
        _rope("rope_axes_T65536", "bf16", 32, 4, 65536, 32, "halves", 3, True, False),
        # fine-tuning in f32 with odd head counts, neighbouring channels paired
        _rope("rope_train_f32_T333", "f32", 3, 1, 333, 64, "neighbours", 1, False, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "attention", "step", "rope", "rope"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "rope":
        hq = _log_int(rng, 1, 32)
        rotary = rng.choice([HEAD, HEAD, 64, 32, 2 * rng.randrange(1, 65)])
        return {"op": kind, "dtype": dtype, "hq": hq, "hk": rng.choice([hq, _log_int(rng, 1, hq)]),
                "rows": _log_int(rng, 1, 32768), "rotary": rotary, "pairs": rng.choice(["halves", "neighbours"]),
                "axes": rng.choice([1, 1, 3]), "packed": rng.random() < 0.5, "train": rng.random() < 0.5}
    hq = _log_int(rng, 1, 16)
    hv = hq * rng.choice([1, 1, 2, 2, 3, 4])
    if kind == "step":
        return {"op": kind, "dtype": dtype, "state": rng.choice(["f32", "f32", "bf16"]), "hq": hq, "hv": hv,
                "n": _log_int(rng, 1, max(1, 8192 // hv))}
    train = rng.random() < 0.5
    most = 65536 * 32 if dtype == "bf16" else 4096 * 32  # tokens times value heads
    total = _log_int(rng, 1, min(65536, (most // 8 if train else most) // hv))
    n = min(_log_int(rng, 1, 64), total)
    cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    return {"op": kind, "dtype": dtype, "hq": hq, "hv": hv, "lens": ",".join(map(str, lens)), "train": train,
            "init": rng.random() < 0.6}


def _lens(case):
    return [int(v) for v in case["lens"].split(",")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, sigma=1.0, to=torch.float32):
        return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(to)

    s = {"case": case}
    if case["op"] == "rope":
        rows, hq, hk = case["rows"], case["hq"], case["hk"]
        if case["packed"]:  # q and k where the projection has left them, in rows with v's channels
            both = normal(rows, (hq + 2 * hk) * HEAD, to=dtype)
            s["q"] = both[:, :hq * HEAD].unflatten(1, (hq, HEAD))
            s["k"] = both[:, hq * HEAD:(hq + hk) * HEAD].unflatten(1, (hk, HEAD))
        else:
            s["q"], s["k"] = normal(rows, hq, HEAD, to=dtype), normal(rows, hk, HEAD, to=dtype)
        s["q_weight"] = torch.rand(HEAD, generator=gen, device="cuda") + 0.5
        s["k_weight"] = torch.rand(HEAD, generator=gen, device="cuda") + 0.5
        half = case["rotary"] // 2
        s["inv_freq"] = (BASE ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        if case["axes"] == 1:
            # rows of a batch, anywhere up to a context of 2^20
            s["positions"] = torch.randint(0, 1 << 20, (rows,), generator=gen, device="cuda", dtype=torch.int32)
            s["pair_axis"] = None
        else:
            # time, height, width; the axes in turn over the pairs
            s["positions"] = torch.randint(0, 1 << 17, (case["axes"], rows), generator=gen, device="cuda",
                                           dtype=torch.int32)
            s["pair_axis"] = (torch.arange(half, device="cuda") % case["axes"]).to(torch.int32)
        if case["train"]:
            s["dq"], s["dk"] = normal(rows, hq, HEAD, to=dtype), normal(rows, hk, HEAD, to=dtype)
        return s

    hq, hv = case["hq"], case["hv"]
    # log-decays that halve from head to head in a geometric row, as slopes of heads are laid out
    slopes = 2.0 ** (-8.0 * (torch.arange(hv, device="cuda") + 1) / hv)
    s["decay"] = -slopes * (0.75 + 0.5 * torch.rand(hv, generator=gen, device="cuda"))
    s["scale"] = HEAD ** -0.5
    if case["op"] == "step":
        n = case["n"]
        s["q"], s["k"] = normal(n, hq, HEAD, to=dtype), normal(n, hq, HEAD, to=dtype)
        s["v"] = normal(n, hv, HEAD, to=dtype)
        s["state"] = normal(n + 3, hv, HEAD, HEAD, to=DTYPES[case["state"]])
        s["slots"] = torch.randperm(n + 3, generator=gen, device="cuda")[:n].to(torch.int32)
        return s
    lens = _lens(case)
    total = sum(lens)
    s["q"], s["k"] = normal(total, hq, HEAD, to=dtype), normal(total, hq, HEAD, to=dtype)
    s["v"] = normal(total, hv, HEAD, to=dtype)
    s["s0"] = normal(len(lens), hv, HEAD, HEAD) if case["init"] else None
    bounds = [0]
    for n in lens:
        bounds.append(bounds[-1] + n)
    s["cu"] = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    if case["train"]:
        s["dout"] = normal(total, hv, HEAD, to=dtype)
        s["dfinal"] = normal(len(lens), hv, HEAD, HEAD) if case["init"] else None
    return s


# ---- plain forms -------------------------------------------------------------


def _powers(decay, n):
    """exp(decay_h n) in 32 bits, [H, ...] for whole numbers n; zero where n is negative."""
    n = n.unsqueeze(0)
    e = torch.exp(decay.double().view(-1, *[1] * (n.dim() - 1)) * n.clamp(min=0).double())
    return torch.where(n >= 0, e, 0.0).float()


def _plain_attention(s):
    case, decay, scale = s["case"], s["decay"], s["scale"]
    lens, hq, hv = _lens(case), case["hq"], case["hv"]
    dev, n_seq = s["q"].device, len(lens)
    # the chunks of all sequences: where each starts and ends
    counts = [-(-n // CHUNK) for n in lens]
    nc = sum(counts)
    cu = s["cu"].long()
    seq = torch.repeat_interleave(torch.arange(n_seq, device=dev), torch.tensor(counts, device=dev), output_size=nc)
    ahead = torch.tensor([sum(counts[:i]) for i in range(n_seq)], device=dev)
    start = cu[seq] + (torch.arange(nc, device=dev) - ahead[seq]) * CHUNK
    end = torch.minimum(start + CHUNK, cu[seq + 1])
    at = torch.arange(CHUNK, device=dev)
    rows = start[:, None] + at
    held = rows < end[:, None]
    rows = rows.clamp(max=s["q"].shape[0] - 1)

    def chunks(x):  # [T, h, 128] -> [hv, nc, CHUNK, 128] with zeros behind a sequence's end
        x = torch.where(held[:, :, None, None], x[rows].float(), 0.0).permute(2, 0, 1, 3)
        return x.repeat_interleave(hv // x.shape[0], 0)

    def tokens(x, heads):  # and back, the heads of a group summed
        x = x.unflatten(0, (heads, hv // heads)).sum(1) if heads != hv else x
        return x.permute(1, 2, 0, 3)[held].to(s["q"].dtype)

    q, k, v = chunks(s["q"]), chunks(s["k"]), chunks(s["v"])
    inside = _powers(decay, at[:, None] - at)[:, None]  # from key j to query i of a chunk
    into = _powers(decay, at + 1)[:, None, :, None]  # from a chunk's entry to query i
    onto = _powers(decay, torch.where(held, end[:, None] - 1 - rows, -1))[..., None]  # from key j to the chunk's end
    same = seq[:, None] == seq
    between = _powers(decay, torch.where(same, start[:, None] - end, -1))  # from a chunk's end to another's entry
    first = seq[:, None] == torch.arange(n_seq, device=dev)
    after = _powers(decay, torch.where(first, start[:, None] - cu[:-1], -1))  # from a sequence's start to a chunk
    left = _powers(decay, torch.where(first, cu[1:] - end[:, None], -1))  # from a chunk's end to the sequence's end
    whole = _powers(decay, cu[1:] - cu[:-1])[:, :, None]

    def flat(x):
        return x.flatten(2)

    def states(x):
        return x.unflatten(2, (HEAD, HEAD))

    added = flat((k * onto).transpose(2, 3) @ v)
    entry = between @ added
    final = left.transpose(1, 2) @ added
    if s["s0"] is not None:
        s0 = flat(s["s0"].transpose(0, 1))
        entry = entry + after @ s0
        final = final + whole * s0
    entry = states(entry)
    out = ((q @ k.transpose(2, 3)) * inside) @ v + (q * into) @ entry
    res = {"out": tokens(out * scale, hv), "final": states(final).transpose(0, 1)}
    if not case["train"]:
        return res
    do = chunks(s["dout"]) * scale
    dadded = flat((q * into).transpose(2, 3) @ do)  # the gradient of a chunk's entry state by the chunk itself
    dexit = between.transpose(1, 2) @ dadded
    ds0 = after.transpose(1, 2) @ dadded
    if s["dfinal"] is not None:
        df = flat(s["dfinal"].transpose(0, 1))
        dexit = dexit + left @ df
        ds0 = ds0 + whole * df
    dexit = states(dexit)
    dp = (do @ v.transpose(2, 3)) * inside
    p = (q @ k.transpose(2, 3)) * inside
    dq = dp @ k + (do @ entry.transpose(2, 3)) * into
    dk = dp.transpose(2, 3) @ q + (v @ dexit.transpose(2, 3)) * onto
    dv = p.transpose(2, 3) @ do + (k @ dexit) * onto
    res |= {"dq": tokens(dq, hq), "dk": tokens(dk, hq), "dv": tokens(dv, hv)}
    if s["s0"] is not None:
        res["ds0"] = states(ds0).transpose(0, 1)
    return res


def _plain_step(s):
    g = s["case"]["hv"] // s["case"]["hq"]
    q, k, v = s["q"].float().repeat_interleave(g, 1), s["k"].float().repeat_interleave(g, 1), s["v"].float()
    slots = s["slots"].long()
    new = torch.exp(s["decay"])[:, None, None] * s["state"][slots].float() + k[..., None] * v[..., None, :]
    s["state"][slots] = new.to(s["state"].dtype)
    out = (q[..., None] * new).sum(2) * s["scale"]
    return {"out": out.to(s["q"].dtype), "state": s["state"]}


def _angles(s):
    """cos and sin [T, 1, rotary / 2] in 64 bits: a far position times a frequency has few bits behind the point."""
    pos, axis = s["positions"], s["pair_axis"]
    per_pair = pos[:, None] if axis is None else pos[axis.long()].T
    angle = (per_pair.double() * s["inv_freq"].double())[:, None]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _pairs(x, case):
    r = case["rotary"]
    if case["pairs"] == "halves":
        return x[..., :r // 2], x[..., r // 2:r]
    return x[..., 0:r:2], x[..., 1:r:2]


def _joined(a, b, x, case):
    r = case["rotary"]
    turned = torch.cat([a, b], -1) if case["pairs"] == "halves" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_rope(s):
    case = s["case"]
    cos, sin = _angles(s)
    out = {}
    for name in ("q", "k"):
        x, w = s[name].float(), s[name + "_weight"]
        rstd = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        xhat = x * rstd
        n = xhat * w
        a, b = _pairs(n, case)
        out[name] = _joined(a * cos - b * sin, a * sin + b * cos, n, case).to(s[name].dtype)
        if case["train"]:
            dy = s["d" + name].float()
            a, b = _pairs(dy, case)
            dn = _joined(a * cos + b * sin, b * cos - a * sin, dy, case)
            u = dn * w
            dx = rstd * (u - xhat * (u * xhat).mean(-1, keepdim=True))
            out["d" + name] = dx.to(s[name].dtype)
            out["d" + name + "_weight"] = (dn * xhat).sum((0, 1))
    return out


# ---- the library's calls -----------------------------------------------------


def _own_attention(gdn, s):
    out, final = gdn.gdn_linear_attention(s["q"], s["k"], s["v"], s["decay"], s["scale"], initial_state=s["s0"],
                                          cu_seqlens=s["cu"])
    res = {"out": out, "final": final}
    if s["case"]["train"]:
        dq, dk, dv, ds0 = gdn.gdn_linear_attention_bwd(s["dout"], s["q"], s["k"], s["v"], s["decay"], s["scale"],
                                                       initial_state=s["s0"], cu_seqlens=s["cu"],
                                                       dfinal_state=s["dfinal"])
        res |= {"dq": dq, "dk": dk, "dv": dv}
        if s["s0"] is not None:
            res["ds0"] = ds0
    return res


def _own_step(gdn, s):
    out = gdn.gdn_linear_attention_step(s["q"], s["k"], s["v"], s["decay"], s["scale"], s["state"],
                                        state_indices=s["slots"])
    return {"out": out, "state": s["state"]}


def _own_rope(gdn, s):
    neighbours = s["case"]["pairs"] == "neighbours"
    args = (s["q_weight"], s["k_weight"], s["inv_freq"], s["positions"])
    q, k = gdn.gdn_qk_norm_rope(s["q"], s["k"], *args, pair_axis=s["pair_axis"], interleaved=neighbours, eps=EPS)
    res = {"q": q, "k": k}
    if s["case"]["train"]:
        dq, dk, dqw, dkw = gdn.gdn_qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], *args,
                                                    pair_axis=s["pair_axis"], interleaved=neighbours, eps=EPS)
        res |= {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    return res


def run(state):
    op = state["case"]["op"]
    if own:
        from gated_deltanet_chunked_gb300 import gdn

        return {"attention": _own_attention, "step": _own_step, "rope": _own_rope}[op](gdn, state)
    return {"attention": _plain_attention, "step": _plain_step, "rope": _plain_rope}[op](state)


# ---- what a pass cannot do without -------------------------------------------


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rope":
        el, half = case["rows"] * (case["hq"] + case["hk"]) * HEAD, case["rotary"] // 2
        # x in, y out, positions, frequencies, weights; a training step takes dy and x again, gives dx and the
        # weights' gradients
        bytes_ = el * e * 2 + case["rows"] * case["axes"] * 4 + half * 4 + 2 * HEAD * 4
        flops = el * 8
        if case["train"]:
            bytes_ += el * e * 2 + 2 * HEAD * 4
            flops += el * 14
        return {"bytes": bytes_, "flops": flops}
    hq, hv = case["hq"], case["hv"]
    if case["op"] == "step":
        n = case["n"]
        held = 4 if case["state"] == "f32" else 2
        return {"bytes": n * (hv * HEAD * HEAD * held * 2 + (2 * hq + 2 * hv) * HEAD * e + 4) + hv * 4,
                "flops": n * hv * HEAD * HEAD * 5}
    lens = _lens(case)
    total, states = sum(lens), len(lens) * hv * HEAD * HEAD * 4
    bytes_ = total * (2 * hq + 2 * hv) * HEAD * e + states * (2 if case["init"] else 1) + hv * 4
    # a token's update and its product with the state
    flops = total * hv * HEAD * HEAD * 4
    if case["train"]:
        # dout in; dq, dk, dv out; dfinal in and ds0 out
        bytes_ += total * (2 * hq + 2 * hv) * HEAD * e + (states * 2 if case["init"] else 0)
        # the gradient state's update and the products for dq, dk and dv
        flops += total * hv * HEAD * HEAD * 8
    return {"bytes": bytes_, "flops": flops}


# ---- definitions in 64 bits --------------------------------------------------


def _exact_attention(case, s):
    """Token by token."""
    g = case["hv"] // case["hq"]
    keep = torch.exp(s["decay"].double())[:, None, None]
    q = (s["q"].double() * s["scale"]).repeat_interleave(g, 1)[..., None]  # columns [T, hv, 128, 1]
    k = s["k"].double().repeat_interleave(g, 1)[..., None]
    v = s["v"].double()[:, :, None, :]  # rows
    lens, hv, dev = _lens(case), case["hv"], q.device
    out, final = torch.empty_like(v), []
    train = case["train"]
    if train:
        do = s["dout"].double()[:, :, None, :]
        dq, dk, dv, ds0 = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), []
    t = 0
    for n, length in enumerate(lens):
        state = torch.zeros(hv, HEAD, HEAD, dtype=torch.float64, device=dev)
        if s["s0"] is not None:
            state.copy_(s["s0"][n])
        for i in range(t, t + length):
            state.mul_(keep)
            state.addcmul_(k[i], v[i])
            torch.matmul(q[i].transpose(1, 2), state, out=out[i])
            if train:
                torch.matmul(state, do[i].transpose(1, 2), out=dq[i])
        final.append(state)
        if train:
            state = torch.zeros(hv, HEAD, HEAD, dtype=torch.float64, device=dev)
            if s["dfinal"] is not None:
                state.copy_(s["dfinal"][n])
            for i in range(t + length - 1, t - 1, -1):
                state.addcmul_(q[i], do[i])
                torch.matmul(state, v[i].transpose(1, 2), out=dk[i])
                torch.matmul(k[i].transpose(1, 2), state, out=dv[i])
                state.mul_(keep)
            ds0.append(state)
        t += length
    res = {"out": out[:, :, 0], "final": torch.stack(final)}
    if train:
        grouped = (case["hq"], g)
        res |= {"dq": (dq[..., 0] * s["scale"]).unflatten(1, grouped).sum(2),
                "dk": dk[..., 0].unflatten(1, grouped).sum(2), "dv": dv[:, :, 0]}
        if s["s0"] is not None:
            res["ds0"] = torch.stack(ds0)
    return res


def _exact_rope(case, s):
    """Pairs as complex numbers; the gradients through torch's own differentiation."""
    pos = s["positions"].double().reshape(-1, case["rows"])
    half, r = case["rotary"] // 2, case["rotary"]
    axis = s["pair_axis"].long() if s["pair_axis"] is not None else torch.zeros(half, dtype=torch.long, device=pos.device)
    angle = torch.einsum("ap,at->tp", (torch.arange(pos.shape[0], device=pos.device)[:, None] == axis).double()
                         * s["inv_freq"].double(), pos)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    res = {}
    for name in ("q", "k"):
        x = s[name].double().contiguous().requires_grad_(case["train"])
        w = s[name + "_weight"].double().requires_grad_(case["train"])
        n = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / HEAD + EPS) * w
        z = n[..., :r].unflatten(-1, (2, half)).transpose(-1, -2) if case["pairs"] == "halves" \
            else n[..., :r].unflatten(-1, (half, 2))
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
        z = z.transpose(-1, -2) if case["pairs"] == "halves" else z
        y = torch.cat([z.flatten(-2), n[..., r:]], -1)
        res[name] = y.detach()
        if case["train"]:
            res["d" + name], res["d" + name + "_weight"] = torch.autograd.grad(y, [x, w], s["d" + name].double())
    return res


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(case, s)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    g = case["hv"] // case["hq"]
    idx = s["slots"].long()
    old = s["state"].double()
    new = torch.einsum("h,nhij->nhij", torch.exp(s["decay"].double()), old.index_select(0, idx))
    new += torch.einsum("nhi,nhj->nhij", s["k"].double().repeat_interleave(g, 1), s["v"].double())
    out = torch.einsum("nhi,nhij->nhj", s["q"].double().repeat_interleave(g, 1), new) * s["scale"]
    return {"out": out, "state": old.index_copy(0, idx, new)}
