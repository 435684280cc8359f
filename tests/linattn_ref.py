"""Linear attention with a decay for each head, its decode step, and the norm
and rotation of queries and keys, from their definitions in 64 bits, each with a
bound on what the kernels' arithmetic may be off by, element by element.

u = 2^-24 is half a step of f32 relative to the value, H[dtype] the half step of
an output's own rounding. M is the same sum taken over magnitudes (a majorant).

Attention. An output is a sum over earlier tokens j of lambda^(i-j) (a_i b_j) c_j.
f32: a product a_i b_j has 128 terms in one chain at most, the state's product
too, a block of 32 tokens another 33; a decay is off by 5u, and taken once for
each block of 32 that a term's age spans (two roundings more each): with at most
100 blocks 128 + 128 + 33 + 7 * 100 < 1024, so 1024 u M.
bf16: the decayed scores and the state, as an operand, are rounded to bf16:
2^-8 M together, as each term passes one of the two. What else there is is f32
and counted as above; the tensor cores add 16 products and the accumulator to a
common exponent (17u a step at most, 64 steps a chunk of 128 tokens), and a state
is kept by a decay every chunk (8u): 2048 u M for 30 chunks. States are not
rounded: theirs alone.

Step. lambda S + k v: three roundings and the decay's 5u; o sums 128 of them.

Norm and rotation. sum x^2 and its root: 16u + 4u, two products: 24u of n. The
angle is off by 2^-22 = 4u, sine and cosine by 4u more: 8u (|n_a| + |n_b|), and
two roundings of the sum. Backward: the same turn, a mean over 128 channels
(32u) of magnitudes, and the root's 20u twice: 100u of the majorant. Sums over
rows: one chain of at most 128 rows a thread, then 16 + 456 partial sums in
chains and trees: 700u.
"""
import numpy as np
import torch

u = 2.0 ** -24
H = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = 2.0 ** -120


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def assert_within(x, ref, bound, what):
    x = x.detach().cpu().double().numpy()
    assert x.shape == ref.shape, f"{what}: shape {x.shape} for {ref.shape}"
    assert np.isfinite(x).all(), f"{what}: not finite"
    if x.size:
        off = np.abs(x - ref) / (bound + TINY)
        w = np.unravel_index(int(np.argmax(off)), off.shape)
        assert off[w] <= 1.0, f"{what} at {w}: off by {abs(x[w] - ref[w]):.3e} where {bound[w]:.3e} is allowed (ref {ref[w]:.6e})"


def _walk(a, b, c, decay, state, against, entry):
    """out_t = a_t S, S = lambda S + b_t^T c_t over the tokens of one sequence, in time or against it; with ``entry``
    the state is decayed before the first token too. Returns out, its majorant, the last state and its majorant."""
    keep = np.exp(decay)[:, None, None]
    S, M = state.copy(), np.abs(state)
    out, mout = np.empty_like(c), np.empty_like(c)
    order = range(len(c) - 1, -1, -1) if against else range(len(c))
    for n, t in enumerate(order):
        if n or entry:
            S, M = keep * S, keep * M
        S = S + b[t][:, :, None] * c[t][:, None, :]
        M = M + np.abs(b[t])[:, :, None] * np.abs(c[t])[:, None, :]
        out[t] = np.einsum("hi,hij->hj", a[t], S)
        mout[t] = np.einsum("hi,hij->hj", np.abs(a[t]), M)
    return out, mout, S, M


def attention(d, lens, dtype):
    """{name: (value, bound)} of out, final, dq, dk, dv and ds0; d holds q, k, v, dout, s0, dfinal, decay, scale."""
    q, k, v, do, decay, scale = (f64(d[n]) if n != "scale" else d[n] for n in ("q", "k", "v", "dout", "decay", "scale"))
    T, hq, hv, N = len(q), q.shape[1], v.shape[1], len(lens)
    g = hv // hq
    qe, ke = np.repeat(q, g, 1), np.repeat(k, g, 1)
    zero = np.zeros((N, hv, 128, 128))
    s0 = zero if d["s0"] is None else f64(d["s0"])
    df = zero if d["dfinal"] is None else f64(d["dfinal"])
    flip = lambda s: s.transpose(0, 2, 1)
    full = {n: (np.zeros((T, hv, 128)), np.zeros((T, hv, 128))) for n in ("out", "dq", "dk", "dv")}
    fin, ds0 = (s0.copy(), np.abs(s0)), (df.copy(), np.abs(df))
    keep = np.exp(decay)[:, None, None]
    t = 0
    for n, length in enumerate(lens):
        r = slice(t, t + length)
        t += length
        if not length:
            continue
        for name, a, b, c, s, against in (("out", qe, ke, v, s0[n], False), ("dq", do, v, ke, flip(s0[n]), False),
                                          ("dv", ke, qe * scale, do, df[n], True),
                                          ("dk", v, do * scale, qe, flip(df[n]), True)):
            x, m, S, M = _walk(a[r], b[r], c[r], decay, s, against, not against)
            f = scale if not against else 1.0
            full[name][0][r], full[name][1][r] = x * f, m * f
            if name == "out":
                fin[0][n], fin[1][n] = S, M
            if name == "dv":
                ds0[0][n], ds0[1][n] = keep * S, keep * M
    half = H[dtype]
    res = {}
    for name, (x, m) in full.items():
        if name in ("dq", "dk"):
            x, m = (z.reshape(T, hq, g, 128).sum(2) for z in (x, m))
        err = (1024 * u if dtype == torch.float32 else half * (1 + half) + 2048 * u) * m
        res[name] = (x, err + half * (np.abs(x) + err))
    state = (1024 if dtype == torch.float32 else 2048) * u
    res["final"] = (fin[0], state * fin[1])
    res["ds0"] = (ds0[0], state * ds0[1])
    return res


def step(d, dtype, state_dtype):
    """(out, bound), (state rows, bound) for the sequences in order; d holds q, k, v, decay, scale, state (their rows)."""
    q, k, v, decay, S = (f64(d[n]) for n in ("q", "k", "v", "decay", "state"))
    g = v.shape[1] // q.shape[1]
    q, k = np.repeat(q, g, 1), np.repeat(k, g, 1)
    keep = np.exp(decay)[:, None, None]
    kv = k[..., None] * v[:, :, None, :]
    new, mag = keep * S + kv, keep * np.abs(S) + np.abs(kv)
    out = d["scale"] * np.einsum("nhi,nhij->nhj", q, new)
    m = abs(d["scale"]) * np.einsum("nhi,nhij->nhj", np.abs(q), mag)
    half, hs = H[dtype], H[state_dtype]
    return (out, half * np.abs(out) + (1 + half) * 140 * u * m), (new, hs * np.abs(new) + 9 * u * mag)


def _pairs(x, r, interleaved):
    return (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])


def _join(a, b, x, r, interleaved):
    y = x.copy()
    p, q = _pairs(y, r, interleaved)
    p[...], q[...] = a, b
    return y


def rope(x, w, dy, inv_freq, positions, pair_axis, interleaved, eps, dtype):
    """{y, dx, dw: (value, bound)} of one of q and k [T, H, 128]; w None: 1."""
    x, dy = f64(x), f64(dy)
    w = np.ones(128) if w is None else f64(w)
    f, pos = f64(inv_freq), positions.cpu().numpy().astype(np.float64).reshape(-1, len(x))
    r = 2 * len(f)
    axis = np.zeros(len(f), int) if pair_axis is None else pair_axis.cpu().numpy()
    # angles in 80 bits: a position of 31 bits leaves a double 22 behind the point
    angle = pos[axis].T.astype(np.longdouble) * f.astype(np.longdouble)
    cos, sin = (fn(angle).astype(np.float64)[:, None, :] for fn in (np.cos, np.sin))
    rstd = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xhat = x * rstd
    n = xhat * w
    half = H[dtype]
    a, b = _pairs(n, r, interleaved)
    y = _join(a * cos - b * sin, a * sin + b * cos, n, r, interleaved)
    both = np.abs(a) + np.abs(b)
    err = 24 * u * np.abs(n)
    err = _join(34 * u * both, 34 * u * both, err, r, interleaved)
    res = {"y": (y, err + half * (np.abs(y) + err))}
    a, b = _pairs(dy, r, interleaved)
    dn = _join(a * cos + b * sin, b * cos - a * sin, dy, r, interleaved)
    both = np.abs(a) + np.abs(b)
    mag = _join(both, both, np.abs(dy), r, interleaved)
    uu, mu = dn * w, mag * np.abs(w)
    dx = rstd * (uu - xhat * (uu * xhat).mean(-1, keepdims=True))
    err = 100 * u * rstd * (mu + np.abs(xhat) * (mu * np.abs(xhat)).mean(-1, keepdims=True))
    res["dx"] = (dx, err + half * (np.abs(dx) + err))
    res["dw"] = ((dn * xhat).sum((0, 1)), 700 * u * (mag * np.abs(xhat)).sum((0, 1)))
    return res
