"""Linear attention over long sequences, a few heads at a time: the definition in 64 bits by chunks on the inputs' own
device, and normwise bounds, which see errors far below those that a bound on every element allows.

u = 2^-24. Roundings of random sign add up as the square root of their number:

* f32 results and all states: fewer than 2^14 roundings in a row (a term's own sums, and one for every block of 32 or 128
  tokens that it ages by), 2^7 u of the norm. The tensor cores may cut instead of rounding, 2 u a step at most, all to one
  side: 32 steps of a chunk's sum are 64 u.
* bf16 outputs: the decayed scores, the state as an operand and the output are rounded, each by 2^-8 of a value at most. A
  significand anywhere in [1, 2) has 2^-8 / sqrt(3) times the root mean square of 1 / significand, 0.736: 1.66e-3. The
  first two are of different parts of the output: together 1.66e-3 of its norm, with its own rounding 2.35e-3. The bound is
  2^-8 = 3.9e-3.
"""
import torch

u = 2.0 ** -24
F32_NORM = 2 ** 7 * u
NORM = {torch.float32: F32_NORM, torch.bfloat16: 2.0 ** -8}


def walk(a, b, c, decay, state, against=False, entry=True, chunk=128):
    """out_t = a_t S, S = lambda S + b_t^T c_t over [T, 128] of one head in 64 bits, against time if asked for; with
    ``entry`` the state is decayed before the first token too. Returns out and the last state."""
    if against:
        a, b, c = a.flip(0), b.flip(0), c.flip(0)
    S, out = state.double().clone(), torch.empty(c.shape, dtype=torch.float64, device=c.device)
    decay = float(decay)
    for t in range(0, len(c), chunk):
        x, y, z = (v[t:t + chunk].double() for v in (a, b, c))
        n = torch.arange(len(x), device=c.device, dtype=torch.float64)
        first = 0 if t == 0 and not entry else 1
        power = lambda e: torch.exp(decay * e)
        age = n[:, None] - n
        inside = torch.where(age >= 0, power(age.clamp(min=0)), 0.0)
        out[t:t + chunk] = ((x @ y.T) * inside) @ z + (x @ S) * power(n + first)[:, None]
        S = S * power(n[-1] + first) + (y * power(n[-1] - n)[:, None]).T @ z
    return (out.flip(0) if against else out), S


def sequence(d, q, k, v, dout, s0, df, decay):
    """{name: tensor} of one sequence: one query and key head [T, 128] and its value heads [T, g, 128]; s0 and df
    [g, 128, 128] or None."""
    scale, g = d["scale"], v.shape[1]
    zero = torch.zeros(g, 128, 128, dtype=torch.float64, device=q.device)
    s0, df = zero if s0 is None else s0, zero if df is None else df
    res = {"out": [], "final": [], "dv": [], "ds0": []}
    dq = dk = 0.0
    for h in range(g):
        out, final = walk(q, k, v[:, h], decay[h], s0[h])
        res["out"].append(out * scale)
        res["final"].append(final)
        dq = dq + walk(dout[:, h], v[:, h], k, decay[h], s0[h].T)[0] * scale
        dv, last = walk(k, q.double() * scale, dout[:, h], decay[h], df[h], True, False)
        res["dv"].append(dv)
        res["ds0"].append(last * torch.exp(decay[h].double()))
        dk = dk + walk(v[:, h], dout[:, h].double() * scale, q, decay[h], df[h].T, True, False)[0]
    res = {n: torch.stack(x, 1 if n in ("out", "dv") else 0) for n, x in res.items()}
    return res | {"dq": dq, "dk": dk}


def assert_near(x, ref, bound, what):
    assert x.shape == ref.shape and torch.isfinite(x).all(), what
    off = ((x.double() - ref).norm() / ref.norm()).item()
    assert off <= bound, f"{what}: {off:.3e} of the norm where {bound:.3e} is allowed"


def compare(got, d, lens, dtype, heads):
    """Every sequence and each value head of the query and key heads ``heads``, normwise."""
    g = d["v"].shape[1] // d["q"].shape[1]
    t = 0
    for n, length in enumerate(lens):
        r, t = slice(t, t + length), t + length
        for h in heads:
            vh = slice(h * g, (h + 1) * g)
            state = lambda name: None if d[name] is None else d[name][n, vh]
            ref = sequence(d, d["q"][r, h], d["k"][r, h], d["v"][r, vh], d["dout"][r, vh], state("s0"), state("dfinal"),
                           d["decay"][vh])
            for name, x in got.items():
                if x is None:
                    continue
                what = f"{name} of sequence {n}, head {h}"
                if name in ("dq", "dk"):
                    assert_near(x[r, h], ref[name], NORM[dtype], what)
                elif name in ("final", "ds0"):
                    for i in range(g):
                        assert_near(x[n, h * g + i], ref[name][i], F32_NORM, what)
                else:
                    for i in range(g):
                        assert_near(x[r, h * g + i], ref[name][:, i], NORM[dtype], what)
