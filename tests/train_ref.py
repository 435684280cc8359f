"""The training operators from their definitions in 64 bits, each with a bound
on what 32-bit arithmetic may be off by, element by element.

The bounds count roundings and nothing else. u = 2^-24 is half a step of f32
relative to the value, U[dtype] the half step of an output's own rounding.

Recurrence. s_t is a sum of terms x_j a_{j+1} ... a_t. A decay costs expf's
error (2 steps = 4u) and the product or fma that takes it up to 2u more in a
scan that multiplies decays together first, and joins segments: 6u for every
factor, below EPS_REC = 8u. Summed over the terms that is E_t = a_t E_{t-1} +
EPS_REC M_t with the majorant M_t = a_t M_{t-1} + |x_t|. The same holds for ds
in reverse. dg = a s_{t-1} ds adds the errors of its factors, and a sum over
128 channels in f32 at most 128u of the sum of magnitudes.

Norms. A sum of D elements over threads that hold at most 16 each, then at
most 10 levels of shuffles: at most SUM = 32u of the sum of magnitudes
(with the scaling by 1/D and the products).
"""
import numpy as np
import torch

u = 2.0 ** -24
EPS_REC = 8 * u
SUM = 32 * u
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = 2.0 ** -126  # values below are flushed or lose bits in either type


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def assert_within(x, ref, bound, what):
    """Every element of x within `bound` of `ref`; where ref is not finite, x is the same."""
    x = x.detach().cpu().double().numpy()
    assert x.shape == ref.shape, f"{what}: shape {x.shape} for {ref.shape}"
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(x), np.isnan(ref)), f"{what}: NaN in other places"
    assert np.array_equal(x[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)]), f"{what}: infinities differ"
    off = np.abs(x[fine] - ref[fine]) / (bound[fine] + TINY)
    if off.size:
        worst = int(np.argmax(off))
        assert off[worst] <= 1.0, (f"{what}: off by {abs(x[fine][worst] - ref[fine][worst]):.3e} where "
                                   f"{bound[fine][worst]:.3e} is allowed (ref {ref[fine][worst]:.6e})")


def recurrence(x, g, h0, lens, dout=None, dfinal=None, dtype=None):
    """{name: (value, bound)} of out, final and, with dout, dx, dg, dh0; x [T, H, C], g [T, H] or [T, H, C], f64."""
    head = g.ndim == 2
    a = np.exp(g)
    a = np.broadcast_to(a[:, :, None], x.shape) if head else a
    half = U[dtype]
    n = len(lens)
    zero = np.zeros((n, *x.shape[1:]))
    h0 = zero if h0 is None else h0
    s, M, E = np.empty_like(x), np.empty_like(x), np.empty_like(x)
    before, Mb, Eb = np.empty_like(x), np.empty_like(x), np.empty_like(x)
    final, Mf, Ef = h0.copy(), np.abs(h0), np.zeros_like(zero)
    t = 0
    for i, length in enumerate(lens):
        for t in range(t, t + length):
            before[t], Mb[t], Eb[t] = final[i], Mf[i], Ef[i]
            final[i] = a[t] * final[i] + x[t]
            Mf[i] = a[t] * Mf[i] + np.abs(x[t])
            Ef[i] = a[t] * Ef[i] + EPS_REC * Mf[i]
            s[t], M[t], E[t] = final[i], Mf[i], Ef[i]
        t += length > 0
    res = {"out": (s, half * np.abs(s) + (1 + half) * E), "final": (final, Ef)}
    if dout is None:
        return res
    dfinal = zero if dfinal is None else dfinal
    ds, Ed, Md = np.empty_like(x), np.empty_like(x), np.empty_like(x)
    dh0, Eh = dfinal.copy(), np.zeros_like(zero)
    end = sum(lens)
    for i in reversed(range(n)):
        e, me, ee = dfinal[i], np.abs(dfinal[i]), np.zeros_like(dfinal[i])
        for t in range(end - 1, end - lens[i] - 1, -1):
            ds[t], Md[t] = dout[t] + e, np.abs(dout[t]) + me
            Ed[t] = ee + EPS_REC * Md[t]
            e, me, ee = a[t] * ds[t], a[t] * Md[t], a[t] * (Ed[t] + EPS_REC * Md[t])
        if lens[i]:
            dh0[i], Eh[i] = e, ee
        end -= lens[i]
    dg = a * before * ds
    Eg = a * (np.abs(before) * Ed + Eb * np.abs(ds) + Eb * Ed) + EPS_REC * np.abs(dg)
    if head:
        Eg = Eg.sum(-1) + 128 * u * np.abs(dg).sum(-1)
        dg = dg.sum(-1)
        bg = Eg
    else:
        bg = half * np.abs(dg) + (1 + half) * Eg
    res |= {"dx": (ds, half * np.abs(ds) + (1 + half) * Ed), "dg": (dg, bg), "dh0": (dh0, Eh)}
    return res


def layernorm(x, w, b, eps, dtype):
    """y, mean and rstd of [R, D] rows in f64, each (value, bound)."""
    half = U[dtype]
    D = x.shape[1]
    w = np.ones(D) if w is None else w
    b = np.zeros(D) if b is None else b
    mean = x.mean(1, keepdims=True)
    c = x - mean
    var = (c * c).mean(1, keepdims=True)
    rstd = 1 / np.sqrt(var + eps)
    e_mean = SUM * np.abs(x).mean(1, keepdims=True)
    # the squares about a mean that is off by d: var + d^2; each centred value rounds once more (2u of its square)
    e_c = e_mean + u * (np.abs(c) + e_mean)
    e_var = (SUM + 2 * u) * (var + 2 * e_mean ** 2) + e_mean ** 2 + 2 * u * np.sqrt(var) * e_mean
    e_rstd = rstd * (e_var / (var + eps) * 0.5 + 4 * u) * 1.01
    y = c * rstd * w + b
    e_y = np.abs(w) * (rstd * e_c + np.abs(c) * e_rstd + e_c * e_rstd + 2 * u * np.abs(c) * rstd) + 2 * u * (
        np.abs(c * rstd * w) + np.abs(y))
    return {"y": (y, half * np.abs(y) + (1 + half) * e_y), "mean": (mean[:, 0], e_mean[:, 0]),
            "rstd": (rstd[:, 0], e_rstd[:, 0])}


def layernorm_bwd(dy, x, mean, rstd, w, dtype):
    """dx, dweight, dbias from the f32 mean and rstd that the call is given."""
    half = U[dtype]
    R, D = x.shape
    w = np.ones(D) if w is None else w
    xhat = (x - mean[:, None]) * rstd[:, None]
    e_x = 2 * u * np.abs(xhat)  # one subtraction of given values, one product
    g = dy * w
    s1, s2 = g.mean(1, keepdims=True), (g * xhat).mean(1, keepdims=True)
    m1, m2 = np.abs(g).mean(1, keepdims=True), np.abs(g * xhat).mean(1, keepdims=True)
    e1, e2 = (SUM + u) * m1, (SUM + 4 * u) * m2
    r = rstd[:, None]
    dx = r * (g - s1 - xhat * s2)
    e_dx = r * (e1 + np.abs(xhat) * e2 + e_x * (np.abs(s2) + e2) + 6 * u * (np.abs(g) + np.abs(s1) + np.abs(xhat * s2)))
    # rows: at most R additions in any order
    n = (R + 8) * u
    dw, db = (dy * xhat).sum(0), dy.sum(0)
    return {"dx": (dx, half * np.abs(dx) + (1 + half) * e_dx), "dweight": (dw, n * np.abs(dy * xhat).sum(0)),
            "dbias": (db, n * np.abs(dy).sum(0))}


def gate_bwd(dy, o, z, w, eps, dtype):
    """do, dz, dweight of the output gate on [rows, 128] f64."""
    half = U[dtype]
    C = o.shape[1]
    r = 1 / np.sqrt((o * o).mean(1, keepdims=True) + eps)
    n = o * r
    sig = 1 / (1 + np.exp(-z))
    silu = z * sig
    up = dy * w * silu
    m = (up * n).mean(1, keepdims=True)
    do = r * (up - n * m)
    # r: SUM of the squares (halved by the root) and 4u; sig: expf 4u, add and quotient 3u; products: u each
    e_r = SUM / 2 + 4 * u
    e_up = 12 * u
    e_m = (SUM + e_r + e_up + 2 * u) * np.abs(up * n).mean(1, keepdims=True)
    e_do = np.abs(do) * e_r + r * (np.abs(up) * e_up + np.abs(n) * e_m + np.abs(n * m) * e_r
                                   + 3 * u * (np.abs(up) + np.abs(n * m)))
    dsilu = sig + silu * (1 - sig)
    dz = dy * n * w * dsilu
    # 1 - sig is off by sig's own error (8u) and a rounding, times |silu|
    e_ds = 8 * u * np.abs(sig) + np.abs(silu) * (10 * u + 10 * u * np.abs(1 - sig)) + 2 * u * np.abs(dsilu)
    e_dz = np.abs(dy * n * w) * e_ds + np.abs(dz) * (e_r + 4 * u)
    t = dy * n * silu
    e_dw = (np.abs(t) * (e_r + 12 * u + (o.shape[0] + 4) * u)).sum(0)
    return {"do": (do, half * np.abs(do) + (1 + half) * e_do), "dz": (dz, half * np.abs(dz) + (1 + half) * e_dz),
            "dweight": (t.sum(0), e_dw)}
