"""Host-side checks of the training operators, without a GPU: refusals of the
C ABI and of the binding, size queries, and the references of the GPU tests
(their gradients against differences)."""
import ctypes

import numpy as np
import pytest
import torch

import train_ref as R
from gated_deltanet_chunked_gb300 import gdn

FAKE = 1 << 20  # 16-byte aligned, never dereferenced by the checks
P = ctypes.c_void_p


def problem(**kw):
    base = dict(batch=1, seqlen=0, num_seqs=2, total_tokens=256, hq=1, hv=4, dk=128, dv=128,
                io_dtype=gdn.GDN_DT_BF16, flags=0, num_state_slots=0)
    return gdn.GdnProblem(**{**base, **kw})


def ptr(v):
    return None if v is None else P(v)


def fwd(p, x=FAKE, g=FAKE, s0=None, cu=FAKE, out=2 * FAKE, fin=None, states=None):
    return gdn.load().gdn_linear_recurrence(ctypes.byref(p), ptr(x), ptr(g), ptr(s0), ptr(cu), ptr(out), ptr(fin),
                                            ptr(states), None)


def bwd(p, dout=FAKE, x=2 * FAKE, g=3 * FAKE, states=FAKE, s0=None, dfin=None, cu=FAKE, dx=4 * FAKE, dg=5 * FAKE,
        dinit=None):
    return gdn.load().gdn_linear_recurrence_bwd(ctypes.byref(p), ptr(dout), ptr(x), ptr(g), ptr(states), ptr(s0),
                                                ptr(dfin), ptr(cu), ptr(dx), ptr(dg), ptr(dinit), None)


CHANNEL = gdn.GDN_FLAG_GATE_CHANNEL


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("kw,code", [
    (dict(hv=0), gdn.GDN_EINVAL),
    (dict(dv=0), gdn.GDN_EINVAL),
    (dict(dv=64), gdn.GDN_EUNSUPPORTED),
    (dict(io_dtype=3), gdn.GDN_EINVAL),
    (dict(num_seqs=0), gdn.GDN_EINVAL),
    (dict(total_tokens=-1), gdn.GDN_EINVAL),
    (dict(flags=2), gdn.GDN_EUNSUPPORTED),
    (dict(flags=CHANNEL | 4), gdn.GDN_EUNSUPPORTED),
    (dict(total_tokens=(1 << 31) - 1), gdn.GDN_EINVAL),
])
def test_recurrence_rejects_bad_problems(call, kw, code):
    assert call(problem(**kw)) == code


def test_recurrence_rejects_bad_pointers():
    for kw in (dict(x=None), dict(g=None), dict(out=None), dict(x=FAKE + 4), dict(out=FAKE + 8), dict(g=FAKE + 2),
               dict(s0=FAKE + 4), dict(cu=FAKE + 2), dict(fin=FAKE + 8), dict(states=FAKE + 4), dict(out=FAKE),
               dict(s0=FAKE, fin=FAKE)):
        assert fwd(problem(), **kw) == gdn.GDN_EINVAL, kw
    assert fwd(problem(flags=CHANNEL), g=FAKE + 4) == gdn.GDN_EINVAL  # per channel: 16 bytes
    assert fwd(problem(), cu=None) == gdn.GDN_EINVAL                   # dense: batch != num_seqs
    assert fwd(problem(batch=2, seqlen=100), cu=None) == gdn.GDN_EINVAL
    for kw in (dict(dout=None), dict(x=None), dict(g=None), dict(states=None), dict(dx=None), dict(dg=None),
               dict(dout=FAKE + 4), dict(dx=4 * FAKE + 8), dict(dg=FAKE + 2), dict(dfin=FAKE + 4),
               dict(dinit=FAKE + 8), dict(dx=FAKE), dict(dx=2 * FAKE), dict(dg=3 * FAKE), dict(dg=4 * FAKE),
               dict(dfin=FAKE, dinit=FAKE)):
        assert bwd(problem(), **kw) == gdn.GDN_EINVAL, kw


def test_states_size():
    size = lambda **kw: int(gdn.load().gdn_linear_recurrence_states_size(ctypes.byref(problem(**kw))))
    assert size(total_tokens=0) == 0
    assert size(total_tokens=1) == size(total_tokens=64) == 4 * 128 * 4
    assert size(total_tokens=65) == 2 * 4 * 128 * 4
    assert size(dv=64) == 0


def test_recurrence_step_rejects_bad_arguments():
    def step(x=FAKE, g=FAKE, st=2 * FAKE, idx=None, out=3 * FAKE, **kw):
        p = problem(**{**dict(batch=4, seqlen=1, num_seqs=4, total_tokens=4, num_state_slots=4), **kw})
        return gdn.load().gdn_linear_recurrence_step(ctypes.byref(p), ptr(x), ptr(g), ptr(st), ptr(idx), ptr(out),
                                                     None)

    for kw in (dict(total_tokens=5), dict(num_state_slots=3), dict(num_state_slots=-1, idx=FAKE), dict(hv=0),
               dict(x=None), dict(g=None), dict(st=None), dict(out=None), dict(x=FAKE + 4), dict(st=FAKE + 4),
               dict(out=FAKE + 8), dict(idx=FAKE + 2), dict(out=2 * FAKE), dict(io_dtype=2),
               dict(flags=CHANNEL, g=FAKE + 8)):
        assert step(**kw) == gdn.GDN_EINVAL, kw
    assert step(dv=64) == gdn.GDN_EUNSUPPORTED
    assert step(flags=1) == gdn.GDN_EUNSUPPORTED


def test_layernorm_rejects_bad_arguments():
    lib = gdn.load()

    def norm(x=FAKE, w=FAKE, b=FAKE, eps=1e-5, y=FAKE, mean=None, rstd=None, **kw):
        p = problem(**{**dict(dv=100), **kw})
        return lib.gdn_layernorm(ctypes.byref(p), ptr(x), ptr(w), ptr(b), ctypes.c_float(eps), ptr(y), ptr(mean),
                                 ptr(rstd), None)

    for kw in (dict(x=None), dict(y=None), dict(x=FAKE + 2), dict(w=FAKE + 4), dict(b=FAKE + 8), dict(eps=-1.0),
               dict(eps=float("nan")), dict(mean=FAKE + 2), dict(rstd=FAKE + 1), dict(dv=0), dict(io_dtype=5),
               dict(total_tokens=-1)):
        assert norm(**kw) == gdn.GDN_EINVAL, kw
    assert norm(dv=16385) == gdn.GDN_EUNSUPPORTED

    def back(dy=FAKE, x=FAKE, mean=FAKE, rstd=FAKE, w=None, dx=FAKE, dw=FAKE, db=FAKE, ws=FAKE, nbytes=None, **kw):
        p = problem(**{**dict(dv=100), **kw})
        need = lib.gdn_layernorm_bwd_workspace_size(ctypes.byref(p))
        return lib.gdn_layernorm_bwd(ctypes.byref(p), ptr(dy), ptr(x), ptr(mean), ptr(rstd), ptr(w), ptr(dx), ptr(dw),
                                     ptr(db), ptr(ws), ctypes.c_size_t(need if nbytes is None else nbytes), None)

    for kw in (dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(dx=None), dict(ws=None),
               dict(ws=FAKE + 16), dict(nbytes=255), dict(dw=FAKE + 4), dict(db=FAKE + 8), dict(w=FAKE + 4),
               dict(dy=FAKE + 2), dict(dx=FAKE + 8), dict(mean=FAKE + 2), dict(dv=-1)):
        assert back(**kw) == gdn.GDN_EINVAL, kw
    assert back(dv=20000) == gdn.GDN_EUNSUPPORTED


def test_outputs_in_one_place_are_refused():
    lib, p = gdn.load(), ctypes.byref(problem(dv=100))
    a, b = ptr(FAKE), ptr(2 * FAKE)
    assert lib.gdn_layernorm(p, a, a, a, ctypes.c_float(1e-5), a, b, b, None) == gdn.GDN_EINVAL
    assert lib.gdn_layernorm_bwd(p, a, a, a, a, a, a, b, b, a, ctypes.c_size_t(1 << 30), None) == gdn.GDN_EINVAL
    assert fwd(problem(flags=CHANNEL), g=2 * FAKE, out=2 * FAKE) == gdn.GDN_EINVAL


def test_layernorm_workspace_size_covers_every_partial_row():
    size = lambda r, d: int(gdn.load().gdn_layernorm_bwd_workspace_size(ctypes.byref(problem(total_tokens=r, dv=d))))
    assert size(1, 100) >= 2 * 100 * 4 and size(1, 100) % 256 == 0
    assert size(10 ** 6, 4096) == size(10 ** 7, 4096)  # bounded: it does not grow with the rows
    assert size(10 ** 6, 4096) <= 2 * 1216 * 4096 * 4
    assert size(0, 100) == 0 and size(5, 20000) == 0


def test_gate_backward_rejects_bad_arguments():
    lib = gdn.load()

    def back(dy=FAKE, o=FAKE, z=FAKE, w=FAKE, eps=1e-6, do=FAKE, dz=2 * FAKE, dw=FAKE, ws=FAKE, nbytes=None, **kw):
        p = problem(**kw)
        need = lib.gdn_gated_rmsnorm_bwd_workspace_size(ctypes.byref(p))
        return lib.gdn_gated_rmsnorm_bwd(ctypes.byref(p), ptr(dy), ptr(o), ptr(z), ptr(w), ctypes.c_float(eps),
                                         ptr(do), ptr(dz), ptr(dw), ptr(ws),
                                         ctypes.c_size_t(need if nbytes is None else nbytes), None)

    for kw in (dict(dy=None), dict(o=None), dict(z=None), dict(w=None), dict(do=None), dict(dz=None), dict(dz=FAKE),
               dict(dy=FAKE + 2), dict(w=FAKE + 4), dict(dw=FAKE + 4), dict(ws=None), dict(ws=FAKE + 64),
               dict(nbytes=0), dict(eps=-1.0), dict(eps=float("nan")), dict(hv=0), dict(dv=0), dict(io_dtype=9)):
        assert back(**kw) == gdn.GDN_EINVAL, kw
    assert back(dv=64) == gdn.GDN_EUNSUPPORTED


def test_binding_refuses_wrong_tensors():
    bf = torch.bfloat16
    x, gh = torch.zeros(70, 2, 128, dtype=bf), torch.zeros(70, 2)
    cu, st = torch.tensor([0, 30, 70], dtype=torch.int32), torch.zeros(2, 2, 128)
    rec, back = gdn.gdn_linear_recurrence, gdn.gdn_linear_recurrence_bwd
    bad = [
        lambda: rec(x, gh),                                        # packed without offsets
        lambda: rec(x, gh.to(bf), cu_seqlens=cu),                  # gates per head are f32
        lambda: rec(x, x.float(), cu_seqlens=cu),                  # gates per channel have x's type
        lambda: rec(x, gh[:, :1].contiguous(), cu_seqlens=cu),
        lambda: rec(x, gh, cu_seqlens=cu.long()),
        lambda: rec(x, gh, cu_seqlens=cu, initial_state=st[:1]),
        lambda: rec(x, gh, cu_seqlens=cu, final_state=st.to(bf)),
        lambda: rec(x, gh, cu_seqlens=cu, out=x[:69]),
        lambda: rec(x, gh, cu_seqlens=cu, states=torch.zeros(1, 2, 128)),
        lambda: rec(x.half(), gh, cu_seqlens=cu),
        lambda: back(x, x, gh, None, cu_seqlens=cu),
        lambda: back(x.float(), x, gh, st, cu_seqlens=cu),
        lambda: back(x, x, gh, st[:1], cu_seqlens=cu),
        lambda: back(x, x, gh, st, cu_seqlens=cu, dg=x),
        lambda: back(x, x, gh, st, cu_seqlens=cu, dfinal_state=st[:, :1]),
        lambda: gdn.gdn_linear_recurrence_step(x, gh, st.to(bf)),
        lambda: gdn.gdn_linear_recurrence_step(x, gh, st[..., :64].contiguous()),
        lambda: gdn.gdn_linear_recurrence_step(x, gh, st, state_indices=torch.zeros(3, dtype=torch.int32)),
        lambda: gdn.gdn_layernorm(x, weight=torch.ones(64)),
        lambda: gdn.gdn_layernorm(x, weight=torch.ones(128, dtype=bf)),
        lambda: gdn.gdn_layernorm(x, out=x.float()),
        lambda: gdn.gdn_layernorm(torch.zeros(3, 0)),
        lambda: gdn.gdn_layernorm(torch.tensor(1.0)),
        lambda: gdn.gdn_layernorm_bwd(x, x, gh[:, :1], gh),
        lambda: gdn.gdn_layernorm_bwd(x, x, gh, gh.to(bf)),
        lambda: gdn.gdn_gated_rmsnorm_bwd(x, x.float(), x, torch.ones(128), 1e-6),
        lambda: gdn.gdn_gated_rmsnorm_bwd(x, x, x, torch.ones(64), 1e-6),
        lambda: gdn.gdn_gated_rmsnorm_bwd(x, x, x, torch.ones(128), 1e-6, dz=x[:1]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    ok = [
        lambda: rec(x, gh, cu_seqlens=cu),
        lambda: back(x, x, gh, st, cu_seqlens=cu),
        lambda: gdn.gdn_linear_recurrence_step(x, gh, torch.zeros(70, 2, 128)),
        lambda: gdn.gdn_layernorm(x),
        lambda: gdn.gdn_layernorm_bwd(x, x, gh, gh),
        lambda: gdn.gdn_gated_rmsnorm_bwd(x, x, x, torch.ones(128), 1e-6),
    ]
    for call in ok:  # right but for the device
        with pytest.raises(ValueError, match="CUDA"):
            call()


# ---- the references' gradients, against central differences -------------------

STEP = 1e-5


def check_gradient(loss, value, grad, rng, what, picks=12):
    """A smooth function's central difference is off by about STEP^2 times its third derivative and by the loss's
    rounding over STEP: both below 1e-7 of a gradient of order 1 to 10 here."""
    flat, g = value.reshape(-1), grad.reshape(-1)
    for i in rng.choice(flat.size, min(picks, flat.size), replace=False):
        keep = flat[i]
        flat[i] = keep + STEP
        up = loss()
        flat[i] = keep - STEP
        down = loss()
        flat[i] = keep
        diff = (up - down) / (2 * STEP)
        assert abs(diff - g[i]) <= 1e-6 * max(1.0, abs(g[i])), (what, i, diff, g[i])


@pytest.mark.parametrize("head", [True, False])
def test_recurrence_reference_gradients(head):
    rng = np.random.default_rng(0)
    lens, hv, C = [5, 0, 1, 9], 2, 6
    T = sum(lens)
    x, dout = rng.standard_normal((2, T, hv, C))
    g = -rng.random((T, hv) if head else (T, hv, C))
    h0, dfinal = rng.standard_normal((2, len(lens), hv, C))
    ref = lambda: R.recurrence(x, g, h0, lens, dout, dfinal, torch.float32)

    def loss():
        r = R.recurrence(x, g, h0, lens, dtype=torch.float32)
        return (r["out"][0] * dout).sum() + (r["final"][0] * dfinal).sum()

    r = ref()
    for name, v in (("dx", x), ("dg", g), ("dh0", h0)):
        check_gradient(loss, v, r[name][0], rng, name)


def test_layernorm_reference_gradients():
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((2, 4, 7))
    w, b = rng.standard_normal((2, 7))

    def loss():
        return (R.layernorm(x, w, b, 1e-3, torch.float32)["y"][0] * dy).sum()

    f = R.layernorm(x, w, b, 1e-3, torch.float32)
    r = R.layernorm_bwd(dy, x, f["mean"][0], f["rstd"][0], w, torch.float32)
    for name, v in (("dx", x), ("dweight", w), ("dbias", b)):
        check_gradient(loss, v, r[name][0], rng, name)


def test_gate_reference_gradients():
    import oracle

    rng = np.random.default_rng(2)
    o, z, dy = rng.standard_normal((3, 3, 128))
    w = rng.standard_normal(128)

    def loss():
        n = o / np.sqrt((o * o).mean(1, keepdims=True) + 1e-3)
        return (n * w * z / (1 + np.exp(-z)) * dy).sum()

    r = R.gate_bwd(dy, o, z, w, 1e-3, torch.float32)
    for name, v in (("do", o), ("dz", z), ("dweight", w)):
        check_gradient(loss, v, r[name][0], rng, name)
    # the same function as the forward pass's oracle (f32 inputs there)
    o32, z32, w32 = (torch.from_numpy(v).float() for v in (o[:, None], z[:, None], w))
    y = oracle.gated_rmsnorm(o32, z32, w32, 1e-3).reshape(3, 128)
    n = o / np.sqrt((o * o).mean(1, keepdims=True) + 1e-3)
    assert np.allclose(y, n * w * z / (1 + np.exp(-z)), rtol=1e-5, atol=1e-6)
