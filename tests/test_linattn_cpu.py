"""Host-side checks of linear attention, its decode step and the norm and rotation of queries and keys, without a GPU:
refusals of the C ABI and of the binding, size queries, and the GPU tests' references against each other."""
import ctypes

import numpy as np
import pytest
import torch

import linattn_ref as R
from gated_deltanet_chunked_gb300 import gdn
from test_training_overlap_cpu import check, spread
from test_training_cpu import FAKE, problem, ptr

NO_GPU = not torch.cuda.is_available()
T, HQ, HV, N = 96, 2, 4, 3
KW = dict(total_tokens=T, num_seqs=N, hq=HQ, hv=HV)
QK, ROWS, STATES, HEADS, CU = T * HQ * 128 * 2, T * HV * 128 * 2, N * HV * 128 * 128 * 4, HV * 4, (N + 1) * 4
f = ctypes.c_float


def size(fn, **kw):
    return int(getattr(gdn.load(), fn)(ctypes.byref(problem(**{**KW, **kw}))))


def fwd(q=FAKE, k=FAKE, v=FAKE, dec=FAKE, s0=None, cu=FAKE, out=2 * FAKE, fin=None, ws=64 * FAKE, nbytes=None, **kw):
    need = size("gdn_linear_attention_workspace_size", **kw) if nbytes is None else nbytes
    return gdn.load().gdn_linear_attention(ctypes.byref(problem(**{**KW, **kw})), ptr(q), ptr(k), ptr(v), ptr(dec),
                                           f(0.1), ptr(s0), ptr(cu), ptr(out), ptr(fin), ptr(ws),
                                           ctypes.c_size_t(need), None)


def bwd(dout=FAKE, q=FAKE, k=FAKE, v=FAKE, dec=FAKE, s0=None, df=None, cu=FAKE, gq=2 * FAKE, gk=3 * FAKE, gv=4 * FAKE,
        d0=None, ws=64 * FAKE, nbytes=None, **kw):
    need = size("gdn_linear_attention_bwd_workspace_size", **kw) if nbytes is None else nbytes
    return gdn.load().gdn_linear_attention_bwd(ctypes.byref(problem(**{**KW, **kw})), ptr(dout), ptr(q), ptr(k), ptr(v),
                                               ptr(dec), f(0.1), ptr(s0), ptr(df), ptr(cu), ptr(gq), ptr(gk), ptr(gv),
                                               ptr(d0), ptr(ws), ctypes.c_size_t(need), None)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("kw,code", [
    (dict(hv=0), gdn.GDN_EINVAL), (dict(hq=0), gdn.GDN_EINVAL), (dict(hq=3), gdn.GDN_EINVAL),
    (dict(hq=8), gdn.GDN_EINVAL), (dict(dv=64), gdn.GDN_EUNSUPPORTED), (dict(dk=256), gdn.GDN_EUNSUPPORTED),
    (dict(io_dtype=2), gdn.GDN_EINVAL), (dict(num_seqs=0), gdn.GDN_EINVAL), (dict(total_tokens=-1), gdn.GDN_EINVAL),
    (dict(flags=4), gdn.GDN_EUNSUPPORTED), (dict(total_tokens=(1 << 31) - 1), gdn.GDN_EINVAL),
    (dict(hv=1 << 20, hq=1, total_tokens=1 << 20), gdn.GDN_EINVAL),
])
def test_bad_problems(call, kw, code):
    assert call(nbytes=1 << 40, **kw) == code


def test_bad_pointers():
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(dec=None), dict(out=None), dict(ws=None),
               dict(q=FAKE + 8), dict(k=FAKE + 2), dict(v=FAKE + 4), dict(dec=FAKE + 2), dict(s0=FAKE + 4),
               dict(cu=FAKE + 2), dict(out=2 * FAKE + 8), dict(fin=FAKE + 8), dict(ws=64 * FAKE + 128), dict(nbytes=100),
               dict(cu=None)):
        assert fwd(**kw) == gdn.GDN_EINVAL, kw
    assert fwd(nbytes=size("gdn_linear_attention_workspace_size") - 1) == gdn.GDN_EINVAL
    for kw in (dict(dout=None), dict(q=None), dict(gq=None), dict(gk=None), dict(gv=None), dict(dec=None), dict(ws=None),
               dict(dout=FAKE + 8), dict(gq=2 * FAKE + 4), dict(df=FAKE + 4), dict(d0=FAKE + 8), dict(nbytes=255)):
        assert bwd(**kw) == gdn.GDN_EINVAL, kw


def test_workspace_sizes():
    for fn in ("gdn_linear_attention_workspace_size", "gdn_linear_attention_bwd_workspace_size"):
        assert size(fn, dv=64) == 0 and size(fn, num_seqs=0) == 0 and size(fn, total_tokens=0) > 0
        for dtype in (gdn.GDN_DT_F32, gdn.GDN_DT_BF16):
            # monotone enough that a caller's largest shape is not the smallest workspace, and never huge: the sums of
            # segments are at most one state for every 32 tokens
            for t in (1, 127, 128, 5000, 70000):
                n = size(fn, total_tokens=t, io_dtype=dtype)
                assert n % 256 == 0 and n <= 1 << 20 | 3 * ((t // 32 + N) * HV * 65536 + t * HV * 512) + 65536


def test_shared_memory_is_refused():
    lib, p = gdn.load(), ctypes.byref(problem(**KW))
    ws = size("gdn_linear_attention_workspace_size")
    assert ws < 2 << 20 and ws % 16 == 0
    sizes = dict(q=QK, k=QK, v=ROWS, dec=HEADS, s0=STATES, cu=CU, out=ROWS, fin=STATES, ws=ws)
    call = lambda q, k, v, dec, s0, cu, out, fin, ws: lib.gdn_linear_attention(
        p, ptr(q), ptr(k), ptr(v), ptr(dec), f(0.1), ptr(s0), ptr(cu), ptr(out), ptr(fin), ptr(ws),
        ctypes.c_size_t(sizes["ws"]), None)
    check(call, spread(sizes), sizes, names=["out", "fin"])
    wb = size("gdn_linear_attention_bwd_workspace_size")
    sizes = dict(do=ROWS, q=QK, k=QK, v=ROWS, dec=HEADS, s0=STATES, df=STATES, cu=CU, dq=QK, dk=QK, dv=ROWS, d0=STATES)
    call = lambda do, q, k, v, dec, s0, df, cu, dq, dk, dv, d0: lib.gdn_linear_attention_bwd(
        p, ptr(do), ptr(q), ptr(k), ptr(v), ptr(dec), f(0.1), ptr(s0), ptr(df), ptr(cu), ptr(dq), ptr(dk), ptr(dv),
        ptr(d0), ptr(1 << 30), ctypes.c_size_t(wb), None)
    check(call, spread(sizes), sizes, names=["dq", "dk", "dv", "d0"])


def test_step_refusals():
    def step(q=FAKE, k=FAKE, v=FAKE, dec=FAKE, st=16 * FAKE, idx=None, out=2 * FAKE, **kw):
        p = problem(**{**dict(batch=4, seqlen=1, num_seqs=4, total_tokens=4, num_state_slots=4, hq=2, hv=4), **kw})
        return gdn.load().gdn_linear_attention_step(ctypes.byref(p), ptr(q), ptr(k), ptr(v), ptr(dec), f(0.1), ptr(st),
                                                    ptr(idx), ptr(out), None)

    for kw in (dict(total_tokens=5), dict(num_state_slots=3), dict(num_state_slots=-1, idx=FAKE), dict(hv=0),
               dict(hq=3), dict(q=None), dict(k=None), dict(v=None), dict(dec=None), dict(st=None), dict(out=None),
               dict(q=FAKE + 4), dict(st=16 * FAKE + 8), dict(out=FAKE + 8), dict(idx=FAKE + 2), dict(out=16 * FAKE),
               dict(out=FAKE), dict(st=FAKE), dict(io_dtype=2), dict(dec=FAKE + 1)):
        assert step(**kw) == gdn.GDN_EINVAL, kw
    assert step(dv=64) == gdn.GDN_EUNSUPPORTED
    assert step(flags=2) == gdn.GDN_EUNSUPPORTED


def rope_call(back=False, q=FAKE, k=2 * FAKE, q_weight=3 * FAKE, k_weight=4 * FAKE, inv_freq=5 * FAKE, positions=6 * FAKE,
              pair_axis=7 * FAKE, oq=8 * FAKE, ok=9 * FAKE, gq=10 * FAKE, gk=11 * FAKE, dqw=None, dkw=None, ws=None, nbytes=0,
              **kw):
    r = gdn.GdnQkRope(**{**dict(q_stride=256, k_stride=128, out_q_stride=256, out_k_stride=128, dout_q_stride=256,
                                dout_k_stride=128, eps=1e-6, tokens=64, hq=2, hk=1, rotary=128, axes=1, interleaved=0,
                                io_dtype=gdn.GDN_DT_BF16), **kw})
    lib, inputs = gdn.load(), [ptr(x) for x in (q, k, q_weight, k_weight, inv_freq, positions, pair_axis)]
    if not back:
        return lib.gdn_qk_norm_rope(ctypes.byref(r), *inputs, ptr(oq), ptr(ok), None)
    return lib.gdn_qk_norm_rope_bwd(ctypes.byref(r), ptr(gq), ptr(gk), *inputs, ptr(oq), ptr(ok), ptr(dqw), ptr(dkw),
                                    ptr(ws), ctypes.c_size_t(nbytes), None)


@pytest.mark.parametrize("back", [False, True])
def test_rope_refusals(back):
    bad = [dict(tokens=-1), dict(hq=0), dict(hk=0), dict(rotary=3), dict(rotary=-2), dict(rotary=130), dict(axes=0),
           dict(axes=9), dict(io_dtype=7), dict(eps=-1.0), dict(eps=float("nan")), dict(q=None), dict(k=None),
           dict(q=FAKE + 8), dict(oq=None), dict(ok=9 * FAKE + 2), dict(q_stride=255), dict(q_stride=128),
           dict(out_q_stride=128), dict(out_q_stride=257), dict(q_stride=-256), dict(q_stride=1 << 62), dict(q_weight=3 * FAKE + 2),
           dict(inv_freq=None), dict(positions=None), dict(positions=6 * FAKE + 1), dict(pair_axis=7 * FAKE + 2),
           dict(oq=9 * FAKE), dict(oq=FAKE + 16), dict(oq=2 * FAKE), dict(ok=FAKE), dict(ok=6 * FAKE), dict(oq=5 * FAKE),
           dict(oq=FAKE, out_q_stride=512)]  # q's place, but rows further apart
    for kw in bad:
        assert rope_call(back, **kw) == gdn.GDN_EINVAL, kw
    if back:
        assert rope_call(True, dqw=12 * FAKE) == gdn.GDN_EINVAL  # no workspace
        for kw in (dict(dqw=FAKE), dict(dkw=8 * FAKE), dict(dqw=12 * FAKE, dkw=12 * FAKE), dict(dqw=12 * FAKE + 2),
                   dict(dqw=12 * FAKE, ws=8 * FAKE), dict(dqw=12 * FAKE, ws=20 * FAKE + 128)):
            assert rope_call(True, **{**dict(ws=20 * FAKE, nbytes=1 << 30), **kw}) == gdn.GDN_EINVAL, kw
    if NO_GPU:  # nothing wrong: ends at the device status word
        for kw in (dict(), dict(oq=FAKE), dict(ok=2 * FAKE), dict(rotary=0, inv_freq=None, positions=None),
                   dict(q_weight=None, k_weight=None, pair_axis=None), dict(tokens=0, q=None, k=None, oq=None, ok=None),
                   # q and k in one projection's rows of 384 channels, outputs over them
                   dict(q_stride=384, k=FAKE + 512, k_stride=384, oq=FAKE, out_q_stride=384, ok=FAKE + 512,
                        out_k_stride=384)):
            assert rope_call(back, **kw) == gdn.GDN_ECUDA, kw
    # k's output over q's part of the rows
    assert rope_call(back, q_stride=384, k=FAKE + 512, k_stride=384, ok=FAKE + 256,
                     out_k_stride=384) == gdn.GDN_EINVAL


def test_binding_refusals():
    z = torch.zeros
    q, v, dec = z(4, 2, 128), z(4, 4, 128), z(4)
    cu = z(2, dtype=torch.int32)
    for bad in (lambda: gdn.gdn_linear_attention(q, q, v, dec, 1.0),                       # no batch dimension
                lambda: gdn.gdn_linear_attention(q, q, v, dec, 1.0, cu_seqlens=cu),        # on the CPU
                lambda: gdn.gdn_linear_attention(q, q[:3], v, dec, 1.0, cu_seqlens=cu),
                lambda: gdn.gdn_linear_attention(q, q, v[:3], dec, 1.0, cu_seqlens=cu),
                lambda: gdn.gdn_linear_attention(q, q, v, dec[:3], 1.0, cu_seqlens=cu),
                lambda: gdn.gdn_linear_attention(q, q, v, dec.double(), 1.0, cu_seqlens=cu),
                lambda: gdn.gdn_linear_attention(q, q, v, dec, 1.0, cu_seqlens=cu.long()),
                lambda: gdn.gdn_linear_attention(q, q, v, dec, 1.0, cu_seqlens=cu, initial_state=z(1, 4, 128, 64)),
                lambda: gdn.gdn_linear_attention(q.half(), q.half(), v.half(), dec, 1.0, cu_seqlens=cu),
                lambda: gdn.gdn_linear_attention(z(2, 4, 128).transpose(0, 1), q, v, dec, 1.0, cu_seqlens=cu),
                lambda: gdn.gdn_linear_attention_bwd(v[:2], q, q, v, dec, 1.0, cu_seqlens=cu),
                lambda: gdn.gdn_linear_attention_step(q, q, v, dec, 1.0, z(4, 4, 128)),
                lambda: gdn.gdn_linear_attention_step(q, q, v, dec, 1.0, z(4, 4, 128, 128))):
        with pytest.raises(ValueError):
            bad()
    fr, pos = z(64), z(4, dtype=torch.int32)
    for bad in (lambda: gdn.gdn_qk_norm_rope(q, q, None, None, fr, pos),                   # on the CPU
                lambda: gdn.gdn_qk_norm_rope(q, q, None, None, z(65), pos),
                lambda: gdn.gdn_qk_norm_rope(q, q, None, None, fr, pos.long()),
                lambda: gdn.gdn_qk_norm_rope(q, q, None, None, fr, pos[:3]),
                lambda: gdn.gdn_qk_norm_rope(q, q, z(64), None, fr, pos),
                lambda: gdn.gdn_qk_norm_rope(q, q[:2], None, None, fr, pos),
                lambda: gdn.gdn_qk_norm_rope(q, q, None, None, fr, z(3, 4, dtype=torch.int32)),  # no pair_axis
                lambda: gdn.gdn_qk_norm_rope(z(4, 2, 64), q, None, None, fr, pos),
                lambda: gdn.gdn_qk_norm_rope(z(2, 4, 128).transpose(0, 1), q, None, None, fr, pos),  # heads apart
                lambda: gdn.gdn_qk_norm_rope(z(4, 2, 256)[..., ::2], q, None, None, fr, pos)):
        with pytest.raises(ValueError):
            bad()


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(0)
    lens, hq, hv = [3, 0, 4], 1, 2
    t = lambda *s: torch.tensor(rng.standard_normal(s))
    d = {"q": t(7, hq, 128), "k": t(7, hq, 128), "v": t(7, hv, 128), "dout": t(7, hv, 128), "s0": t(3, hv, 128, 128),
         "dfinal": t(3, hv, 128, 128), "decay": torch.tensor([-0.3, -1.0]).double(), "scale": 0.2}
    R.H[torch.float64] = 2.0 ** -53
    ref = R.attention(d, lens, torch.float64)

    def loss(d):
        r = R.attention(d, lens, torch.float64)
        return (r["out"][0] * d["dout"].numpy()).sum() + (r["final"][0] * d["dfinal"].numpy()).sum()

    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("s0", "ds0")):
        way = t(*d[name].shape)
        ends = [loss({**d, name: d[name] + s * 1e-4 * way}) for s in (1, -1)]
        want = (ref[grad][0] * way.numpy()).sum()
        assert abs((ends[0] - ends[1]) / 2e-4 - want) <= 1e-6 * abs(want) + 1e-6, name
