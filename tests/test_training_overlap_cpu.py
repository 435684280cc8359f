"""Refusals, by the C ABI, of tensors of the training operators that share memory. Addresses are never dereferenced:
every call that would run is made without a GPU only, where it ends at the device status word."""
import ctypes

import pytest
import torch

from gated_deltanet_chunked_gb300 import gdn
from test_training_cpu import CHANNEL, problem, ptr

NO_GPU = not torch.cuda.is_available()
MB = 1 << 20
EPS = ctypes.c_float(1e-5)


def check(call, places, sizes, pairs_allowed=(), names=None):
    """Each pair of (output, other): the other's last 16 bytes, then its first, in the output's first and last are
    refused, and the next free place is not."""
    for o in names:
        for other in places:
            if other == o:
                continue
            tail = places[other] + sizes[other] - 16
            for at in (tail, places[other] - sizes[o] + 16, places[other]):
                if at == places[other] and (o, other) in pairs_allowed:
                    continue
                assert call(**{**places, o: at}) == gdn.GDN_EINVAL, (o, other, at - places[other])
            if NO_GPU:
                for at in (places[other] + sizes[other], places[other] - sizes[o]):
                    others = [k for k in places if k not in (o, other)]
                    if all(at + sizes[o] <= places[k] or places[k] + sizes[k] <= at for k in others):
                        assert call(**{**places, o: at}) == gdn.GDN_ECUDA, (o, other, at - places[other])
    if NO_GPU:
        assert call(**places) == gdn.GDN_ECUDA
        for o, other in pairs_allowed:
            assert call(**{**places, o: places[other]}) == gdn.GDN_ECUDA, (o, other)


def spread(sizes):
    assert all(v < 2 * MB and v % 16 == 0 for v in sizes.values())
    return {k: (4 * i + 8) * MB for i, k in enumerate(sizes)}


T, HV, N = 96, 4, 3
ROWS, HEADS, STATES = T * HV * 128 * 2, T * HV * 4, N * HV * 128 * 4
CKPT, CU = 2 * HV * 128 * 4, (N + 1) * 4


@pytest.mark.parametrize("flags", [0, CHANNEL], ids=["head", "channel"])
def test_recurrence(flags):
    g = ROWS if flags else HEADS
    lib, p = gdn.load(), ctypes.byref(problem(num_seqs=N, total_tokens=T, hv=HV, flags=flags))
    sizes = dict(x=ROWS, g=g, s0=STATES, cu=CU, out=ROWS, fin=STATES, states=CKPT)
    check(lambda x, g, s0, cu, out, fin, states: lib.gdn_linear_recurrence(
        p, ptr(x), ptr(g), ptr(s0), ptr(cu), ptr(out), ptr(fin), ptr(states), None),
        spread(sizes), sizes, names=["out", "fin", "states"])
    sizes = dict(dout=ROWS, x=ROWS, g=g, states=CKPT, s0=STATES, dfin=STATES, cu=CU, dx=ROWS, dg=g, d0=STATES)
    check(lambda dout, x, g, states, s0, dfin, cu, dx, dg, d0: lib.gdn_linear_recurrence_bwd(
        p, ptr(dout), ptr(x), ptr(g), ptr(states), ptr(s0), ptr(dfin), ptr(cu), ptr(dx), ptr(dg), ptr(d0), None),
        spread(sizes), sizes, names=["dx", "dg", "d0"])


def test_recurrence_step():
    p = ctypes.byref(problem(batch=4, seqlen=1, num_seqs=4, total_tokens=4, num_state_slots=6, flags=CHANNEL))
    lib, el = gdn.load(), 4 * 4 * 128 * 2
    sizes = dict(x=el, g=el, state=6 * 4 * 128 * 4, idx=16, out=el)
    check(lambda x, g, state, idx, out: lib.gdn_linear_recurrence_step(p, ptr(x), ptr(g), ptr(state), ptr(idx),
                                                                       ptr(out), None),
          spread(sizes), sizes, pairs_allowed=[("out", "x")], names=["out", "state"])


def test_norm():
    prob = problem(total_tokens=100, dv=200)
    lib, p, rows, stats, cols = gdn.load(), ctypes.byref(prob), 100 * 200 * 2, 400, 800
    sizes = dict(x=rows, w=cols, b=cols, y=rows, mean=stats, rstd=stats)
    check(lambda x, w, b, y, mean, rstd: lib.gdn_layernorm(p, ptr(x), ptr(w), ptr(b), EPS, ptr(y), ptr(mean),
                                                           ptr(rstd), None),
          spread(sizes), sizes, pairs_allowed=[("y", "x")], names=["y", "mean", "rstd"])
    ws = int(lib.gdn_layernorm_bwd_workspace_size(p))
    sizes = dict(dy=rows, x=rows, mean=stats, rstd=stats, w=cols, dx=rows, ws=ws)
    place = spread({**sizes, "dw": cols, "db": cols})

    def back(dy, x, mean, rstd, w, dx, ws, dw=place["dw"], db=place["db"]):
        return lib.gdn_layernorm_bwd(p, ptr(dy), ptr(x), ptr(mean), ptr(rstd), ptr(w), ptr(dx), ptr(dw), ptr(db),
                                     ptr(ws), ctypes.c_size_t(sizes["ws"]), None)

    where = {k: place[k] for k in sizes}
    check(back, where, sizes, pairs_allowed=[("dx", "dy"), ("dx", "x")], names=["dx"])
    for kw in (dict(dw=place["dx"] + rows - 16), dict(db=place["dx"] - cols + 16), dict(dw=place["db"] + 16),
               dict(dw=place["ws"]), dict(db=place["ws"] + ws - 16), dict(ws=place["w"] - ws // 256 * 256 + 256)):
        assert back(**{**where, **kw}) == gdn.GDN_EINVAL, kw
    if NO_GPU:
        assert back(**where, **dict(dw=place["w"])) == gdn.GDN_ECUDA


def test_gate_backward():
    lib, p = gdn.load(), ctypes.byref(problem(total_tokens=T, hv=HV))
    ws = int(lib.gdn_gated_rmsnorm_bwd_workspace_size(p))
    sizes = dict(dy=ROWS, o=ROWS, z=ROWS, w=512, do=ROWS, dz=ROWS)
    place = spread({**sizes, "dw": 512, "ws": ws})

    def back(dy, o, z, w, do, dz, dw=place["dw"], ws_=place["ws"]):
        return lib.gdn_gated_rmsnorm_bwd(p, ptr(dy), ptr(o), ptr(z), ptr(w), EPS, ptr(do), ptr(dz), ptr(dw), ptr(ws_),
                                         ctypes.c_size_t(ws), None)

    where = {k: place[k] for k in sizes}
    check(back, where, sizes, pairs_allowed=[(d, i) for d in ("do", "dz") for i in ("dy", "o", "z")],
          names=["do", "dz"])
    for kw in (dict(dw=place["do"] + ROWS - 16), dict(dw=place["ws"]), dict(ws_=place["dz"]), dict(ws_=place["o"])):
        assert back(**where, **kw) == gdn.GDN_EINVAL, kw
