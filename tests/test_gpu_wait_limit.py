"""Bounded waits of the training operators that run out, under test.

The limit of a wait is lowered to less than a copy or another CTA's answer
takes, so that waits run out at places that differ from call to call. Every
such call ends, leaves GDN_ETIMEOUT and a context that can be used; a call
that leaves GDN_OK all the same has the bits of an undisturbed one, and so has
the first call with the default limit."""
import contextlib

import pytest
import torch

import test_gpu_layernorm as norm
import test_gpu_linrec as linrec
from gated_deltanet_chunked_gb300 import gdn

pytestmark = pytest.mark.gpu

LIMITS = [1, 1, 1, 200, 400, 800, 1600, 5000, 1]


@contextlib.contextmanager
def wait_limit(ns):
    gdn.gdn_set_wait_limit_ns(ns)
    try:
        yield
        torch.cuda.synchronize()
    finally:
        gdn.gdn_set_wait_limit_ns(0)


def disturbed(call, ref):
    """Statuses of calls under LIMITS; their results are compared where the status is GDN_OK."""
    seen = []
    for ns in LIMITS:
        with wait_limit(ns):
            res = call()
        seen.append(gdn.gdn_get_device_status())
        assert seen[-1] in (gdn.GDN_OK, gdn.GDN_ETIMEOUT)
        if seen[-1] == gdn.GDN_OK:
            assert all(torch.equal(res[k], ref[k]) for k in ref if ref[k] is not None), ns
    res = call()
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    assert all(torch.equal(res[k], ref[k]) for k in ref if ref[k] is not None)
    return seen


@linrec.DTYPES
@linrec.GATES
@pytest.mark.parametrize("hv,lens", [(1, [9000, 0, 11000]), (3, [20000]), (32, [2500, 1, 1500]), (160, [300, 41])],
                         ids=["one_head", "three_heads", "all_sms", "single_ctas"])
def test_recurrence(cuda, hv, lens, gate, dtype):
    d = linrec.to(linrec.make(71, lens, hv, dtype, gate, True), cuda)
    ref = linrec.run(d)
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    seen = disturbed(lambda: linrec.run(d), ref)
    if hv < 160:  # the CTAs of a cluster wait for each other many times
        assert gdn.GDN_ETIMEOUT in seen


def test_recurrence_with_bad_offsets(cuda):
    d = linrec.to(linrec.make(72, [5000], 2, torch.bfloat16, "channel", False), cuda)
    bad = torch.tensor([0, 4000, 3000, 5000], dtype=torch.int32, device=cuda)
    out = torch.full_like(d["x"], 2.0)
    with wait_limit(1):
        gdn.gdn_linear_recurrence(d["x"], d["g"], cu_seqlens=bad, out=out)
    assert gdn.gdn_get_device_status() == gdn.GDN_EDEVICE_INPUT
    assert (out == 2).all()


def test_recurrence_beside_an_undisturbed_one(cuda):
    """A call that gives up does not reach one that runs at the same time."""
    sets = [linrec.to(linrec.make(73 + i, [6000, 900], 4, torch.bfloat16, gate, True), cuda)
            for i, gate in enumerate(("channel", "head"))]
    ref = linrec.run(sets[1])
    streams = [torch.cuda.Stream(cuda) for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        with wait_limit(1):
            with torch.cuda.stream(streams[0]):
                linrec.run(sets[0])
            gdn.gdn_set_wait_limit_ns(0)  # a launch keeps the limit that it was given
            with torch.cuda.stream(streams[1]):
                res = linrec.run(sets[1])
        assert gdn.gdn_get_device_status() in (gdn.GDN_OK, gdn.GDN_ETIMEOUT)
        assert all(torch.equal(res[k], ref[k]) for k in ref)


@norm.DTYPES
@pytest.mark.parametrize("rows,width", [(2000, 16383), (700, 9001), (500, 16384), (3, 12345)])
def test_norm(cuda, rows, width, dtype):
    """Rows on two CTAs (of aligned widths the backward pass alone)."""
    d = {k: v.to(cuda) for k, v in norm.make(74, rows, width, dtype).items()}
    ref = norm.run(d, cuda)
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    seen = disturbed(lambda: norm.run(d, cuda), ref)
    if rows >= 500:  # a pair waits many times
        assert gdn.GDN_ETIMEOUT in seen
