"""Waits that run out in segments of one to three chunks, whose tiles are all asked for before any wait: the copies still
under way land before the CTA ends, so that the shared memory of the CTAs that follow on its SM stays theirs."""
import pytest
import torch

import test_gpu_linattn as la
from gated_deltanet_chunked_gb300 import gdn
from test_gpu_wait_limit import disturbed, wait_limit

pytestmark = pytest.mark.gpu

LENS = {"one_chunk": [128, 1, 100], "two_chunks": [256, 200, 0, 129], "three_chunks": [384, 257, 300]}


@pytest.mark.parametrize("hq,hv", [(1, 2), (16, 32)], ids=["few", "all_sms"])
@pytest.mark.parametrize("lens", list(LENS.values()), ids=list(LENS))
def test_few_chunks(cuda, lens, hq, hv):
    d = la.to(la.make(41, lens, hq, hv, torch.bfloat16, True), cuda)
    ref = la.run(d)
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    assert gdn.GDN_ETIMEOUT in disturbed(lambda: la.run(d), ref)


def test_beside_an_undisturbed_call(cuda):
    """A call that gives up does not reach one that runs at the same time, or the one behind it."""
    sets = [la.to(la.make(42 + i, [250, 700, 128], 8, 16, torch.bfloat16, True), cuda) for i in range(2)]
    ref = [la.run(s) for s in sets]
    streams = [torch.cuda.Stream(cuda) for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        with wait_limit(1):
            with torch.cuda.stream(streams[0]):
                la.run(sets[0])
            gdn.gdn_set_wait_limit_ns(0)  # a launch keeps the limit that it was given
            with torch.cuda.stream(streams[0]):
                behind = la.run(sets[0])
            with torch.cuda.stream(streams[1]):
                beside = la.run(sets[1])
        assert gdn.gdn_get_device_status() in (gdn.GDN_OK, gdn.GDN_ETIMEOUT)
        la.same(behind, ref[0])
        la.same(beside, ref[1])
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
