"""Bounded waits of linear attention's bf16 kernels that run out, under test: every such call ends and leaves
GDN_ETIMEOUT and a context that can be used."""
import pytest
import torch

import test_gpu_linattn as la
from gated_deltanet_chunked_gb300 import gdn
from test_gpu_wait_limit import disturbed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hv,lens", [(1, 2, [3000, 0, 500]), (16, 32, [700, 1, 900])], ids=["few", "all_sms"])
def test_linear_attention(cuda, hq, hv, lens):
    d = la.to(la.make(31, lens, hq, hv, torch.bfloat16, True), cuda)
    ref = la.run(d)
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    assert gdn.GDN_ETIMEOUT in disturbed(lambda: la.run(d), ref)
