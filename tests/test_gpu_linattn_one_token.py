"""An infinity or NaN in one token's row of one tensor: which rows of the results it may reach, all others bit for bit as
without it.

out and dq of a token are sums over the tokens up to it, dk and dv over those from it on; a row of the token's own operand
(q in out, dout in dq, v in dk, k in dv) is in that row alone. With bf16 one operand of each sum (v in out, k in dq, q in dk,
dout in dv) reaches up to 127 places to the other side, too."""
import pytest
import torch

import test_gpu_linattn as la
from gated_deltanet_chunked_gb300 import gdn

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
# result: (its own operand, the operand that reaches both sides with bf16, the other one, in time)
SUMS = {"out": ("q", "v", "k", True), "dq": ("dout", "k", "v", True), "dk": ("v", "q", "dout", False),
        "dv": ("k", "dout", "q", False)}


def reached(name, tensor, dtype, at, first, last):
    """Rows [from, to) of result ``name`` that row ``at`` of ``tensor`` may reach, in the sequence [first, last)."""
    own, both, other, in_time = SUMS[name]
    if tensor == own:
        return at, at + 1
    if tensor not in (both, other):
        return at, at
    slack = 127 if tensor == both and dtype == BF16 else 0
    return (max(at - slack, first), last) if in_time else (first, min(at + 1 + slack, last))


@la.DTYPES
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [30, 77, 200, 349, 530, 549])
def test_one_token(cuda, dtype, value, at):
    lens = [30, 320, 200]  # sequences of several segments, one that ends inside a chunk and a block
    first, last = (30, 350) if at < 350 else (350, 550)
    n = 1 if at < 350 else 2
    d = la.make(60, lens, 2, 2, dtype, True)
    clean = la.run(la.to(d, cuda))
    for tensor in ("q", "k", "v", "dout"):
        c = la.to({**d, tensor: d[tensor].clone()}, cuda)
        c[tensor][at, 0] = value
        res = la.run(c)
        for name in SUMS:
            lo, hi = reached(name, tensor, dtype, at, first, last)
            keep = torch.ones(res[name].shape[:2], dtype=torch.bool, device=cuda)
            keep[lo:hi, 0] = False
            assert torch.equal(res[name][keep], clean[name][keep]), (name, tensor)
            if hi > lo:
                assert not torch.isfinite(res[name][at, 0]).all(), (name, tensor)
        for name, by in (("final", ("k", "v")), ("ds0", ("q", "dout"))):
            keep = torch.ones(3, 2, dtype=torch.bool, device=cuda)
            if tensor in by:
                keep[n, 0] = False
                assert not torch.isfinite(res[name][n, 0]).all(), (name, tensor)
            assert torch.equal(res[name][keep], clean[name][keep]), (name, tensor)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
