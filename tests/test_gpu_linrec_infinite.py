"""An infinite value in a sequence of the gated linear recurrence: the state is not finite from there to the sequence's
end (infinite, or NaN once a product of decays that underflowed has met it), and nothing else changes."""
import pytest
import torch

import test_gpu_linrec as linrec
from gated_deltanet_chunked_gb300 import gdn

pytestmark = pytest.mark.gpu


@linrec.DTYPES
@linrec.GATES
def test_a_state_of_infinity(cuda, gate, dtype):
    lens, at, head, channel = [40, 3000, 50], 540, 1, 7
    d = linrec.to(linrec.make(81, lens, 2, dtype, gate, True), cuda)
    clean = linrec.run(d)
    d["x"][at, head, channel] = float("inf")
    res = linrec.run(d)
    assert gdn.gdn_read_device_status() == gdn.GDN_OK
    end = lens[0] + lens[1]
    own = res["out"][at:end, head, channel]
    assert own[0] == float("inf") and not torch.isfinite(own).any()
    assert not torch.isfinite(res["final"][1, head, channel])
    for k in ("dx", "dh0"):  # they do not depend on x
        assert torch.equal(res[k], clean[k]), k
    res["out"][at:end, head, channel] = clean["out"][at:end, head, channel]
    res["final"][1, head, channel] = clean["final"][1, head, channel]
    where = (slice(at + 1, end), head) + ((channel,) if gate == "channel" else ())
    assert not torch.isfinite(res["dg"][where]).any()
    res["dg"][where] = clean["dg"][where]
    for k in ("out", "final", "dg"):
        assert torch.equal(res[k], clean[k]), k
