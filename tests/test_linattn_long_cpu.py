"""The reference of linear attention over long sequences: against the one that goes token by token, and what its bounds
refuse."""
import pytest
import torch

import linattn_long_ref as L
import linattn_ref as R

F32, BF16 = torch.float32, torch.bfloat16
LENS = [300, 1, 129]


def inputs(dtype, hq=2, hv=4):
    gen = torch.Generator().manual_seed(3)
    normal = lambda *shape: torch.randn(shape, generator=gen)
    T, N = sum(LENS), len(LENS)
    d = {"q": normal(T, hq, 128), "k": normal(T, hq, 128), "v": normal(T, hv, 128), "dout": normal(T, hv, 128)}
    d = {k: x.to(dtype) for k, x in d.items()}
    return d | {"s0": normal(N, hv, 128, 128), "dfinal": normal(N, hv, 128, 128), "scale": 0.1,
                "decay": torch.tensor([-0.5, -0.01, 0.0, -float("inf")])[:hv]}


def exact(d, dtype):
    return {k: torch.from_numpy(v) for k, (v, _) in R.attention(d, LENS, dtype).items()}


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_token_by_token(dtype):
    d = inputs(dtype)
    d["decay"][3] = -30.0  # (-inf times no tokens is no number in the chunks' powers)
    ref = exact(d, dtype)
    t = 0
    for n, length in enumerate(LENS):
        r, t = slice(t, t + length), t + length
        for h in range(2):
            vh = slice(2 * h, 2 * h + 2)
            got = L.sequence(d, d["q"][r, h], d["k"][r, h], d["v"][r, vh], d["dout"][r, vh], d["s0"][n, vh],
                             d["dfinal"][n, vh], d["decay"][vh])
            want = {"out": ref["out"][r, vh], "dv": ref["dv"][r, vh], "dq": ref["dq"][r, h], "dk": ref["dk"][r, h],
                    "final": ref["final"][n, vh], "ds0": ref["ds0"][n, vh]}
            for name, x in want.items():
                off = ((got[name] - x).norm() / x.norm()).item()
                assert off <= 1e-12, (name, n, h, off)


def test_what_the_bounds_refuse():
    d = inputs(BF16)
    d["decay"][3] = -30.0
    ref = exact(d, BF16)
    rounded = {k: x.to(F32 if k in ("final", "ds0") else BF16) for k, x in ref.items()}
    L.compare(rounded, d, LENS, BF16, [0, 1])
    for name, x in rounded.items():
        few = x.to(BF16).to(x.dtype) if name in ("final", "ds0") else (x.float() * (1 + 2.0 ** -7)).to(BF16)
        for wrong in (torch.zeros_like(x), few):
            with pytest.raises(AssertionError):
                L.compare({name: wrong}, d, LENS, BF16, [0, 1])
