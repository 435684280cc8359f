"""Angles of the rotation at far positions, taken back from the rotated channels.

A head of ones under no eps is its own norm; with a weight of 1 on the first channel of a pair and 0 on the second the pair
becomes (cos t, sin t), whose angle is off by t's own error, 2^-22 radian at most, and by sine's and cosine's: one step of
a value below 1 each, 2^-24, together sqrt(2) 2^-24 on the unit circle."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from gated_deltanet_chunked_gb300 import gdn

pytestmark = pytest.mark.gpu

# frequencies and positions whose parts' products in whole turns leave remainders that add up to nearly half a turn
PAIRS = [
    ("0x1.aeb9680000000p-6", -1664266146), ("0x1.4d4ed40000000p-6", -1493573560), ("0x1.1860040000000p-6", 1763627106),
    ("0x1.f70adc0000000p-7", -2019590083), ("0x1.2bbd020000000p-4", -459263975), ("0x1.2824d80000000p-6", -1407590266),
    ("0x1.308ef40000000p-4", 455077925), ("0x1.6169040000000p-2", -430497784), ("0x1.7b38d20000000p-6", -1426435987),
    ("0x1.2294c40000000p-6", 1691967627), ("0x1.4e45640000000p-5", -1644617660), ("0x1.3514540000000p-6", -2050703207),
    ("0x1.77a4940000000p-6", -2060230572), ("0x1.203b620000000p-3", -246489075), ("0x1.7b38d20000000p-6", -1951436714),
    ("0x1.5e468e0000000p-4", -1631973341), ("0x1.e8b64e0000000p-6", 1223176251), ("0x1.35c9860000000p-5", -1239801812),
    ("0x1.fb503e0000000p-1", -82776061), ("0x1.e900840000000p-3", -1980653557),
]
PI = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)


def angle_of(pos, freq):
    """pos * freq less whole turns."""
    t = Fraction(int(pos)) * Fraction(float(freq))
    return float(t - round(t / (2 * PI)) * 2 * PI)


def off(cuda, freqs, positions, interleaved):
    """|angle - position * frequency| of token i's pair i."""
    n = len(freqs)
    f = torch.tensor(freqs, dtype=torch.float32)
    pos = torch.tensor(positions, dtype=torch.int64).to(torch.int32)
    x = torch.ones(n, 1, 128, device=cuda)
    first = torch.arange(n) * 2 if interleaved else torch.arange(n)
    second = first + (1 if interleaved else n)
    w = torch.ones(128)
    w[second] = 0
    q, k = gdn.gdn_qk_norm_rope(x, x.clone(), w.to(cuda), w.to(cuda), f.to(cuda), pos.to(cuda), interleaved=interleaved,
                                eps=0.0)
    assert torch.equal(q, k) and (q[:, 0, -1] == 1).all()  # a channel behind the rotated ones is the norm itself
    q = q[:, 0].cpu().double().numpy()
    i = np.arange(n)
    got = np.arctan2(q[i, second.numpy()], q[i, first.numpy()])
    d = got - np.array([angle_of(p, v) for p, v in zip(pos.tolist(), f.tolist())])
    return np.abs(d - 2 * np.pi * np.rint(d / (2 * np.pi)))


BOUND = 2.0 ** -22 + 2 ** 0.5 * 2.0 ** -24


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
def test_remainders_that_add_up(cuda, interleaved):
    e = off(cuda, [float.fromhex(f) for f, _ in PAIRS], [p for _, p in PAIRS], interleaved)
    assert (e <= BOUND).all(), e.max() * 2 ** 24


@pytest.mark.parametrize("top", [1.0, 64.0])
def test_anywhere(cuda, top):
    rng = np.random.default_rng(int(top))
    for _ in range(40):
        freqs = (top * 2.0 ** -rng.uniform(0, 20, 60)).astype(np.float32).tolist()
        e = off(cuda, freqs, rng.integers(-2 ** 31, 2 ** 31, 60).tolist(), False)
        assert (e <= BOUND).all(), e.max() * 2 ** 24
