"""gdn_layernorm of rows whose offset is large beside their deviations.

With u = 2^-24, D elements, c the values about the mean and S = 32u the error
of a sum over the threads (train_ref): a first mean is off by e0 = S mean|x|,
the values about it by u (|c| + e0); their own mean, which corrects the first,
is then known to ed = (S + 4u) (mean|c| + e0), and nothing else depends on the
offset. Values about the corrected mean are off by ec = 2u (|c| + e0) + ed; the
squares, corrected by the square of the first mean's error, by
(S + 6u) (var + e0^2) + 2 e0 ed. The mean is rounded once. Where the mean is
not above 4 deviations (of the row, or of its half on two CTAs, whose mean and
deviation differ from the row's), it need not be corrected: there e0 is at
most S (mean|c| + |mean|), and stays in the mean and, squared, in the
squares."""
import numpy as np
import pytest
import torch

import train_ref as R
from gated_deltanet_chunked_gb300 import gdn

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5


def reference(x, w, b, dtype):
    u, S, half = R.u, R.SUM, R.U[dtype]
    mean = x.mean(1, keepdims=True)
    c = x - mean
    mean += c.mean(1, keepdims=True)  # what 64 bits left
    c = x - mean
    var = (c * c).mean(1, keepdims=True)
    rstd = 1 / np.sqrt(var + EPS)
    e0 = S * np.abs(x).mean(1, keepdims=True)
    near = mean ** 2 < 64 * var  # 16 of a row; with room for a half's
    ed = (S + 4 * u) * (np.abs(c).mean(1, keepdims=True) + e0) + near * e0
    ec = 2 * u * (np.abs(c) + e0) + ed
    ev = 1.01 * ((S + 6 * u) * (var + e0 ** 2) + 2 * e0 * ed + near * e0 ** 2)
    er = rstd * (0.5 * ev / (var + EPS) + 4 * u) * 1.01
    y = c * rstd * w + b
    ey = np.abs(w) * (rstd * ec + np.abs(c) * er + ec * er + 2 * u * np.abs(c) * rstd) + 2 * u * (
        np.abs(c * rstd * w) + np.abs(y))
    return {"y": (y, half * np.abs(y) + (1 + half) * ey), "mean": (mean[:, 0], u * np.abs(mean[:, 0]) + 1.01 * ed[:, 0]),
            "rstd": (rstd[:, 0], er[:, 0])}


def rows(width, dtype):
    gen = torch.Generator().manual_seed(width)
    normal = torch.randn(9, width, generator=gen)
    x = torch.empty(9, width)
    x[0] = 1000.0
    x[1] = -1.0 / 3.0
    x[2] = 1000.0 + 1e-3 * normal[2]
    x[3] = 3e4 + 0.05 * normal[3]
    x[4] = -777.0 + 0.5 * normal[4]
    x[5] = torch.where(normal[5] > 0, 1000.0, 1004.0)  # neighbours in bf16
    x[6] = torch.where(normal[6] > 0, 1000.0, 1000.0 + 2.0 ** -14)  # neighbours in f32
    x[7] = 12345.0
    x[7, width // 2] += 0.25
    x[8] = normal[8]
    return x.to(dtype), torch.randn(width, generator=gen) + 1, torch.randn(width, generator=gen)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("width", [3, 77, 100, 384, 1000, 1001, 2000, 4097, 6000, 9001, 12000, 16383, 16384])
def test_errors_are_small_beside_the_deviations(cuda, width, dtype):
    x, w, b = rows(width, dtype)
    ref = reference(R.f64(x), R.f64(w), R.f64(b), dtype)
    y, mean, rstd = gdn.gdn_layernorm(x.to(cuda), w.to(cuda), b.to(cuda), EPS, save_stats=True)
    for name, t in (("y", y), ("mean", mean), ("rstd", rstd)):
        R.assert_within(t, *ref[name], name)


@pytest.mark.parametrize("width", [100, 1000, 9001, 16384])
def test_constant_rows_without_eps(cuda, width):
    """var is 0 and not below: 1 / sqrt(0) is infinite, and no NaN comes from a negative square."""
    x = torch.tensor([1000.0, 1.0 / 3.0, 0.1, 7e4]).reshape(4, 1).repeat(1, width).to(cuda)
    _, mean, rstd = gdn.gdn_layernorm(x, eps=0.0, save_stats=True)
    assert torch.equal(mean, x[:, 0])  # ed is far below half a step
    e0 = R.SUM * R.f64(x[:, 0])
    ev = 1.01 * ((R.SUM + 6 * R.u) * e0 ** 2 + 2 * e0 * (R.SUM + 4 * R.u) * e0)
    assert (R.f64(rstd) >= 0.99 / np.sqrt(ev)).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("width", [1, 8, 9, 100, 600, 1001, 9001, 12000])
def test_backward_of_a_mean_whose_normalised_value_overflows(cuda, width, dtype):
    """mean * rstd is infinite, every normalised value finite: what a thread holds outside the row reaches no sum."""
    gen = torch.Generator().manual_seed(width)
    level = torch.tensor(1.5e36, dtype=dtype)
    x = level.repeat(5, width)
    dy, w = torch.randn(5, width, generator=gen).to(dtype), torch.randn(width, generator=gen) + 1
    mean, rstd = level.float().repeat(5), torch.full((5,), 316.0)
    res = gdn.gdn_layernorm_bwd(dy.to(cuda), x.to(cuda), mean.to(cuda), rstd.to(cuda), w.to(cuda))
    ref = R.layernorm_bwd(R.f64(dy), R.f64(x), R.f64(mean), R.f64(rstd), R.f64(w), dtype)
    for name, t in zip(("dx", "dweight", "dbias"), res):
        R.assert_within(t, *ref[name], name)
