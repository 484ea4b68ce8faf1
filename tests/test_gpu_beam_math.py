"""The beam selection's exponential and logarithm (pairs of fp32) against float64.

Bounds, from the roundings.  e^x: r = x - n ln 2 is exact after the first part of ln 2 and
rounds once after the second, which is off by 2^-25 of 2.1e-4: 2^-26 + 116 x 2.1e-4 x 2^-25
= 1.07 x 2^-26 for |r| < 0.35.  The polynomial q r^2 is below 0.07, q below 0.57: q's last
step rounds by 2^-25, the earlier ones by a third of that, times r^2; q r by 2^-27, times
r; q r^2 and its sum with the rest of 1 + r by 2^-28 each: 0.8 x 2^-26.  Terms left out
2^-32.  Of e^r >= 0.707: (1.07 + (0.8 + 0.02) x 1.415) 2^-26 = 2.24 x 2^-26.  ln y:
fp32's l within 1 ulp or 2^-22 of a value up to 89, then l + (y e^-l - 1), off as
e^-l is and by half the square of l's error, (2^-18)^2 / 2."""
import math

import pytest
import torch

import mla_latent_decode_gb300 as mla
from mla_latent_decode_gb300 import build

pytestmark = pytest.mark.gpu
EXP = 2.24 * 2.0 ** -26
LOG = EXP + 2.0 ** -37 + 2.0 ** -40


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


def _inputs(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    v = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    k = n // 2
    x = torch.cat([-80 * u[:k], -torch.exp(-40 * u[k:]) * 3]).float()
    y = torch.cat([torch.exp(79 * v[:k]), 1 + torch.exp(-17 * v[k:])]).float()
    return x, y


@pytest.mark.parametrize("seed", range(4))
def test_against_float64(seed):
    x, y = _inputs(1 << 22, seed)
    e, l = mla.debug_beam_math(x, y)
    want = torch.exp(x.double())
    live = x > -80
    assert bool((e[~live] == 0).all())
    assert float(((e - want).abs() / want)[live].max()) <= EXP
    assert float((l - torch.log(y.double())).abs().max()) <= LOG


def test_ends():
    ln2 = math.log(2.0)
    x = [0.0, -0.0, -80.0, -79.99999, -80.00001, -1000.0, -math.inf, math.nan]
    x += [-(n + d) * ln2 for n in range(115) for d in (0.4999999, 0.5, 0.5000001, 0.0)]
    # (y up to e^79, where e^-l is not 0 yet: a sum of exponentials has 2^31 terms at most)
    y = [1.0, math.nextafter(1.0, 2.0) + 2.0 ** -23, 2.0, 65536.0, 2.0 ** 31, 2e34]
    y += [1.0 + 2.0 ** -k for k in range(23)]
    y += [1.0] * (len(x) - len(y))
    x = torch.tensor(x, dtype=torch.float32, device="cuda")
    y = torch.tensor(y, dtype=torch.float32, device="cuda")
    e, l = mla.debug_beam_math(x, y)
    assert e[:2].tolist() == [1.0, 1.0] and bool(e[7].isnan()) and float(l[0]) == 0.0
    want = torch.where(x > -80, torch.exp(x.double()), 0.0)
    live = want > 0
    assert bool((e[~live & ~x.isnan()] == 0).all())
    assert float(((e - want).abs() / want)[live].max()) <= EXP
    assert float((l - torch.log(y.double())).abs().max()) <= LOG
    mla.debug_beam_math(x[:0], y[:0])


def test_refusals():
    x = torch.zeros(4, device="cuda")
    for bad in (torch.zeros(3, device="cuda"), torch.zeros(4, device="cuda", dtype=torch.float64), torch.zeros(4)):
        with pytest.raises(ValueError):
            mla.debug_beam_math(x, bad)
