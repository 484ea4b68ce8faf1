"""Rows that are not finite in the residual RMS norm: a NaN or an infinity shows in
every output that depends on it, in E4M3 as a NaN scale with NaN codes, as the
definition in 64 bits has it; finite rows beside them keep test_gpu_add_rms_norm's
tolerances.
"""
import numpy as np
import pytest
import torch

import mla_latent_decode_gb300 as mla
from latent_ref import f64
from mla_latent_decode_gb300 import build
from test_gpu_add_rms_norm import _check, _rows

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


def _definition(x, res, w, groups):
    """(y, |y|'s maximum per group): NaN wherever the formula gives one."""
    with np.errstate(all="ignore"):
        h = f64(x) + (f64(res) if res is not None else 0.0)
        y = h / np.sqrt((h * h).mean(1, keepdims=True) + EPS) * f64(w)
        return y, np.abs(y).reshape(len(y), groups, -1).max(-1)


# whole vectors; rows shifted alike (odd d); by element (arrays off a boundary differently)
@pytest.mark.parametrize("d,group,pad", [
    (1536, 0, 0), (1536, 128, 0), (7168, 32, 0), (1531, 0, 0), (640, 0, 1), (640, 128, 4), (7168, 0, 0)])
@pytest.mark.parametrize("n", [8, 700])  # a thread per vector; several vectors a thread
@pytest.mark.parametrize("where", ["x", "residual"])
def test_nan_and_infinity_show(n, d, group, pad, where):
    x, w, res = _rows(n, d, 1, pad), (1 + 0.3 * _rows(1, d, 2)[0].float()).bfloat16(), _rows(n, d, 3, pad)
    hit = x if where == "x" else res
    hit[1, 0] = float("nan")
    hit[2, d - 1] = float("inf")
    hit[4, d // 2] = -float("inf")
    hit[5, 7], hit[5, 11] = float("inf"), float("nan")
    x[6, 3], res[6, 3] = float("inf"), -float("inf")
    bad = [1, 2, 4, 5, 6]
    fine = [r for r in range(n) if r not in bad]
    out, res_out = torch.empty((n, d), dtype=torch.bfloat16, device="cuda"), torch.empty_like(res)
    _, out8, scales, _ = mla.add_rms_norm(x, w, res, EPS, out=out, e4m3=True, group=group, residual_out=res_out)
    y, amax = _definition(x, res, w, scales.shape[1])
    s, codes = f64(scales), out8.view(torch.uint8).cpu().numpy()
    assert np.array_equal(np.isnan(s), np.isnan(amax))
    assert np.isnan(amax[bad]).any(1).all()
    lost = np.repeat(np.isnan(amax), d // amax.shape[1], 1)
    assert np.all((codes & 0x7F)[lost] == 0x7F) and not np.any((codes & 0x7F)[~lost] == 0x7F)
    zero = np.repeat(amax == 0, d // amax.shape[1], 1)  # beside an infinity: finite / inf
    assert np.all(codes[zero] & 0x7F == 0) and np.all(s[amax == 0] == 0)
    assert np.array_equal(np.isnan(f64(out)), np.isnan(y))
    with np.errstate(invalid="ignore"):
        assert np.array_equal(f64(res_out)[bad], f64((x + res)[bad]), equal_nan=True)
    pick = lambda t: t[fine]
    _check(pick(x), pick(res), w, EPS, (pick(out), pick(out8.view(torch.uint8)), pick(scales), pick(res_out)))


def test_weight_that_is_not_finite():
    """A NaN weight: its column, and with a scale per group the group it lies in."""
    n, d = 5, 512
    x, w = _rows(n, d, 4), _rows(1, d, 5)[0].contiguous()
    w[200] = float("nan")
    out = torch.empty_like(x)
    _, out8, scales, _ = mla.add_rms_norm(x, w, None, EPS, out=out, e4m3=True, group=64)
    want = torch.zeros((n, 8), dtype=torch.bool)
    want[:, 200 // 64] = True
    assert torch.equal(scales.isnan().cpu(), want)
    assert torch.equal(out8.float().isnan().cpu(), want.repeat_interleave(64, 1))
    assert torch.equal(out.isnan().cpu(), (torch.arange(d) == 200).expand(n, d))
