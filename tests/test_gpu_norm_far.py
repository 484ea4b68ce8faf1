"""The residual RMS norm of finite rows whose squares leave fp32's range: against
the definition in 64 bits with test_gpu_add_rms_norm's tolerances.
"""
import pytest
import torch

import mla_latent_decode_gb300 as mla
from mla_latent_decode_gb300 import build
from test_gpu_add_rms_norm import _check, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


@pytest.mark.parametrize("d,group", [(1536, 0), (7168, 128), (1531, 0), (16384, 64)])
@pytest.mark.parametrize("n", [6, 700])
@pytest.mark.parametrize("residual", [True, False])
def test_rows_above_the_square_root_of_the_range(n, d, group, residual):
    """Rows of 2^60 to 2^120 beside ordinary ones."""
    x, w = _rows(n, d, 1), (1 + 0.3 * _rows(1, d, 2)[0].float()).bfloat16()
    res = _rows(n, d, 3) if residual else None
    for r, power in enumerate((60, 64, 66, 100, 120)):
        x[r] = (x[r].double() * 2.0 ** power).to(torch.bfloat16)
        if residual and power != 66:  # there x alone
            res[r] = (res[r].double() * 2.0 ** power).to(torch.bfloat16)
    out = torch.empty_like(x)
    keep = None if res is None else res.clone()
    got = mla.add_rms_norm(x, w, res, 1e-6, out=out, e4m3=True, group=group)
    _check(x, keep, w, 1e-6, got)


@pytest.mark.parametrize("power", [-50, -64, -80, -110])
@pytest.mark.parametrize("d", [512, 7001])
def test_small_rows_without_eps(power, d):
    n = 5
    x, w = _rows(n, d, 4), _rows(1, d, 5)[0].contiguous()
    x[1:] = (x[1:].double() * 2.0 ** power).to(torch.bfloat16)
    out = torch.empty_like(x)
    _check(x, None, w, 0.0, mla.add_rms_norm(x, w, None, 0.0, out=out, e4m3=True))


def test_zeros_without_eps_are_not_a_number():
    """0 / 0, as the formula has it; with an eps, zeros."""
    x, w = torch.zeros((2, 256), dtype=torch.bfloat16, device="cuda"), torch.ones(256).bfloat16().cuda()
    out, out8, scales, _ = mla.add_rms_norm(x, w, None, 0.0, out=torch.empty_like(x), e4m3=True)
    assert out.isnan().all() and scales.isnan().all() and out8.float().isnan().all()
    out, out8, scales, _ = mla.add_rms_norm(x, w, None, 1e-6, out=out, e4m3=True)
    assert not out.any() and not scales.any() and not out8.view(torch.uint8).any()
