"""The append at magnitudes whose squares or quotients leave fp32's range: finite
rows are stored as the definition has them, or saturate with their sign.
"""
import numpy as np
import pytest
import torch

import mla_latent_decode_gb300 as mla
from latent_ref import E4M3, NOPE, ROW, decode4, e4m3_values, encode, f64, sure, table
from mla_latent_decode_gb300 import build
from test_gpu_append import _inputs, _pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("power", [59, 63, 64, 100, 120, -64, -70, -100])
def test_norm_of_far_rows(kind, power):
    """Without eps the norm of x 2^k is that of x: powers of two change no rounding,
    so every stored byte is the same, though the squares leave fp32's range."""
    n = 9
    rows, weight, _, pos = _inputs(n, 0, 21)
    rows = torch.randn(rows.shape, generator=torch.Generator().manual_seed(22)).clamp(-8, 8).bfloat16().cuda()
    far = rows.clone()
    far[:, :NOPE] *= 2.0 ** power
    assert far.isfinite().all()
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    tab = table(5000).cuda()
    kept = []
    for r in (rows, far):
        kv, scale = _pool(kind, 64)
        mla.kv_append(r, slots, pos, tab, kv, scale, norm_weight=weight, eps=0.0)
        kept.append((kv.view(torch.uint8), scale))
    assert torch.equal(kept[0][0], kept[1][0])
    assert kind == "bf16" or torch.equal(kept[0][1], kept[1][1])


def test_norm_of_one_large_value():
    """One huge value among ordinary ones, with eps: it alone is left of the row."""
    rows = torch.ones((2, ROW)).bfloat16().cuda()
    rows[0, 5], rows[1, 300] = 2.0 ** 127, -(2.0 ** 66)
    kv, _ = _pool("bf16", 64)
    slots, pos = torch.arange(2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    w = torch.ones(NOPE).bfloat16().cuda()
    mla.kv_append(rows, slots, pos, table(1).cuda(), kv, None, norm_weight=w)
    x = f64(rows)[:, :NOPE]
    want = x / np.sqrt((x * x).mean(1, keepdims=True) + 1e-6)
    got = f64(kv[:2])[:, :NOPE]
    # 2^-17 of the norm and 2^-8 of bf16; below fp32's normal range, 2^-133 (bf16's last step)
    assert np.all(np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -17) * np.abs(want) + 2.0 ** -133)


@pytest.mark.parametrize("g", [2.0 ** -60, 2.0 ** -85, 2.0 ** -120, 2.0 ** -140, 2.0 ** -149])
def test_far_values_saturate_with_their_sign(g):
    """Without the norm: values some 2^200 times the factor, of either sign."""
    rows = torch.full((1, ROW), 3e38).bfloat16().cuda()
    rows[0, 1::2] = -3e38
    kv, _ = _pool("fp4", 64)
    at, pos = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.kv_append(rows, at, pos, table(1).cuda(), kv, torch.full((1,), g, device="cuda"))
    raw = kv[0].cpu().numpy()
    assert np.all(raw[:256] == 0xF7)          # +6 and -6
    assert np.all(raw[256:288] == 0x7E)       # 448
    sign = np.where(np.arange(64) % 2, 0x80, 0)
    assert np.all(raw[288:] == 0x7E | sign)


@pytest.mark.parametrize("g", [2.0 ** 125, 2.0 ** 126, 1.5 * 2.0 ** 127])
def test_large_factors(g):
    """Six times the factor is past fp32's range: blocks still get their scales."""
    n = 6
    rows = torch.randn((n, ROW), generator=torch.Generator().manual_seed(23)).clamp(-3, 3)
    rows = (rows.double() * 2.0 ** 126).float().bfloat16().cuda()
    assert rows.isfinite().all()
    kv, _ = _pool("fp4", 64)
    at, pos = torch.arange(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    gd = torch.full((1,), g, device="cuda")
    mla.kv_append(rows, at, pos, table(1).cuda(), kv, gd)
    raw, x = kv[:n].cpu().numpy(), f64(rows)
    quo = np.abs(x[:, :NOPE].reshape(n, 32, 16)).max(-1) / (6 * g)
    fixed = sure(quo, E4M3, 2.0 ** -17)
    assert fixed.mean() > 0.9 and quo.min() > 2.0 ** -6
    assert np.array_equal(raw[:, 256:288][fixed], encode(quo, E4M3)[fixed])
    step = np.repeat(e4m3_values(raw[:, 256:288]) * g, 16, 1)
    got = decode4(raw, g)
    # within half of E2M1's widest step of the block's, or the saturated last part of it
    assert np.all(np.abs(got[:, :NOPE] - x[:, :NOPE]) <= step)
