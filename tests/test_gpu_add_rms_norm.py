"""GPU parity of the residual RMS norm (mla_add_rms_norm) with the float64
definition.

Tolerances, from the roundings: h = x + residual is rounded to fp32 once
(2^-24); the sum of squares is at most 32 + 10 additions deep, so y stays within
2^-18 relative; a bf16 output adds 2^-8.  A code must equal the definition's,
on the stored scale, wherever a 2^-17 change of the quotient would not move it.
"""
import numpy as np
import pytest
import torch

import mla_latent_decode_gb300 as mla
from latent_ref import E4M3, e4m3_values, encode, f64, sure
from mla_latent_decode_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


def _rows(n, d, seed, pad=0):
    t = torch.randn((n, d + pad), generator=torch.Generator().manual_seed(seed))
    return t.bfloat16().cuda()[:, pad:]


def _check(x, res, w, eps, got):
    out, out8, scales, res_out = got
    h = f64(x) + (f64(res) if res is not None else 0.0)
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * f64(w)
    if res is not None:
        assert np.all(np.abs(f64(res_out) - h) <= (2.0 ** -8 + 2.0 ** -24) * np.abs(h))
    if out is not None:
        assert np.all(np.abs(f64(out) - y) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(y))
    if out8 is not None:
        n, d = y.shape
        s = f64(scales)
        groups = y.reshape(n, s.shape[1], -1)
        amax = np.abs(groups).max(-1)
        assert np.all(np.abs(s - amax / 448) <= 2.0 ** -17 * amax / 448)
        codes = out8.view(torch.uint8).cpu().numpy()
        sw = np.repeat(s, groups.shape[2], 1)
        q = np.where(sw > 0, y / np.where(sw > 0, sw, 1.0), 0.0)
        fixed = sure(q, E4M3, 2.0 ** -17)
        assert fixed.mean() > 0.99 or y.size < 100
        assert np.array_equal((codes & 0x7F)[fixed], encode(q, E4M3)[fixed])
        err = np.abs(e4m3_values(codes) * sw - y)
        assert np.all(err <= 2.0 ** -4 * np.abs(y) + 2.0 ** -10 * sw + 2.0 ** -17 * np.abs(y))


@pytest.mark.parametrize("n,d,group", [
    (1, 1, 0), (3, 8, 0), (2, 100, 0), (5, 576, 64), (7, 1536, 128), (80, 7168, 0),
    (33, 7168, 128), (4, 4000, 32), (2, 8200, 0), (3, 16384, 128), (2, 32768, 0), (2, 31, 0)])
@pytest.mark.parametrize("residual", [True, False])
def test_matches_definition(n, d, group, residual):
    x, w = _rows(n, d, 1), (1 + 0.3 * _rows(1, d, 2)[0].float()).bfloat16()
    res = 3 * _rows(n, d, 3) if residual else None
    res_out = torch.empty_like(res) if residual else None
    out = torch.empty((n, d), dtype=torch.bfloat16, device="cuda")
    keep = None if res is None else res.clone()
    got = mla.add_rms_norm(x, w, res, 1e-5, out=out, e4m3=True, group=group, residual_out=res_out)
    _check(x, res, w, 1e-5, got)
    assert res is None or torch.equal(res, keep)


@pytest.mark.parametrize("pad", [1, 4, 8])
def test_strided_and_misaligned_rows(pad):
    n, d = 6, 640
    x, w, res = _rows(n, d, 4, pad), _rows(1, d, 5)[0].contiguous(), _rows(n, d, 6, pad)
    wide8 = torch.zeros((n, d + 2 * pad), dtype=torch.uint8, device="cuda")
    wide = torch.zeros((n, d + 2 * pad), dtype=torch.bfloat16, device="cuda")
    out, out8 = wide[:, pad:pad + d], wide8[:, pad:pad + d]
    scales = torch.full((n, 9), -1.0, device="cuda")[:, 2:7]
    got = mla.add_rms_norm(x, w, res.clone(), out=out, out8=out8, scales=scales, group=128)
    _check(x, res, w, 1e-6, got)
    for t in (wide, wide8):
        assert int((t[:, :pad] != 0).sum()) == 0 and int((t[:, pad + d:] != 0).sum()) == 0


def test_in_place_zeros_and_one_output():
    n, d = 9, 1536
    x, w, res = _rows(n, d, 7), _rows(1, d, 8)[0].contiguous(), _rows(n, d, 9)
    x[2] = 0
    res[2] = 0
    x[4] *= 2.0 ** 60  # the square of such a value stays in fp32
    x0, res0 = x.clone(), res.clone()
    out, out8, scales, res_out = mla.add_rms_norm(x, w, res, out=x)  # both in place
    assert out is x and res_out is res and out8 is None and scales is None
    _check(x0, res0, w, 1e-6, (out, None, None, res_out))
    _, out8, scales, _ = mla.add_rms_norm(x0, w, None, e4m3=True)
    assert float(scales[2]) == 0 and int(out8.view(torch.uint8)[2].max()) == 0
    _check(x0, None, w, 1e-6, (None, out8, scales, None))
    assert mla.add_rms_norm(x0[:0], w)[0].shape == (0, d)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    again = mla.add_rms_norm(x0, w, res0.clone(), stream=s)[0]
    s.synchronize()
    assert torch.equal(again, out)


def test_many_rows():
    """More rows than a grid dimension of 65535 would hold."""
    n, d = 70001, 64
    x, w = _rows(n, d, 10), _rows(1, d, 11)[0].contiguous()
    got = mla.add_rms_norm(x, w, None, e4m3=True, out=torch.empty_like(x), group=32)
    _check(x, None, w, 1e-6, got)


@pytest.mark.parametrize("n,d", [(9, 1), (17, 7), (16, 9), (700, 1531), (700, 5003), (400, 7001), (3, 32761), (2, 32759)])
@pytest.mark.parametrize("off", [0, 3])
def test_rows_shifted_alike(n, d, off):
    """Odd lengths: every row at another distance from a vector's boundary, the
    same in all arrays, and nothing written outside the rows."""
    def frame(k, dtype):
        flat = torch.zeros(off + n * d + 16, dtype=dtype, device="cuda")
        if k is not None:
            flat[off:off + n * d] = _rows(1, n * d, k)[0]
        return flat, flat[off:off + n * d].view(n, d)

    (_, x), (_, res), w = frame(20, torch.bfloat16), frame(21, torch.bfloat16), _rows(1, d, 22)[0].contiguous()
    keep = res.clone()
    flat, out = frame(None, torch.bfloat16)
    flat8, out8 = frame(None, torch.uint8)
    got = mla.add_rms_norm(x, w, res, out=out, out8=out8)
    _check(x, keep, w, 1e-6, got)
    for t in (flat, flat8):
        assert int((t[:off] != 0).sum()) == 0 and int((t[off + n * d:] != 0).sum()) == 0
    # arrays that are not shifted alike
    other = torch.zeros(n * d + 1, dtype=torch.bfloat16, device="cuda")[1:].view(n, d)
    _check(x, keep, w, 1e-6, mla.add_rms_norm(x, w, keep.clone(), out=other, e4m3=True))


@pytest.mark.parametrize("d", [7168, 7167])
def test_more_values_than_32_bits_count(d):
    n = 300_001
    assert n * d > 1 << 31
    x = torch.zeros((n, d), dtype=torch.bfloat16, device="cuda")
    last, w = _rows(5, d, 30), _rows(1, d, 31)[0].contiguous()
    x[-5:] = last
    _, out8, scales, _ = mla.add_rms_norm(x, w, None, e4m3=True)
    _check(last, None, w, 1e-6, (None, out8[-5:], scales[-5:], None))
    assert not out8[:5].view(torch.uint8).any()
