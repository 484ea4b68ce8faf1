"""Decode over the 4-bit cache where a long tail of small probabilities is what the
output consists of: one token holds the maximum and a value of zero, tens of
thousands lie 17 to 19 nats below it and all point the same way.

A probability reaches the second product as f16, the row's maximum at 2^6 or more,
so it is off by 2^-11 of itself or, where that is more, by half of f16's last
step: 2^-25 / 2^6 of the maximum, which is a bound of 2^-31 |v| for each token.
"""
import numpy as np
import pytest
import torch

import mla_latent_decode_gb300 as mla
from latent_ref import E4M3, encode, f64
from mla_latent_decode_gb300 import build
from test_gpu_fp4_decode import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


def tail_case(q, H, L, at):
    """Scores from the RoPE key alone; token `at` of the request is the sink."""
    case = Case(1, q, H, [L], seed=40, g=2.0 ** -4)
    case.q_nope[:] = 0
    case.q_rope[:] = 0
    case.q_rope[..., 0] = 9.0   # the sink's score
    case.q_rope[..., 1] = 1.0   # spreads the tail over two nats
    r = np.random.default_rng(41)
    kv = case.kv_host[case.r2t_host[0, :L]]
    kv[:, :256] = r.integers(0x1, 0x8, (L, 256)) * 0x11  # values of one sign
    kv[:, 256:288] = encode(1.0, E4M3)
    kv[:, 288:] = 0
    kv[:, 289] = encode(r.uniform(0.0, 448.0, L), E4M3)  # up to 2 nats: 28 * SCALE
    kv[at, :256] = 0
    kv[at, 288] = encode(480.0, E4M3)                    # 9 * 28 * SCALE = 18.2 nats
    kv[at, 289] = encode(230.0, E4M3)
    case.kv_host[case.r2t_host[0, :L]] = kv
    case.up()
    return case


def check_tail(case, O, LSE, S):
    L = case.lens[0]
    P = -(-L // 64)
    for s in range(S):
        t0, t1 = s * P // S * 64, min((s + 1) * P // S * 64, L)
        heads = [0, case.H - 1]
        ref, lse, A, E, vmax = case.expect(0, t0, t1, heads)
        got = f64(O[s, 0, 0][:, heads]).reshape(ref.shape)
        floor = (t1 - t0) * 2.0 ** -31 * vmax
        tol = (2.0 ** -11 + 2.0 ** -12 + E[:, None] * 2.0 ** -14) * A + floor
        assert np.abs(ref).min() > 4 * floor  # the bound would notice a lost tail
        assert np.all(np.abs(got - ref) <= tol), (s, (np.abs(got - ref) / tol).max())
        gl = f64(LSE[s, 0, 0][:, heads]).reshape(lse.shape)
        assert np.all(np.abs(gl - lse) <= E * 2.0 ** -15 + 2.0 ** -18)


@pytest.mark.parametrize("H", [16, 32, 64, 96])
@pytest.mark.parametrize("at", [0, 9000])
def test_long_tail_few_rows(H, at):
    case = tail_case(1, H, 20011, at)
    O, LSE = case.run(1)
    assert case.status == 0
    check_tail(case, O, LSE, 1)


@pytest.mark.parametrize("q,H", [(1, 97), (2, 96), (5, 96)])
@pytest.mark.parametrize("at", [0, 9000])
@pytest.mark.parametrize("S", [1, 3])
def test_long_tail_clusters(q, H, at, S):
    """More than 96 rows; parts without the sink have the tail as their maximum."""
    case = tail_case(q, H, 20011, at)
    O, LSE = case.run(S)
    assert case.status == 0
    check_tail(case, O, LSE, S)


@pytest.mark.parametrize("q,H", [(1, 16), (1, 96), (5, 96)])
def test_rising_maxima_keep_the_tail(q, H):
    """Sinks that rise by two nats along the context: sums and outputs are rescaled
    again and again, by references that lie below the maxima they come from."""
    case = tail_case(q, H, 6011, 6000)
    rows = case.r2t_host[0, 100:6000:600]
    case.kv_host[rows, :256] = 0
    case.kv_host[rows, 288] = encode(44.8 * np.arange(10), E4M3)
    case.up()
    O, LSE = case.run(1)
    assert case.status == 0
    check_tail(case, O, LSE, 1)
