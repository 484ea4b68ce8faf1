"""Decode over the 4-bit cache where the factor of a row's scores leaves fp32's
range: pools with a very small or very large factor, queries of zeros, and more
rows than one CTA takes at far magnitudes.  Tolerances of test_gpu_fp4_decode.
"""
import numpy as np
import pytest
import torch

import mla_latent_decode_gb300 as mla
from mla_latent_decode_gb300 import build
from test_gpu_fp4_decode import Case, check

pytestmark = pytest.mark.gpu
ROWS = [(2, 5), (3, 32), (3, 43), (5, 96)]  # 10, 96, 129 and 480 rows


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


@pytest.mark.parametrize("q,H", ROWS)
@pytest.mark.parametrize("g", [2.0 ** -30, 2.0 ** -40, 2.0 ** -60, 2.0 ** -90])
def test_zero_queries_with_a_small_factor(q, H, g):
    """A row of zeros (or of tiny values) weighs what it sees alike; masked tokens
    in its tiles stay masked."""
    case = Case(2, q, H, [200, 70], seed=50, g=g)
    case.q_nope[:, 0], case.q_rope[:, 0] = 0, 0
    case.q_nope[0, 1] *= 2.0 ** -110
    case.q_rope[0, 1] *= 2.0 ** -110
    case.up()
    O, LSE = case.run(2)
    check(case, O, LSE, 2, heads=[0, H - 1])


@pytest.mark.parametrize("q,H", ROWS)
@pytest.mark.parametrize("q_scale,g", [(1e-20, 1.0), (1e18, 1e-18), (1.0, 2.0 ** -60), (30.0, 0.0625)])
def test_magnitudes(q, H, q_scale, g):
    case = Case(2, q, H, [200, 70], seed=51, q_scale=q_scale, g=g)
    O, LSE = case.run(2)
    check(case, O, LSE, 2, heads=[0, H - 1])


@pytest.mark.parametrize("q,H", ROWS)
def test_zero_scores_under_a_large_factor(q, H):
    """Keys of zeros score 0 whatever the queries and the factor are."""
    case = Case(1, q, H, [300], seed=52, q_scale=1e30, g=1e20)
    case.kv_host[case.r2t_host[0, :300], 256:] = 0
    case.up()
    O, LSE = case.run(1)
    check(case, O, LSE, 1, heads=[0, H - 1])
