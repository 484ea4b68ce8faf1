"""Prompt chunks over the 4-bit cache: far more query rows a request than drafts
have, most of them masked from most of the chunk, against the definition in 64
bits with the tolerances of test_gpu_fp4_decode.
"""
import numpy as np
import pytest
import torch

import mla_latent_decode_gb300 as mla
from mla_latent_decode_gb300 import build
from test_gpu_fp4_decode import Case, check

pytestmark = pytest.mark.gpu
# (queries, heads, lengths): 1000 to 3000 rows, chunks that open the context and later ones
CHUNKS = [(64, 16, [64, 700]), (200, 5, [200, 333, 1000]), (33, 33, [50, 129]), (300, 10, [301])]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


@pytest.mark.parametrize("q,H,lens", CHUNKS)
@pytest.mark.parametrize("S", [1, 3])
def test_chunk_in_clusters(q, H, lens, S):
    case = Case(len(lens), q, H, lens, seed=60 + q)
    O, LSE = case.run(S)
    assert case.status == 0
    check(case, O, LSE, S, heads=[0, H - 1])


@pytest.mark.parametrize("q,H,lens", CHUNKS)
def test_chunk_in_row_groups(q, H, lens):
    """The same in groups of 96 rows, one CTA each, in any order."""
    case = Case(len(lens), q, H, lens, seed=60 + q)
    S, U = 2, -(-q * H // 96)
    order = np.random.default_rng(1).permutation(len(lens) * S * U)
    O, LSE = case.run(S, work=order)
    assert case.status == 0
    check(case, O, LSE, S, heads=[0, H - 1])


@pytest.mark.parametrize("q,H,lens", CHUNKS[:2])
def test_chunk_as_planned_and_merged(q, H, lens):
    case = Case(len(lens), q, H, lens, seed=61 + q)
    S, bnd, work, _ = mla.plan_sched(len(lens), q, H, lens, kv_dtype="fp4_e2m1")
    O, LSE = case.run(S, bnd=bnd, work=work)
    assert case.status == 0
    check(case, O, LSE, S, bnd=bnd, heads=[0, H - 1])


def test_chunk_with_limits_of_any_order():
    """kv_limit as a tree of drafts has it: not rising along the queries."""
    q, H, lens = 40, 12, [500, 90]
    lim = np.random.default_rng(2).integers(-3, 520, (2, q))
    lim[0, 5], lim[1, 7], lim[1, 8] = 0, 500, 1
    case = Case(2, q, H, lens, limits=lim.tolist(), seed=62)
    for kw in (dict(), dict(work=np.arange(2 * 2 * -(-q * H // 96)))):
        O, LSE = case.run(2, **kw)
        assert case.status == 0
        check(case, O, LSE, 2, heads=[0, H - 1])


def test_nan_token_within_a_chunk():
    """Only the queries at and after a broken token see it."""
    q, H, L = 100, 3, 230
    for work in (None, np.arange(-(-q * H // 96))):
        case = Case(1, q, H, [L], seed=63)
        O, LSE = case.run(1, work=work)
        at = L - q + 60  # seen by queries 60 and later
        case.kv_host[case.r2t_host[0, at], 256:] = 0x7F
        case.up()
        O2, LSE2 = case.run(1, work=work)
        assert torch.equal(O[:, :, :, :60], O2[:, :, :, :60]) and torch.equal(LSE[..., :60, :], LSE2[..., :60, :])
        assert O2[:, :, :, 60:].isnan().all() and LSE2[..., 60:, :].isnan().all()
