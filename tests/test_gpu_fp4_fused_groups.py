"""decode_fused over row groups of 96 rows: the merge of the very parts that
decode_partial writes, counters left zero, and its time beside the two launches'.
"""
import numpy as np
import pytest
import torch

import mla_latent_decode_gb300 as mla
from mla_latent_decode_gb300 import build
from test_gpu_fp4_decode import SCALE, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


# rows a request: 97 to 1000, one to eleven groups, counters shared by two groups or not
@pytest.mark.parametrize("q,H", [(1, 97), (1, 128), (2, 96), (3, 86), (3, 128), (5, 96), (8, 77), (10, 100)])
@pytest.mark.parametrize("S,shards", [(1, 1), (3, 1), (2, 2)])
def test_groups_merge_in_one_launch(q, H, S, shards):
    B = 2
    case = Case(B, q, H, [300, 70, 129, 500][:B * shards], shards=shards, seed=70 + H)
    U = -(-q * H // 96)
    work = np.random.default_rng(H).permutation(B * shards * S * U).astype(np.int32)
    O, LSE = case.run(S, work=work)
    out, lse = mla.lse_combine(O, LSE)
    counters = mla.fused_counters(B, q, H, "cuda")
    for _ in range(2):
        got, got_lse = mla.decode_fused(case.qn, case.qr, case.kv, case.gd, case.r2t, case.sl, None, S, SCALE,
                                        num_shards=shards, counters=counters, work=torch.from_numpy(work).cuda())
        assert torch.equal(got, out) and torch.equal(got_lse, lse)
        assert not counters.any()
