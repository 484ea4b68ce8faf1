"""Appended rows that hold a NaN read back as NaN where they did, in every format,
and a decode shows them to the rows that see them.
"""
import numpy as np
import pytest
import torch

import mla_latent_decode_gb300 as mla
from latent_ref import NOPE, ROW, table
from mla_latent_decode_gb300 import build
from test_gpu_append import _inputs, _pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("norm", [True, False])
def test_nan_stays(kind, norm):
    rows, weight, _, pos = _inputs(6, 0, 31)
    rows = rows.contiguous()
    rows[1, 100], rows[3, NOPE + 9] = float("nan"), float("nan")  # a latent's value; a RoPE value
    rows[4, :NOPE] = float("nan")
    if norm:
        rows[5, 200] = float("inf")  # inf / inf
    kv, scale = _pool(kind, 64)
    ref, ref_scale = _pool(kind, 64)
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    tab = table(5000).cuda()
    mla.kv_append(rows, slots, pos, tab, kv, scale, norm_weight=weight if norm else None)
    clean = rows.nan_to_num(0.5, posinf=0.5)
    mla.kv_append(clean, slots, pos, tab, ref, ref_scale, norm_weight=weight if norm else None)
    back, was = mla.kv_read(kv, slots, scale), mla.kv_read(ref, slots, ref_scale)
    nan = back.isnan().cpu()
    assert torch.equal(back[[0, 2]], was[[0, 2]]) and not nan[[0, 2]].any()
    assert kind != "fp8" or scale[:6].isfinite().all()
    block = 16 if kind == "fp4" else 1
    want = torch.zeros((6, ROW), dtype=torch.bool)
    want[1, 100 // block * block:100 // block * block + block] = True
    if norm:
        want[1, :NOPE] = True  # the root of the row
        want[5, 200 // block * block:200 // block * block + block] = True
    want[3, NOPE + 8:NOPE + 10] = True  # the pair turns together
    want[4, :NOPE] = True
    assert torch.equal(nan, want)


def test_decode_shows_an_appended_nan():
    """One broken token of a 4-bit cache: NaN for the queries that see it."""
    from test_gpu_fp4_decode import Case
    for q, H in ((3, 16), (3, 60)):
        case = Case(1, q, H, [130], seed=71)
        O, LSE = case.run(1)
        rows = torch.randn((1, ROW), generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
        rows[0, 3] = float("nan")
        at = torch.tensor([int(case.r2t_host[0, 128])], dtype=torch.int32, device="cuda")  # seen by queries 1 and 2
        mla.kv_append(rows, at, torch.zeros(1, dtype=torch.int32, device="cuda"), table(1).cuda(), case.kv, case.gd,
                      norm_weight=torch.ones(NOPE).bfloat16().cuda())
        O2, LSE2 = case.run(1)
        assert torch.equal(O[:, :, :, 0], O2[:, :, :, 0]) and torch.equal(LSE[..., 0, :], LSE2[..., 0, :])
        assert O2[:, :, :, 1:].isnan().all() and LSE2[..., 1:, :].isnan().all()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_a_row_of_nothing_but_nan(kind):
    rows = torch.full((2, ROW), float("nan")).bfloat16().cuda()
    rows[1] = 0
    kv, scale = _pool(kind, 64)
    slots, pos = torch.arange(2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    mla.kv_append(rows, slots, pos, table(1).cuda(), kv, scale)
    back = mla.kv_read(kv, slots, scale)
    assert back[0].isnan().all() and not back[1].any()
    assert kind != "fp8" or not scale[:2].any()
