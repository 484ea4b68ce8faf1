"""Attention within packed prompts (mla_prefill): which outputs are finite depends on the
inputs alone, not on where a plan cuts the keys into parts.

By the definition a value that is not finite makes the outputs of its dim NaN or infinite
in the rows that see it, however small its probability; a row that sees only keys with
s = -inf has out = 0 and lse = -inf, and a row that sees such keys among others sees their
values with probability 0, and 0 x inf is NaN."""
import math

import pytest
import torch

import mla_latent_decode_gb300 as mla
from mla_latent_decode_gb300 import build

pytestmark = pytest.mark.gpu
SCALE = 192.0 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


def _inputs(lq, lk, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    return dict(q_nope=randn(lq, H, 128), q_rope=randn(lq, H, 64), k_nope=randn(lk, H, 128), v=randn(lk, H, 128),
                k_rope=randn(lk, 64))


def _run(x, lq, lk, H, sms, ctas, causal=True):
    work, parts = mla.plan_prefill([lq], [lk], H, num_sms=sms, ctas=ctas, causal=causal)
    cu_q, cu_kv = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (lq, lk))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = mla.prefill(**x, cu_q=cu_q, cu_kv=cu_kv, work=torch.from_numpy(work).cuda(), sm_scale=SCALE,
                           num_parts=parts, status=status, causal=causal)
    assert int(status.item()) == 0
    return out, lse, parts


@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("low_first", [True, False])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_values_of_vanishing_probability(bad, low_first, ctas):
    """A part whose scores lie more than 104 below another's weighs nothing, but what it holds counts."""
    lq, lk, H = 70, 6000, 16
    x = _inputs(lq, lk, H, 1)
    x["q_nope"][:] = 4.0
    low = slice(0, lk // 2) if low_first else slice(lk // 2, lk)
    x["k_nope"][:] = 8.0
    x["k_nope"][low] = -8.0                                  # (scores 2 x 4096 x SCALE = 591 below)
    at = low.start + 700
    x["v"][at, 3, 5] = bad
    x["v"][at + 1, 7, 100] = bad
    whole, whole_lse, none = _run(x, lq, lk, H, 1, ctas)
    cut, cut_lse, parts = _run(x, lq, lk, H, 300, ctas)
    assert none == 0 and parts > 0
    want = torch.ones_like(whole, dtype=torch.bool)
    want[:, 3, 5] = want[:, 7, 100] = False
    assert torch.equal(whole.isfinite(), want)
    assert torch.equal(cut.isfinite(), want)
    assert bool(whole_lse.isfinite().all() and cut_lse.isfinite().all())


@pytest.mark.parametrize("ctas", [1, 2])
def test_values_of_probability_zero(ctas):
    """Keys with s = -inf in one part, others elsewhere; the last queries' own tokens among them."""
    lq, lk, H = 70, 6000, 16
    x = _inputs(lq, lk, H, 2)
    x["q_nope"][:] = x["q_nope"].abs() + 0.125
    for span in (slice(0, 2500), slice(lk - lq, lk)):
        x["k_nope"][span, :, 0] = -math.inf
    x["v"][100, 3, 5] = math.nan
    x["v"][lk - 30, 4, 6] = math.inf                         # seen by the last 30 rows
    whole, whole_lse, _ = _run(x, lq, lk, H, 1, ctas)
    cut, cut_lse, parts = _run(x, lq, lk, H, 300, ctas)
    assert parts > 0
    want = torch.ones_like(whole, dtype=torch.bool)
    want[:, 3, 5] = False
    want[-30:, 4, 6] = False
    assert torch.equal(whole.isfinite(), want)
    assert torch.equal(cut.isfinite(), want)
    # the same scores; probabilities and outputs rounded to bf16 on either side, 4 x 2^-8 of values
    # below 6; sums of up to 6000 / 4 terms in a row
    assert bool(((whole.float() - cut.float()).abs()[want] <= 4 * 2.0 ** -8 * 6).all())
    assert bool(((whole_lse - cut_lse).abs() <= 2.0 ** -12).all())


@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("lk,sms", [(200, 1), (6000, 1), (6000, 300)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_rows_that_see_only_impossible_keys(bad, lk, sms, ctas):
    """out = 0 and lse = -inf, whatever the values hold and wherever they stand."""
    lq, H = 100, 16
    x = _inputs(lq, lk, H, 3)
    x["q_nope"][:] = x["q_nope"].abs() + 0.125
    x["k_nope"][:, 2, 0] = -math.inf
    x["k_nope"][:, 5, 0] = -math.inf
    for t in (3, lk - lq + 10, lk - 1):
        x["v"][t, 2] = bad
        x["v"][t, 4, 9] = bad                                # a head with ordinary keys
    out, lse, _ = _run(x, lq, lk, H, sms, ctas)
    for h in (2, 5):
        assert bool((out[:, h] == 0).all()) and bool((lse[:, h] == -math.inf).all())
    other = out[:, 4]
    assert not bool(other[:, 9].isfinite().any())
    assert bool(other[:, :9].isfinite().all() and other[:, 10:].isfinite().all())
