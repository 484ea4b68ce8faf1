"""Attention within packed prompts (mla_prefill) over hundreds of units a CTA of which some
have values to clean and others have not: sequences without keys, and prefixes of whole
tiles that every row sees.  What is noted of a unit's values is told apart from other
units' and read before it is wiped."""
import math

import numpy as np
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


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


# (queries, keys, prefix): cleaned, whole tiles that all rows see, none at all, more queries than keys
CLEANED, WHOLE, EMPTY, FEW = (5, 5, 0), (4, 128, 128), (3, 0, 0), (6, 2, 0)
MIXES = {
    "every other": [CLEANED, WHOLE] * 30,
    "none between": [CLEANED, EMPTY] * 30,
    "runs": [EMPTY] * 20 + [CLEANED] * 14 + [WHOLE] * 12 + [CLEANED, EMPTY, FEW, WHOLE] * 4,
    "rare": [WHOLE, EMPTY] * 26 + [CLEANED] + [EMPTY] * 10,
}


@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("ctas", [1, 2])
def test_cleaned_units_among_others(mix, ctas):
    lq, lk, pre = (list(x) for x in zip(*MIXES[mix]))
    H = 1200                                       # 60 sequences: more than 200 units a CTA
    g = torch.Generator(device="cuda").manual_seed(ctas)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    Tq, Tk = sum(lq), sum(lk)
    x = dict(q_nope=randn(Tq, H, 128), q_rope=randn(Tq, H, 64), k_nope=randn(Tk, H, 128), v=randn(Tk, H, 128),
             k_rope=randn(Tk, 64))
    starts_q, starts_k = np.concatenate([[0], np.cumsum(lq)]), np.concatenate([[0], np.cumsum(lk)])
    for n, kind in enumerate(MIXES[mix]):
        for i, bad in enumerate((math.nan, math.inf, -math.inf)):
            for h in range((7 * n + i) % 5, H, 5):
                if kind == CLEANED:
                    x["v"][int(starts_k[n]) + 1 + i, h, (n + h + i) % 128] = bad
    work, parts = mla.plan_prefill(lq, lk, H, prefix=pre, ctas=ctas)
    assert parts == 0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    prefix = torch.tensor(pre, dtype=torch.int32, device="cuda")
    args = dict(x, cu_q=_cu(lq), cu_kv=_cu(lk), work=torch.from_numpy(work).cuda(), sm_scale=SCALE, prefix=prefix,
                status=status)
    out = torch.full((Tq, H, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Tq, H), 3.0, device="cuda")
    mla.prefill(**args, out=out, lse_out=lse)
    assert int(status.item()) == 0
    for n in range(len(lq)):
        qs, ks = slice(int(starts_q[n]), int(starts_q[n + 1])), slice(int(starts_k[n]), int(starts_k[n + 1]))
        got, got_lse = out[qs].double(), lse[qs].double()
        if lk[n] == 0:
            assert bool((got == 0).all()) and bool((got_lse == -math.inf).all())
            continue
        q = torch.cat([x["q_nope"][qs], x["q_rope"][qs]], -1).double().transpose(0, 1)
        k = torch.cat([x["k_nope"][ks], x["k_rope"][ks, None].expand(-1, H, -1)], -1).double().transpose(0, 1)
        v = x["v"][ks].double().transpose(0, 1)
        i, t = torch.arange(lq[n], device="cuda")[:, None], torch.arange(lk[n], device="cuda")[None]
        see = (t < pre[n]) | (t <= lk[n] - lq[n] + i)
        s = torch.where(see, SCALE * (q @ k.transpose(1, 2)), -math.inf)
        want_lse = torch.logsumexp(s, -1)
        p = torch.where((want_lse == -math.inf)[..., None], 0.0, torch.exp(s - want_lse[..., None]))
        want = torch.stack([torch.where(see[r][:, None], p[:, r, :, None] * v, 0.0).sum(1) for r in range(lq[n])], 1)
        want = want.transpose(0, 1)
        assert torch.equal(got.isnan(), want.isnan()), n
        assert torch.equal(got[want.isinf()], want[want.isinf()]), n
        fine = want.isfinite()
        # probabilities and outputs rounded to bf16, 2^-8 each of values below 6 (scores' and sums'
        # fp32 roundings are below a hundredth of that)
        assert bool(((got - want).abs()[fine] <= 2.02 * 2.0 ** -8 * 6).all()), n
        live = want_lse.T.isfinite()
        assert torch.equal(got_lse.isfinite(), live)
        assert bool(((got_lse - want_lse.T).abs()[live] <= 2.0 ** -11).all()), n
    again = torch.full_like(out, 3.0)
    mla.prefill(**args, out=again, lse_out=lse)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
