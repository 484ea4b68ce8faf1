"""GPU parity of the attention within packed prompts (mla_prefill) with the
float64 definition.

Tolerances, from the roundings.  A score is a sum of 192 products in fp32: within
d = 200 * 2^-24 * scale * sum |q_i k_i|, and the exponent's own arithmetic adds
4 * 2^-24 |s| (scaling, difference) and the exponential 2^-21, so a probability is
within (2 d + 8 * 2^-24 max |s| + 2^-20) of itself before it is rounded to bf16
(2^-8).  Sums over n keys add n 2^-24.  The output is sum p v, within that of
sum p |v|, rounded to bf16 (2^-8).  The lse is within the same bound without the
bf16 rounding (those are summed in fp32) plus 2^-22 of itself.
"""
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


def _inputs(lq, lk, H, seed=0, spare=0, wide=True):
    """Random inputs; with `wide` they are views into a projection's rows."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    Tq, Tk = sum(lq) + spare, sum(lk) + spare

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    if wide:
        q, kv, rows = randn(Tq, H, 192), randn(Tk, H, 256), randn(Tk, 576)
        return dict(q_nope=q[..., :128], q_rope=q[..., 128:], k_nope=kv[..., :128], v=kv[..., 128:],
                    k_rope=rows[:, 512:])
    return dict(q_nope=randn(Tq, H, 128), q_rope=randn(Tq, H, 64), k_nope=randn(Tk, H, 128),
                v=randn(Tk, H, 128), k_rope=randn(Tk, 64))


def _visible(lq, lk, pre, causal):
    i = torch.arange(lq, device="cuda")[:, None]
    t = torch.arange(lk, device="cuda")[None]
    if not causal:
        return torch.ones((lq, lk), dtype=torch.bool, device="cuda")
    return (t < pre) | (t <= lk - lq + i)


def _reference(x, lq, lk, pre, causal, scale=SCALE):
    """out, lse and their bounds for every row of the packed sequences, float64."""
    H = x["q_nope"].shape[1]
    outs = []
    qa = ka = 0
    for n in range(len(lq)):
        qs, ks = slice(qa, qa + lq[n]), slice(ka, ka + lk[n])
        qa, ka = qa + lq[n], ka + lk[n]
        q = torch.cat([x["q_nope"][qs], x["q_rope"][qs]], -1).double().transpose(0, 1)
        k = torch.cat([x["k_nope"][ks], x["k_rope"][ks, None].expand(-1, H, -1)], -1).double().transpose(0, 1)
        v = x["v"][ks].double().transpose(0, 1)
        see = _visible(lq[n], lk[n], pre[n] if pre else 0, causal)
        s = torch.where(see, scale * (q @ k.transpose(1, 2)), -math.inf)
        d = 200 * 2.0 ** -24 * scale * (q.abs() @ k.abs().transpose(1, 2)).masked_fill(~see, 0).amax(-1) \
            if lk[n] else torch.zeros((H, lq[n]), dtype=torch.float64, device="cuda")
        top = torch.where(see, s.abs(), 0.0).amax(-1) if lk[n] else torch.zeros_like(d)
        lse = torch.logsumexp(s, -1) if lk[n] else torch.full_like(d, -math.inf)
        p = torch.where(see, torch.exp(s - lse[..., None]), 0.0)
        p = torch.where((lse == -math.inf)[..., None], 0.0, p)
        # rows of a NaN score are NaN; values that a row does not see do not count
        o = torch.stack([torch.where(see[i][:, None], p[:, i, :, None] * v, 0.0).sum(1) for i in range(lq[n])], 1) \
            if not bool(v.isfinite().all()) else p @ v
        rel = 2 * d + 8 * 2.0 ** -24 * top + 2.0 ** -20 + lk[n] * 2.0 ** -24
        tol = 2.0 ** -8 * o.abs() * (1 + 2.0 ** -7) + (2.0 ** -8 + rel)[..., None] * (p @ v.abs().nan_to_num(0, 0, 0))
        outs.append((o.transpose(0, 1), lse.T, tol.transpose(0, 1), (rel + 2.0 ** -22 * lse.abs().nan_to_num(0, 0, 0)).T))
    return tuple(torch.cat([o[i] for o in outs]) for i in range(4))


def _run(x, lq, lk, pre, causal, scale=SCALE, plan=None, ctas=0, **more):
    H = x["q_nope"].shape[1]
    work, parts = plan or mla.plan_prefill(lq, lk, H, prefix=pre, causal=causal, ctas=ctas)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    prefix = None if pre is None else torch.tensor(pre, dtype=torch.int32, device="cuda")
    out, lse = mla.prefill(**x, cu_q=_cu(lq), cu_kv=_cu(lk), work=torch.from_numpy(work).cuda(), sm_scale=scale,
                           prefix=prefix, causal=causal, num_parts=parts, status=status, **more)
    assert int(status.item()) == 0
    return out, lse, parts


def _check(x, lq, lk, pre, causal, scale=SCALE, **more):
    out, lse, parts = _run(x, lq, lk, pre, causal, scale, **more)
    o, l, tol, ltol = _reference(x, lq, lk, pre, causal, scale)
    n = sum(lq)
    got = out[:n].double()
    nan = o.isnan()
    assert torch.equal(got.isnan(), nan)
    inf = o.isinf()
    assert torch.equal(got[inf], o[inf])
    fine = ~nan & ~inf
    assert bool(((got - o).abs() <= tol)[fine].all()), float(((got - o).abs() / tol)[fine].max())
    empty = l == -math.inf
    assert torch.equal(lse[:n] == -math.inf, empty)
    fine = ~empty & ~l.isnan()
    assert torch.equal(lse[:n].isnan(), l.isnan())
    assert bool(((lse[:n].double() - l).abs() <= ltol)[fine].all())
    return out, lse, parts


@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("lq,lk,pre,H,causal", [
    ([1], [1], None, 1, True),
    ([17], [17], None, 16, True),
    ([127, 128, 129], [127, 128, 129], None, 3, True),
    ([255, 256, 257], [255, 256, 257], None, 2, True),
    ([600], [600], None, 5, True),
    ([1, 3, 130, 0, 64], [900, 3, 400, 0, 1000], None, 4, True),       # context in the cache, an empty sequence
    ([200, 300], [200, 300], [64, 299], 3, True),                      # prefixes, one inside a tile
    ([200, 300, 5], [200, 300, 500], [200, 1000, 0], 3, True),         # a prefix of all, one past the end
    ([150, 70], [20, 0], None, 2, True),                               # more queries than keys: rows that see none
    ([150, 70], [20, 0], [20, 5], 2, True),
    ([100, 260], [300, 129], None, 2, False),                          # in full
    ([1] * 40, list(range(1, 41)), None, 8, True),
    ([512, 511, 1030], [512, 640, 1030], [0, 513, 700], 2, True),      # around a pair's block
])
def test_matches_the_definition(lq, lk, pre, H, causal, ctas):
    _check(_inputs(lq, lk, H), lq, lk, pre, causal, ctas=ctas)


@pytest.mark.parametrize("ctas", [1, 2])
def test_many_units_a_cta(ctas):
    """CTAs take over units that have not started, with and without keys, cleaned values and parts."""
    lens = [300, 1, 64, 129, 0, 513, 40, 257] * 4
    ctx = [0, 700, 0, 128, 3, 0, 0, 1] * 4
    pre = [0, 0, 64, 5, 0, 600, 40, 0] * 4
    lk = [a + c for a, c in zip(lens, ctx)]
    lk[7] = 0                                                          # rows that see nothing, between others
    x = _inputs(lens, lk, 24, seed=2)
    x["v"][500, 3, 7] = math.inf
    x["v"][2000, 20, 100] = math.nan
    _check(x, lens, lk, pre, True, ctas=ctas)


@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("lq,lk,H", [([200], [9000], 2), ([64, 300], [5000, 12000], 1), ([1], [20000], 3)])
def test_keys_cut_into_parts(lq, lk, H, ctas):
    x = _inputs(lq, lk, H, seed=3, wide=False)
    *_, parts = _check(x, lq, lk, None, True, ctas=ctas)
    assert parts > 1


def test_every_cut_is_the_same_sum():
    """Plans for few and many SMs cut differently; each is within the bound."""
    lq, lk, H = [300, 10], [3000, 1500], 2
    x = _inputs(lq, lk, H, seed=5)
    seen = set()
    for sms in (1, 4, 16, 64, 300):
        for ctas in (1, 2):
            plan = mla.plan_prefill(lq, lk, H, num_sms=sms, ctas=ctas)
            _check(x, lq, lk, None, True, plan=plan)
            seen.add(plan[1])
    assert len(seen) > 1


@pytest.mark.parametrize("ctas", [1, 2])
def test_large_scores_and_their_order(ctas):
    """Maxima that rise through the sequence, fall, or sit on one key: the reference moves."""
    lq, lk, H = [300], [300], 3
    x = _inputs(lq, lk, H, seed=6, wide=False)
    ramp = torch.linspace(0.0, 12.0, 300, device="cuda")
    x["k_nope"][:, 0] = (x["k_nope"][:, 0].float() + ramp[:, None]).bfloat16()
    x["k_nope"][:, 1] = (x["k_nope"][:, 1].float() + ramp.flip(0)[:, None]).bfloat16()
    x["k_nope"][7, 2] = 30.0
    x["q_nope"] = x["q_nope"].abs()
    _check(x, lq, lk, None, True, ctas=ctas)


@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_keys_and_values_that_a_row_does_not_see(bad, ctas):
    """A token's key and value reach the rows that see it and no other, whatever they hold."""
    lq, lk, pre, H = [200, 90, 40], [200, 350, 40], [0, 0, 40], 2
    x = _inputs(lq, lk, H, seed=7, spare=64, wide=False)
    clean, _, _ = _run(x, lq, lk, pre, True, ctas=ctas)
    x["v"][130, 0, 5] = bad            # sequence 0, seen from row 130 on
    x["v"][199, 1, 127] = bad          # its last token, seen by its last row
    x["v"][200 + 300, 1, 64] = bad     # sequence 1: context and drafts
    x["k_nope"][150, 1, 3] = math.nan
    x["v"][sum(lk):] = math.nan        # behind the last sequence
    x["k_nope"][sum(lk):] = math.nan
    x["k_rope"][sum(lk):] = math.nan
    out, _, _ = _check(x, lq, lk, pre, True, ctas=ctas)
    assert torch.equal(out[:130], clean[:130])
    assert torch.equal(out[290:330], clean[290:330])


@pytest.mark.parametrize("ctas", [1, 2])
def test_ends_of_many_sequences(ctas):
    """Launches of many units load sequences' ends in boxes of 32 rows; what is left of other
    tiles in shared memory, NaN among it, reaches no row."""
    lens = [1, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 160, 200, 255, 257]
    lk = [n + c for n, c in zip(lens, [0, 7, 64, 0, 31, 1, 95, 33, 0, 128, 2, 96, 0, 40, 8, 0, 63])]
    x = _inputs(lens, lk, 40, seed=4, spare=32)
    g = torch.Generator().manual_seed(5)
    for name in ("k_nope", "v"):
        for _ in range(12):
            t, h = int(torch.randint(sum(lk), (1,), generator=g)), int(torch.randint(40, (1,), generator=g))
            x[name][t, h, int(torch.randint(128, (1,), generator=g))] = math.nan
    for name in ("k_nope", "v", "k_rope"):
        x[name][sum(lk):] = math.nan
    for name in ("q_nope", "q_rope"):
        x[name][sum(lens):] = math.nan
    _check(x, lens, lk, None, True, ctas=ctas)
    _check(x, lens, lk, [0, 9] * 8 + [3], True, ctas=ctas)


def test_broken_values_in_hundreds_of_units_a_cta():
    """Notes on cleaned values are told apart over more units than their tags have numbers."""
    lens, H = [5] * 60, 1200
    x = _inputs(lens, lens, H, seed=8, wide=False)
    for n in range(60):
        for i, bad in enumerate((math.nan, math.inf, -math.inf)):
            x["v"][5 * n + 1 + i, (37 * n + 400 * i) % H, (n + i) % 128] = bad
    _check(x, lens, lens, None, True, ctas=1)


def test_rows_behind_the_last_sequence_stay():
    lq, lk, H = [100], [100], 2
    x = _inputs(lq, lk, H, spare=50)
    out = torch.full((150, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((150, H), 9.0, device="cuda")
    _check(x, lq, lk, None, True, out=out, lse_out=lse)
    assert bool((out[100:] == 7.0).all()) and bool((lse[100:] == 9.0).all())


def test_small_and_large_scales():
    lq = lk = [140]
    for scale in (1e-8, 3.0):
        _check(_inputs(lq, lk, 2, seed=9), lq, lk, None, True, scale=scale)


def test_nothing_to_do():
    x = _inputs([], [], 2, spare=3)
    out = torch.full((3, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    _run(x, [], [], None, True, out=out)
    _run(x, [0, 0], [1, 2], None, True, out=out)
    assert bool((out == 5.0).all())


@pytest.mark.parametrize("ctas", [1, 2])
def test_bad_work_and_lengths_are_reported(ctas):
    lq = lk = [100, 30]
    x = _inputs(lq, lk, 2)
    work, _ = mla.plan_prefill(lq, lk, 2, ctas=ctas)

    def status_of(work, cu_q=_cu(lq), cu_kv=_cu(lk), num_parts=0):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        mla.prefill(**x, cu_q=cu_q, cu_kv=cu_kv, work=torch.from_numpy(work).cuda(), sm_scale=SCALE,
                    num_parts=num_parts, status=status)
        return int(status.item())

    assert status_of(work) == 0
    for column, value in ((0, 2), (0, -1), (1, 1), (1, -1), (2, 1), (2, -1), (3, 0), (3, 33), (5, 5), (5, -1),
                          (6, 0), (6, 9), (7, 256)):
        bad = work.copy()
        bad[0, ..., column] = value
        assert status_of(bad) == mla.STATUS_BAD_WORK, (column, value)
    bad = work.copy()
    bad[0, ..., 2:5] = 0, 2, 3
    assert status_of(bad, num_parts=2 * ctas) == mla.STATUS_BAD_WORK
    assert status_of(work, cu_q=_cu([100, 31])) == mla.STATUS_BAD_LENGTH
    assert status_of(work, cu_kv=_cu([131, 0])) == mla.STATUS_BAD_LENGTH
    assert status_of(work, cu_kv=_cu([-1, 50])) == mla.STATUS_BAD_LENGTH


@pytest.mark.parametrize("ctas", [1, 2])
def test_captured_and_on_another_stream(ctas):
    lq, lk, H = [300, 20], [4000, 20], 2
    x = _inputs(lq, lk, H, seed=11)
    want, want_lse, parts = _run(x, lq, lk, None, True, ctas=ctas)
    assert parts > 1
    work, parts = mla.plan_prefill(lq, lk, H, ctas=ctas)
    work, cu_q, cu_kv = torch.from_numpy(work).cuda(), _cu(lq), _cu(lk)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = mla.prefill(**x, cu_q=cu_q, cu_kv=cu_kv, work=work, sm_scale=SCALE, num_parts=parts, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = mla.prefill(**x, cu_q=cu_q, cu_kv=cu_kv, work=work, sm_scale=SCALE, num_parts=parts)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
