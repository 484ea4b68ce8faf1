"""GPU parity of the beam selection (mla_beam_select) with the float64
definition: tokens and parents exactly, scores within the roundings.

A score is c + (x - lse) in fp64, rounded to fp32 (2^-24 of itself); the lse's sum
of exponentials is in fp32: a term's exponent is a rounded difference times a
rounded log2(e) (2^-23 |x - max|, at most 2^-16 for the terms within 128 of the
maximum, the others are 0), the exponential 2^-21, and the sums are up to 64 + 10
additions deep per thread, warp and block (2^-17): 2^-15 in all, of a sum.  The order
of two beams' tokens is the definition's where their scores differ by more than
that, so the inputs keep them apart.
"""
import math

import pytest
import torch

import mla_latent_decode_gb300 as mla
from mla_latent_decode_gb300 import build

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -15


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


def _reference(logits, scores, k, finished, end):
    """Scores fp64, rows and tokens int64 [B, k]."""
    B, W, V = logits.shape
    x = logits.double().cpu()
    c = scores.double().cpu()
    lse = torch.logsumexp(x, -1)
    s = c[..., None] + (x - lse[..., None])
    whole = lse.isfinite() & c.isfinite()
    s = torch.where(whole[..., None], s, -math.inf)
    if finished is not None:
        done = finished.cpu().bool()
        s[done] = -math.inf
        for b, w in done.nonzero().tolist():
            if math.isfinite(float(c[b, w])):
                s[b, w, end] = c[b, w]
    best, at = torch.sort(s.reshape(B, -1), dim=1, descending=True, stable=True)
    at = at[:, :k]
    return best[:, :k], at // V + W * torch.arange(B)[:, None], at % V


def _check(logits, scores, k, finished=None, end=0, status=0):
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, rows, tokens = mla.beam_select(logits, scores, k, finished=finished, end_token=end, status=word)
    want, r, t = _reference(logits, scores, k, finished, end)
    assert int(word.item()) == status
    got = got.cpu().double()
    live = want > -math.inf
    assert torch.equal(got > -math.inf, live)
    assert bool(((got - want).abs() <= TOL + 2.0 ** -23 * want.abs())[live].all())
    assert torch.equal(rows.cpu().long(), r)
    assert torch.equal(tokens.cpu().long(), t)


def _inputs(B, W, V, dtype=torch.bfloat16, seed=0):
    g = torch.Generator().manual_seed(seed)
    logits = (3 * torch.randn((B, W, V), generator=g)).to(dtype).cuda()
    scores = (-5 * torch.rand((B, W), generator=g)).cuda()
    return logits, scores


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("B,W,V,k", [
    (1, 1, 1, 1), (1, 2, 1, 2), (2, 1, 7, 7), (1, 3, 5, 15), (3, 4, 100, 8), (2, 5, 1003, 10), (1, 4, 32000, 8),
    (2, 3, 65537, 64), (1, 32, 2000, 64), (9, 2, 511, 1)])
def test_matches_the_definition(B, W, V, k, dtype):
    logits, scores = _inputs(B, W, V, dtype)
    _check(logits, scores, k)


@pytest.mark.parametrize("V", [131072, 262145])
def test_large_vocabularies(V):
    logits, scores = _inputs(2, 3, V)
    _check(logits, scores, 6)


@pytest.mark.parametrize("k", [1, 24, 25, 64])
def test_parts_of_many_tiles(k):
    """So many requests that a warp has more tiles of a row than are looked at together."""
    V = 1200001
    g = torch.Generator().manual_seed(k)
    rows = torch.empty((4, 1, V))
    rows[0, 0] = 3 * torch.randn(V, generator=g)
    rows[1, 0] = torch.round(2 * torch.randn(V, generator=g))         # ties in every tile
    rows[2, 0] = torch.sort(torch.randn(V, generator=g)).values       # the best at the end
    rows[3, 0] = -math.inf
    rows[3, 0, torch.randint(V, (40,), generator=g)] = 1.5
    rows = rows.bfloat16()
    scores = -torch.rand((4, 1), generator=g)
    want, r, t = _reference(rows.cuda(), scores.cuda(), k, None, 0)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, parents, tokens = mla.beam_select(rows.cuda().repeat(40, 1, 1), scores.cuda().repeat(40, 1), k, status=word)
    assert int(word.item()) == 0
    live = want > -math.inf
    for b in range(160):
        assert torch.equal(tokens[b].cpu().long(), t[b % 4])
        assert bool((parents[b] == b).all())
        assert bool(((got[b].cpu().double() - want[b % 4]).abs() <= TOL + 2.0 ** -23 * want[b % 4].abs())[live[b % 4]].all())
        assert torch.equal(got[b].cpu() > -math.inf, live[b % 4])


@pytest.mark.parametrize("B,W", [(1, 32), (100, 17), (160, 32), (170, 8)])
def test_many_rows_a_warp(B, W):
    """Clusters with fewer warps than rows."""
    logits, scores = _inputs(B, W, 300, torch.float16, seed=B)
    _check(logits, scores, 40)


@pytest.mark.parametrize("B", [37, 45, 57, 79, 120])
def test_clusters_of_every_size(B):
    # eight CTAs a request down to two, by how many requests there are
    logits, scores = _inputs(B, 3, 24001, torch.float16, seed=B)
    logits[B // 2] = logits[B // 2].round()  # ties across the CTAs' parts
    logits[B // 3] = logits[B // 3, :1]
    scores[B // 3] = 0
    _check(logits, scores, 33)


def test_rows_at_odd_addresses():
    logits, scores = _inputs(2, 3, 1200)
    for off in (1, 3, 5):
        _check(logits[:, :, off:off + 1001], scores, 9)
    _check(logits[:, 1:, 7:], scores[:, 1:].contiguous(), 4)


def test_ties_go_to_the_lowest_position():
    logits, scores = _inputs(2, 4, 40000)
    logits = torch.round(logits.float()).bfloat16()     # few values, many of each
    logits[1] = logits[1, 0]                            # all beams alike
    scores[1] = -1.0
    _check(logits, scores, 40)
    _check(torch.zeros_like(logits), torch.zeros_like(scores), 64)
    logits[0, :, 20000:] = -0.0
    logits[0, :, :20000] = 0.0
    _check(logits, torch.zeros_like(scores), 16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("W,V,scale", [(32, 1003, 0.1), (7, 24001, 1.0), (3, 131071, 3.0), (9, 333, 30.0)])
def test_equal_rows_that_start_anywhere(W, V, scale, dtype):
    row = (scale * torch.randn(V, generator=torch.Generator().manual_seed(V))).to(dtype)
    row[V // 2] = row.max()                             # equal values within a row, too
    logits = row.expand(2, W, V).contiguous().cuda()
    _check(logits, torch.full((2, W), -2.0, device="cuda"), 50)


@pytest.mark.parametrize("descending", [False, True])
def test_sorted_vocabularies(descending):
    """Every value above those before it, or all the best in a few threads' hands."""
    x = torch.sort(torch.randn((2, 2, 50000), generator=torch.Generator().manual_seed(1)), dim=-1,
                   descending=descending).values.cuda()
    _check(x, torch.tensor([[0.0, -0.3], [-1.0, -1.1]], device="cuda"), 64)
    x[:, :, 3000:] = -math.inf
    _check(x, torch.tensor([[0.0, -0.3], [-1.0, -1.1]], device="cuda"), 16)


def test_masked_vocabularies():
    logits, scores = _inputs(3, 4, 30000, torch.float32, seed=4)
    keep = torch.rand(logits.shape, generator=torch.Generator().manual_seed(5)).cuda() < 0.001
    masked = logits.masked_fill(~keep, -math.inf)
    _check(masked, scores, 16)
    few = torch.full_like(logits, -math.inf)
    few[0, 1, 77] = 1.0
    few[0, 3, [5, 900]] = 2.0                       # three continuations, then the lowest positions
    few[1, 0, 29999] = 0.0
    _check(few, scores, 12)
    low = torch.finfo(torch.float32).min
    _check(logits.masked_fill(~keep, low), scores, 16)


def test_finished_and_dead_beams():
    logits, scores = _inputs(3, 5, 2000, seed=6)
    done = torch.zeros((3, 5), dtype=torch.bool, device="cuda")
    done[0, 2] = done[1, :4] = done[2] = True
    _check(logits, scores, 10, finished=done, end=1999)
    _check(logits, scores, 10, finished=done.to(torch.uint8), end=0)
    scores[:, 1:] = -math.inf                       # the first step: one beam counts
    _check(logits, scores, 10)
    _check(logits, scores, 10, finished=done, end=3)
    scores[:] = -math.inf
    _check(logits, scores, 7)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_broken_beams_end(bad):
    logits, scores = _inputs(2, 4, 3000, seed=7)
    logits[0, 2, 2999] = bad
    _check(logits, scores, 8, status=mla.STATUS_BAD_SCORE)
    logits, scores = _inputs(2, 4, 3000, seed=8)
    scores[1, 0] = bad
    _check(logits, scores, 8, status=mla.STATUS_BAD_SCORE)
    scores[:] = math.nan
    _check(logits, scores, 8, status=mla.STATUS_BAD_SCORE)


def test_far_logits():
    logits, scores = _inputs(1, 2, 5000, torch.float32, seed=9)
    logits[0, 0] += 3e4
    logits[0, 1] -= 3e4
    # lse and logit are rounded to fp32 steps of 2^-9 near 3e4: the scores follow the stored logits
    _check(logits, scores, 8)
    logits[0, 0, 123] = 3.3e38
    logits[0, 1, 17] = -3.3e38
    _check(logits, scores, 8)


def test_captured_and_repeated():
    logits, scores = _inputs(4, 4, 20000, seed=10)
    want = [t.clone() for t in mla.beam_select(logits, scores, 8)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = mla.beam_select(logits, scores, 8)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_requests():
    mla.beam_select(torch.empty((0, 3, 10), device="cuda"), torch.empty((0, 3), device="cuda"), 4)
