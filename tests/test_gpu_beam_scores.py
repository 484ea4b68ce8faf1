"""GPU parity of the beam selection's scores (mla_beam_select) where beams are close to
each other: confident beams, whose sums of exponentials are 1 and a few millionths, and
equal rows whose logits rise from tile to tile.

Tolerance of a score, from the kernel's roundings, for a row with probabilities p_i:
a term's exponent is a difference and a product, 2^-24 of itself each, over one or
more hops (to the lane's maximum at the time, to its later ones, to the warp's) whose
lengths add up to |x_i - max|, and log2(e) itself is off by 2^-25: 2^-23 (1 + 2^-2) sum p_i |x_i - max|.
Every hop's exponential is within 2^-22 and its product rounds by 2^-24, the hops at
most 2 and one for every tile of a part.  A tile's terms meet in 16 + 2 additions at
most, a lane's tiles in a compensated sum, lanes in 5 additions after one of its parts
and a product: 25 x 2^-24.  The rest is in pairs of fp32 or in fp64 (below 2^-40); the
score is rounded to fp32, 2^-24 of itself.
"""
import math

import pytest
import torch

import mla_latent_decode_gb300 as mla
from mla_latent_decode_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


def _select(logits, scores, k):
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, rows, tokens = mla.beam_select(logits, scores, k, status=word)
    assert int(word.item()) == 0
    return got.double().cpu(), rows.cpu().tolist(), tokens.cpu().tolist()


def _exact(logits, scores):
    """Scores [B, W, V] in fp64, and every row's bound but the last rounding."""
    x = logits.double().cpu()
    lse = torch.logsumexp(x, -1, keepdim=True)
    p = torch.exp(x - lse)
    far = (x.amax(-1, keepdim=True) - x).masked_fill(p == 0, 0.0)
    tile = 1024 if logits.dtype is torch.float32 else 2048
    hops = 2 + 1 + -(-x.shape[-1] // tile)
    bound = 1.25 * 2.0 ** -23 * (p * far).sum(-1) + hops * 1.25 * 2.0 ** -22 + 25 * 2.0 ** -24 + 2.0 ** -40
    return scores.double().cpu()[..., None] + (x - lse), bound


def _check(logits, scores, k):
    B, W, V = logits.shape
    got, rows, tokens = _select(logits, scores, k)
    want, bound = _exact(logits, scores)
    best = torch.sort(want.reshape(B, -1), dim=1, descending=True).values[:, :k]
    for b in range(B):
        for i in range(k):
            w = rows[b][i] - b * W
            own = float(want[b, w, tokens[b][i]])
            tol = float(bound[b, w]) + 2.0 ** -24 * abs(own)
            assert abs(float(got[b, i]) - own) <= tol, (b, i, float(got[b, i]), own, tol)
            assert own >= float(best[b, i]) - 2 * float(bound[b].max())
        assert len(set(zip(rows[b], tokens[b]))) == k


def _peaked(V, seconds, dtype=torch.bfloat16):
    """Rows with one token at 20, one below it and the rest at -20."""
    x = torch.full((1, len(seconds), V), -20.0)
    x[..., 0] = 20.0
    x[0, :, 1] = torch.tensor(seconds)
    return x.to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("V", [1000, 1001, 24003])
def test_confident_beams_keep_their_own_sums(V, dtype):
    # sums 1 + 6.14e-6 and 1 + 3.73e-6 (+ V e^-40), 2.4e-6 apart; the two tokens meet in one
    # lane's first additions, so a sum is off by 2^-24 and a few parts in 10^7 of 6e-6
    logits = _peaked(V, [8.0, 7.5], dtype)
    scores = torch.zeros((1, 2), device="cuda")
    got, rows, tokens = _select(logits, scores, 2)
    assert rows == [[1, 0]] and tokens == [[0, 0]]
    want, _ = _exact(logits, scores)
    assert abs(float(got[0, 0]) - float(want[0, 1, 0])) < 2.0 ** -22
    assert abs(float(got[0, 1]) - float(want[0, 0, 0])) < 2.0 ** -22
    _check(logits, scores, 4)


@pytest.mark.parametrize("V", [512, 1003])
def test_sums_a_little_apart_are_a_chain_of_rows(V):
    """Three rows, each near the next: no row takes another's sum."""
    for seconds in ([8.5, 8.0, 7.0], [7.0, 8.0, 8.5], [8.0, 7.0, 8.5]):
        logits = _peaked(V, seconds)
        _, rows, _ = _select(logits, torch.zeros((1, 3), device="cuda"), 3)
        assert rows[0] == sorted(range(3), key=lambda w: seconds[w])


@pytest.mark.parametrize("W", [2, 5, 17, 32])
@pytest.mark.parametrize("V", [4096, 4097])
def test_many_confident_beams(W, V):
    seconds = [20.0 + math.log(1e-6 * (1 + (7 * w) % W)) for w in range(W)]   # sums 1e-6 apart, off by 2^-23 at most
    logits = _peaked(V, seconds, torch.float32)
    got, rows, _ = _select(logits, torch.zeros((1, W), device="cuda"), W)
    want = [math.log1p(math.exp(s - 20.0)) for s in seconds]
    assert rows[0] == sorted(range(W), key=lambda w: want[w])
    assert all(abs(float(got[0, i]) + want[w]) < 2.0 ** -22 for i, w in enumerate(rows[0]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("place", [1, 5000, 9002])
def test_rows_that_differ_in_one_place(place, dtype):
    """Equal but for one logit, wherever rows start: the smaller sum is the better beam."""
    g = torch.Generator().manual_seed(place)
    row = torch.randn(9003, generator=g) - 12.0
    row[17] = 4.0
    logits = row.expand(2, 7, 9003).clone()
    # terms e^-11 and e^-11.5 of a sum of about 1.002: 6.6e-6 apart, a sum off by less than 20 x 2^-24
    logits[..., place] = -7.5
    logits[0, 1::2, place] = -7.0
    logits[1, 3, place] = -7.0                                      # one row among equal ones
    logits = logits.to(dtype).cuda()
    scores = torch.zeros((2, 7), device="cuda")
    got, rows, tokens = _select(logits, scores, 7)
    assert rows[0] == [0, 2, 4, 6, 1, 3, 5] and tokens[0] == [17] * 7
    assert rows[1] == [7 + w for w in (0, 1, 2, 4, 5, 6, 3)] and tokens[1] == [17] * 7
    assert len(set(got[1, :6].tolist())) == len(set(got[0, :4].tolist())) == len(set(got[0, 4:].tolist())) == 1
    _check(logits, scores, 7)


@pytest.mark.parametrize("B,W,V", [(2, 3, 40001), (160, 2, 70003), (3, 32, 9999)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_equal_rows_of_rising_logits_tie(B, W, V, dtype):
    """Every tile has a new maximum, and rows start at other places modulo 16 bytes."""
    row = torch.linspace(-0.5, 0.5, V).to(dtype)
    logits = row.expand(B, W, V).contiguous().cuda()
    got, rows, tokens = _select(logits, torch.zeros((B, W), device="cuda"), 2 * W)
    order = torch.sort(row.double(), descending=True, stable=True).indices
    top = [int(t) for t in order[:2]]
    for b in (0, B // 2, B - 1):
        if float(row[top[0]]) > float(row[top[1]]):
            assert rows[b] == [b * W + w for w in range(W)] * 2
            assert tokens[b] == [top[0]] * W + [top[1]] * W
        else:
            equal = (row == row[top[0]]).nonzero()[:, 0].tolist()
            assert list(zip(rows[b], tokens[b])) == [(b * W + w, t) for w in range(W) for t in equal][:2 * W]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("B,W,V,k", [(2, 4, 32000, 8), (3, 5, 10007, 16), (1, 16, 2048, 33), (20, 3, 50257, 6)])
def test_scores_within_the_roundings(B, W, V, k, dtype):
    g = torch.Generator().manual_seed(V)
    logits = (3 * torch.randn((B, W, V), generator=g)).to(dtype).cuda()
    logits[0, 0] = torch.sort(logits[0, 0].float()).values.to(dtype)
    _check(logits, (-5 * torch.rand((B, W), generator=g)).cuda(), k)


def test_equal_rows_through_strides():
    """Rows of a wider buffer: starts that agree modulo 16 bytes and starts that do not."""
    row = (2 * torch.randn(3001, generator=torch.Generator().manual_seed(3))).bfloat16()
    row[1234] = 20.0
    for wide in (3001, 3008, 3013):
        logits = torch.full((2, 9, wide), 50.0, dtype=torch.bfloat16)
        logits[..., :3001] = row
        logits[..., 9] = -0.0
        logits[1, 4, 9] = 0.0                                        # the same value
        logits = logits.cuda()[..., :3001]
        got, rows, _ = _select(logits, torch.full((2, 9), -1.0, device="cuda"), 9)
        assert rows == [list(range(9)), list(range(9, 18))]
        assert all(len(set(got[b].tolist())) == 1 for b in range(2))
