"""The prompts' planner (mla_plan_prefill): its cuts are those of a list schedule written out
plainly, and it costs the host less than a layer of what it plans."""
import heapq
import random
import time

import numpy as np
import pytest

import mla_latent_decode_gb300 as mla
from mla_latent_decode_gb300 import build

CUTS = (1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 28, 32)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


def _plan(lq, lk, pre, H, causal, ctas, sms):
    """(expected end, {(sequence, block): parts}) of a form, in fiftieths of a key tile."""
    rows, tile, fixed = (128, 50, 85) if ctas == 1 else (512, 39, 110)
    slots = 2 * sms if ctas == 1 else max(sms // 2, 1)
    tiles = []
    for q, k, p in zip(lq, lk, pre):
        ends = [min(r + rows, q) - 1 for r in range(0, q, rows)]
        tiles.append([-(-(min(k, max(p, k - q + 1 + e, 0)) if causal else k) // 128) for e in ends])
    blocks = sum(map(len, tiles))
    longest = max((t for x in tiles for t in x), default=0)
    limit = max(longest, 1)

    def parts_of(t, limit):
        return max(1, min(-(-t // limit), 32))

    end = (sum(map(sum, tiles)) * tile + blocks * fixed) * H / slots + longest * tile / 2
    if 0 < blocks * H < 8 * slots:
        order = sorted(range(len(tiles)), key=lambda n: -(tiles[n][-1] if tiles[n] else -1))
        best = None
        for cut in CUTS:
            limit = max(-(-longest // cut), 1)
            if cut > 1 and limit < 4:
                break
            free, last, sum_, merged = [0] * slots, 0, 0, 0
            for n in order:
                for _ in range(H):
                    for t in reversed(tiles[n]):
                        parts = parts_of(t, limit)
                        merged += parts * (rows // 128) if parts > 1 else 0
                        for s in range(parts):
                            cost = fixed + tile * (t * (s + 1) // parts - t * s // parts)
                            at = free[0] + cost
                            heapq.heapreplace(free, at)
                            last, sum_ = max(last, at), sum_ + cost
            end = (last + sum_ / slots) / 2 + (150 + 0.4 * merged if merged else 0)
            if best is None or end < best[0]:
                best = end, limit
        end, limit = best
    return end, {(n, b): parts_of(t, limit) for n, x in enumerate(tiles) for b, t in enumerate(x)}


@pytest.mark.parametrize("seed", range(40))
def test_cuts_are_those_of_the_list_schedule(seed):
    r = random.Random(seed)
    N, H = r.randint(1, 9), r.choice([1, 2, 5, 16])
    lq = [r.choice([0, 1, 100, 128, r.randint(1, 2500)]) for _ in range(N)]
    lk = [q + r.choice([0, r.randint(0, 2000), r.randint(0, 40000)]) for q in lq]
    pre = [r.choice([0, r.randint(0, k)]) for k in lk]
    causal, sms = r.random() < 0.8, r.choice([1, 20, 152])
    single, pair = (_plan(lq, lk, pre, H, causal, c, sms) for c in (1, 2))
    for ctas in (0, 1, 2):
        work, slots = mla.plan_prefill(lq, lk, H, prefix=pre, causal=causal, ctas=ctas, num_sms=sms)
        work = work.reshape(len(work), work.size // 8 // max(len(work), 1), 8)
        form = ctas or (2 if pair[0] < single[0] else 1)
        want = (single, pair)[form - 1][1]
        if len(work):
            assert work.shape[1] == form
        assert {(n, b): of for n, b, _, of in work[:, 0, :4].tolist()} == want
        used = sum(p for p in want.values() if p > 1) * (1 if form == 1 else 4)
        assert slots == -(-used // 2)


@pytest.mark.parametrize("lq,lk,H", [
    ([8191], [8191], 16), ([8192], [100000], 8), ([512] * 16, [40000] * 16, 16), ([2000] * 8, [30000] * 8, 16),
    ([2300], [32000], 128), ([250] * 8, [20000] * 8, 128), ([1100] * 16, [32000] * 16, 16), ([2000] * 8, [200000] * 8, 8)])
def test_a_plan_costs_less_than_a_layer(lq, lk, H):
    """Every step is planned.  0.04 to 0.35 ms, where a heap step for every head's part took 4 to 28;
    a layer of the smallest, 8191 tokens x 16 heads, is 0.2 ms of products."""
    best = 1.0
    for _ in range(8):
        start = time.perf_counter()
        mla.plan_prefill(lq, lk, H, num_sms=152)
        best = min(best, time.perf_counter() - start)
    assert best < 1.5e-3


def test_far_lengths_and_many_sms():
    """Costs beyond the schedule's ring, more slots than jobs, and no job at all."""
    for lq, lk, H, sms in (([1], [0x7fffff00], 3, 152), ([300, 1], [2000000, 3], 128, 152), ([5], [9], 1, 0x7fffffff),
                           ([0, 0], [5, 0], 4, 152), ([700], [100], 2, 1)):
        work, slots = mla.plan_prefill(lq, lk, H, num_sms=sms)
        work = work.reshape(len(work), work.size // 8 // max(len(work), 1), 8)[:, :1].reshape(-1, 8)
        block = work[0, 7] if len(work) else 128
        assert sorted({(n, b) for n, b in work[:, :2].tolist()}) == [
            (n, b) for n, q in enumerate(lq) for b in range(-(-q // block))]
        for n, b, part, of in work[:, :4].tolist():
            assert 0 <= part < of <= mla.PREFILL_MAX_PARTS
        assert np.all(work[:, 3] <= 32) and slots >= 0
