"""GPU parity of the decode over the 4-bit latent cache with the float64
definition, on the tensor-core path and on the CUDA cores.

Bounds, from the roundings.  The stored values and the queries enter the
products exactly; a score's sum of 576 products in at most 24-bit (tensor
cores: about 21-bit) steps is off by at most 2^-16 of sum |q_d k_d| sm_scale
(E below), and the exponential and its argument by 2^-19 of |score| <= E more.
So LSE is within E 2^-15 + 2^-18.  Each probability carries that relative error and, on
the tensor cores, one rounding to f16 (2^-11 relative; those below 2^-14 of the
row's largest, 2^-24 absolute), so an fp32 part is within (2^-11 + 2^-12 + E 2^-14)
A of the definition, A = sum p |v| (the rescaled accumulator adds 2^-12), plus
2^-20 of the row's largest |v| for the probabilities under f16's normal range;
a bf16 part adds 2^-8.
"""
import numpy as np
import pytest
import torch

import mla_latent_decode_gb300 as mla
from latent_ref import attend, decode4, f64, random_pool
from mla_latent_decode_gb300 import build

pytestmark = pytest.mark.gpu
SCALE = 192.0 ** -0.5
G = 0.0625


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


class Case:
    """Queries, a paged 4-bit pool (unused slots all NaN codes) and tables."""

    def __init__(self, B, q, H, lens, seed=0, shards=1, g=G, q_scale=1.0, limits=None):
        self.B, self.q, self.H, self.shards, self.g = B, q, H, shards, g
        r = np.random.default_rng(seed)
        self.lens = list(lens)
        V = B * shards
        pages = [-(-L // 64) for L in self.lens]
        self.slots = (1 + sum(pages)) * 64
        kv = random_pool(self.slots, seed + 1, g)
        perm = r.permutation(sum(pages)) + 1
        self.stride = max(1, max(pages)) * 64
        r2t = np.zeros((V, self.stride), np.int32)
        used = np.zeros(self.slots, bool)
        at = 0
        for v in range(V):
            own = perm[at:at + pages[v]]
            at += pages[v]
            t = np.arange(pages[v] * 64)
            r2t[v, :len(t)] = own[t // 64] * 64 + t % 64
            used[r2t[v, :self.lens[v]]] = True
        kv[~used] = 0xFF
        self.kv_host, self.r2t_host = kv, r2t
        gen = torch.Generator().manual_seed(seed)
        self.q_nope = (q_scale * torch.randn((B, q, H, 512), generator=gen)).bfloat16()
        self.q_rope = (q_scale * torch.randn((B, q, H, 64), generator=gen)).bfloat16()
        self.limits = limits
        self.up()

    def up(self):
        self.kv = torch.from_numpy(self.kv_host).cuda()
        self.r2t = torch.from_numpy(self.r2t_host).cuda()
        self.sl = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.kl = None if self.limits is None else torch.tensor(self.limits, dtype=torch.int32, device="cuda")
        self.qn, self.qr = self.q_nope.cuda(), self.q_rope.cuda()
        self.gd = torch.full((1,), self.g, device="cuda")

    def sees(self, v, i):
        n = self.limits[v][i] if self.limits is not None else self.lens[v] - self.q + 1 + i
        return max(0, min(self.lens[v], n))

    def run(self, S, bnd=None, work=None, **kw):
        bnd = None if bnd is None else torch.as_tensor(bnd, dtype=torch.int32).cuda()
        work = None if work is None else torch.as_tensor(work, dtype=torch.int32).cuda()
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = mla.decode_partial(self.qn, self.qr, self.kv, self.gd, self.r2t, self.sl, self.kl, S, SCALE,
                                 num_shards=self.shards, split_pages=bnd, work=work, status=st, **kw)
        torch.cuda.synchronize()
        self.status = int(st.item())
        return out

    def expect(self, v, t0, t1, heads):
        """(O, LSE, A, E, vmax) of request v's query rows of `heads` over [t0, t1)."""
        b = v % self.B
        k = decode4(self.kv_host[self.r2t_host[v, t0:t1]], self.g)
        vis = np.array([[t0 + t < self.sees(v, i) for t in range(t1 - t0)]
                        for i in range(self.q) for _ in heads]).reshape(self.q * len(heads), t1 - t0)
        x = [f64(t[b][:, heads]).reshape(self.q * len(heads), -1) for t in (self.q_nope, self.q_rope)]
        out = attend(x[0], x[1], k, vis, SCALE)
        vmax = np.where(vis.any(0)[:, None], np.abs(k[:, :512]), 0).max(initial=0.0)
        return (*out, vmax)


def check(case, O, LSE, S, bnd=None, heads=None, requests=None, bf16=False):
    heads = list(range(case.H)) if heads is None else heads
    Of, Lf = f64(O), f64(LSE)
    for v in range(case.B * case.shards) if requests is None else requests:
        c, b = divmod(v, case.B)
        P = -(-case.lens[v] // 64)
        for s in range(S):
            p0, p1 = (s * P // S, (s + 1) * P // S) if bnd is None else (bnd[v][s], bnd[v][s + 1])
            t0, t1 = p0 * 64, min(p1 * 64, case.lens[v])
            t1 = max(t0, t1)
            ref, lse, A, E, vmax = case.expect(v, t0, t1, heads)
            got = Of[s, c, b][:, heads].reshape(ref.shape)
            gl = Lf[s, c, b][:, heads].reshape(lse.shape)
            empty = np.isneginf(lse)
            assert np.array_equal(np.isneginf(gl), empty), (v, s)
            assert np.all(got[empty] == 0), (v, s)
            live = ~empty
            assert np.isfinite(got[live]).all() and np.isfinite(gl[live]).all(), (v, s)
            dl = np.abs(gl - lse)[live]
            assert np.all(dl <= E[live] * 2.0 ** -15 + 2.0 ** -18), (v, s, dl.max())
            tol = (2.0 ** -11 + 2.0 ** -12 + E[:, None] * 2.0 ** -14) * A + 2.0 ** -20 * vmax
            if bf16:
                tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
            err = np.abs(got - ref)
            assert np.all(err[live] <= tol[live]), (v, s, (err[live] / np.maximum(tol[live], 1e-30)).max())


CASES = {
    "one_token": dict(B=1, q=1, H=1, lens=[1]),
    "tiny": dict(B=1, q=1, H=16, lens=[256]),
    "page_edges": dict(B=6, q=1, H=3, lens=[63, 64, 65, 127, 128, 129]),
    "zero_and_short": dict(B=5, q=5, H=7, lens=[0, 1, 3, 5, 300]),
    "heads96_q5": dict(B=2, q=5, H=96, lens=[1000, 333]),
    "rows_255_to_257": dict(B=1, q=1, H=257, lens=[700]),
    "rows_128": dict(B=2, q=2, H=64, lens=[513, 640]),
    "rows_129": dict(B=1, q=3, H=43, lens=[1281]),
    "long": dict(B=1, q=2, H=8, lens=[20011]),
    "heads16_q1": dict(B=9, q=1, H=16, lens=[4097, 2000, 31, 640, 3, 1, 999, 64, 2500]),
    "rows_17": dict(B=2, q=1, H=17, lens=[777, 128]),
    "rows_32_q4": dict(B=3, q=4, H=8, lens=[1000, 65, 3]),
    "rows_30_long": dict(B=1, q=5, H=6, lens=[9001]),
    "heads33_q1": dict(B=3, q=1, H=33, lens=[900, 65, 1025]),
}


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("S", [1, 3])
@pytest.mark.parametrize("name", CASES)
def test_partial_matches_definition(name, S, simt):
    case = Case(seed=len(name), **CASES[name])
    O, LSE = case.run(S, simt=simt)
    assert case.status == 0
    heads = None if case.H <= 16 else sorted({0, 1, case.H // 2, case.H - 2, case.H - 1})
    check(case, O, LSE, S, heads=heads)


@pytest.mark.parametrize("q_scale,g", [(1e-20, 1.0), (30.0, 0.0625), (1e18, 1e-18), (1.0, 2.0 ** -60)])
def test_magnitudes(q_scale, g):
    """Queries and the pool's factor far from 1: the row scale keeps the f16
    query exact and the scores' factor is fp32."""
    case = Case(2, 2, 5, [200, 70], seed=3, q_scale=q_scale, g=g)
    O, LSE = case.run(2)
    check(case, O, LSE, 2)


def test_query_range_within_a_row():
    """Elements 2^-24 of the row's largest and below still count exactly."""
    case = Case(1, 1, 4, [100], seed=5)
    case.q_nope[..., 3] = 512.0
    case.q_nope[..., 4:200] *= 2.0 ** -20
    case.q_rope *= 2.0 ** -25
    case.kv_host[:, 1] &= 0x0F  # element 3 of every row is 0
    case.up()
    O, LSE = case.run(1)
    check(case, O, LSE, 1)


def test_zero_queries_and_zero_rows():
    case = Case(2, 1, 3, [130, 64], seed=6)
    case.q_nope[0], case.q_rope[0] = 0, 0
    case.kv_host[:, 256:] = np.where(np.arange(case.slots)[:, None] % 3 == 0, 0, case.kv_host[:, 256:])
    case.up()
    O, LSE = case.run(1)
    check(case, O, LSE, 1)


def test_parts_of_any_length_and_work_order():
    case = Case(3, 5, 96, [1500, 640, 70], seed=7)
    bnd = [[0, 0, 7, 24], [0, 10, 10, 10], [0, 1, 2, 2]]
    O, LSE = case.run(3, bnd=bnd)
    check(case, O, LSE, 3, bnd=bnd, heads=[0, 50, 95])
    U = -(-5 * 96 // 256)
    order = np.random.default_rng(0).permutation(3 * 3 * U)
    O2, LSE2 = case.run(3, bnd=bnd, work=order)
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)
    bad = order.copy()
    bad[2] = 3 * 3 * U
    case.run(3, bnd=bnd, work=bad)
    assert case.status == mla.STATUS_BAD_WORK


def test_shards_and_limits_with_empty_rows():
    """Eight token-interleaved shards, short ones empty for some queries."""
    from mla_latent_decode_gb300 import synth
    B, q, S8 = 2, 5, 8
    loc = [synth.shard_lengths(L, q, S8, s) for s in range(S8) for L in (1000, 9)]
    case = Case(B, q, 24, [l for l, _ in loc], shards=S8, limits=[m for _, m in loc], seed=8)
    O, LSE = case.run(1)
    check(case, O, LSE, 1, heads=[0, 23])
    lim = [[0, 3, 64, 65, 200], [200, 0, 0, 1, 128]]
    case = Case(2, 5, 9, [200, 130], limits=lim, seed=9)
    O, LSE = case.run(2)
    check(case, O, LSE, 2)


@pytest.mark.parametrize("simt", [False, True])
def test_masked_tokens_hold_anything(simt):
    """NaN scales and RoPE codes in a draft token: rows that see it are NaN,
    the others are bitwise those of a cache without them."""
    case = Case(1, 5, 40, [200], seed=10)
    O, LSE = case.run(2, simt=simt)
    slot = case.r2t_host[0, 198]  # seen by queries 3 and 4
    case.kv_host[slot, 256:288] = 0x7F
    case.kv_host[slot, 288:] = 0xFF
    case.up()
    O2, LSE2 = case.run(2, simt=simt)
    assert torch.equal(O[:, :, :, :3], O2[:, :, :, :3]) and torch.equal(LSE[..., :3, :], LSE2[..., :3, :])
    if not simt:
        assert LSE2[1, 0, 0, 3:].isnan().all() and O2[1, 0, 0, 3:].isnan().all()


@pytest.mark.parametrize("shape", [dict(B=1, q=1, H=9), dict(B=1, q=1, H=70), dict(B=1, q=2, H=96)])
def test_rows_that_saw_nan_stay_nan(shape):
    """A context that opens with NaN tokens and goes on finite: NaN throughout."""
    case = Case(lens=[900], seed=15, **shape)
    case.kv_host[case.r2t_host[0, :200], 256:288] = 0x7F
    case.up()
    O, LSE = case.run(1)
    assert O.isnan().all() and LSE.isnan().all()


@pytest.mark.parametrize("simt", [False, True])
def test_bad_pages_read_as_zeros_and_lengths_are_clamped(simt):
    case = Case(2, 1, 20, [300, 200], seed=11)
    host = case.r2t_host.copy()
    case.r2t_host[0, 64:128] = -64            # negative
    case.r2t_host[0, 128:192] += 32           # not a page boundary
    case.r2t_host[1, 0:64] = case.slots       # past the pool
    case.up()
    O, LSE = case.run(1, simt=simt)
    assert case.status == mla.STATUS_BAD_SLOT
    case.r2t_host = host.copy()
    for v, a in ((0, 64), (0, 128), (1, 0)):
        case.kv_host[case.r2t_host[v, a:a + 64]] = 0
    check(case, O, LSE, 1)
    case.lens[1] = case.stride + 999
    case.up()
    case.run(1, simt=simt)
    assert case.status & mla.STATUS_BAD_LENGTH


ROWS = [dict(B=2, q=1, H=16, lens=[1300, 70]), dict(B=2, q=3, H=9, lens=[640, 2]),
        dict(B=2, q=2, H=60, lens=[1000, 129]), dict(B=2, q=5, H=96, lens=[700, 64])]


@pytest.mark.parametrize("shape", ROWS)
def test_bf16_parts(shape):
    case = Case(seed=20, **shape)
    O, LSE = case.run(2, part_dtype=torch.bfloat16)
    assert O.dtype == torch.bfloat16 and case.status == 0
    check(case, O, LSE, 2, heads=[0, case.H - 1], bf16=True)
    O32, LSE32 = case.run(2)
    assert torch.equal(O, O32.bfloat16()) and torch.equal(LSE, LSE32)


@pytest.mark.parametrize("shape", ROWS)
def test_one_launch_equals_two(shape):
    """decode_fused and decode_scratch merge the very parts of decode_partial."""
    case = Case(seed=21, **shape)
    S, bnd, work, _ = mla.plan_sched(case.B, case.q, case.H, case.lens, kv_dtype="fp4_e2m1")
    S, bnd = (S, bnd) if S > 1 else (2, None)
    bnd = None if bnd is None else torch.as_tensor(bnd, dtype=torch.int32).cuda()
    O, LSE = case.run(S, bnd=bnd)
    out, lse = mla.lse_combine(O, LSE)
    args = (case.qn, case.qr, case.kv, case.gd, case.r2t, case.sl, None, S, SCALE)
    counters = mla.fused_counters(case.B, case.q, case.H, "cuda")
    for _ in range(2):  # the counters are left zero
        out2, lse2 = mla.decode_fused(*args, split_pages=bnd, counters=counters)
        assert torch.allclose(out2.float(), out.float(), rtol=2.0 ** -7, atol=1e-6)
        assert torch.allclose(lse2, lse, rtol=1e-6, atol=1e-6, equal_nan=True)
        assert int(counters.abs().sum()) == 0
    out3, lse3 = mla.decode_scratch(*args, split_pages=bnd)
    assert torch.equal(out3, out2) and torch.equal(lse3, lse2)


def test_rising_maxima_rescale():
    """Scores that grow along the context: the references rise tile by tile."""
    for shape in (dict(B=1, q=1, H=5), dict(B=1, q=2, H=60)):
        case = Case(lens=[1500], seed=22, q_scale=0.05, **shape)
        t = np.arange(1500)
        rows = case.r2t_host[0, :1500]
        case.kv_host[rows, 256:288] = np.minimum(16 + t // 16, 0x7E)[:, None]
        case.kv_host[rows, :256] &= 0x77
        case.q_nope = case.q_nope.abs()
        case.up()
        O, LSE = case.run(2)
        check(case, O, LSE, 2, heads=[0, case.H - 1])


def test_side_stream_equals_default_stream():
    case = Case(3, 5, 96, [900, 64, 333], seed=12)
    O, LSE = case.run(2)
    s = torch.cuda.Stream()
    O2, LSE2 = case.run(2, stream=s)
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)


def test_combined_result():
    """Parts merged: the scheduler's plan against the unsplit definition."""
    lens = [3000, 17, 1, 640, 5000]
    case = Case(5, 1, 96, lens, seed=13)
    S, bnd, work, _ = mla.plan_sched(5, 1, 96, lens, kv_dtype="fp4_e2m1")
    O, LSE = case.run(S, bnd=bnd, work=work)
    out, lse = mla.lse_combine(O, LSE)
    heads = [0, 47, 95]
    for b, L in enumerate(lens):
        ref, rl, A, E, vmax = case.expect(b, 0, L, heads)
        tol = (2.0 ** -10 + E[:, None] * 2.0 ** -13) * A + 2.0 ** -20 * vmax + 2.0 ** -8 * np.abs(ref)
        assert np.all(np.abs(f64(out[b][:, heads]).reshape(ref.shape) - ref) <= tol), b
        assert np.all(np.abs(f64(lse[b][:, heads]).reshape(-1) - rl) <= E * 2.0 ** -14 + 2.0 ** -17), b


def test_append_then_decode():
    """Rows written by kv_append, attended as they were stored."""
    from latent_ref import table
    case = Case(2, 3, 16, [130, 70], seed=14)
    gen = torch.Generator().manual_seed(3)
    rows = torch.randn((200, 576), generator=gen).bfloat16().cuda()
    slots = torch.tensor([s for v, L in enumerate(case.lens) for s in case.r2t_host[v, :L]], dtype=torch.int32).cuda()
    pos = torch.arange(200, dtype=torch.int32).cuda()
    case.kv.fill_(0xFF)
    w = torch.ones(512).bfloat16().cuda()
    qr = mla.kv_append(rows[:200], slots, pos, table(256).cuda(), case.kv, case.gd, norm_weight=w)
    assert qr is None
    case.kv_host = case.kv.cpu().numpy()
    O, LSE = case.run(1)
    assert case.status == 0
    check(case, O, LSE, 1)
