"""Decode over the 4-bit cache at 33 to 97 query rows a request: every width of
the one-CTA kernel and both sides of its limits, against the definition in 64
bits with the tolerances of test_gpu_fp4_decode.
"""
import numpy as np
import pytest
import torch

import mla_latent_decode_gb300 as mla
from mla_latent_decode_gb300 import build
from test_gpu_fp4_decode import Case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


@pytest.mark.parametrize("q,H,lens", [
    (1, 34, [1, 63, 64, 65, 1025]),
    (1, 48, [3000, 2]),
    (1, 64, [129, 700]),
    (5, 13, [0, 1, 4, 5, 900]),
    (1, 65, [128, 641]),
    (5, 16, [2000, 3, 70]),
    (1, 95, [1281]),
    (1, 96, [5000, 64, 1, 999]),
    (3, 32, [193, 2]),
    (1, 97, [300]),
])
@pytest.mark.parametrize("S", [1, 4])
def test_partial_matches_definition(q, H, lens, S):
    case = Case(len(lens), q, H, lens, seed=30 + H)
    O, LSE = case.run(S)
    assert case.status == 0
    check(case, O, LSE, S, heads=sorted({0, 1, H // 2, H - 2, H - 1}))


@pytest.mark.parametrize("q,H", [(1, 60), (5, 19)])
def test_long_contexts(q, H):
    """Hundreds of pages: every ring turns round many times, the page table's
    entries are fetched 32 at a time."""
    case = Case(1, q, H, [13003], seed=31)
    O, LSE = case.run(1)
    assert case.status == 0
    check(case, O, LSE, 1, heads=[0, H - 1])


@pytest.mark.parametrize("q,H", [(2, 31), (5, 18)])
def test_masked_tokens_hold_anything(q, H):
    """NaN scales and RoPE codes in a draft token: rows that see it are NaN, the
    others are bitwise those of a cache without them."""
    case = Case(1, q, H, [200], seed=32)
    O, LSE = case.run(2)
    slot = case.r2t_host[0, 199]  # seen by the last query only
    case.kv_host[slot, 256:288] = 0x7F
    case.kv_host[slot, 288:] = 0xFF
    case.up()
    O2, LSE2 = case.run(2)
    assert torch.equal(O[:, :, :, :-1], O2[:, :, :, :-1]) and torch.equal(LSE[..., :-1, :], LSE2[..., :-1, :])
    assert LSE2[1, 0, 0, -1].isnan().all() and O2[1, 0, 0, -1].isnan().all()


@pytest.mark.parametrize("H", [50, 90])
def test_bad_pages_read_as_zeros(H):
    case = Case(2, 1, H, [300, 200], seed=33)
    host = case.r2t_host.copy()
    case.r2t_host[0, 64:128] = -64            # negative
    case.r2t_host[0, 128:192] += 32           # not a page boundary
    case.r2t_host[1, 0:64] = case.slots       # past the pool
    case.up()
    O, LSE = case.run(1)
    assert case.status == mla.STATUS_BAD_SLOT
    case.r2t_host = host
    for v, a in ((0, 64), (0, 128), (1, 0)):
        case.kv_host[case.r2t_host[v, a:a + 64]] = 0
    check(case, O, LSE, 1, heads=[0, H - 1])


@pytest.mark.parametrize("q,H", [(5, 12), (5, 17)])
def test_limits_with_empty_rows(q, H):
    lim = [[0, 3, 64, 65, 200], [130, 0, 0, 1, 128]]
    case = Case(2, q, H, [200, 130], limits=lim, seed=34)
    O, LSE = case.run(2)
    check(case, O, LSE, 2, heads=[0, H - 1])


@pytest.mark.parametrize("q,H", [(1, 64), (1, 96)])
def test_rising_maxima_rescale(q, H):
    case = Case(1, q, H, [1500], seed=35, q_scale=0.05)
    t, rows = np.arange(1500), case.r2t_host[0, :1500]
    case.kv_host[rows, 256:288] = np.minimum(16 + t // 16, 0x7E)[:, None]
    case.kv_host[rows, :256] &= 0x77
    case.q_nope = case.q_nope.abs()
    case.up()
    O, LSE = case.run(2)
    check(case, O, LSE, 2, heads=[0, H - 1])


@pytest.mark.parametrize("H", [40, 96])
def test_plan_and_one_launch(H):
    """The scheduler's plan with its work list; the fused merge of the same parts."""
    lens = [3000, 17, 1, 640, 5000]
    case = Case(5, 1, H, lens, seed=36)
    S, bnd, work, _ = mla.plan_sched(5, 1, H, lens, kv_dtype="fp4_e2m1")
    O, LSE = case.run(S, bnd=bnd, work=work)
    check(case, O, LSE, S, bnd=bnd, heads=[0, H - 1])
    out, lse = mla.lse_combine(O, LSE)
    bnd_d = torch.as_tensor(bnd, dtype=torch.int32).cuda()
    out2, lse2 = mla.decode_scratch(case.qn, case.qr, case.kv, case.gd, case.r2t, case.sl, None, S, 192.0 ** -0.5,
                                    split_pages=bnd_d)
    # the same fp32 parts, merged in another order, rounded to bf16
    assert torch.allclose(out2.float(), out.float(), rtol=2.0 ** -7, atol=1e-6)
    assert torch.allclose(lse2, lse, rtol=1e-6, atol=1e-6)


@pytest.mark.parametrize("q,H", [(1, 16), (1, 64), (1, 96), (5, 96)])
def test_pool_past_32_bit_offsets(q, H):
    """The same pages at the end of a pool of 4.6 GB: bitwise the same results."""
    case = Case(2, q, H, [700, 130], seed=40)
    O, LSE = case.run(2)
    slots = 13_000_000 // 64 * 64
    shift = slots - case.kv.shape[0] // 64 * 64
    big = torch.zeros((slots, mla.FP4_ROW_BYTES), dtype=torch.uint8, device="cuda")
    big[shift:shift + case.kv.shape[0]] = case.kv[:slots - shift]
    assert shift * mla.FP4_ROW_BYTES > 1 << 32
    case.kv, case.r2t = big, case.r2t + shift
    O2, LSE2 = case.run(2)
    assert case.status == 0
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)


@pytest.mark.parametrize("q,H", [(1, 16), (1, 64), (1, 96), (5, 96)])
def test_a_query_row_that_is_not_finite_stays_alone(q, H):
    case = Case(1, q, H, [333], seed=41)
    O, LSE = case.run(2)
    case.q_nope[0, 0, 3, 7] = float("nan")
    case.q_rope[0, 0, 5, 1] = float("inf")
    case.up()
    O2, LSE2 = case.run(2)
    assert LSE2[:, 0, 0, 0, 3].isnan().all() and O2[:, 0, 0, 0, 3].isnan().all()
    rest = [h for h in range(H) if h not in (3, 5)]
    assert torch.equal(O[:, :, :, :, rest], O2[:, :, :, :, rest])
    assert torch.equal(LSE[:, :, :, :, rest], LSE2[:, :, :, :, rest])


@pytest.mark.parametrize("q,H,lens", [
    (3, 128, [300, 1]), (5, 96, [64]), (1, 97, [900, 0, 65]), (2, 100, [700, 40, 129]), (8, 128, [2000]), (1, 192, [500])])
def test_row_groups_of_a_work_list(q, H, lens):
    """A work list of one unit per 96 rows: the one-CTA kernel in groups of rows,
    against the definition and, merged in the launch, against its own parts."""
    case = Case(len(lens), q, H, lens, seed=50)
    S, U = 3, -(-q * H // 96)
    P = [-(-L // 64) for L in lens]
    bnd = [[s * p // S for s in range(S)] + [p] for p in P]
    order = np.random.default_rng(1).permutation(S * len(lens) * U)
    O, LSE = case.run(S, bnd=bnd, work=order)
    assert case.status == 0
    check(case, O, LSE, S, bnd=bnd, heads=sorted({0, 1, H // 2, H - 2, H - 1}))
    out, lse = mla.lse_combine(O, LSE)
    dev = dict(split_pages=torch.as_tensor(bnd, dtype=torch.int32).cuda(),
               work=torch.as_tensor(order, dtype=torch.int32).cuda())
    args = (case.qn, case.qr, case.kv, case.gd, case.r2t, case.sl, None, S, 192.0 ** -0.5)
    counters = mla.fused_counters(case.B, q, H, "cuda")
    for _ in range(2):
        out2, lse2 = mla.decode_fused(*args, counters=counters, **dev)
        assert torch.allclose(out2.float(), out.float(), rtol=2.0 ** -7, atol=1e-6)
        assert torch.allclose(lse2, lse, rtol=1e-6, atol=1e-6, equal_nan=True)
        assert int(counters.abs().sum()) == 0


def test_short_work_is_planned_in_row_groups():
    lens = [300, 170]
    case = Case(2, 3, 128, lens, seed=51)
    S, bnd, work, _ = mla.plan_sched(2, 3, 128, lens, kv_dtype="fp4_e2m1")
    assert len(work) == 2 * S * 4
    O, LSE = case.run(S, bnd=bnd, work=work)
    assert case.status == 0
    check(case, O, LSE, S, bnd=bnd, heads=[0, 64, 127])
    case.run(S, bnd=bnd, work=[len(work)] + list(work[1:]))
    assert case.status == mla.STATUS_BAD_WORK
