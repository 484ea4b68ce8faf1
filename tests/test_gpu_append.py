"""GPU parity of the cache append and read (mla_kv_append, mla_kv_read) with the
float64 definition.

Tolerances, from the roundings: the norm's fp32 sum, root and products stay
within 2^-18 relative (16 + 5 additions deep, each 2^-24, halved by the root,
and five more roundings); a rotation within 2^-22 (|a| + |b|); a bf16 result
adds 2^-8 relative.  A stored code must equal the definition's wherever a 2^-17
relative change of its quotient would not move it (the norm's bound, and the
scale's own rounding), and everywhere it is within one code's half step of the
value.
"""
import numpy as np
import pytest
import torch

import mla_latent_decode_gb300 as mla
from latent_ref import (E2M1, E4M3, NOPE, ROW, decode4, e4m3_values, encode, f64,
                        random_pool, rotate, sure, table)
from mla_latent_decode_gb300 import build

pytestmark = pytest.mark.gpu
REL = 2.0 ** -17
G = 0.0625


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


def _pool(kind, slots):
    if kind == "bf16":
        return torch.full((slots, 576), 7.0, dtype=torch.bfloat16, device="cuda"), None
    if kind == "fp8":
        return (torch.full((slots, 576), 0x7F, dtype=torch.uint8, device="cuda"),
                torch.full((slots,), -1.0, device="cuda"))
    return (torch.full((slots, 352), 0x55, dtype=torch.uint8, device="cuda"),
            torch.full((1,), G, device="cuda"))


def _inputs(n, H, seed, stride=ROW, q_pad=0):
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn((n, stride), generator=g)
    if n > 2:
        wide[1] *= 1e-20
        wide[2] = 0.0
    if n > 4:
        wide[3] *= 3e4
        wide[4, 5] = 4000.0
    rows = wide.bfloat16().cuda()[:, stride - ROW:]
    weight = (1 + 0.2 * torch.randn(NOPE, generator=g)).bfloat16().cuda()
    q = torch.randn((n, H, 64 + q_pad), generator=g).bfloat16().cuda()[:, :, q_pad:]
    pos = torch.randint(0, 5000, (n,), generator=g).int()
    return rows, weight, q, pos.cuda()


def _expect(rows, weight, pos, tab, interleaved, eps):
    x = f64(rows)
    c = x[:, :NOPE]
    if weight is not None:
        c = c / np.sqrt((c * c).mean(1, keepdims=True) + eps) * f64(weight)
    t = f64(tab)[pos.cpu().numpy()]
    r = rotate(x[:, NOPE:], t[:, :32], t[:, 32:], interleaved)
    a = np.abs(x[:, NOPE:])
    other = a[:, np.arange(64) ^ 1] if interleaved else np.roll(a, 32, 1)
    slack = np.concatenate([REL * np.abs(c), 2.0 ** -22 * (a + other)], 1)
    return np.concatenate([c, r], 1), slack, t


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("n,H,stride,q_pad,norm", [
    (1, 1, 576, 0, True), (5, 96, 640, 128, True), (9, 3, 584, 8, False),
    (67, 65, 576, 0, True), (300, 0, 704, 0, True)])
def test_append_matches_definition(kind, interleaved, n, H, stride, q_pad, norm):
    rows, weight, q, pos = _inputs(n, H, n, stride, q_pad)
    weight = weight if norm else None
    eps = 1e-6
    tab = table(5000).cuda()
    kv, scale = _pool(kind, 1024)
    before = kv.clone()
    slots = torch.randperm(1024)[:n].int().cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = mla.kv_append(rows, slots, pos, tab, kv, scale, norm_weight=weight, eps=eps,
                          q_rope=q if H else None, interleaved=interleaved, status=st)
    back = mla.kv_read(kv, slots, scale, status=st)
    assert int(st.item()) == 0
    want, slack, t = _expect(rows, weight, pos, tab, interleaved, eps)
    at = slots.long()
    left = torch.ones(1024, dtype=torch.bool, device="cuda")
    left[at] = False
    assert torch.equal(kv[left].view(torch.uint8), before[left].view(torch.uint8)), \
        "rows of other slots changed"
    got = f64(back)
    if kind == "bf16":
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + slack + 1e-39)
        assert torch.equal(back, kv[at])
    elif kind == "fp8":
        s = f64(scale[at])
        amax = np.abs(want).max(1)
        assert np.all(np.abs(s - amax / 448) <= REL * amax / 448 + slack.max(1) / 448 + 1e-44)
        codes = kv[at].cpu().numpy()
        val = e4m3_values(codes)
        assert np.isfinite(val).all()
        safe = np.where(s > 0, s, 1.0)[:, None]
        # half a step of the code, or of the smallest code, and the slack
        err = np.abs(val * s[:, None] - want)
        assert np.all(err <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * s[:, None] + slack)
        quo = np.where(s[:, None] > 0, want / safe, 0.0)
        fixed = sure(quo, E4M3, 2 * REL) & (slack <= 2 * REL * np.abs(want))
        assert fixed.mean() > 0.9 or n < 3
        assert np.array_equal((codes & 0x7F)[fixed], encode(quo, E4M3)[fixed])
        assert np.all(np.abs(got - val * s[:, None]) <= 2.0 ** -8 * np.abs(val * s[:, None]) + 1e-39)
    else:
        raw = kv[at].cpu().numpy()
        c, blocks = want[:, :NOPE], want[:, :NOPE].reshape(n, 32, 16)
        quo = np.abs(blocks).max(-1) / (6 * G)
        fixed = sure(quo, E4M3, REL)
        # without the norm the maxima are bf16 values, some of them exact ties
        assert fixed.mean() > (0.99 if norm else 0.9) or n < 3
        assert np.array_equal(raw[:, 256:288][fixed], encode(quo, E4M3)[fixed])
        s = e4m3_values(raw[:, 256:288])
        step = np.repeat(s * G, 16, 1)
        cq = np.where(step > 0, c / np.where(step > 0, step, 1.0), 0.0)
        code = np.stack([raw[:, :256] & 15, raw[:, :256] >> 4], -1).reshape(n, NOPE)
        fixed = sure(cq, E2M1, REL)
        assert fixed.mean() > 0.99 or n < 3
        assert np.array_equal((code & 7)[fixed], encode(cq, E2M1)[fixed])
        neg = (c < 0) & (code & 7 != 0)
        assert np.array_equal((code & 8 != 0) & (code & 7 != 0), neg)
        r = want[:, NOPE:] / G
        fixed = sure(r, E4M3, REL) & (slack[:, NOPE:] <= REL * np.abs(want[:, NOPE:]))
        assert fixed.mean() > 0.8 or n < 3
        assert np.array_equal((raw[:, 288:] & 0x7F)[fixed], encode(r, E4M3)[fixed])
        val = decode4(raw, G)
        assert np.all(np.abs(got - val) <= 2.0 ** -8 * np.abs(val) + 2.0 ** -22 * np.abs(val))
    if H:
        x = f64(q)
        ref = rotate(x, t[:, None, :32], t[:, None, 32:], interleaved)
        a = np.abs(x)
        other = a[..., np.arange(64) ^ 1] if interleaved else np.roll(a, 32, -1)
        assert np.all(np.abs(f64(q_out) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * (a + other))


def test_queries_rotate_in_place():
    rows, weight, q, pos = _inputs(7, 5, 3)
    tab = table(5000).cuda()
    slots = torch.arange(7, dtype=torch.int32, device="cuda")
    for interleaved in (True, False):
        kv, scale = _pool("fp4", 64)
        apart = mla.kv_append(rows, slots, pos, tab, kv, scale, norm_weight=weight, q_rope=q,
                              interleaved=interleaved)
        own = q.clone()
        mla.kv_append(rows, slots, pos, tab, kv, scale, norm_weight=weight, q_rope=own, q_out=own,
                      interleaved=interleaved)
        assert torch.equal(apart, own)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_bad_slots_and_positions_are_skipped_and_reported(kind):
    rows, weight, q, pos = _inputs(6, 2, 4)
    tab = table(5000).cuda()
    kv, scale = _pool(kind, 64)
    ref_kv, ref_scale = _pool(kind, 64)
    good = torch.tensor([3, 9, 12, 60, 1, 5], dtype=torch.int32, device="cuda")
    ref_q = mla.kv_append(rows, good, pos, tab, ref_kv, ref_scale, norm_weight=weight, q_rope=q)
    slots, bad_pos = good.clone(), pos.clone()
    slots[1], slots[3], bad_pos[4] = -1, 64, 5000
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full_like(q, 9.0)
    mla.kv_append(rows, slots, bad_pos, tab, kv, scale, norm_weight=weight, q_rope=q, q_out=q_out,
                  status=st)
    assert int(st.item()) == mla.STATUS_BAD_SLOT | mla.STATUS_BAD_POSITION
    empty, _ = _pool(kind, 64)
    for i, s in enumerate(good.tolist()):
        want = empty if i in (1, 3, 4) else ref_kv
        assert torch.equal(kv[s].view(torch.uint8), want[s].view(torch.uint8)), i
        assert torch.equal(q_out[i], torch.full_like(q[i], 9.0) if i == 4 else ref_q[i]), i
    st.zero_()
    back = mla.kv_read(ref_kv, slots, ref_scale, status=st)
    assert int(st.item()) == mla.STATUS_BAD_SLOT
    full = mla.kv_read(ref_kv, good, ref_scale)
    full[1] = 0
    full[3] = 0
    assert torch.equal(back, full)


def test_saturation_and_far_offsets():
    """Values beyond 2688 g and 448 g saturate; a pool row past 2^31 bytes is
    addressed in 64 bits."""
    slots = (1 << 31) // 352 + 70
    kv = torch.zeros((slots, 352), dtype=torch.uint8, device="cuda")
    g = torch.full((1,), 2.0 ** -10, device="cuda")
    rows = torch.full((1, 576), 900.0).bfloat16().cuda()
    rows[0, 1::2] = -900.0
    at = torch.tensor([slots - 1], dtype=torch.int32, device="cuda")
    tab = torch.zeros((1, 64), device="cuda")
    tab[:, :32] = 1.0
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.kv_append(rows, at, pos, tab, kv, g)
    got = f64(mla.kv_read(kv, at, g))[0]
    sign = np.where(np.arange(576) % 2, -1.0, 1.0)
    assert np.array_equal(got[:512], sign[:512] * 2688 * 2.0 ** -10)
    assert np.array_equal(got[512:], sign[512:] * 448 * 2.0 ** -10)
    assert int(kv[:-1].sum()) == 0


def test_every_code_reads_back():
    """All 256 x (sign, code, scale) combinations of a block and of a RoPE code."""
    kv = random_pool(256, 1)
    kv[:, :256] = np.arange(256)[:, None]
    kv[:, 256:288] = (np.arange(256)[:, None] + 8 * np.arange(32)) % 0x7F
    kv[:, 288:] = np.arange(64) + 64 * (np.arange(256)[:, None] % 4)
    t = torch.from_numpy(kv).cuda()
    got = f64(mla.kv_read(t, torch.arange(256, dtype=torch.int32, device="cuda"),
                          torch.ones(1, device="cuda")))
    want = decode4(kv, 1.0)
    assert np.array_equal(got, want, equal_nan=True)


def test_side_stream_and_empty():
    rows, weight, q, pos = _inputs(40, 3, 5)
    tab = table(5000).cuda()
    slots = torch.arange(40, dtype=torch.int32, device="cuda")
    kv, scale = _pool("fp4", 64)
    mla.kv_append(rows, slots, pos, tab, kv, scale, norm_weight=weight)
    kv2, _ = _pool("fp4", 64)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    mla.kv_append(rows, slots, pos, tab, kv2, scale, norm_weight=weight, stream=s)
    s.synchronize()
    assert torch.equal(kv, kv2)
    before = kv.clone()
    mla.kv_append(rows[:0], slots[:0], pos[:0], tab, kv, scale, norm_weight=weight)
    assert mla.kv_read(kv, slots[:0], scale).shape == (0, 576)
    assert torch.equal(kv, before)


@pytest.mark.parametrize("width,dtype", [(352, torch.uint8), (576, torch.uint8), (576, torch.bfloat16)])
def test_pool_past_32_bit_offsets(width, dtype):
    """Rows at the end of a pool of more than 2^32 bytes, and back."""
    slots = ((1 << 32) // (width * dtype.itemsize) // 64 + 2) * 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    rows = torch.randn((70, 576), generator=gen, device="cuda").bfloat16()
    pos = torch.arange(70, dtype=torch.int32, device="cuda")
    back = []
    for total in (128, slots):
        pool = torch.zeros((total, width), dtype=dtype, device="cuda")
        scale = None if dtype == torch.bfloat16 else torch.full((total if width == 576 else 1,), 0.0625, device="cuda")
        at = torch.arange(total - 70, total, dtype=torch.int32, device="cuda")
        mla.kv_append(rows, at, pos, table(128).cuda(), pool, scale)
        back.append(mla.kv_read(pool, at, scale))
        assert int((pool[:total - 70] != 0).sum()) == 0 if total == 128 else not pool[:64].any()
        del pool
    assert torch.equal(*back) and back[0].float().abs().max() > 1
