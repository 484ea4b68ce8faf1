"""Refusals of the 4-bit cache's entry points and their neighbours, on the host
before any launch (no GPU needed): error codes of the C ABI with made-up
aligned addresses, and the binding's checks of shapes, types and strides.
"""
import ctypes

import numpy as np
import pytest
import torch

import mla_latent_decode_gb300 as mla
from latent_ref import E2M1, E4M3, decode4, e4m3_values, encode, random_pool
from mla_latent_decode_gb300 import build

ARG, UNSUP, ALIGN = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mla.library()


def P(x):
    return None if x is None else ctypes.c_void_p(x)


def append(lib, **over):
    a = dict(rows=16, stride=576, n=4, w=16, eps=1e-6, slots=16, pos=16, tab=16, mp=10, il=1, kv=16,
             dt=2, ks=16, ns=64, q=16, qt=192, qh=64, qo=16, ot=192, oh=64, H=3, st=None)
    a.update(over)
    return lib.mla_kv_append(P(a["rows"]), a["stride"], a["n"], P(a["w"]), a["eps"], P(a["slots"]), P(a["pos"]),
                             P(a["tab"]), a["mp"], a["il"], P(a["kv"]), a["dt"], P(a["ks"]), a["ns"], P(a["q"]),
                             a["qt"], a["qh"], P(a["qo"]), a["ot"], a["oh"], a["H"], P(a["st"]), None)


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), ARG), (dict(rows=None), ARG), (dict(slots=None), ARG), (dict(pos=None), ARG),
    (dict(tab=None), ARG), (dict(kv=None), ARG), (dict(dt=3), ARG), (dict(ks=None), ARG),
    (dict(dt=1, ks=None), ARG), (dict(ns=0), ARG), (dict(ns=1 << 31), ARG), (dict(mp=0), ARG),
    (dict(stride=568), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG),
    (dict(H=-1), ARG), (dict(q=None), ARG), (dict(qo=None), ARG), (dict(qh=32), ARG), (dict(qt=8), ARG),
    (dict(rows=24), ALIGN), (dict(stride=577), ALIGN), (dict(w=8), ALIGN), (dict(slots=2), ALIGN),
    (dict(tab=4), ALIGN), (dict(kv=8), ALIGN), (dict(q=8), ALIGN), (dict(qh=65), ALIGN), (dict(oh=68), ALIGN),
    (dict(st=2), ALIGN), (dict(n=0), 0), (dict(n=0, rows=None), 0)])
def test_append_arguments(lib, over, code):
    assert append(lib, **over) == code
    if code:
        assert lib.mla_last_error_string()


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), ARG), (dict(kv=None), ARG), (dict(dt=5), ARG), (dict(ks=None), ARG), (dict(slots=None), ARG),
    (dict(out=None), ARG), (dict(stride=575), ARG), (dict(stride=580), ALIGN), (dict(out=8), ALIGN), (dict(n=0), 0)])
def test_read_arguments(lib, over, code):
    a = dict(kv=16, dt=2, ks=16, ns=64, slots=16, n=4, out=16, stride=576, st=None)
    a.update(over)
    assert lib.mla_kv_read(P(a["kv"]), a["dt"], P(a["ks"]), a["ns"], P(a["slots"]), a["n"], P(a["out"]),
                           a["stride"], P(a["st"]), None) == code


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), ARG), (dict(d=0), ARG), (dict(d=32769), UNSUP), (dict(group=16), ARG), (dict(group=256), ARG),
    (dict(d=100, group=32), ARG), (dict(eps=-1e-6), ARG), (dict(x=None), ARG), (dict(w=None), ARG),
    (dict(out=None, out8=None), ARG), (dict(res=None), ARG), (dict(ro=None), ARG), (dict(sc=None), ARG),
    (dict(xs=100), ARG), (dict(os=100), ARG), (dict(ss=0), ARG), (dict(group=64, ss=2), ARG),
    (dict(x=1), ALIGN), (dict(sc=2), ALIGN), (dict(n=0), 0)])
def test_norm_arguments(lib, over, code):
    a = dict(x=16, xs=256, res=16, rs=256, ro=16, ros=256, w=16, eps=1e-6, n=4, d=256, out=16, os=256, out8=16,
             o8s=256, sc=16, ss=4, group=0)
    a.update(over)
    assert lib.mla_add_rms_norm(P(a["x"]), a["xs"], P(a["res"]), a["rs"], P(a["ro"]), a["ros"], P(a["w"]), a["eps"],
                                a["n"], a["d"], P(a["out"]), a["os"], P(a["out8"]), a["o8s"], P(a["sc"]), a["ss"],
                                a["group"], None) == code


def test_decode_refuses_fp4_without_its_factor(lib):
    p = P
    args = lambda ks, dt: (p(16), p(16), p(16), p(ks), dt, 4096, p(16), 64, p(16), None, 1, 5, 96, 1, 64, 0.07, 1,
                           None, None, 0, p(16), p(16), None, None)
    assert lib.mla_decode_partial(*args(None, 2)) == ARG
    assert lib.mla_decode_partial(*args(16, 3)) == ARG
    assert lib.mla_decode_partial(*args(20, 2)) == ALIGN
    wrong = list(args(16, 2))
    wrong[18], wrong[19] = p(16), 7  # a work list of the wrong length
    assert lib.mla_decode_partial(*wrong) == ARG
    assert lib.mla_kv_write(p(16), 4, p(16), p(16), 2, p(16), 64, None, None) == ARG


def test_planner_takes_fp4(lib):
    lens = [100_000] * 16
    S, bnd, work, eff = mla.plan_sched(16, 5, 96, lens, num_sms=152, kv_dtype="fp4_e2m1")
    assert S >= 1 and bnd.shape == (16, S + 1) and sorted(work) == list(range(len(work)))


def test_binding_refuses_shapes_types_and_strides():
    bf, i32 = torch.bfloat16, torch.int32
    rows, slots, pos = torch.zeros((4, 576), dtype=bf), torch.zeros(4, dtype=i32), torch.zeros(4, dtype=i32)
    tab, kv, g = torch.zeros((8, 64)), torch.zeros((64, 352), dtype=torch.uint8), torch.ones(1)
    ok = dict(rows=rows, slots=slots, positions=pos, cos_sin=tab, kv=kv, kv_scale=g)
    for bad in (dict(rows=rows.float()), dict(rows=rows[:, :575]), dict(rows=torch.zeros((576, 4), dtype=bf).T),
                dict(slots=slots.long()), dict(positions=pos[:3]), dict(cos_sin=tab[:, :32]),
                dict(cos_sin=tab.double()), dict(kv=kv[:, :300]), dict(kv_scale=g.double()),
                dict(kv=torch.zeros((64, 576), dtype=torch.uint8)),  # E4M3: one scale per slot
                dict(norm_weight=torch.zeros(511, dtype=bf)), dict(norm_weight=torch.zeros(512)),
                dict(q_rope=torch.zeros((4, 2, 32), dtype=bf)), dict(q_rope=torch.zeros((3, 2, 64), dtype=bf)),
                dict(q_rope=torch.zeros((4, 64, 2), dtype=bf).transpose(1, 2))):
        with pytest.raises(ValueError):
            mla.kv_append(**{**ok, **bad})
    with pytest.raises(TypeError):
        mla.kv_append(**{**ok, "kv": kv.float()})
    with pytest.raises(ValueError):
        mla.kv_read(kv, slots, g, out=torch.zeros((3, 576), dtype=bf))
    with pytest.raises(ValueError):
        mla.kv_read(kv, slots.long(), g)
    x, w = torch.zeros((4, 64), dtype=bf), torch.zeros(64, dtype=bf)
    for bad in (dict(x=x[0]), dict(x=x.float()), dict(weight=w[:63]), dict(residual=x[:3]),
                dict(residual_out=x), dict(out=x.float()), dict(out8=x), dict(out8=torch.zeros((3, 64), dtype=torch.uint8)),
                dict(out8=torch.zeros((4, 64), dtype=torch.uint8), scales=torch.zeros(4))):
        with pytest.raises((ValueError, IndexError)):
            mla.add_rms_norm(**{**dict(x=x, weight=w), **bad})


def test_binding_refuses_fp4_decode_layouts():
    bf = torch.bfloat16
    ok = dict(q_nope=torch.zeros((2, 1, 4, 512), dtype=bf), q_rope=torch.zeros((2, 1, 4, 64), dtype=bf),
              kv=torch.zeros((64, 352), dtype=torch.uint8), kv_scale=torch.ones(1),
              req_to_token=torch.zeros((2, 64), dtype=torch.int32), seq_lens=torch.ones(2, dtype=torch.int32),
              kv_limit=None, num_splits=1, sm_scale=0.07)
    for bad in (dict(q_nope=ok["q_nope"].float()), dict(q_rope=torch.zeros((2, 1, 4, 128), dtype=bf)[..., ::2]),
                dict(q_rope=torch.zeros((2, 1, 3, 64), dtype=bf)), dict(kv_scale=None),
                dict(kv_scale=torch.ones(1, dtype=torch.float64)), dict(seq_lens=torch.ones(2, dtype=torch.int64)),
                dict(kv=torch.zeros((64, 704), dtype=torch.uint8)[:, ::2]),
                dict(req_to_token=torch.zeros((2, 64), dtype=torch.int64))):
        for call in (mla.decode_partial, mla.decode_fused, mla.decode_scratch):
            with pytest.raises(ValueError):
                call(**{**ok, **bad})


def test_reference_formats():
    """The tests' own codecs against torch's E4M3 and the E2M1 value set."""
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(e4m3_values(codes.numpy()), want, equal_nan=True)
    x = torch.randn(20000, dtype=torch.float64).float() * 30
    got = torch.from_numpy(encode(x.double().numpy(), E4M3)).to(torch.uint8)
    assert torch.equal(got, x.abs().to(torch.float8_e4m3fn).view(torch.uint8))
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0]
    assert list(E2M1[encode(ties, E2M1)]) == [0, 1, 1, 2, 2, 4, 4, 6]
    kv = random_pool(3, 0)
    row = decode4(kv, 2.0)
    assert row[1, 0] == 2.0 * E2M1[kv[1, 0] & 7] * (-1 if kv[1, 0] & 8 else 1) * e4m3_values(kv[1, 256])
    assert row[2, 575] == 2.0 * e4m3_values(kv[2, 351])


@pytest.mark.parametrize("H,L,wide", [(16, 100000, True), (96, 100000, True), (97, 100000, False), (16, 64, False)])
def test_plan_spreads_one_request_over_every_sm(H, L, wide):
    """One CTA per part up to 96 rows, so up to 160 parts; clusters stay at 64."""
    S, bnd, work, _ = mla.plan_sched(1, 1, H, [L], num_sms=152, kv_dtype="fp4_e2m1")
    assert (S > 64) == wide and S <= 160
    assert bnd.shape == (1, S + 1) and bnd[0, 0] == 0 and bnd[0, -1] == -(-L // 64) and (np.diff(bnd[0]) >= 0).all()
    assert sorted(work) == list(range(S))
    assert mla.plan_parts(1, 1, H, [L], num_sms=152, kv_dtype="fp4_e2m1")[0] <= 160


@pytest.mark.parametrize("B,q,H,L,groups", [
    (2, 3, 128, 300, True), (1, 5, 96, 64, True), (16, 5, 96, 100000, False), (1, 5, 96, 100000, False)])
def test_plan_takes_row_groups_for_short_work(B, q, H, L, groups):
    S, bnd, work, _ = mla.plan_sched(B, q, H, [L] * B, num_sms=152, kv_dtype="fp4_e2m1")
    U = -(-q * H // (96 if groups else 256))
    assert sorted(work) == list(range(B * S * U))
    assert bnd.shape == (B, S + 1) and (bnd[:, 0] == 0).all() and (bnd[:, -1] == -(-L // 64)).all()


def test_append_of_no_tokens_with_queries(lib):
    """n = 0 is a no-op: an empty tensor's address is NULL, whatever H is."""
    assert append(lib, n=0, q=None, qo=None) == 0
    assert append(lib, n=0, q=None, qo=None, rows=None, slots=None, pos=None) == 0
    assert append(lib, n=0, H=-1) == ARG and append(lib, n=0, kv=None) == ARG


def test_binding_appends_no_tokens_with_queries(lib, monkeypatch):
    monkeypatch.setattr(mla, "_launch", lambda t, stream, fn, *args: mla._check(fn(*args, None)))
    bf, i32 = torch.bfloat16, torch.int32
    kv, g = torch.zeros((64, 352), dtype=torch.uint8), torch.ones(4)
    rows, ids = torch.zeros((0, 576), dtype=bf), torch.zeros(0, dtype=i32)
    got = mla.kv_append(rows, ids, ids, torch.zeros((8, 64)), kv, g, q_rope=torch.zeros((5, 3, 64), dtype=bf)[:0])
    assert got.shape == (0, 3, 64) and got.dtype == bf


@pytest.mark.parametrize("capacity", [1 << 62, (1 << 63) - 1, 1 << 40])
def test_plan_takes_any_capacity(lib, capacity):
    """The capacity bounds what is written; it is not a size to allocate."""
    B, q, H = 2, 3, 128
    bnd, work = (ctypes.c_int32 * (B * 65))(), (ctypes.c_int32 * (B * 64 * 4))()
    S, n, eff = ctypes.c_int(), ctypes.c_int64(), ctypes.c_float()
    lens = (ctypes.c_int32 * B)(300, 300)
    rc = lib.mla_plan_sched(B, q, H, 1, 2, lens, 152, 8, bnd, ctypes.byref(S), work, capacity, ctypes.byref(n),
                            ctypes.byref(eff))
    want = mla.plan_sched(B, q, H, [300] * B, num_sms=152, kv_dtype="fp4_e2m1")
    assert rc == 0 and S.value == want[0] and list(work[:n.value]) == list(want[2])
    assert list(bnd[:B * (S.value + 1)]) == list(want[1].reshape(-1))


def _decode_args(**over):
    bf = torch.bfloat16
    a = dict(q_nope=torch.zeros((2, 3, 4, 512), dtype=bf), q_rope=torch.zeros((2, 3, 4, 64), dtype=bf),
             kv=torch.zeros((64, 352), dtype=torch.uint8), kv_scale=torch.ones(4),
             req_to_token=torch.zeros((2, 64), dtype=torch.int32), seq_lens=torch.ones(2, dtype=torch.int32),
             kv_limit=None, num_splits=2, sm_scale=0.07)
    a.update(over)
    return a


I32, F32 = torch.int32, torch.float32
COMMON = [
    ("seq_lens", torch.ones(1, dtype=I32)), ("req_to_token", torch.zeros((1, 64), dtype=I32)),
    ("req_to_token", torch.zeros(128, dtype=I32)),
    ("kv_limit", torch.ones((2, 3), dtype=torch.int64)), ("kv_limit", torch.ones((2, 2), dtype=I32)),
    ("kv_limit", torch.ones((3, 2), dtype=I32).T),
    ("split_pages", torch.zeros((2, 3), dtype=torch.int64)), ("split_pages", torch.zeros((2, 2), dtype=I32)),
    ("split_pages", torch.zeros((2, 6), dtype=I32)[:, ::2]),
    ("work", torch.zeros(4, dtype=torch.int64)), ("work", torch.zeros(8, dtype=I32)[::2]),
    ("status", torch.zeros(1, dtype=torch.int64)), ("status", torch.zeros(0, dtype=I32))]
N = 2 * 3 * 4
PARTIAL = [("O_part", torch.zeros(2 * N * 512 - 1)), ("O_part", torch.zeros(2 * N * 512, dtype=torch.float16)),
           ("O_part", torch.zeros((2 * N, 1024))[:, :512]), ("LSE_part", torch.zeros(2 * N - 1)),
           ("LSE_part", torch.zeros(2 * N, dtype=torch.bfloat16))]
MERGED = [("out", torch.zeros(N * 512)), ("out", torch.zeros(N * 512 - 1, dtype=torch.bfloat16)),
          ("lse_out", torch.zeros(N, dtype=torch.float64)), ("lse_out", torch.zeros(N - 1))]
FUSED = PARTIAL + MERGED + [("O_part", torch.zeros(2 * N * 512, dtype=torch.bfloat16)),
                            ("counters", torch.zeros(1, dtype=I32)), ("counters", torch.zeros(2, dtype=torch.int64))]


@pytest.mark.parametrize("call,bad", [(c, b) for c, more in (("decode_partial", PARTIAL), ("decode_fused", FUSED),
                                                             ("decode_scratch", MERGED)) for b in COMMON + more],
                         ids=lambda x: x if isinstance(x, str) else f"{x[0]}-{x[1].dtype}-{tuple(x[1].shape)}")
def test_binding_refuses_fp4_decode_buffers(call, bad, monkeypatch):
    """Whatever the kernels read or write by address is refused by name when it is
    too small, of another type or not contiguous."""
    launched = []
    monkeypatch.setattr(mla, "_launch", lambda *a: launched.append(a))
    monkeypatch.setattr(mla, "_on", lambda t: launched.append(t) or mla._HERE_ALREADY)
    monkeypatch.setattr(mla, "_check", lambda rc: rc)
    monkeypatch.setattr(mla, "_stream", lambda s: None)

    class Library:
        def __getattr__(self, name):
            return lambda *a: 0

    monkeypatch.setattr(mla, "library", lambda: Library())
    good = dict(kv_limit=torch.ones((2, 3), dtype=I32), split_pages=torch.zeros((2, 3), dtype=I32),
                work=torch.zeros(4, dtype=I32), status=torch.zeros(1, dtype=I32))
    if call != "decode_scratch":
        good.update(O_part=torch.zeros(2 * N * 512), LSE_part=torch.zeros(2 * N))
    if call != "decode_partial":
        good.update(out=torch.zeros(N * 512, dtype=torch.bfloat16), lse_out=torch.zeros(N))
    if call == "decode_fused":
        good.update(counters=torch.zeros(2, dtype=I32))
    getattr(mla, call)(**_decode_args(**good))
    assert len(launched) == 1
    with pytest.raises(ValueError, match=bad[0]):
        getattr(mla, call)(**_decode_args(**{**good, bad[0]: bad[1]}))
    assert len(launched) == 1


def test_one_launch_over_row_groups_bounds_its_parts(lib):
    """Two groups count in the halves of one counter."""
    p = P
    args = lambda S, shards, work, n: (p(16), p(16), p(16), p(16), 2, 4096, p(16), 64, p(16), None, 1, 2, 64, shards, 64,
                                       0.07, S, None, work, n, p(16), p(16), p(16), p(16), None, None, None)
    assert lib.mla_decode(*args(4096, 16, p(16), 2 * 4096 * 16)) == UNSUP
