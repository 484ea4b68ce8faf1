"""Refusals of the prompts', beams' and pages' entry points on the host before any
launch (no GPU needed), and the prompts' planner against its contract: every block
of every sequence in exactly one set of parts.
"""
import contextlib
import ctypes
import random

import numpy as np
import pytest
import torch

import mla_latent_decode_gb300 as mla
from mla_latent_decode_gb300 import build

ARG, UNSUP, ALIGN = -1, -2, -3
bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return mla.library()


def P(x):
    return None if x is None else ctypes.c_void_p(x)


@pytest.mark.parametrize("over,code", [
    (dict(Tq=-1), ARG), (dict(Tk=-1), ARG), (dict(N=-1), ARG), (dict(nw=-1), ARG), (dict(parts=-1), ARG), (dict(H=0), ARG),
    (dict(H=65536), ARG), (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG),
    (dict(scale=float("inf")), ARG), (dict(ctas=0), ARG), (dict(ctas=3), ARG), (dict(Tq=0x7fffff01), ARG),
    (dict(Tk=0x7fffff01), ARG), (dict(nw=1 << 29), ARG), (dict(qn=None), ARG), (dict(qr=None), ARG), (dict(kn=None), ARG),
    (dict(kr=None), ARG), (dict(v=None), ARG), (dict(cq=None), ARG), (dict(ck=None), ARG), (dict(work=None), ARG),
    (dict(out=None), ARG), (dict(parts=2), ARG), (dict(qt=120), ARG), (dict(qh=64), ARG), (dict(rh=56), ARG),
    (dict(kt=8), ARG), (dict(vh=120), ARG), (dict(krt=56), ARG), (dict(qn=24), ALIGN), (dict(qr=40), ALIGN),
    (dict(kn=8), ALIGN), (dict(v=8), ALIGN), (dict(kr=8), ALIGN), (dict(qt=4 * 192 + 4), ALIGN), (dict(vt=1025), ALIGN),
    (dict(krt=577), ALIGN), (dict(out=48), ALIGN), (dict(cq=2), ALIGN), (dict(ck=2), ALIGN), (dict(pre=2), ALIGN),
    (dict(work=2), ALIGN), (dict(lse=2), ALIGN), (dict(st=2), ALIGN), (dict(parts=2, op=48, lp=16), ALIGN),
    (dict(nw=0), 0), (dict(N=0), 0), (dict(Tq=0), 0)])
def test_prefill_arguments(lib, over, code):
    a = dict(qn=32, qt=4 * 192, qh=192, qr=32, rt=4 * 192, rh=192, Tq=10, kn=32, kt=4 * 256, kh=256, kr=32, krt=576, v=32,
             vt=4 * 256, vh=256, Tk=20, H=4, cq=16, ck=16, pre=None, N=2, causal=1, scale=0.07, work=16, nw=2, ctas=1,
             parts=0, op=None, lp=None, out=32, lse=None, st=None)
    a.update(over)
    assert lib.mla_prefill(P(a["qn"]), a["qt"], a["qh"], P(a["qr"]), a["rt"], a["rh"], a["Tq"], P(a["kn"]), a["kt"], a["kh"],
                           P(a["kr"]), a["krt"], P(a["v"]), a["vt"], a["vh"], a["Tk"], a["H"], P(a["cq"]), P(a["ck"]),
                           P(a["pre"]), a["N"], a["causal"], a["scale"], P(a["work"]), a["nw"], a["ctas"], a["parts"],
                           P(a["op"]), P(a["lp"]), P(a["out"]), P(a["lse"]), P(a["st"]), None) == code
    if code:
        assert lib.mla_last_error_string()


@pytest.mark.parametrize("over,code", [
    (dict(dt=3), ARG), (dict(dt=-1), ARG), (dict(B=-1), ARG), (dict(W=0), ARG), (dict(V=0), ARG), (dict(k=0), ARG),
    (dict(W=1, V=3, k=4, end=2), ARG), (dict(W=33), UNSUP), (dict(k=65), UNSUP), (dict(end=-1), ARG), (dict(end=1000), ARG),
    (dict(bs=999), ARG), (dict(ws=999), ARG), (dict(B=1 << 30), ARG), (dict(x=None), ARG), (dict(c=None), ARG),
    (dict(os=None), ARG), (dict(pa=None), ARG), (dict(to=None), ARG), (dict(x=17), ALIGN), (dict(dt=2, x=18), ALIGN),
    (dict(c=2), ALIGN), (dict(os=2), ALIGN), (dict(pa=2), ALIGN), (dict(to=2), ALIGN), (dict(st=2), ALIGN), (dict(B=0), 0)])
def test_beam_arguments(lib, over, code):
    a = dict(x=16, dt=0, bs=4000, ws=1000, c=16, fin=None, B=3, W=4, V=1000, end=2, k=4, os=16, pa=16, to=16, st=None)
    a.update(over)
    assert lib.mla_beam_select(P(a["x"]), a["dt"], a["bs"], a["ws"], P(a["c"]), P(a["fin"]), a["B"], a["W"], a["V"], a["end"],
                               a["k"], P(a["os"]), P(a["pa"]), P(a["to"]), P(a["st"]), None) == code
    if code:
        assert lib.mla_last_error_string()


@pytest.mark.parametrize("over,code", [
    (dict(R=-1), ARG), (dict(s=0), ARG), (dict(os=0), ARG), (dict(np=0), ARG), (dict(R=4097), UNSUP),
    (dict(np=(1 << 25) + 1), ARG), (dict(s=1 << 31), ARG), (dict(R=4096, s=1 << 25), ARG), (dict(t=None), ARG),
    (dict(l=None), ARG), (dict(r=None), ARG), (dict(f=None), ARG), (dict(o=None), ARG), (dict(lo=None), ARG),
    (dict(c=None), ARG), (dict(o=4096), ARG), (dict(o=4096 + 4 * 127), ARG), (dict(lo=16), ARG), (dict(t=4098), ALIGN),
    (dict(p=2), ALIGN), (dict(k=2), ALIGN), (dict(g=2), ALIGN), (dict(st=2), ALIGN), (dict(R=0), 0)])
def test_fork_arguments(lib, over, code):
    a = dict(t=4096, s=64, l=16, p=None, k=None, g=None, R=2, r=32, np=10, f=48, o=65536, os=64, lo=64, c=80, st=None)
    a.update(over)
    assert lib.mla_pages_fork(P(a["t"]), a["s"], P(a["l"]), P(a["p"]), P(a["k"]), P(a["g"]), a["R"], P(a["r"]), a["np"],
                              P(a["f"]), P(a["o"]), a["os"], P(a["lo"]), P(a["c"]), P(a["st"]), None) == code
    if code:
        assert lib.mla_last_error_string()


@pytest.mark.parametrize("over,code", [
    (dict(R=-1), ARG), (dict(s=0), ARG), (dict(os=0), ARG), (dict(np=0), ARG), (dict(m=-1), ARG),
    (dict(np=(1 << 25) + 1), ARG), (dict(s=1 << 31), ARG), (dict(r=None), ARG), (dict(n=None), ARG), (dict(t=None), ARG),
    (dict(l=None), ARG), (dict(o=None), ARG), (dict(a=None), ARG), (dict(b=None), ARG), (dict(o=4100), ARG),
    (dict(o=4096, os=65), ARG), (dict(l=2), ALIGN), (dict(r=2), ALIGN), (dict(a=2), ALIGN), (dict(n=2), ALIGN),
    (dict(st=2), ALIGN)])
def test_compact_arguments(lib, over, code):
    a = dict(t=4096, s=64, l=16, R=2, r=32, np=10, o=65536, os=64, a=48, b=64, m=4, n=80, st=None)
    a.update(over)
    assert lib.mla_pages_compact(P(a["t"]), a["s"], P(a["l"]), a["R"], P(a["r"]), a["np"], P(a["o"]), a["os"], P(a["a"]),
                                 P(a["b"]), a["m"], P(a["n"]), P(a["st"]), None) == code
    assert lib.mla_last_error_string()


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), ARG), (dict(dt=3), ARG), (dict(ns=63), ARG), (dict(ns=1 << 31), ARG), (dict(kv=None), ARG),
    (dict(s=None), ARG), (dict(d=None), ARG), (dict(dt=1), ARG), (dict(kv=8), ALIGN), (dict(s=2), ALIGN), (dict(d=2), ALIGN),
    (dict(t=2), ALIGN), (dict(c=2), ALIGN), (dict(dt=1, ks=2), ALIGN), (dict(st=2), ALIGN), (dict(n=0), 0)])
def test_copy_arguments(lib, over, code):
    a = dict(kv=16, dt=0, ks=None, ns=640, s=16, d=32, t=None, c=None, n=4, st=None)
    a.update(over)
    assert lib.mla_kv_copy(P(a["kv"]), a["dt"], P(a["ks"]), a["ns"], P(a["s"]), P(a["d"]), P(a["t"]), P(a["c"]), a["n"],
                           P(a["st"]), None) == code


def test_binding_refuses():
    def z(*shape, dtype=bf):
        return torch.zeros(shape, dtype=dtype)

    x = dict(q_nope=z(5, 2, 128), q_rope=z(5, 2, 64), k_nope=z(7, 2, 128), k_rope=z(7, 64), v=z(7, 2, 128),
             cu_q=z(2, dtype=i32), cu_kv=z(2, dtype=i32), work=z(1, 8, dtype=i32), sm_scale=0.07)
    for over in (dict(q_nope=z(5, 2, 64)), dict(q_nope=z(5, 256)), dict(q_rope=z(4, 2, 64)), dict(k_nope=z(7, 3, 128)),
                 dict(v=z(7, 2, 128, dtype=torch.float16)), dict(k_rope=z(7, 32)), dict(k_rope=z(7, 2, 64)),
                 dict(k_nope=z(7, 128, 2).transpose(1, 2)), dict(cu_q=z(2, dtype=torch.int64)), dict(cu_kv=z(3, dtype=i32)),
                 dict(prefix=z(2, dtype=i32)), dict(work=z(8, dtype=i32)), dict(work=z(1, 3, 8, dtype=i32)),
                 dict(work=z(1, 8, dtype=torch.int64)), dict(out=z(5, 2, 64)), dict(lse_out=z(5, 2)),
                 dict(num_parts=2, O_part=z(2, 2, 256, 64, dtype=f32)), dict(status=z(1)), dict(cu_q=z(0, dtype=i32))):
        with pytest.raises(ValueError):
            mla.prefill(**{**x, **over})
    b = dict(logits=z(2, 3, 50), scores=z(2, 3, dtype=f32), k=4)
    for over in (dict(logits=z(6, 50)), dict(logits=z(2, 3, 50, dtype=torch.float64)), dict(logits=z(2, 50, 3).transpose(1, 2)),
                 dict(scores=z(2, 2, dtype=f32)), dict(scores=z(2, 3)), dict(finished=z(2, 2, dtype=torch.bool)),
                 dict(finished=z(2, 3, dtype=i32)), dict(out_scores=z(2, 3, dtype=f32)), dict(parents=z(2, 4)),
                 dict(tokens=z(2, 4, dtype=torch.int64)), dict(status=z(1))):
        with pytest.raises(ValueError):
            mla.beam_select(**{**b, **over})
    f = dict(table=z(2, 128, dtype=i32), lens=z(2, dtype=i32), refs=z(9, dtype=i32), free_count=z(1, dtype=i32))
    for over in (dict(table=z(2, 128)), dict(table=z(128, 2, dtype=i32).T), dict(lens=z(3, dtype=i32)),
                 dict(refs=z(9, dtype=torch.int64)), dict(free_count=z(0, dtype=i32)), dict(parents=z(3, dtype=i32)),
                 dict(keep=z(2)), dict(grow=z(1, dtype=i32)), dict(table_out=z(3, 128, dtype=i32)),
                 dict(lens_out=z(1, dtype=i32)), dict(copies=z(2, 3, dtype=i32))):
        with pytest.raises(ValueError):
            mla.pages_fork(**{**f, **over})
    c = dict(table=f["table"], lens=f["lens"], refs=f["refs"], max_moves=3)
    for over in (dict(src=z(4, dtype=i32)), dict(dst=z(2, dtype=i32)), dict(count=z(1)), dict(lens=z(1, dtype=i32)),
                 dict(table_out=z(2, 128))):
        with pytest.raises(ValueError):
            mla.pages_compact(**{**c, **over})
    k = dict(kv=z(128, 576), src=z(2, dtype=i32), dst=z(2, dtype=i32))
    for over in (dict(kv=z(128, 500)), dict(kv=z(128, 576, dtype=u8), kv_scale=z(4, dtype=f32)), dict(dst=z(3, dtype=i32)),
                 dict(tokens=z(1, dtype=i32)), dict(count=z(1)), dict(src=z(2))):
        with pytest.raises(ValueError):
            mla.kv_copy(**{**k, **over})


def _z(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


CALLS = {
    "prefill": lambda: mla.prefill(_z(5, 2, 128), _z(5, 2, 64), _z(7, 2, 128), _z(7, 64), _z(7, 2, 128), _z(2, dtype=i32),
                                   _z(2, dtype=i32), _z(1, 8, dtype=i32), 0.07),
    "beam_select": lambda: mla.beam_select(_z(2, 3, 50), _z(2, 3, dtype=f32), 4),
    "pages_fork": lambda: mla.pages_fork(_z(2, 128, dtype=i32), _z(2, dtype=i32), _z(9, dtype=i32), _z(1, dtype=i32)),
    "pages_compact": lambda: mla.pages_compact(_z(2, 128, dtype=i32), _z(2, dtype=i32), _z(9, dtype=i32)),
    "kv_copy": lambda: mla.kv_copy(_z(128, 576), _z(2, dtype=i32), _z(2, dtype=i32)),
}


@pytest.mark.parametrize("name", CALLS)
def test_launches_on_the_tensors_device(name, monkeypatch):
    inside, seen = [], []

    @contextlib.contextmanager
    def on(t):
        inside.append(t.device)
        yield
        inside.pop()

    class Library:
        def __getattr__(self, fn):
            return lambda *args: seen.append(list(inside)) or 0

    monkeypatch.setattr(mla, "_on", on)
    monkeypatch.setattr(mla, "_stream", lambda stream: 0)
    monkeypatch.setattr(mla, "library", lambda: Library())
    CALLS[name]()
    assert seen == [[torch.device("cpu")]]


def test_plan_covers_every_block_once():
    r = random.Random(3)
    for _ in range(60):
        N, H = r.randint(0, 12), r.choice([1, 5, 16, 96])
        lq = [r.choice([0, 1, 127, 128, 129, 511, 512, 513, r.randint(1, 5000)]) for _ in range(N)]
        lk = [r.choice([q, q + r.randint(0, 30000), max(0, q - r.randint(0, 200))]) for q in lq]
        pre = [r.randint(0, k + 5) for k in lk] if r.random() < 0.5 else None
        for ctas in (0, 1, 2):
            work, parts = mla.plan_prefill(lq, lk, H, prefix=pre, causal=r.random() < 0.8, ctas=ctas,
                                           num_sms=r.choice([1, 20, 152]))
            one = work.reshape(len(work), -1, 8)
            assert (one == one[:, :1]).all()                    # a pair's CTAs have the same entry
            work = one[:, 0]
            block = 128 if one.shape[1] == 1 else 512
            assert ctas in (0, one.shape[1]) and (work[:, 7] == block).all()
            seen, slots = {}, []
            for i, (n, b, part, of, slot, first, count, _) in enumerate(work.tolist()):
                assert 0 <= b < -(-lq[n] // block) and 0 <= part < of <= mla.PREFILL_MAX_PARTS
                assert first <= i < first + count and (work[first:first + count, 0] == n).all()
                seen.setdefault((n, b), []).append(part)
                assert (slot >= 0) == (of > 1)
                if of > 1:
                    assert slot % (block // 128) == 0
                    if part == 0:
                        slots += range(slot, slot + of * block // 128)
            assert sorted(seen) == [(n, b) for n in range(N) for b in range(-(-lq[n] // block))]
            assert all(p == list(range(len(p))) for p in seen.values())
            assert sorted(slots) == list(range(len(slots))) and parts == -(-len(slots) // 2)


def test_plan_refuses():
    for args in (([-1], [1], 1), ([1], [-1], 1), ([1], [1], 0)):
        with pytest.raises(mla.MlaError):
            mla.plan_prefill(*args)
    with pytest.raises(mla.MlaError):
        mla.plan_prefill([1], [1], 1, ctas=3)
    with pytest.raises(mla.MlaError):
        mla.plan_prefill([1], [1], 1, num_sms=-1)
    with pytest.raises(ValueError):
        mla.plan_prefill([1], [1, 2], 1)
    with pytest.raises(ValueError):
        mla.plan_prefill([1], [1], 1, prefix=[1, 2])
    n, c, parts = ctypes.c_int64(), ctypes.c_int(), ctypes.c_int()
    lens = (ctypes.c_int * 1)(1000)
    out = np.zeros(4, np.int32)
    assert mla.library().mla_plan_prefill(lens, lens, None, 1, 1, 1, 0, 0, out.ctypes.data, 4, ctypes.byref(n), ctypes.byref(c),
                                          ctypes.byref(parts)) == ARG
    assert mla.library().mla_plan_prefill(lens, lens, None, 1, 1, 1, 0, 0, out.ctypes.data, 4, None, ctypes.byref(c),
                                          ctypes.byref(parts)) == ARG
    assert not out.any()
