"""GPU parity of the page table's operators (mla_pages_fork, mla_pages_compact,
mla_kv_copy) with a plain Python model; everything is whole numbers or bytes, so
every comparison is exact."""
import random

import numpy as np
import pytest
import torch

import mla_latent_decode_gb300 as mla
from mla_latent_decode_gb300 import build
from pages_ref import PAGE, compact, counts, fork, pages_of, table_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


def _dev(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _random_rows(r, R, pages, longest, shared):
    """Rows with random lengths; some share the first pages of the row before."""
    names = list(range(1, pages))
    r.shuffle(names)
    rows, lens, at = [], [], 0
    for i in range(R):
        n = r.choice([0, 1, 63, 64, 65, r.randint(0, longest)])
        n = min(n, longest)
        k = 0
        if i and r.random() < shared:
            k = r.randint(0, min(lens[-1], n) // PAGE)
        own = pages_of(n) - k
        rows.append((rows[-1][:k] if k else []) + names[at:at + own])
        lens.append(n)
        at += own
    assert at < pages
    return rows, lens


def _fork(rows, lens, refs, parents, keep, grow, stride, out_stride=None, status=0):
    R = len(rows)
    table = _dev(table_of(rows, stride)).reshape(R, stride)
    d_refs, free = _dev(refs), _dev([int((refs[1:] == 0).sum())])
    out = torch.full((R, out_stride or stride), -5, dtype=torch.int32, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = table.clone()
    t, n, c = mla.pages_fork(table, _dev(lens), d_refs, free, parents=None if parents is None else _dev(parents),
                             keep=None if keep is None else _dev(keep), grow=None if grow is None else _dev(grow),
                             table_out=out, status=word)
    assert int(word.item()) == status
    assert torch.equal(table, before)
    return t.cpu().numpy(), n.cpu().numpy(), c.cpu().numpy(), d_refs.cpu().numpy(), int(free.item())


def _check_fork(rows, lens, refs, parents, keep, grow, stride, out_stride=None):
    R = len(rows)
    t, n, c, got_refs, free = _fork(rows, lens, refs, parents, keep, grow, stride, out_stride)
    new, new_lens, new_refs, copies = fork(rows, lens, refs, parents or list(range(R)), keep or [1 << 30] * R,
                                           grow or [0] * R)
    want = np.full((R, out_stride or stride), -5, np.int32)
    for i, row in enumerate(new):
        e = table_of([row], max(len(row), 1) * PAGE)[0][:min(len(row) * PAGE, want.shape[1])]
        want[i, :len(e)] = e
    assert np.array_equal(n, new_lens)
    assert np.array_equal(c, copies)
    assert np.array_equal(got_refs, new_refs)
    assert np.array_equal(t, want)
    assert free == int((new_refs[1:] == 0).sum())
    return new, new_lens, new_refs


@pytest.mark.parametrize("seed", range(8))
@pytest.mark.parametrize("R,longest", [(1, 200), (3, 130), (17, 700), (130, 900)])
def test_fork_matches_the_model(R, longest, seed):
    r = random.Random(1000 * R + seed)
    pages = R * (2 * pages_of(longest) + 4) + 40
    rows, lens = _random_rows(r, R, pages, longest, 0.5)
    refs = counts(rows, pages)
    for p in r.sample([q for row in rows for q in row] or [1], 1):
        refs[p] += r.randint(0, 1)                      # a holder outside the table
    refs[0] = 1
    stride = PAGE * (pages_of(longest) + 2) + r.choice([0, 1, 4, 30])
    for _ in range(3):
        parents = [r.choice([-1, i, r.randrange(R), r.randrange(R)]) for i in range(R)]
        keep = [r.choice([1 << 30, 0, r.randint(0, longest)]) for _ in range(R)]
        grow = [r.choice([0, 1, 5, 64, 100]) for _ in range(R)]
        grow = [min(g, stride - min(k, lens[p] if p >= 0 else 0)) for g, k, p in zip(grow, keep, parents)]
        expect = fork(rows, lens, refs, parents, keep, grow)
        if expect is None:
            break
        rows, lens, refs = _check_fork(rows, lens, refs, parents, keep, grow, stride)
        lens = [int(n) for n in lens]


def test_fork_with_defaults_and_other_strides():
    rows, lens = [[3, 4], [5]], [100, 64]
    refs = counts(rows, 20)
    _check_fork(rows, lens, refs, None, None, None, 256)
    _check_fork(rows, lens, refs, None, None, [1, 1], 256, 200)
    _check_fork(rows, lens, refs, [1, 0], None, [0, 3], 129, 301)
    _check_fork(rows, lens, refs, [0, 0], None, [1, 1], 256)


def test_prompt_for_many_beams_and_a_long_row():
    rows, lens = [list(range(1, 1001))] + [[]] * 63, [64000 - 30] + [0] * 63
    refs = counts(rows, 70000)
    refs[0] = 1
    _check_fork(rows, lens, refs, [0] * 64, None, [700] * 64, PAGE * 1012)
    _check_fork(rows, lens, refs, [-1] * 64, None, [64000] + [20] * 63, PAGE * 1012)


def test_more_rows_than_threads():
    R = 1500
    rows, lens = [[1 + i] for i in range(R)], [1 + i % 64 for i in range(R)]
    refs = counts(rows, 2 * R + 100)
    r = random.Random(3)
    _check_fork(rows, lens, refs, [r.randrange(R) for _ in range(R)], None, [r.randint(0, 60) for _ in range(R)], 128)


def test_free_pages_far_up_the_pool():
    """More pages in use than one round of the search looks at."""
    pages = 200000
    refs = np.ones(pages, np.int32)
    refs[[70000, 131071, 131072, 199990, 199999]] = 0
    rows = [[10, 11], [12]]
    _check_fork(rows, [128, 10], refs, [0, 0], None, [100, 60], 512)
    t, n, c, got, free = _fork(rows, [128, 10], refs, [0, 0], None, [200, 200], 512, status=mla.STATUS_NO_PAGES)
    assert np.array_equal(got, refs) and free == 5 and not n.any() and (c[:2] == -1).all() and not c[2].any()


@pytest.mark.parametrize("what,status", [
    (dict(parents=[0, 2]), "BAD_PARENT"), (dict(parents=[-2, 0]), "BAD_PARENT"), (dict(keep=[-1, 5]), "BAD_LENGTH"),
    (dict(grow=[0, -1]), "BAD_LENGTH"), (dict(grow=[0, 193]), "BAD_LENGTH"), (dict(lens=[100, 257]), "BAD_LENGTH"),
    (dict(lens=[-1, 64]), "BAD_LENGTH"), (dict(rows=[[3, 50], [5]]), "BAD_SLOT"), (dict(rows=[[3, 0], [5]]), "BAD_SLOT")])
def test_fork_refuses_as_a_whole(what, status):
    a = dict(rows=[[3, 4], [5]], lens=[100, 64], parents=[0, 1], keep=None, grow=[1, 1])
    a.update(what)
    refs = counts([[3, 4], [5]], 20)
    t, n, c, got, free = _fork(a["rows"], a["lens"], refs, a["parents"], a["keep"], a["grow"], 256,
                               status=getattr(mla, "STATUS_" + status))
    assert np.array_equal(got, refs) and free == int((refs[1:] == 0).sum())
    assert not n.any() and (c[:2] == -1).all() and not c[2].any()


def test_full_pages_outside_the_pool_are_reported():
    refs = counts([[3], [5]], 20)
    _, _, _, got, _ = _fork([[3], [50]], [64, 64], refs, [0, 0], None, [0, 0], 128, status=mla.STATUS_BAD_SLOT)
    assert got[3] == 2 and got[5] == 1


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("R,pages", [(1, 30), (5, 300), (60, 3000), (9, 100000)])
def test_compact_matches_the_model(R, pages, seed):
    r = random.Random(seed * 77 + R)
    names = r.sample(range(1, pages), min(pages // 2, 2500))
    rows, lens, at = [], [], 0
    for i in range(R):
        n = r.randint(0, len(names) * PAGE // R)
        rows.append(names[at:at + pages_of(n)])
        lens.append(n)
        at += pages_of(n)
    if R > 2:
        rows[2], lens[2] = list(rows[1]), lens[1]       # shared pages
    refs = counts(rows, pages)
    refs[0] = 1
    stride = PAGE * (max(len(row) for row in rows) + 1) + r.choice([0, 3])
    for limit in (pages, r.randint(0, 40)):
        new, new_refs, src, dst = compact(rows, refs, limit)
        for in_place in (False, True):
            table = _dev(table_of(rows, stride)).reshape(R, stride)
            before = table.clone()
            d_refs = _dev(refs)
            word = torch.zeros(1, dtype=torch.int32, device="cuda")
            out = table if in_place else torch.full_like(table, -7)
            t, s, d, count = mla.pages_compact(table, _dev(lens), d_refs, max_moves=limit, table_out=out, status=word)
            m = len(src)
            assert int(word.item()) == 0 and int(count.item()) == m
            assert s[:m].tolist() == src and d[:m].tolist() == dst
            assert bool((s[m:] == -1).all()) and bool((d[m:] == -1).all())
            assert np.array_equal(d_refs.cpu().numpy(), new_refs)
            assert np.array_equal(t.cpu().numpy(), table_of(new, stride))
            assert in_place or torch.equal(table, before)


def test_compact_without_rows_and_bad_lengths():
    refs = _dev([1, 0, 0, 2, 0, 1])
    t, s, d, count = mla.pages_compact(torch.zeros((0, 64), dtype=torch.int32, device="cuda"), _dev([]), refs)
    assert refs.tolist() == [1, 1, 2, 0, 0, 0] and s.tolist() == [5, 3, -1, -1, -1, -1] and count.item() == 2
    assert d.tolist() == [1, 2, -1, -1, -1, -1]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    refs = _dev([1, 0, 1, 1])
    table = _dev(table_of([[2], [3]], 64))
    t, *_ = mla.pages_compact(table, _dev([65, 64]), refs, table_out=table.clone(), status=word)
    assert word.item() == mla.STATUS_BAD_LENGTH
    assert np.array_equal(t.cpu().numpy(), table_of([[2], [1]], 64))


def _pool(kind, pages):
    g = torch.Generator().manual_seed(pages)
    if kind == "bf16":
        return torch.randn((pages * PAGE, 576), generator=g).bfloat16().cuda(), None
    raw = torch.randint(0, 256, (pages * PAGE, 576 if kind == "fp8" else 352), generator=g, dtype=torch.uint8).cuda()
    return raw, torch.rand(pages * PAGE if kind == "fp8" else 1, generator=g).cuda()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_copy(kind):
    pool, scale = _pool(kind, 40)
    raw, sc = pool.view(torch.uint8).clone(), None if scale is None else scale.clone()
    src, dst, tokens = [1, 5, -1, 7, 2, 9, 11, 12], [20, 21, 22, -1, 23, 9, 24, 25], [64, 1, 64, 64, 0, 64, 63, 99]
    mla.kv_copy(pool, _dev(src), _dev(dst), scale, tokens=_dev(tokens))
    for s, d, n in zip(src, dst, tokens):
        n = min(n, 64)
        if s < 0 or d < 0 or s == d:
            continue
        raw[d * 64:d * 64 + n] = raw[s * 64:s * 64 + n]
        if kind == "fp8":
            sc[d * 64:d * 64 + n] = sc[s * 64:s * 64 + n]
    assert torch.equal(pool.view(torch.uint8), raw)
    assert scale is None or torch.equal(scale, sc)


def test_copy_by_count_and_outside_the_pool():
    pool, _ = _pool("bf16", 12)
    want = pool.clone()
    want[9 * 64:10 * 64] = want[64:128]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.kv_copy(pool, _dev([1, 2, 3]), _dev([9, 10, 11]), count=_dev([1]), status=word)
    assert torch.equal(pool, want) and word.item() == 0
    mla.kv_copy(pool, _dev([1, 2]), _dev([9, 10]), count=_dev([-3]), status=word)
    mla.kv_copy(pool, _dev([12, 1]), _dev([1, 12]), status=word)
    assert torch.equal(pool, want) and word.item() == mla.STATUS_BAD_SLOT
    mla.kv_copy(pool, _dev([]), _dev([]), status=word)


def test_copy_past_32_bit_offsets():
    pages = (1 << 32) // (64 * 1152) + 40
    pool = torch.zeros((pages * PAGE, 576), dtype=torch.bfloat16, device="cuda")
    x = torch.randn((PAGE, 576), device="cuda").bfloat16()
    pool[64:128] = x
    mla.kv_copy(pool, _dev([1]), _dev([pages - 1]))
    mla.kv_copy(pool, _dev([pages - 1]), _dev([2]))
    assert torch.equal(pool[-64:], x) and torch.equal(pool[128:192], x) and not bool(pool[192:-64].any())


def test_captured_fork_and_copy():
    rows, lens = [[3, 4], [5, 6]], [100, 90]
    refs = counts(rows, 64)
    table, d_lens = _dev(table_of(rows, 256)), _dev(lens)
    pool, _ = _pool("bf16", 64)
    start, free0 = _dev(refs), _dev([int((refs[1:] == 0).sum())])
    d_refs, free, parents, grow = start.clone(), free0.clone(), _dev([1, 1]), _dev([1, 1])
    out = torch.zeros_like(table)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d_refs.copy_(start)
        free.copy_(free0)
        t, n, c = mla.pages_fork(table, d_lens, d_refs, free, parents=parents, grow=grow, table_out=out)
        mla.kv_copy(pool, c[0], c[1], tokens=c[2])
    new, new_lens, new_refs, copies = fork(rows, lens, refs, [1, 1], [999] * 2, [1, 1])
    want = pool.clone()
    s, d, k = copies[:, 1]
    want[d * 64:d * 64 + k] = want[s * 64:s * 64 + k]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert n.tolist() == new_lens and np.array_equal(c.cpu().numpy(), copies)
        assert np.array_equal(d_refs.cpu().numpy(), new_refs) and torch.equal(pool, want)
