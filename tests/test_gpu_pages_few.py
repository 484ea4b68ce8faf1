"""The page table's fork (mla_pages_fork) where the count of free pages says more than the
pool has: the status is set, every row's length covers pages that it holds, and nothing is
to be copied for a row that got no page."""
import random

import numpy as np
import pytest
import torch

import mla_latent_decode_gb300 as mla
from mla_latent_decode_gb300 import build
from pages_ref import PAGE, counts, pages_of, table_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


def _dev(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("R,spare", [(2, 0), (5, 3), (40, 20), (700, 100)])
def test_rows_hold_what_they_got(R, spare, seed):
    r = random.Random(seed * 100 + R)
    rows, lens, at = [], [], 1
    for _ in range(R):
        n = r.choice([10, 64, 100, 200])
        rows.append(list(range(at, at + pages_of(n))))
        lens.append(n)
        at += pages_of(n)
    pages = at + spare
    refs = counts(rows, pages)
    refs[0] = 1
    parents = [r.randrange(R) for _ in range(R)]
    grow = [r.choice([0, 1, 70, 150]) for _ in range(R)]
    stride = 8 * PAGE
    said = 100 * R
    d_refs, free = _dev(refs), _dev([said])
    out = torch.full((R, stride), -5, dtype=torch.int32, device="cuda")
    copies = torch.full((3, R), 12345, dtype=torch.int32, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, n, c = mla.pages_fork(_dev(table_of(rows, stride)), _dev(lens), d_refs, free, parents=_dev(parents), grow=_dev(grow),
                             table_out=out, copies=copies, status=word)
    t, n, c, after = t.cpu().numpy(), n.cpu().numpy(), c.cpu().numpy(), d_refs.cpu().numpy()
    kept = [lens[p] for p in parents]
    claims = {}
    for i, p in enumerate(parents):
        claims.setdefault(p, i)                              # all take all of the row: the first is the heir
    need = [pages_of(k + g) - k // PAGE - (k % PAGE > 0 and claims[p] == i)
            for i, (k, g, p) in enumerate(zip(kept, grow, parents))]
    short = sum(need) > spare
    assert int(word.item()) == (mla.STATUS_NO_PAGES if short else 0)
    new = list(range(at, pages))
    held = np.zeros(pages, np.int32)
    for i, (k, g, p) in enumerate(zip(kept, grow, parents)):
        mine = list(rows[p][:k // PAGE])
        got, new = new[:need[i]], new[need[i]:]
        copied = k % PAGE > 0 and claims[p] != i
        if copied and got:
            assert c[:, i].tolist() == [rows[p][k // PAGE], got[0], k % PAGE]
        else:
            assert c[:, i].tolist() == [-1, -1, 0], (i, c[:, i])
        if k % PAGE and not copied:
            mine.append(rows[p][k // PAGE])
        mine += got
        assert n[i] == min(k + g, len(mine) * PAGE)
        full = table_of([mine], max(len(mine), 1) * PAGE)[0][:len(mine) * PAGE]
        assert np.array_equal(t[i, :n[i]], full[:n[i]])
        for q in mine:
            held[q] += 1
    assert np.array_equal(after[1:], held[1:])
    given = min(sum(need), spare)
    freed = int(((refs[1:] > 0) & (after[1:] == 0)).sum())
    assert int(free.item()) == said - given + freed
