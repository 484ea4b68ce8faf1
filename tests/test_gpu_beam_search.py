"""The operators of beam search together: the example's loop (prompts, selection,
page tables, copies, decode) against the same model on every beam's own tokens,
dense and in float64, after every step.

Tolerance: what the cache path rounds to bf16 on the way to a logit are the latent
row, the query, the absorbed query (or k and v in the prompt), the probabilities,
the output and its projection, each by at most 2^-8 of itself, and the embedding's
products that the dense form shares.  Scores are below about 4, so rounded operands
move a probability by at most 4 x 3 x 2^-8, 5%; with the output's own roundings
the logits differ by at most 8% of their norm.  An E4M3 row adds 2^-4 and a 4-bit
block's values up to a sixth (half a step of 1 at 3), in each of its two uses.  A row that
read another beam's cache, or lost a page, differs by its own norm.
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))

import beam_search  # noqa: E402
import mla_latent_decode_gb300 as mla  # noqa: E402
from fp4_layer import QK, ROPE, SM_SCALE  # noqa: E402
from mla_latent_decode_gb300 import build  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


def _rotate(x, rotation):
    """x [T, ..., 64] interleaved pairs, rotation [T, 64]: cosines, sines."""
    cos, sin = rotation[:, :32], rotation[:, 32:]
    while cos.dim() < x.dim():
        cos, sin = cos[:, None], sin[:, None]
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _dense_logits(model, tokens, rotation):
    """The last token's logits in float64."""
    T, H = len(tokens), model.H
    h = model.embed[torch.tensor(tokens, device="cuda")].double()
    q = (h @ model.w_q.double()).view(T, H, QK + ROPE)
    rows = h @ model.w_kv.double()
    latent = rows[:, :512] * torch.rsqrt(rows[:, :512].square().mean(-1, keepdim=True) + 1e-6)
    rot = rotation[:T].double()
    k_rope, q_rope = _rotate(rows[:, 512:], rot), _rotate(q[..., QK:], rot)
    k = torch.einsum("td,hkd->thk", latent, model.w_kc.double())
    v = torch.einsum("td,hdk->thk", latent, model.w_vc.double())
    s = SM_SCALE * (torch.einsum("hk,thk->ht", q[-1, :, :QK], k) + q_rope[-1] @ k_rope.T)
    o = torch.einsum("ht,thk->hk", torch.softmax(s, -1), v)
    return o.reshape(-1) @ model.w_out.double()


@pytest.mark.parametrize("kv,tol", [("bf16", 0.08), ("fp8_e4m3", 0.21), ("fp4_e2m1", 0.42)])
def test_every_beam_reads_its_own_tokens(kv, tol):
    worst, orders = 0.0, set()

    def check(search):
        nonlocal worst
        got = search.logits.reshape(search.B * search.W, -1).double()
        for r, seq in enumerate(search.sequences):
            want = _dense_logits(search.model, seq, search.rotation)
            worst = max(worst, float((got[r] - want).norm() / want.norm()))
        orders.add(tuple(map(tuple, search.sequences[:search.W])))

    search = beam_search.run(steps=9, kv=kv, check=check)
    assert worst < tol, worst
    assert len(orders) == 9
    # the pool: every page is counted once per row that holds it, and none is lost
    rows = [search.table[r, :n:64].cpu() // 64 for r, n in enumerate(search.host_lens)]
    held = torch.zeros_like(search.refs.cpu())
    for row in rows:
        held[row.long()] += 1
    assert torch.equal(held[1:], search.refs.cpu()[1:])
    assert int(search.free.item()) == int((search.refs[1:] == 0).sum())
    live = int((held[1:] > 0).sum())
    assert int(search.refs.nonzero().max()) == live          # compacted
    # and the beams that stayed still read the same
    tokens = torch.tensor([s[-1] for s in search.sequences], device="cuda")
    search._fork(None, torch.tensor([0] * search.W + [1] * search.W, dtype=torch.int32, device="cuda"))
    search.host_lens = [n + (n > 0) for n in search.host_lens]
    slots = search.table.gather(1, (search.lens - 1).clamp(min=0).long()[:, None])
    assert bool((slots[search.W:] >= 64).all())
    search.lens[:search.W] = 1                                # (any page: their logits are not looked at)
    search.host_lens[:search.W] = [1] * search.W
    search.table[:search.W, :64] = torch.arange(64, dtype=torch.int32, device="cuda")
    search.forward(tokens)
    got = search.logits[1].double()
    for w in range(search.W):
        want = _dense_logits(search.model, search.sequences[search.W + w] + [int(tokens[search.W + w])], search.rotation)
        assert float((got[w] - want).norm() / want.norm()) < tol


def test_beams_come_in_order_and_differ():
    seen = []
    search = beam_search.run(steps=6, check=lambda s: seen.append((s.scores.clone(), [list(x) for x in s.sequences])))
    for scores, sequences in seen:
        flat = scores.view(-1).tolist()
        for b in range(2):
            assert flat[b * 4:b * 4 + 4] == sorted(flat[b * 4:b * 4 + 4], reverse=True)
            assert len(set(map(tuple, sequences[b * 4:b * 4 + 4]))) == 4
    assert search.scores.isfinite().all()
