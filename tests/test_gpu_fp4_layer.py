"""The operators together: the example's sublayer over a 4-bit and a bf16 cache,
chunked prefill against single tokens, and a captured graph replayed.
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))

import fp4_layer  # noqa: E402
import mla_latent_decode_gb300 as mla  # noqa: E402
from mla_latent_decode_gb300 import build  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mla.library()


def test_sublayer_over_four_bits_stays_near_bf16():
    """E2M1 with a scale per 16 values keeps Gaussian latents to about 10% (a
    step of 1/2 to 2 of 6 times the block's largest / 6); attention averages
    many of them, so the outputs differ by at most that order."""
    four, full = fp4_layer.run(fp4=True).float(), fp4_layer.run(fp4=False).float()
    rel = float((four - full).norm() / full.norm())
    assert 0.0 < rel < 0.25


@pytest.mark.parametrize("H", [16, 96])
def test_prefill_chunks_equal_single_tokens(H):
    """The same rows whether a prompt is appended and attended in chunks of 50
    (more query rows, another kernel) or one token at a time."""
    a = fp4_layer.run(B=1, H=H, hidden=256, prompt=100, steps=0)
    b = fp4_layer.run(B=1, H=H, hidden=256, prompt=0, steps=100)
    rel = float((a.float() - b.float()).norm() / b.float().norm())
    assert rel < 0.02  # bf16 projections of differently batched products


def test_captured_step_replays():
    """Norm, append, decode and combine in one CUDA graph, replayed on new inputs."""
    B, H, L, d = 3, 16, 300, 512
    gen = torch.Generator(device="cuda").manual_seed(1)

    def randn(*s):
        return torch.randn(s, generator=gen, device="cuda").bfloat16()

    cache = fp4_layer.Cache(B, 512, True)
    cache.grow(L - 1)
    prior = randn(B * (L - 1), 576)
    table = fp4_layer.rotation_table(512)
    slots0 = cache.table[:, :L - 1].reshape(-1).contiguous()
    pos0 = torch.arange(L - 1, device="cuda", dtype=torch.int32).repeat(B)
    mla.kv_append(prior, slots0, pos0, table, cache.kv, cache.scale)
    slots, pos = cache.grow(1)
    x, w, res = randn(B, d), randn(d), randn(B, d)
    rows, q_nope, q_rope = randn(B, 576), randn(B, 1, H, 512), randn(B, H, 64)
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    out8 = torch.empty((B, d), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((B, 1), device="cuda")

    def once():
        mla.add_rms_norm(x, w, res, residual_out=torch.empty_like(res), out8=out8, scales=scales)
        q = mla.kv_append(rows, slots, pos, table, cache.kv, cache.scale, q_rope=q_rope)
        O, LSE = mla.decode_partial(q_nope, q.view(B, 1, H, 64), cache.kv, cache.scale, cache.table,
                                    lens, None, 2, fp4_layer.SM_SCALE)
        return mla.lse_combine(O, LSE)

    once()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out, lse = once()
    torch.cuda.current_stream().wait_stream(side)
    for k in range(2):
        rows.copy_(randn(B, 576))
        q_rope.copy_(randn(B, H, 64))
        x.copy_(randn(B, d))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone(), out8.view(torch.uint8).clone(), scales.clone()
        want_out, want_lse = once()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want_out) and torch.equal(got[1], want_lse)
        assert torch.equal(got[2], out8.view(torch.uint8)) and torch.equal(got[3], scales)
