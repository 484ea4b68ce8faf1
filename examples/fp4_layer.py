"""One MLA attention sublayer over a 4-bit latent cache, step by step as a
serving loop runs it:

    residual norm (E4M3) -> projections -> append to the cache -> absorbed
    decode over the cache -> combine -> per-head output projection

with random weights and a page table that grows by one page at a time.  The
same steps over a bf16 cache show what holding the cache in 4 bits costs.

    python examples/fp4_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mla_latent_decode_gb300 as mla  # noqa: E402

PAGE, NOPE, ROPE, QK = mla.PAGE_SIZE, 512, 64, 128
SM_SCALE = 192.0 ** -0.5


class Layer:
    """Random weights: hidden -> per-head queries (128 + 64) and the latent row."""

    def __init__(self, hidden, H, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def w(*shape, fan):
            return (torch.randn(shape, generator=g, device=device) / fan ** 0.5).bfloat16()

        self.H = H
        self.norm = torch.ones(hidden, dtype=torch.bfloat16, device=device)
        self.kv_norm = torch.ones(NOPE, dtype=torch.bfloat16, device=device)
        self.w_q = w(hidden, H * (QK + ROPE), fan=hidden)
        self.w_kv = w(hidden, NOPE + ROPE, fan=hidden)
        self.w_kc = w(H, QK, NOPE, fan=QK)
        self.w_vc = w(H, NOPE, QK, fan=NOPE)
        self.w_o = w(H * QK, hidden, fan=H * QK)


class Cache:
    """A paged pool of B requests, bf16 or 4 bits, pages handed out in turn."""

    def __init__(self, B, max_tokens, fp4, device="cuda"):
        self.pages = -(-max_tokens // PAGE)
        slots = (1 + B * self.pages) * PAGE
        self.scale = torch.full((1,), 0.0625, device=device) if fp4 else None
        self.kv = torch.zeros((slots, mla.FP4_ROW_BYTES if fp4 else mla.ROW_DIM), device=device,
                              dtype=torch.uint8 if fp4 else torch.bfloat16)
        # page p of request b is page 1 + p * B + b of the pool
        t = torch.arange(self.pages * PAGE, dtype=torch.int32)
        b = torch.arange(B, dtype=torch.int32)[:, None]
        self.table = ((1 + t // PAGE * B + b) * PAGE + t % PAGE).to(device)
        self.kv_dtype = "fp4_e2m1" if fp4 else "bf16"
        self.length = 0

    def grow(self, q_len):
        """Slots and positions of the next q_len tokens of every request."""
        at = torch.arange(self.length, self.length + q_len, device=self.table.device)
        self.length += q_len
        slots = self.table[:, at].reshape(-1).contiguous()
        return slots, at.to(torch.int32).repeat(self.table.shape[0])


def rotation_table(max_pos, device="cuda"):
    """fp32 [max_pos, 64]: 32 cosines and 32 sines per position, angles in float64."""
    freq = 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64) / ROPE)
    angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


def step(layer, cache, table, x, residual, status):
    """x, residual bf16 [B * q_len, hidden] -> (output of the sublayer, residual)."""
    B, H = cache.table.shape[0], layer.H
    q_len = x.shape[0] // B
    _, x8, scales, residual = mla.add_rms_norm(x, layer.norm, residual.clone(), e4m3=True)
    h = (x8.float() * scales).bfloat16()
    q = (h @ layer.w_q).view(B * q_len, H, QK + ROPE)
    slots, positions = cache.grow(q_len)
    q_rope = mla.kv_append(h @ layer.w_kv, slots, positions, table, cache.kv, cache.scale,
                           norm_weight=layer.kv_norm, q_rope=q[..., QK:], status=status)
    q_nope = mla.absorb_q(q[..., :QK].contiguous().view(B, q_len, H, QK), layer.w_kc, status=status)
    lens = [cache.length] * B
    S, pages, work, _ = mla.plan_sched(B, q_len, H, lens, kv_dtype=cache.kv_dtype)
    dev = x.device
    parts, lse_parts = mla.decode_partial(
        q_nope, q_rope.view(B, q_len, H, ROPE), cache.kv, cache.scale, cache.table,
        torch.tensor(lens, dtype=torch.int32, device=dev), None, S, SM_SCALE, status=status,
        split_pages=torch.from_numpy(pages).to(dev), work=torch.from_numpy(work).to(dev))
    o, _ = mla.lse_combine(parts, lse_parts)
    o = mla.project_out(o, layer.w_vc, status=status)
    return o.view(B * q_len, H * QK) @ layer.w_o, residual


def run(B=2, H=16, hidden=1536, prompt=200, steps=8, seed=0, fp4=True):
    """Prefill `prompt` tokens in chunks, then decode one at a time; the
    sublayer's outputs of every token, bf16 [B, prompt + steps, hidden]."""
    layer, cache = Layer(hidden, H, seed), Cache(B, prompt + steps, fp4)
    table = rotation_table(prompt + steps)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn((B, prompt + steps, hidden), generator=g, device="cuda").bfloat16()
    out, at = [], 0
    while at < prompt + steps:
        n = min(50, prompt - at) if at < prompt else 1
        chunk = x[:, at:at + n].reshape(B * n, hidden)
        y, _ = step(layer, cache, table, chunk, torch.zeros_like(chunk), status)
        out.append(y.view(B, n, hidden))
        at += n
    if int(status.item()):
        raise RuntimeError(f"device status {int(status.item())}")
    return torch.cat(out, 1)


def main():
    four, full = run(fp4=True).float(), run(fp4=False).float()
    rel = float((four - full).norm() / full.norm())
    print(f"4-bit cache against bf16 cache: relative difference {rel:.3f} of the sublayer's output")


if __name__ == "__main__":
    main()
