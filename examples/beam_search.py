"""Beam search of a one-layer model over a paged latent cache, step by step as a
serving loop runs it:

    prompts:  append to the cache -> attention within the packed prompts -> logits
    a step:   selection over beams and vocabulary -> page table of the chosen
              beams -> copy of the pages that two of them would write -> append ->
              absorbed decode -> combine -> output projection -> logits

with random weights.  Beams of a request share its prompt's pages; a beam that
goes on alone keeps its pages, one that goes on twice has only its last page copied.
At the end the first request leaves and the pool is compacted.

    python examples/beam_search.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import mla_latent_decode_gb300 as mla  # noqa: E402
from fp4_layer import Layer, QK, ROPE, SM_SCALE, rotation_table  # noqa: E402

PAGE = mla.PAGE_SIZE


class Model(Layer):
    """One attention sublayer between an embedding and an output matrix."""

    def __init__(self, hidden, H, vocab, seed=0, device="cuda"):
        super().__init__(hidden, H, seed, device)
        g = torch.Generator(device=device).manual_seed(seed + 100)
        self.embed = torch.randn((vocab, hidden), generator=g, device=device).bfloat16()
        self.w_out = (torch.randn((H * QK, vocab), generator=g, device=device) * (6 / (H * QK) ** 0.5)).bfloat16()


class Search:
    """The beams of B requests, W rows each, over one layer's pool."""

    def __init__(self, model, prompts, W, steps, kv="bf16", device="cuda"):
        self.model, self.W, self.B, self.kv_type = model, W, len(prompts), kv
        self.dev, R = device, len(prompts) * W
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        longest = max(len(p) for p in prompts) + steps
        pages = 2 + sum(-(-len(p) // PAGE) for p in prompts) + R * (2 + -(-steps // PAGE))
        width = {"bf16": mla.ROW_DIM, "fp8_e4m3": mla.ROW_DIM, "fp4_e2m1": mla.FP4_ROW_BYTES}[kv]
        self.pool = torch.zeros((pages * PAGE, width), device=device,
                                dtype=torch.bfloat16 if kv == "bf16" else torch.uint8)
        self.scale = {"bf16": None, "fp8_e4m3": torch.zeros(pages * PAGE, device=device),
                      "fp4_e2m1": torch.full((1,), 0.0625, device=device)}[kv]
        self.rotation = rotation_table(longest)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=device)
        self.free = torch.full((1,), pages - 1, dtype=torch.int32, device=device)
        stride = (-(-longest // PAGE) + 1) * PAGE
        # two tables, used in turn: a step reads the one and writes the other
        self.table = torch.zeros((R, stride), dtype=torch.int32, device=device)
        self.other = torch.zeros_like(self.table)
        self.lens = torch.zeros(R, dtype=torch.int32, device=device)
        self.host_lens = [0] * R
        self.sequences = [[] for _ in range(R)]
        self.done = torch.zeros((self.B, W), dtype=torch.bool, device=device)
        self._prompts(prompts)

    def _ints(self, x):
        return torch.tensor(x, dtype=torch.int32, device=self.dev)

    def _fork(self, parents, grow):
        """Rows go on as their parents' (None: their own), with room for `grow` tokens."""
        table, lens, copies = mla.pages_fork(self.table, self.lens, self.refs, self.free, parents=parents, grow=grow,
                                             table_out=self.other, status=self.status)
        mla.kv_copy(self.pool, copies[0], copies[1], self.scale, tokens=copies[2], status=self.status)
        self.table, self.other, self.lens = table, self.table, lens

    def _project(self, tokens, slots, positions):
        """Append the tokens; returns their queries, rotated."""
        h = self.model.embed[tokens]
        q = (h @ self.model.w_q).view(len(tokens), self.model.H, QK + ROPE)
        q_rope = mla.kv_append(h @ self.model.w_kv, slots, positions, self.rotation, self.pool, self.scale,
                               norm_weight=self.model.kv_norm, q_rope=q[..., QK:], status=self.status)
        return q[..., :QK], q_rope

    def _prompts(self, prompts):
        """A request's first row takes the prompt; its other rows start at the first step."""
        B, W, m, H = self.B, self.W, self.model, self.model.H
        lens = [len(p) for p in prompts]
        self._fork(self._ints([-1] * (B * W)), self._ints([lens[r // W] if r % W == 0 else 0 for r in range(B * W)]))
        slots = torch.cat([self.table[b * W, :n] for b, n in enumerate(lens)])
        positions = self._ints([i for n in lens for i in range(n)])
        q_nope, q_rope = self._project(torch.tensor(sum(prompts, []), device=self.dev), slots, positions)
        rows = mla.kv_read(self.pool, slots, self.scale, status=self.status)
        latent = rows[:, :512]
        k_nope = torch.einsum("td,hkd->thk", latent, m.w_kc).contiguous()
        v = torch.einsum("td,hdk->thk", latent, m.w_vc).contiguous()
        work, parts = mla.plan_prefill(lens, lens, H)
        cu = self._ints([sum(lens[:b]) for b in range(B + 1)])
        out, _ = mla.prefill(q_nope, q_rope, k_nope, rows[:, 512:], v, cu, cu, torch.from_numpy(work).to(self.dev),
                             SM_SCALE, num_parts=parts, status=self.status)
        self.logits = (out[(cu[1:] - 1).long()].view(B, -1) @ m.w_out)[:, None]      # [B, 1, vocab]
        self.scores = torch.zeros((B, 1), device=self.dev)
        self.first = True
        for b, p in enumerate(prompts):
            self.sequences[b * W] = list(p)
            self.host_lens[b * W] = len(p)

    def step(self, end_token):
        """Choose every request's beams and run them; returns their tokens [B, W]."""
        B, W, m, H = self.B, self.W, self.model, self.model.H
        self.scores, parents, tokens = mla.beam_select(self.logits, self.scores, W, end_token=end_token,
                                                       finished=None if self.first else self.done, status=self.status)
        if self.first:
            parents, self.first = parents * W, False  # (one row a request so far)
        else:
            self.done = self.done.view(-1)[parents.long()]
        self.done = self.done | (tokens == end_token)
        rows = parents.view(-1)
        self._fork(rows, self._ints([1] * (B * W)))
        at = rows.tolist()  # the host follows, for the plan and the texts
        self.sequences = [self.sequences[p] + [t] for p, t in zip(at, tokens.view(-1).tolist())]
        self.host_lens = [self.host_lens[p] + 1 for p in at]
        self.forward(tokens.view(-1))
        return tokens

    def forward(self, tokens):
        """Append one token to every row and leave the next logits."""
        B, W, m, H = self.B, self.W, self.model, self.model.H
        R = B * W
        positions = self.lens - 1
        slots = self.table.gather(1, positions.long()[:, None]).view(-1)
        q_nope, q_rope = self._project(tokens, slots, positions)
        q = mla.absorb_q(q_nope.reshape(R, 1, H, QK).contiguous(), m.w_kc, status=self.status)
        S, pages, work, _ = mla.plan_sched(R, 1, H, self.host_lens, kv_dtype=self.kv_type)
        parts, lse = mla.decode_partial(q, q_rope.view(R, 1, H, ROPE), self.pool, self.scale, self.table, self.lens,
                                        None, S, SM_SCALE, status=self.status,
                                        split_pages=torch.from_numpy(pages).to(self.dev),
                                        work=torch.from_numpy(work).to(self.dev))
        o, _ = mla.lse_combine(parts, lse)
        o = mla.project_out(o, m.w_vc, status=self.status)
        self.logits = (o.view(R, H * QK) @ m.w_out).view(B, W, -1)

    def leave(self, request):
        """A request's rows give their pages back, and the pool closes its holes."""
        R = self.B * self.W
        gone = [r // self.W == request for r in range(R)]
        self._fork(self._ints([-1 if g else r for r, g in enumerate(gone)]), None)
        self.host_lens = [0 if g else n for n, g in zip(self.host_lens, gone)]
        _, src, dst, count = mla.pages_compact(self.table, self.lens, self.refs, table_out=self.table, status=self.status)
        mla.kv_copy(self.pool, src, dst, self.scale, count=count, status=self.status)


def run(lengths=(70, 200), W=4, steps=20, H=16, hidden=256, vocab=1000, kv="bf16", seed=0, check=None):
    """Search; `check(search)` is called with the rows' sequences and logits after every step."""
    model = Model(hidden, H, vocab, seed)
    g = torch.Generator().manual_seed(seed + 1)
    prompts = [torch.randint(3, vocab, (n,), generator=g).tolist() for n in lengths]
    search = Search(model, prompts, W, steps + 1, kv)
    for _ in range(steps):
        search.step(end_token=2)
        if check is not None:
            check(search)
    search.leave(0)
    if int(search.status.item()):
        raise RuntimeError(f"device status {int(search.status.item())}")
    return search


def main():
    search = run()
    live = int((search.refs[1:] > 0).sum())
    print(f"{search.B} requests x {search.W} beams; best scores {search.scores[:, 0].tolist()}; "
          f"{live} pages hold the second request's beams, the highest {int(search.refs.nonzero().max())}")


if __name__ == "__main__":
    main()
