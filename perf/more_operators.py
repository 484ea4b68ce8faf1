"""Cases of the operators around the latent cache's decode, for timing and comparison.

Four operators of a serving loop that starts from prompts and may branch:

* ``prefill``: attention within packed prompts before absorption (queries and keys of 128 + 64 dims
  per head with one RoPE key for all heads, values of 128), each sequence by itself, its queries at
  the end of its keys, causal with an optional prefix that every query sees, or in full;
* ``beam``: the k best continuations over all beams and the vocabulary;
* ``fork``: the page table behind a step of beam search (rows taken over, shared, ended, started and
  grown, pages counted, freed and handed out), then the copy of the pages that two rows would write;
* ``compact``: live pages moved from the top of the pool into its holes, table and pool.

Where ``own`` is false ``run`` computes in elementary torch operations; where it is true it makes the
calls a user makes.
"""
import math
import random

import torch

own = False

NOPE, ROPE, VALUE, PAGE = 128, 64, 128, 64
SM_SCALE = 1.0 / math.sqrt(192.0)
ROW_BYTES = {"bf16": 1152, "fp8": 576, "fp4": 352}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one short prompt, a tensor-parallel share of the heads: latency counts
        dict(name="prefill_tiny", op="prefill", N=1, H=16, lo=17, hi=17, ctx_lo=0, ctx_hi=0, prefix=0.0, causal=True, len_seed=0),
        # many short documents with a prefix that is seen from everywhere, all 96 heads
        dict(name="prefill_documents", op="prefill", N=64, H=96, lo=33, hi=700, ctx_lo=0, ctx_hi=0, prefix=0.5, causal=True, len_seed=1),
        # ragged prompts of one batch, few heads
        dict(name="prefill_packed", op="prefill", N=24, H=16, lo=101, hi=6001, ctx_lo=0, ctx_hi=0, prefix=0.0, causal=True, len_seed=2),
        # chunks of a few hundred tokens against long contexts already in the cache: few rows, long keys
        dict(name="prefill_chunk", op="prefill", N=3, H=16, lo=200, hi=300, ctx_lo=8000, ctx_hi=32000, prefix=0.0, causal=True, len_seed=3),
        # one long prompt, all 96 heads: the largest
        dict(name="prefill_long", op="prefill", N=1, H=96, lo=8191, hi=8191, ctx_lo=0, ctx_hi=0, prefix=0.0, causal=True, len_seed=4),
        # one request's beams: latency
        dict(name="beam_one", op="beam", B=1, W=4, V=32000, k=8, dtype="bf16", finished=0.0, allowed=1.0, first=False),
        # a batch's step, odd vocabulary, fp32 logits, some beams at their end
        dict(name="beam_step", op="beam", B=16, W=5, V=100003, k=10, dtype="fp32", finished=0.2, allowed=1.0, first=False),
        # a large batch: bound by the logits' bytes
        dict(name="beam_batch", op="beam", B=64, W=16, V=131072, k=16, dtype="bf16", finished=0.1, allowed=1.0, first=False),
        # one request with four beams
        dict(name="fork_one", op="fork", groups=1, W=4, lo=300, hi=300, own_tokens=40, kv="bf16", keep=False, fresh=0, len_seed=5),
        # a batch of beams over long prompts with rejected drafts and new requests, 4-bit pool
        dict(name="fork_batch", op="fork", groups=32, W=8, lo=2000, hi=16000, own_tokens=1500, kv="fp4", keep=True, fresh=9, len_seed=6),
        # a small pool after a few requests ended
        dict(name="compact_small", op="compact", R=6, lo=500, hi=3001, gone=0.3, kv="bf16", moves=64, len_seed=7),
        # a large pool, half of its requests gone
        dict(name="compact_large", op="compact", R=200, lo=2000, hi=24001, gone=0.5, kv="fp4", moves=8192, len_seed=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "beam", "fork", "compact"])
    if op == "prefill":
        while True:
            lo = _log(rng, 1, 3000)
            ctx = rng.random() < 0.4
            ctx_lo = _log(rng, 1, 8000) if ctx else 0
            case = dict(op=op, N=_log(rng, 1, 64), H=rng.choice([rng.randint(1, 128), 16, 96]), lo=lo, hi=_log(rng, lo, 8191),
                        ctx_lo=ctx_lo, ctx_hi=_log(rng, ctx_lo, 32000) if ctx else 0, prefix=rng.choice([0.0, 0.0, 0.5]),
                        causal=rng.random() < 0.85, len_seed=rng.randint(100, 1 << 30))
            lq, lk, _ = _sequences(case)
            if sum(a * b for a, b in zip(lq, lk)) * case["H"] <= 6.4e9 and sum(lk) * case["H"] < 4.0e6:
                return case
    if op == "beam":
        W, V = rng.randint(1, 16), _log(rng, 100, 260000)
        B = min(_log(rng, 1, 64), max(1, (64 * 16 * 131072) // (W * V)))
        return dict(op=op, B=B, W=W, V=V, k=rng.choice([W, 2 * W, rng.randint(1, 64)]),
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]) if B * W * V < 6e7 else "bf16",
                    finished=rng.choice([0.0, 0.2]), allowed=rng.choice([1.0, 1.0, 0.001]), first=rng.random() < 0.2)
    if op == "fork":
        lo = _log(rng, 1, 4000)
        return dict(op=op, groups=_log(rng, 1, 32), W=rng.randint(1, 8), lo=lo, hi=_log(rng, lo, 16000), own_tokens=_log(rng, 1, 1500),
                    kv=rng.choice(["bf16", "fp8", "fp4"]), keep=rng.random() < 0.5, fresh=rng.randint(0, 9),
                    len_seed=rng.randint(100, 1 << 30))
    lo, kv = _log(rng, 1, 4000), rng.choice(["bf16", "fp8", "fp4", "fp4"])
    share = 352 / ROW_BYTES[kv]  # pools of about the same bytes
    return dict(op=op, R=_log(rng, 2, int(200 * share)), lo=lo, hi=_log(rng, lo, 24001), gone=rng.uniform(0.1, 0.7), kv=kv,
                moves=_log(rng, 16, int(8192 * share)), len_seed=rng.randint(100, 1 << 30))


def _sequences(case):
    """Query lengths, key lengths and prefixes of a packed batch."""
    r = random.Random(case["len_seed"])
    lq = [_log(r, case["lo"], case["hi"]) for _ in range(case["N"])]
    ctx = [_log(r, case["ctx_lo"], case["ctx_hi"]) if case["ctx_hi"] else 0 for _ in lq]
    lk = [a + c for a, c in zip(lq, ctx)]
    return lq, lk, [r.randint(0, b) if r.random() < case["prefix"] else 0 for b in lk]


def _visible(case):
    """Pairs (query, key) of one head."""
    pairs = 0
    for lq, lk, pre in zip(*_sequences(case)):
        pairs += sum(min(lk, max(pre, lk - lq + 1 + i)) for i in range(lq)) if case["causal"] else lq * lk
    return pairs


def _pages(tokens):
    return -(-tokens // PAGE)


def _fork_rows(case):
    """The rows of a beam step on the host: page lists, lengths, parents, kept and new tokens, pool size."""
    r = random.Random(case["len_seed"])
    G, W = case["groups"], case["W"]
    rows, lens, at = [], [], 1
    for _ in range(G):
        prompt = _pages(_log(r, case["lo"], case["hi"]))
        shared = list(range(at, at + prompt))
        at += prompt
        for _ in range(W):
            more = r.randint(1, case["own_tokens"])
            rows.append(shared + list(range(at, at + _pages(more))))
            lens.append(prompt * PAGE + more)
            at += _pages(more)
    R = G * W
    parents = [g * W + min(r.randrange(W), r.randrange(W)) for g in range(G) for _ in range(W)]
    grow = [r.choice([1, 1, 1, 5]) for _ in range(R)]
    keep = [max(0, lens[p] - r.randint(0, 4)) if case["keep"] else lens[p] for p in parents]
    for i in r.sample(range(R), min(case["fresh"], R // 2)):
        parents[i], grow[i] = -1, _log(r, 20, 2000)
    spare = sum(_pages(x) for x in grow) + 2 * R + 16
    return rows, lens, parents, keep, grow, at + spare + at // 8


def _compact_rows(case):
    """The rows of a pool where a share of the requests has ended: page lists, lengths, pool size."""
    r = random.Random(case["len_seed"])
    lens = [_log(r, case["lo"], case["hi"]) for _ in range(case["R"])]
    total = 1 + sum(_pages(n) for n in lens)
    gone = [r.random() < case["gone"] for _ in lens]
    if all(gone):
        gone[0] = False
    return lens, gone, total + total // 16


def work(case):
    if case["op"] == "prefill":
        lq, lk, _ = _sequences(case)
        H = case["H"]
        nbytes = sum(lq) * H * (2 * (NOPE + ROPE) + 2 * VALUE + 4) + sum(lk) * (H * 2 * (NOPE + VALUE) + 2 * ROPE)
        return dict(bytes=nbytes, flops=2 * (NOPE + ROPE + VALUE) * H * _visible(case))
    if case["op"] == "beam":
        n = case["B"] * case["W"]
        live = case["B"] if case["first"] else n
        return dict(bytes=live * case["V"] * (4 if case["dtype"] == "fp32" else 2) + n * 5 + case["B"] * case["k"] * 12,
                    flops=live * case["V"] * 3)
    if case["op"] == "fork":
        rows, lens, parents, keep, grow, pages = _fork_rows(case)
        kept = [min(k, lens[p]) if p >= 0 else 0 for k, p in zip(keep, parents)]
        seen, copied = set(), 0
        for k, p in zip(kept, parents):
            copied += k % PAGE if p in seen else 0
            seen.add(p)
        nbytes = 4 * sum(kept) + 4 * PAGE * sum(_pages(k + g) for k, g in zip(kept, grow)) + 8 * pages + 2 * copied * ROW_BYTES[case["kv"]]
        return dict(bytes=nbytes, flops=0)
    lens, gone, pages = _compact_rows(case)
    live = sum(_pages(n) for n, g in zip(lens, gone) if not g)
    moves = min(case["moves"], int(live * (1 - live / pages)))  # about the live pages above the boundary
    return dict(bytes=8 * pages + 8 * PAGE * live + moves * 2 * PAGE * ROW_BYTES[case["kv"]], flops=0)


# ---------------------------------------------------------------- prepare
def _pool(kv, pages, gen, dev):
    """A pool of random rows; 4-bit and 8-bit rows are random codes (no NaN among the E4M3 ones)."""
    slots = pages * PAGE
    if kv == "bf16":
        return torch.randn((slots, 576), generator=gen, device=dev, dtype=torch.bfloat16), None
    raw = torch.randint(0, 127, (slots, ROW_BYTES[kv]), generator=gen, device=dev, dtype=torch.uint8)
    if kv == "fp8":
        return raw, torch.rand(slots, generator=gen, device=dev)
    return raw, torch.full((1,), 0.0625, device=dev)


def _table(page_lists, stride_pages, dev):
    flat = torch.zeros((len(page_lists), stride_pages), dtype=torch.int32)
    for i, p in enumerate(page_lists):
        flat[i, :len(p)] = torch.tensor(p, dtype=torch.int32)
    base = flat.to(dev)[:, :, None] * PAGE + torch.arange(PAGE, device=dev, dtype=torch.int32)
    held = torch.tensor([len(p) for p in page_lists], device=dev)
    live = torch.arange(stride_pages, device=dev) < held[:, None]
    return torch.where(live[:, :, None], base, 0).reshape(len(page_lists), -1).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed * 6151 + 29)
    host = random.Random(seed * 31 + 7)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    s = dict(case)
    if case["op"] == "prefill":
        lq, lk, pre = _sequences(case)
        H, Tq, Tk = case["H"], sum(lq), sum(lk)

        def randn(*shape):
            return torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)

        # the projections' outputs: queries next to their RoPE part, keys next to values, the RoPE key in its row
        q, kv, rows = randn(Tq, H, NOPE + ROPE), randn(Tk, H, NOPE + VALUE), randn(Tk, 576)
        s.update(q_nope=q[..., :NOPE], q_rope=q[..., NOPE:].contiguous(), k_nope=kv[..., :NOPE], v=kv[..., NOPE:], k_rope=rows[:, 512:],
                 lens=(lq, lk, pre), prefix=ints(pre) if any(pre) else None)
        for name, n in (("cu_q", lq), ("cu_kv", lk)):
            s[name] = ints([sum(n[:i]) for i in range(len(n) + 1)])
        if own:
            import mla_latent_decode_gb300 as mla
            # the plan and the outputs' buffers that a serving loop keeps for a step's layers
            plan, parts = mla.plan_prefill(lq, lk, H, prefix=pre if any(pre) else None, causal=case["causal"])
            s.update(plan=torch.from_numpy(plan).to(dev), parts=parts,
                     O_part=torch.empty((max(parts, 1), H, 256, VALUE), device=dev), LSE_part=torch.empty((max(parts, 1), H, 256), device=dev),
                     out=torch.empty((Tq, H, VALUE), dtype=torch.bfloat16, device=dev), lse=torch.empty((Tq, H), device=dev))
    elif case["op"] == "beam":
        B, W, V = case["B"], case["W"], case["V"]
        dtype = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[case["dtype"]]
        x = torch.empty((B, W, V), dtype=dtype, device=dev)
        for b in range(B):
            x[b] = 2.5 * torch.randn((W, V), generator=gen, device=dev)
            if case["allowed"] < 1:  # constrained decoding: most tokens ruled out
                x[b].masked_fill_(torch.rand((W, V), generator=gen, device=dev) >= case["allowed"], -math.inf)
        c = -8 * torch.rand((B, W), generator=gen, device=dev)
        if case["first"]:  # the first step: the beams are still alike and only one counts
            c[:, 1:] = -math.inf
        s.update(logits=x, scores=c, end_token=min(2, V - 1),
                 done=torch.rand((B, W), generator=gen, device=dev) < case["finished"] if case["finished"] else None,
                 out_scores=torch.empty((B, case["k"]), device=dev), parents=torch.empty((B, case["k"]), dtype=torch.int32, device=dev),
                 tokens=torch.empty((B, case["k"]), dtype=torch.int32, device=dev))
    elif case["op"] == "fork":
        rows, lens, parents, keep, grow, pages = _fork_rows(case)
        names = [0] + host.sample(range(1, pages), pages - 1)
        rows = [[names[p] for p in row] for row in rows]
        refs = [0] * pages
        for row in rows:
            for p in row:
                refs[p] += 1
        refs[0] = 1
        stride = max(max(len(row) for row in rows), max(_pages(k + g) for k, g in zip(keep, grow)), max(_pages(g) for g in grow)) + 2
        table = _table(rows, stride, dev)
        pool, scale = _pool(case["kv"], pages, gen, dev)
        s.update(table=table, lens=ints(lens), parents=ints(parents), keep=ints(keep), grow=ints(grow), refs0=ints(refs),
                 free0=ints([sum(r == 0 for r in refs)]), pool=pool, scale=scale, table_out=torch.zeros_like(table), lens_out=ints([0] * len(rows)))
        s.update(refs=s["refs0"].clone(), free=s["free0"].clone(), copies=torch.zeros((3, len(rows)), dtype=torch.int32, device=dev))
    else:
        lens, gone, pages = _compact_rows(case)
        names = host.sample(range(1, pages), sum(_pages(n) for n in lens))
        rows, at = [], 0
        for n, g in zip(lens, gone):
            rows.append([] if g else names[at:at + _pages(n)])
            at += _pages(n)
        lens = [0 if g else n for n, g in zip(lens, gone)]
        refs = [0] * pages
        for p in [0] + [p for row in rows for p in row]:
            refs[p] = 1
        table = _table(rows, max(len(row) for row in rows) + 1, dev)
        pool, scale = _pool(case["kv"], pages, gen, dev)
        s.update(table=table, lens=ints(lens), refs0=ints(refs), refs=ints(refs), pool=pool, scale=scale, table_out=torch.zeros_like(table),
                 src=torch.zeros(case["moves"], dtype=torch.int32, device=dev), dst=torch.zeros(case["moves"], dtype=torch.int32, device=dev),
                 count=ints([0]))
    return s


# -------------------------------------------------------------------- run
def run(s):
    return {"prefill": _prefill, "beam": _beam, "fork": _fork, "compact": _compact}[s["op"]](s)


def _prefill(s):
    if own:
        import mla_latent_decode_gb300 as mla
        out, lse = mla.prefill(s["q_nope"], s["q_rope"], s["k_nope"], s["k_rope"], s["v"], s["cu_q"], s["cu_kv"], s["plan"], SM_SCALE,
                               prefix=s["prefix"], causal=s["causal"], num_parts=s["parts"], O_part=s["O_part"], LSE_part=s["LSE_part"],
                               out=s["out"], lse_out=s["lse"])
        return dict(out=out, lse=lse)
    H, dev = s["H"], s["v"].device
    out = torch.zeros((s["q_nope"].shape[0], H, VALUE), dtype=torch.bfloat16, device=dev)
    lse = torch.full(out.shape[:2], -math.inf, device=dev)
    qa = ka = 0
    for lq, lk, pre in zip(*s["lens"]):
        qs, ks = slice(qa, qa + lq), slice(ka, ka + lk)
        qa, ka = qa + lq, ka + lk
        sees = (lk - lq + 1 + torch.arange(lq, device=dev)).clamp(min=pre, max=lk) if s["causal"] else torch.full((lq,), lk, device=dev)
        hidden = torch.arange(lk, device=dev) >= sees[:, None]
        step = max(1, min(H, int(6e8 / (lq * lk))))
        for h in range(0, H, step):
            q = torch.cat([s["q_nope"][qs, h:h + step], s["q_rope"][qs, h:h + step]], -1).float().transpose(0, 1)
            k_rope = s["k_rope"][ks].float()[None].expand(q.shape[0], -1, -1)
            k = torch.cat([s["k_nope"][ks, h:h + step].float().transpose(0, 1), k_rope], -1)
            score = torch.bmm(q, k.transpose(1, 2)).mul_(SM_SCALE).masked_fill_(hidden, -math.inf)
            top = score.amax(-1, keepdim=True)
            p = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
            total = p.sum(-1, keepdim=True)
            o = torch.bmm(p, s["v"][ks, h:h + step].float().transpose(0, 1))
            out[qs, h:h + step] = torch.where(total > 0, o / torch.where(total > 0, total, 1.0), 0.0).transpose(0, 1).bfloat16()
            lse[qs, h:h + step] = (top + total.log())[..., 0].T
    return dict(out=out, lse=lse)


def _beam(s):
    if own:
        import mla_latent_decode_gb300 as mla
        scores, parents, tokens = mla.beam_select(s["logits"], s["scores"], s["k"], finished=s["done"], end_token=s["end_token"],
                                                  out_scores=s["out_scores"], parents=s["parents"], tokens=s["tokens"])
        return dict(scores=scores, parents=parents, tokens=tokens)
    B, W, V, k = s["B"], s["W"], s["V"], s["k"]
    scores, where = [], []
    for b in range(B):  # in 64 bits: the order of two beams' tokens hangs on differences of their sums
        x = s["logits"][b].double()
        top = x.amax(-1, keepdim=True)
        lse = top + (x - top).exp().sum(-1, keepdim=True).log()
        x = torch.where(lse.isfinite(), x - lse, -math.inf)  # a beam with nothing allowed has no continuation
        total = s["scores"][b].double()[:, None] + x
        if s["done"] is not None:
            ended = torch.full_like(total, -math.inf)
            ended[:, s["end_token"]] = s["scores"][b].double()
            total = torch.where(s["done"][b][:, None], ended, total)
        best, at = torch.sort(total.reshape(-1), descending=True, stable=True)
        scores.append(best[:k].float())
        where.append(at[:k])
    where = torch.stack(where)
    parents = where // V + W * torch.arange(B, device=where.device)[:, None]
    return dict(scores=torch.stack(scores), parents=parents.int(), tokens=(where % V).int())


def _copy_pages(pool, scale, src, dst, tokens):
    """pool[dst page] = pool[src page], the first `tokens` rows of each."""
    row = torch.arange(PAGE, device=src.device)
    live = row < tokens[:, None]
    a, b = (src[:, None] * PAGE + row)[live], (dst[:, None] * PAGE + row)[live]
    pool[b] = pool[a]
    if scale is not None and scale.numel() > 1:
        scale[b] = scale[a]


def _fork(s):
    s["refs"].copy_(s["refs0"])  # the pool as it stands before the step
    s["free"].copy_(s["free0"])
    if own:
        import mla_latent_decode_gb300 as mla
        table, lens, copies = mla.pages_fork(s["table"], s["lens"], s["refs"], s["free"], parents=s["parents"], keep=s["keep"], grow=s["grow"],
                                             table_out=s["table_out"], lens_out=s["lens_out"], copies=s["copies"])
        mla.kv_copy(s["pool"], copies[0], copies[1], s["scale"], tokens=copies[2])
        return _forked(s, table, lens, copies)
    table, refs = s["table"], s["refs"]
    R, dev = table.shape[0], table.device
    i = torch.arange(R, device=dev)
    alive = s["parents"] >= 0
    p = s["parents"].long().clamp(min=0)
    held = (s["lens"].long() + PAGE - 1) // PAGE
    kept = torch.where(alive, torch.minimum(s["keep"], s["lens"][p]).long(), 0)
    full, part = kept // PAGE, kept % PAGE
    length = kept + s["grow"]
    # the heir of a row: of its children the one that takes most pages, the lowest among equals
    rank = torch.where(alive, (2 * full + (part > 0)) * (R + 1) + R - i, -1)
    best = torch.full((R,), -1, device=dev).scatter_reduce(0, p, rank, "amax")
    heir = alive & (rank == best[p])
    tail = table[p, full * PAGE].long() // PAGE
    stays = heir & (part > 0) & (refs[tail] == 1)
    copied = alive & (part > 0) & ~stays
    have = full + stays
    need = (length + PAGE - 1) // PAGE - have
    first = need.cumsum(0) - need
    new = (refs[1:] == 0).nonzero()[:, 0] + 1
    # the table: what is taken over, then new pages
    pages = table.shape[1] // PAGE
    at = torch.arange(pages, device=dev)
    taken = table[p].reshape(R, pages, PAGE)
    nth = first[:, None] + at - have[:, None]
    base = new[nth.clamp(min=0, max=len(new) - 1)].int()[:, :, None] * PAGE + torch.arange(PAGE, device=dev, dtype=torch.int32)
    out = torch.where((at < have[:, None])[:, :, None], taken, base).reshape(R, -1)
    live = (at < (have + need)[:, None]).repeat_interleave(PAGE, 1)
    s["table_out"].copy_(torch.where(live, out, s["table_out"]))
    s["lens_out"].copy_(length)
    # the counts
    old = table.reshape(R, pages, PAGE)[:, :, 0].long() // PAGE
    refs.index_add_(0, old[at < held[:, None]], torch.full((int(held.sum()),), -1, dtype=torch.int32, device=dev))
    got = s["table_out"].reshape(R, pages, PAGE)[:, :, 0].long() // PAGE
    mine = at < (have + need)[:, None]
    refs.index_add_(0, got[mine], torch.ones(int(mine.sum()), dtype=torch.int32, device=dev))
    s["free"].copy_((refs[1:] == 0).sum())
    src = torch.where(copied, tail, -1)
    dst = torch.where(copied, new[first.clamp(max=len(new) - 1)], -1)
    s["copies"].copy_(torch.stack([src, dst, torch.where(copied, part, 0)]))
    _copy_pages(s["pool"], s["scale"], src[copied], dst[copied], part[copied])
    return _forked(s, s["table_out"], s["lens_out"], s["copies"])


def _pool_values(s):
    """E4M3 codes as values; 4-bit rows as the bytes that were copied."""
    return s["pool"].view(torch.float8_e4m3fn) if s["kv"] == "fp8" else s["pool"]


def _forked(s, table, lens, copies):
    out = dict(table=table, lens=lens, refs=s["refs"], free=s["free"], copies=copies, pool=_pool_values(s))
    return out if s["scale"] is None else dict(out, scale=s["scale"])


def _compact(s):
    s["refs"].copy_(s["refs0"])
    if own:
        import mla_latent_decode_gb300 as mla
        table, src, dst, count = mla.pages_compact(s["table"], s["lens"], s["refs"], table_out=s["table_out"], src=s["src"], dst=s["dst"],
                                                   count=s["count"])
        mla.kv_copy(s["pool"], src, dst, s["scale"], count=count)
    else:
        refs, dev = s["refs"], s["refs"].device
        live = refs > 0
        live[0] = False
        n = int(live.sum())
        at = torch.arange(refs.numel(), device=dev)
        holes = ((at > 0) & (at <= n) & ~live).nonzero()[:, 0]
        high = (live & (at > n)).nonzero()[:, 0].flip(0)
        m = min(len(holes), s["moves"])
        src, dst = high[:m], holes[:m]
        refs[dst] = refs[src]
        refs[src] = 0
        to = at.clone()
        to[src] = dst
        table = s["table"].long()
        here = torch.arange(table.shape[1], device=dev) < (s["lens"].long()[:, None] + PAGE - 1) // PAGE * PAGE
        moved = (to[table // PAGE] * PAGE + table % PAGE).int()
        s["table_out"].copy_(torch.where(here, moved, s["table_out"]))
        s["src"].fill_(-1)
        s["dst"].fill_(-1)
        s["src"][:m], s["dst"][:m] = src.int(), dst.int()
        s["count"].fill_(m)
        _copy_pages(s["pool"], s["scale"], src, dst, torch.full((m,), PAGE, device=dev))
        table, src, dst, count = s["table_out"], s["src"], s["dst"], s["count"]
    out = dict(table=table, refs=s["refs"], src=src, dst=dst, count=count, pool=_pool_values(s))
    return out if s["scale"] is None else dict(out, scale=s["scale"])


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence and request by request; page tables have no computed numbers."""
    if case["op"] in ("fork", "compact"):
        return None
    s = prepare(case, seed)
    if case["op"] == "prefill":
        H = case["H"]
        lq, lk, pre = _sequences(case)
        out, lse = [], []
        for n in range(case["N"]):
            qa, ka = sum(lq[:n]), sum(lk[:n])
            visible = torch.ones((lq[n], lk[n]), dtype=torch.bool, device="cuda")
            if case["causal"]:
                visible = torch.tril(visible, lk[n] - lq[n])
                visible[:, :pre[n]] = True
            o = torch.zeros((lq[n], H, VALUE), dtype=torch.float64, device="cuda")
            total = torch.zeros((lq[n], H), dtype=torch.float64, device="cuda")
            for h in range(H):
                a = s["q_nope"][qa:qa + lq[n], h].double() @ s["k_nope"][ka:ka + lk[n], h].double().T
                a += s["q_rope"][qa:qa + lq[n], h].double() @ s["k_rope"][ka:ka + lk[n]].double().T
                a = torch.where(visible, a / math.sqrt(192.0), -math.inf)
                total[:, h] = torch.logsumexp(a, -1)
                w = torch.exp(a - total[:, h:h + 1])
                o[:, h] = w @ s["v"][ka:ka + lk[n], h].double()
            out.append(o)
            lse.append(total)
        return dict(out=torch.cat(out), lse=torch.cat(lse))
    best = []
    for b in range(case["B"]):
        y = torch.log_softmax(s["logits"][b].double(), -1).nan_to_num(nan=-math.inf) + s["scores"][b].double()[:, None]
        if s["done"] is not None:
            for w in s["done"][b].nonzero()[:, 0].tolist():
                y[w] = -math.inf
                y[w, s["end_token"]] = float(s["scores"][b, w])
        best.append(torch.topk(y.flatten(), case["k"]).values)
    return dict(scores=torch.stack(best), parents=None, tokens=None)
