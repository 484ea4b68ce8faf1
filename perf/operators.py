"""Cases of the 4-bit latent cache and the operators around it, for timing and comparison.

Four operators of one MLA layer's serving step:

* ``attend``: MLA latent decode over a paged cache whose rows are held in 4 bits, with MTP draft
  tokens (query i of a request sees t <= L - q_len + i), merged over its KV parts;
* ``append``: RMS norm of the latent, rotation of the RoPE key and of the queries' RoPE part, and the
  write of the row into the paged pool (bf16, E4M3 or 4 bits), then ``read``: the rows of the context
  back in bf16, as a prefill step needs them for its up-projection;
* ``norm``: residual addition and RMS norm, with the output in E4M3 and its scales.

The 4-bit row (352 bytes): 512 E2M1 codes of c_kv (element 2i in the low half of byte i), 32 E4M3
block scales (16 elements each), 64 E4M3 codes of the RoPE key.  A value is code * block scale * g
(c_kv) or code * g (RoPE key), g one fp32 number of the pool.

Where ``own`` is false ``run`` computes in elementary torch operations in fp32, rounded once at the
end; where it is true it makes the calls a user makes.
"""
import math
import random

import torch

own = False

NOPE, ROPE, ROW, PAGE, ROW4 = 512, 64, 576, 64, 352
EPS = 1e-6
SM_SCALE = 1.0 / math.sqrt(192.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one request without drafts, 16 heads, 256 tokens: the smallest call, where latency counts
        dict(name="attend_tiny", op="attend", B=1, q=1, H=16, lo=256, hi=256, len_seed=0),
        # few heads (a tensor-parallel share), no drafts, odd ragged lengths: bound by the cache's bytes
        dict(name="attend_few_heads", op="attend", B=32, q=1, H=16, lo=2001, hi=60001, len_seed=1),
        # all 96 heads without drafts, many short and medium contexts
        dict(name="attend_no_drafts", op="attend", B=48, q=1, H=96, lo=501, hi=32001, len_seed=2),
        # 24 requests x 5 drafts x 96 heads, 1k to 200k tokens
        dict(name="attend_ragged", op="attend", B=24, q=5, H=96, lo=1000, hi=200000, len_seed=3),
        # 16 requests x 5 drafts x 96 heads x 100k tokens: the largest
        dict(name="attend_dp16", op="attend", B=16, q=5, H=96, lo=100000, hi=100000, len_seed=4),
        # one new token of one request: latency
        dict(name="append_one_fp4", op="append", n=1, H=96, kv="fp4", pairs="interleaved", norm=True, max_pos=4096),
        # a verify step's 16 x 5 tokens
        dict(name="append_step_fp4", op="append", n=80, H=96, kv="fp4", pairs="interleaved", norm=True, max_pos=200000),
        # 128 requests' step into an E4M3 pool, half-split rotation pairs
        dict(name="append_step_fp8", op="append", n=640, H=96, kv="fp8", pairs="halves", norm=True, max_pos=100000),
        # a prefill chunk (odd length) into a bf16 pool, no query rotation here
        dict(name="append_chunk_bf16", op="append", n=16383, H=0, kv="bf16", pairs="interleaved", norm=True, max_pos=100000),
        # a prefill chunk into the 4-bit pool, with its queries
        dict(name="append_chunk_fp4", op="append", n=8191, H=96, kv="fp4", pairs="interleaved", norm=True, max_pos=100000),
        # a verify step's rows, one scale per row
        dict(name="norm_step", op="norm", n=80, d=7168, group=0),
        # a prefill chunk, odd row count, groups of 128
        dict(name="norm_chunk", op="norm", n=16383, d=7168, group=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "norm"])
    if op == "attend":
        H = rng.choice([rng.randint(1, 128), 16, 96])
        q = rng.choice([1, 1, rng.randint(2, 8), 5])
        B = _log(rng, 1, 48)
        lo = _log(rng, 1, 2000)
        hi = _log(rng, lo, 200000)
        # no more work than the largest listed case, and the plain form's scores fit the card
        while B > 1 and (B * hi * q * H > 7.0e8 or B * hi > 3.0e6):
            B = max(1, B // 2)
        return dict(op=op, B=B, q=q, H=H, lo=lo, hi=hi, len_seed=rng.randint(100, 1 << 30))
    if op == "append":
        n = _log(rng, 1, 12000)
        return dict(op=op, n=n, H=rng.choice([0, rng.randint(1, 128), 96]) if n < 8000 else rng.randint(0, 64),
                    kv=rng.choice(["bf16", "fp8", "fp4", "fp4"]), pairs=rng.choice(["interleaved", "halves"]),
                    norm=rng.random() < 0.8, max_pos=_log(rng, max(2, n), 200000))
    group = rng.choice([0, 128])
    n = _log(rng, 1, 16000)
    d = 128 * rng.randint(1, 56) if group else rng.choice([rng.randint(8, 7168), 1536, 512])
    return dict(op=op, n=n, d=d, group=group)


def _lengths(case):
    r = random.Random(case["len_seed"])
    return [_log(r, case["lo"], case["hi"]) for _ in range(case["B"])]


def work(case):
    if case["op"] == "attend":
        lens, q, H = _lengths(case), case["q"], case["H"]
        rows = case["B"] * q * H
        pairs = H * sum(max(0, min(L, L - q + 1 + i)) for L in lens for i in range(q))
        nbytes = sum(lens) * ROW4 + sum(-(-L // PAGE) for L in lens) * 4 + rows * (ROW * 2 + NOPE * 2 + 4)
        return dict(bytes=nbytes, flops=2 * (ROW + NOPE) * pairs)
    if case["op"] == "append":
        n, H = case["n"], case["H"]
        stored = {"bf16": ROW * 2, "fp8": ROW + 4, "fp4": ROW4}[case["kv"]]
        # the new rows in, the stored rows out and in again, the rows in bf16 out; queries in and out
        nbytes = n * (ROW * 2 + 2 * stored + ROW * 2 + ROPE * 4 + 3 * 4) + n * H * ROPE * 4 + NOPE * 2
        return dict(bytes=nbytes, flops=n * (ROW * 8 + H * ROPE * 3))
    n, d, group = case["n"], case["d"], case["group"]
    scales = n * (d // group if group else 1) * 4
    return dict(bytes=n * d * (2 + 2 + 2 + 1) + d * 2 + scales, flops=n * d * 8)


# ------------------------------------------------- the 4-bit and 8-bit formats
def _e2m1(x):
    """Values rounded to E2M1 (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives), ties to even."""
    m = x.abs().clamp(max=6.0)
    fine = torch.round(m * 2) / 2
    mid = torch.round(m)
    wide = torch.round(m / 2) * 2
    return torch.copysign(torch.where(m < 2, fine, torch.where(m < 4, mid, wide)), x)


def _e2m1_codes(v):
    """E2M1 values -> their 4-bit codes."""
    m = v.abs()
    code = torch.where(m < 2, 2 * m, torch.where(m < 4, m + 2, m / 2 + 4)).to(torch.uint8)
    return code | (torch.signbit(v).to(torch.uint8) << 3)


def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _encode4(c, r, g):
    """c [n, 512], r [n, 64] fp32 -> the pool's bytes [n, 352]."""
    n = c.shape[0]
    blocks = c.reshape(n, NOPE // 16, 16)
    s8 = _e4m3(blocks.abs().amax(-1) / (6.0 * g))
    step = (s8.float() * g)[..., None]
    v = _e2m1(torch.where(step > 0, blocks / torch.where(step > 0, step, 1.0), 0.0))
    code = _e2m1_codes(v).reshape(n, NOPE)
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    return torch.cat([packed, s8.view(torch.uint8), _e4m3(r / g).view(torch.uint8)], 1)


def _decode4(rows, g):
    """The pool's bytes [..., 352] -> values [..., 576] fp32."""
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6.], device=rows.device)
    b = rows[..., :256]
    code = torch.stack([b & 15, b >> 4], -1).reshape(*rows.shape[:-1], NOPE)
    s = rows[..., 256:288].view(torch.float8_e4m3fn).float()
    c = lut[code.int()].unflatten(-1, (NOPE // 16, 16)) * (s * g)[..., None]
    r = rows[..., 288:].view(torch.float8_e4m3fn).float() * g
    return torch.cat([c.flatten(-2), r], -1)


# ---------------------------------------------------------------- prepare
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed * 7919 + 17)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    s = dict(case)
    if case["op"] == "attend":
        B, q, H = case["B"], case["q"], case["H"]
        lens = _lengths(case)
        pages = [-(-L // PAGE) for L in lens]
        total = sum(pages)
        perm = (torch.randperm(total, generator=gen, device=dev) + 1).to(torch.int32)
        at = torch.arange(max(pages), device=dev)
        first = torch.tensor([sum(pages[:b]) for b in range(B)], device=dev)
        live = at < torch.tensor(pages, device=dev)[:, None]
        page = torch.where(live, perm[(first[:, None] + at).clamp(max=total - 1)], 0)
        r2t = (page[:, :, None] * PAGE + torch.arange(PAGE, device=dev, dtype=torch.int32)).reshape(B, -1)
        s["g"] = torch.full((1,), 0.0625, device=dev)
        kv = torch.empty(((total + 1) * PAGE, ROW4), dtype=torch.uint8, device=dev)
        for a in range(0, kv.shape[0], 1 << 19):
            x = randn(min(1 << 19, kv.shape[0] - a), ROW)
            kv[a:a + x.shape[0]] = _encode4(x[:, :NOPE], x[:, NOPE:], 0.0625)
        s.update(q_nope=randn(B, q, H, NOPE).bfloat16(), q_rope=randn(B, q, H, ROPE).bfloat16(), kv=kv,
                 r2t=r2t.to(torch.int32).contiguous(), lens=torch.tensor(lens, dtype=torch.int32, device=dev))
        if own:
            # the plan and the workspaces that a serving loop keeps for a step's layers
            import mla_latent_decode_gb300 as mla
            S, bnd, wk, _ = mla.plan_sched(B, q, H, lens, kv_dtype="fp4_e2m1")
            s.update(S=S, bnd=torch.from_numpy(bnd).to(dev), wk=torch.from_numpy(wk).to(dev),
                     O_part=torch.empty((S, 1, B, q, H, NOPE), device=dev),
                     LSE_part=torch.empty((S, 1, B, q, H), device=dev),
                     out=torch.empty((B, q, H, NOPE), dtype=torch.bfloat16, device=dev),
                     lse=torch.empty((B, q, H), device=dev))
    elif case["op"] == "append":
        n, H = case["n"], case["H"]
        slots = -(-n // PAGE) * PAGE + PAGE
        # a projection's output: the latent row next to other columns (rows are strided)
        wide = randn(n, ROW + 64).bfloat16()
        s["rows"] = wide[:, 32:32 + ROW] if n % 2 else wide[:, :ROW].contiguous()
        s["weight"] = (1 + 0.1 * randn(NOPE)).bfloat16() if case["norm"] else None
        s["slots"] = torch.randperm(slots, generator=gen, device=dev)[:n].to(torch.int32)
        s["pos"] = torch.randint(0, case["max_pos"], (n,), generator=gen, device=dev, dtype=torch.int32)
        freq = 10000.0 ** (-torch.arange(0, ROPE, 2, device=dev, dtype=torch.float64) / ROPE)
        angle = torch.arange(case["max_pos"], device=dev, dtype=torch.float64)[:, None] * freq
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["q"] = randn(n, H, ROPE).bfloat16() if H else None
        s["q_out"] = torch.empty_like(s["q"]) if H else None
        width, kind = {"bf16": (ROW, torch.bfloat16), "fp8": (ROW, torch.uint8), "fp4": (ROW4, torch.uint8)}[case["kv"]]
        s["pool"] = torch.zeros((slots, width), dtype=kind, device=dev)
        s["scale"] = {"bf16": None, "fp8": torch.zeros(slots, device=dev), "fp4": torch.full((1,), 0.0625, device=dev)}[case["kv"]]
        s["back"] = torch.empty((n, ROW), dtype=torch.bfloat16, device=dev)
    else:
        n, d = case["n"], case["d"]
        s.update(x=randn(n, d).bfloat16(), res=(2 * randn(n, d)).bfloat16(), weight=(1 + 0.1 * randn(d)).bfloat16())
        s.update(res_out=torch.empty_like(s["res"]), y8=torch.empty((n, d), dtype=torch.float8_e4m3fn, device=dev),
                 scales=torch.empty((n, d // case["group"] if case["group"] else 1), device=dev))
    return s


# -------------------------------------------------------------------- run
def run(s):
    return {"attend": _attend, "append": _append, "norm": _norm}[s["op"]](s)


def _attend(s):
    if own:
        import mla_latent_decode_gb300 as mla
        mla.decode_partial(s["q_nope"], s["q_rope"], s["kv"], s["g"], s["r2t"], s["lens"], None, s["S"], SM_SCALE,
                           O_part=s["O_part"], LSE_part=s["LSE_part"], split_pages=s["bnd"], work=s["wk"])
        out, lse = mla.lse_combine(s["O_part"], s["LSE_part"], out=s["out"], lse_out=s["lse"])
        return dict(out=out, lse=lse)
    B, q, H = s["B"], s["q"], s["H"]
    k = _decode4(s["kv"][s["r2t"].long()], s["g"])                       # [B, T, 576]
    x = torch.cat([s["q_nope"], s["q_rope"]], -1).float().reshape(B, q * H, ROW)
    T = k.shape[1]
    sees = s["lens"][:, None] - q + 1 + torch.arange(q, device=k.device)  # tokens that query i sees
    hidden = torch.arange(T, device=k.device) >= sees[:, :, None]         # [B, q, T]
    score = torch.bmm(x, k.transpose(1, 2)).mul_(SM_SCALE).reshape(B, q, H, T).masked_fill_(hidden[:, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p.reshape(B, q * H, T), k[..., :NOPE]).reshape(B, q, H, NOPE)
    out = torch.where(total > 0, o / torch.where(total > 0, total, 1.0), 0.0).bfloat16()
    return dict(out=out, lse=(top + total.log())[..., 0])


def _rotate(x, cos, sin, pairs):
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs == "interleaved" else (x[..., :ROPE // 2], x[..., ROPE // 2:])
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.stack([u, v], -1).flatten(-2) if pairs == "interleaved" else torch.cat([u, v], -1)


def _append(s):
    if own:
        import mla_latent_decode_gb300 as mla
        mla.kv_append(s["rows"], s["slots"], s["pos"], s["table"], s["pool"], s["scale"], norm_weight=s["weight"], eps=EPS,
                      q_rope=s["q"], q_out=s["q_out"], interleaved=s["pairs"] == "interleaved")
        rows = mla.kv_read(s["pool"], s["slots"], s["scale"], out=s["back"])
        return dict(rows=rows, q=s["q_out"]) if s["H"] else dict(rows=rows)
    x = s["rows"].float()
    c = x[:, :NOPE]
    if s["norm"]:
        c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    t = s["table"][s["pos"].long()]
    cos, sin = t[:, :ROPE // 2], t[:, ROPE // 2:]
    r = _rotate(x[:, NOPE:], cos, sin, s["pairs"])
    at = s["slots"].long()
    if s["kv"] == "bf16":
        s["pool"][at] = torch.cat([c, r], 1).bfloat16()
        rows = s["pool"][at]
    elif s["kv"] == "fp8":
        v = torch.cat([c, r], 1)
        scale = v.abs().amax(-1) / 448.0
        s["pool"][at] = _e4m3(torch.where(scale[:, None] > 0, v / scale[:, None], 0.0)).view(torch.uint8)
        s["scale"][at] = scale
        rows = (s["pool"][at].view(torch.float8_e4m3fn).float() * s["scale"][at][:, None]).bfloat16()
    else:
        s["pool"][at] = _encode4(c, r, s["scale"])
        rows = _decode4(s["pool"][at], s["scale"]).bfloat16()
    if not s["H"]:
        return dict(rows=rows)
    return dict(rows=rows, q=_rotate(s["q"].float(), cos[:, None], sin[:, None], s["pairs"]).bfloat16())


def _norm(s):
    group = s["group"] or s["d"]
    if own:
        import mla_latent_decode_gb300 as mla
        mla.add_rms_norm(s["x"], s["weight"], residual=s["res"], eps=EPS, residual_out=s["res_out"], out8=s["y8"],
                         scales=s["scales"], group=s["group"])
        return dict(y8=s["y8"], scales=s["scales"], res=s["res_out"])
    h = s["x"].float() + s["res"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    y = y.reshape(s["n"], -1, group)
    scale = y.abs().amax(-1, keepdim=True) / 448.0
    y8 = _e4m3(torch.where(scale > 0, y / scale, 0.0)).reshape(s["n"], s["d"])
    return dict(y8=y8, scales=scale[..., 0], res=h.bfloat16())


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """The definitions in 64 bits, request by request; the 8-bit and 4-bit codes have no such value beyond their own."""
    s = prepare(case, seed)
    if case["op"] == "attend":
        B, q, H = case["B"], case["q"], case["H"]
        grid = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2
        out = torch.zeros((B, q, H, NOPE), dtype=torch.float64, device="cuda")
        lse = torch.full((B, q, H), -math.inf, dtype=torch.float64, device="cuda")
        for b, L in enumerate(_lengths(case)):
            raw = s["kv"].index_select(0, s["r2t"][b, :L].long())
            low, high = raw[:, :256] % 16, raw[:, :256] // 16
            code = torch.zeros((L, NOPE), dtype=torch.int64, device="cuda")
            code[:, 0::2], code[:, 1::2] = low.long(), high.long()
            c = grid[code % 8] * (1 - 2 * (code // 8)).double()
            c = c * raw[:, 256:288].contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, 1) * float(s["g"])
            r = raw[:, 288:].contiguous().view(torch.float8_e4m3fn).double() * float(s["g"])
            del code, low, high, raw
            for i in range(q):
                m = min(L, L - q + 1 + i)
                if m <= 0:
                    continue
                a = s["q_nope"][b, i].double() @ c[:m].T + s["q_rope"][b, i].double() @ r[:m].T
                a = a / math.sqrt(192.0)
                lse[b, i] = torch.logsumexp(a, -1)
                out[b, i] = torch.exp(a - lse[b, i][:, None]) @ c[:m]
        return dict(out=out, lse=lse)
    if case["op"] == "append":
        def turn(x):
            z = x.double()
            z = torch.complex(z[..., 0::2], z[..., 1::2]) if case["pairs"] == "interleaved" else torch.complex(z[..., :32], z[..., 32:])
            t = s["table"].double()[s["pos"].long()]
            z = z * torch.complex(t[:, :32], t[:, 32:]).reshape(len(t), *[1] * (z.dim() - 2), 32)
            return torch.view_as_real(z).flatten(-2) if case["pairs"] == "interleaved" else torch.cat([z.real, z.imag], -1)

        x = s["rows"].double()
        c = x[:, :NOPE]
        if case["norm"]:
            c = c / torch.sqrt((c * c).sum(-1, keepdim=True) / NOPE + EPS) * s["weight"].double()
        rows = torch.cat([c, turn(x[:, NOPE:])], 1) if case["kv"] == "bf16" else None
        if case["H"]:
            return dict(rows=rows, q=turn(s["q"]))
        return None if rows is None else dict(rows=rows)
    h = s["x"].double() + s["res"].double()
    y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / case["d"] + EPS) * s["weight"].double()
    top = y.reshape(case["n"], -1, case["group"] or case["d"]).abs().amax(-1)
    return dict(y8=None, scales=top / 448.0, res=h)
