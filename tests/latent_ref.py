"""Plain 64-bit references of the 4-bit latent rows and the operators around
them (numpy / torch float64 on the CPU), written from the formats' definitions:
E4M3 and E2M1 by their value tables, nearest with ties to the even code.
"""
import math

import numpy as np
import torch

NOPE, ROPE, ROW, PAGE, ROW4 = 512, 64, 576, 64, 352


def _table(ebits, mbits, bias, drop):
    """Non-negative values of a small float in code order, the last `drop`
    codes (NaN) left out."""
    n = 1 << (ebits + mbits)
    out = []
    for c in range(n - drop):
        e, m = c >> mbits, c & ((1 << mbits) - 1)
        out.append(m * 2.0 ** (1 - bias - mbits) if e == 0
                   else (1 + m / 2 ** mbits) * 2.0 ** (e - bias))
    return np.array(out)


E4M3 = _table(4, 3, 7, 1)
E2M1 = _table(2, 1, 1, 0)
assert E4M3[-1] == 448 and list(E2M1) == [0, .5, 1, 1.5, 2, 3, 4, 6]


def encode(x, table):
    """Codes (without sign) of |x| rounded to the nearest value, ties to the
    even code, saturated."""
    m = np.abs(np.asarray(x, np.float64))
    mid = (table[1:] + table[:-1]) / 2
    lo = np.searchsorted(mid, m, side="left")    # a tie stays below
    hi = np.searchsorted(mid, m, side="right")   # a tie goes above
    return np.where(lo % 2 == 0, lo, hi)


def sure(x, table, rel=2.0 ** -18):
    """Where the code of x does not depend on a relative error of `rel`."""
    return encode(np.abs(x) * (1 - rel), table) == encode(np.abs(x) * (1 + rel), table)


def e4m3_values(codes):
    codes = np.asarray(codes).astype(np.int64)
    mag = np.append(E4M3, np.nan)[codes & 0x7F]
    return np.where(codes & 0x80, -mag, mag)


def decode4(rows, g):
    """uint8 [..., 352] -> float64 [..., 576]."""
    rows = np.asarray(rows)
    by = rows[..., :256].astype(np.int64)
    code = np.stack([by & 15, by >> 4], -1).reshape(*rows.shape[:-1], NOPE)
    c = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]
    s = np.repeat(e4m3_values(rows[..., 256:288]), 16, -1)
    with np.errstate(invalid="ignore"):
        return np.concatenate([c * s, e4m3_values(rows[..., 288:])], -1) * g


def rotate(x, cos, sin, interleaved):
    """float64 [..., 64] rotated by cos / sin [..., 32]."""
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    u, v = a * cos - b * sin, a * sin + b * cos
    if interleaved:
        return np.stack([u, v], -1).reshape(x.shape)
    return np.concatenate([u, v], -1)


def random_pool(num_slots, seed, g=0.0625):
    """Uniform codes with plausible scales and RoPE codes, uint8 [slots, 352]."""
    r = np.random.default_rng(seed)
    kv = np.empty((num_slots, ROW4), np.uint8)
    kv[:, :256] = r.integers(0, 256, (num_slots, 256))
    kv[:, 256:288] = encode(r.uniform(0.5, 8.0, (num_slots, 32)), E4M3)
    x = r.standard_normal((num_slots, 64)) / g
    kv[:, 288:] = encode(x, E4M3) | np.where(x < 0, 0x80, 0)
    return kv


def attend(q_nope, q_rope, k, visible, sm_scale):
    """One row group over one token range: q [R, 576] parts, k float64 [T, 576],
    visible [R, T] -> (O [R, 512], LSE [R], A [R, 512], E [R]): A = sum p |v|
    and E = the largest sum |q_d k_d| sm_scale of a visible token, for bounds."""
    x = np.concatenate([q_nope, q_rope], -1)
    vis = np.asarray(visible)
    k0 = np.where(vis.any(0)[:, None], k, 0.0)
    s = np.where(vis, x @ k0.T * sm_scale, -np.inf)
    mag = np.where(vis, np.abs(x) @ np.abs(k0).T * sm_scale, 0.0)
    top = s.max(1, initial=-np.inf)
    with np.errstate(divide="ignore", invalid="ignore"):
        p = np.where(vis, np.exp(s - np.where(np.isneginf(top), 0, top)[:, None]), 0.0)
        l = p.sum(1)
        lse = np.where(l > 0, top + np.log(l), -np.inf)
        p = np.where(l[:, None] > 0, p / l[:, None], 0.0)
    return p @ k0[:, :NOPE], lse, p @ np.abs(k0[:, :NOPE]), mag.max(1, initial=0.0)


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def table(max_pos):
    """fp32 [max_pos, 64] cosines and sines, angles in float64."""
    a = np.arange(max_pos)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32))


__all__ = [n for n in dir() if not n.startswith("_")] + ["math"]
