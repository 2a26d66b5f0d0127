"""Plain 64-bit form of the 4-bit KV cache, from the layout and formulas of the C header."""
import math
from fractions import Fraction

import torch


def params(lo: float, hi: float):
    """(scale, zero) of a group in exact arithmetic (Python's fractions), NaN where it has none."""
    d = float(torch.tensor(hi, dtype=torch.float32) - torch.tensor(lo, dtype=torch.float32))
    a = max(abs(lo), abs(hi))
    if not (math.isfinite(d) and math.isfinite(a)):
        return math.nan, math.nan
    least = max(Fraction(d) * 4 / 59, Fraction(a) / 64, Fraction(1, 1 << 120))
    e = math.floor(math.log2(least)) - 8
    while Fraction(2) ** (e + 8) <= least:
        e += 1
    unit = Fraction(2) ** e                       # least = 128..256 units
    scale = math.ceil(least / unit) * unit
    return float(scale), math.floor(4 * Fraction(lo) / scale) / 4


def code(x: float, scale: float, zero: float) -> int:
    """nearest(x / scale - zero), ties to even, in exact arithmetic."""
    return 0 if math.isnan(scale) else min(15, max(0, round(Fraction(x) / Fraction(scale) - Fraction(zero))))


def values(x: torch.Tensor) -> torch.Tensor:
    """What the form holds of x [..., D], group by group and number by number (small inputs)."""
    flat = x.double().cpu().reshape(-1, 32).tolist()
    out = []
    for g in flat:
        bad = any(not math.isfinite(v) for v in g)
        s, z = (math.nan, math.nan) if bad else params(min(g), max(g))
        out.append([s * (code(v, s, z) + z) if not bad else math.nan for v in g])
    return torch.tensor(out, dtype=torch.float64).reshape(x.shape)


def offsets(dh: int, r: int):
    """Of token r: byte and nibble of each key channel and each value channel, bytes of the scales (2 each)."""
    ng = dh // 32
    key, val = [], []
    for c in range(dh):
        g, cc, i = c // 32, c % 32 // 8, c % 8
        key.append((r * dh // 2 + (ng * cc + g) * 4 + i // 2, i % 2))
        j, n = c // 16, c % 8
        val.append((8 * dh + 512 * (j // 4) + 64 * n + 16 * (r % 8 // 2) + 4 * (j % 4) + 2 * (r % 2) + r // 8, c % 16 // 8))
    return key, val, 16 * dh + 4 * ng * r, 16 * dh + 64 * ng + 4 * ng * r


def unpack(pool: torch.Tensor):
    """((codes, scales, zeros) of keys and of values): [pages, heads, tokens, D] and [..., D / 32] in 64 bits."""
    pool = pool.cpu()
    pages, heads, blocks, size = pool.shape
    dh = size // 20
    ng = dh // 32
    out = []
    for which in (0, 1):
        codes, prm = [], []
        for r in range(16):
            o = offsets(dh, r)
            at, nib = (torch.tensor(v) for v in zip(*o[which]))
            codes.append((pool[..., at].int() >> (4 * nib)) & 15)
            start = o[2 + which]
            prm.append(pool[..., start:start + 4 * ng].contiguous().view(torch.bfloat16))
        codes = torch.stack(codes, 3).reshape(pages, heads, 16 * blocks, dh).double()
        prm = torch.stack(prm, 3).reshape(pages, heads, 16 * blocks, 2 * ng).double()
        out.append((codes, prm[..., :ng], prm[..., ng:]))
    return out


def decode(part):
    codes, scale, zero = part
    return (scale[..., None] * (codes.unflatten(-1, (-1, 32)) + zero[..., None])).flatten(-2)


def sequence(table, s, n, part):
    """Rows [n, heads, ...] of sequence s of a tensor [pages, heads, tokens, ...]."""
    tokens = part.shape[2]
    return torch.stack([part[int(table[s, p // tokens]), :, p % tokens] for p in range(n)]) if n else part.new_zeros(
        (0, part.shape[1], *part.shape[3:]))


def attention(q, q_pos, pool, table, scale):
    """(out, mass, room) of queries [n, t, h, dh] in 64 bits: mass = sum_j p_j |v_j| of each output, room what
    fp32 arithmetic may leave of error in it."""
    n, t, h, dh = q.shape
    q, q_pos, table = q.double().cpu(), q_pos.view(n, t).cpu(), table.cpu()
    kp, vp = unpack(pool)
    hkv = pool.shape[1]
    out, mass, room = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
    for i in range(n):
        keys = max(0, int(q_pos[i].max()) + 1)
        k, v = (sequence(table, i, keys, decode(p)) for p in (kp, vp))
        (ks, kz), (vs, vz) = ([sequence(table, i, keys, p[x]) for x in (1, 2)] for p in (kp, vp))
        for a in range(t):
            m = int(q_pos[i, a]) + 1
            for b in range(h if m > 0 else 0):
                g = b // (h // hkv)
                p = torch.softmax(scale * (k[:m, g] @ q[i, a, b]), 0)
                out[i, a, b], mass[i, a, b] = p @ v[:m, g], p @ v[:m, g].abs()
                # scores: products with 16 + code and (zero - 16) times a sum of the query; the groups' sums, their
                # two steps a part and the scale are under 16 operations, each off by 2^-23 (truncation) of this size
                size = ((47 + kz[:m, g].abs()) * ks[:m, g]) @ q[i, a, b].view(-1, 32).abs().sum(1)
                off = 2 * (abs(scale) * 16 * 2.0 ** -23 * size.max() + 2.0 ** -20)  # of a weight; the exponential's 2^-20
                # outputs: the same with 16 + code and zero - 16, a step for 16 keys of a warp (64 of a CTA), then merges
                size = (p @ ((47 + vz[:m, g].abs()) * vs[:m, g])).repeat_interleave(32)
                room[i, a, b] = 2 * off * mass[i, a, b] + (m / 64 + 32) * 2.0 ** -23 * size
    return out, mass, room
