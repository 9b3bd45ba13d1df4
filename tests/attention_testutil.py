"""Plain fp64 forms of the softmax-attention layers' operators, and small helpers, for the tests.

Nothing here comes from the package: the cache's contents are held in logical order
([pages, hkv, page, D] values and scales, lists of pages per sequence) and only ``packed_v`` knows
the value layout of include/gdn.h.
"""
import math

import torch

QMAX = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
TINY = 2.0 ** -100
FORMATS = [torch.int8, torch.float8_e4m3fn]
FORMAT_IDS = ["int8", "e4m3"]
IOS = [torch.bfloat16, torch.float32]
IO_IDS = ["bf16", "fp32"]


def table(max_pos, R, base=1e4):
    f = base ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1))
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def pair_index(R, style):
    """The two elements of each rotated pair."""
    i = torch.arange(R // 2)
    return (i, i + R // 2) if style == "half" else (2 * i, 2 * i + 1)


def rope(x, pos, tab, w, eps, offset, style):
    """fp64 norm, weight and rotation of x [T, heads, D]; also |a| + |b| of each element's pair
    (the scale its rounding errors are measured on)."""
    x = x.double()
    R = tab.shape[1]
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double() + offset
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    ia, ib = pair_index(R, style)
    c, s = tab.double()[pos.long()][:, None].split(R // 2, -1) if R else (None, None)
    out, mag = y.clone(), y.abs()
    if R:
        a, b = y[..., ia], y[..., ib]
        out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return out, mag


def rope_grad(x, pos, tab, w, eps, offset, style, do):
    """fp64 gradients (dx, dw) of <do, rope(x)>, and the magnitudes of the terms summed in each."""
    x, do = x.double(), do.double()
    R, D = tab.shape[1], x.shape[-1]
    w = torch.ones(D, dtype=torch.float64) if w is None else w.double() + offset
    dy, mag = do.clone(), do.abs()
    if R:
        ia, ib = pair_index(R, style)
        c, s = tab.double()[pos.long()][:, None].split(R // 2, -1)
        a, b = do[..., ia], do[..., ib]
        dy[..., ia], dy[..., ib] = a * c + b * s, b * c - a * s
        mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * r
    dn = dy * w
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    dx_mag = r * ((mag * w.abs()) + n.abs() * (mag * w.abs() * n.abs()).mean(-1, keepdim=True))
    return dx, (dy * n).sum((0, 1)), dx_mag, (mag * n.abs()).sum((0, 1))


def values(codes):
    """What codes (int8 or e4m3) stand for before their scale, fp32."""
    return codes.float()


def pick(codes, ids):
    """codes[ids] (8-bit floating point has no indexing on the CPU)."""
    return codes.view(torch.uint8)[ids].view(codes.dtype)


def encode(y, fmt):
    """fp32 y to codes, rounded to nearest even within +-qmax."""
    y = y.float().clamp(-QMAX[fmt], QMAX[fmt])
    return y.round().to(torch.int8) if fmt == torch.int8 else y.to(torch.float8_e4m3fn)


def page_scale(amax, fmt):
    """fp32 scale of pages with that fp32 amax."""
    s = amax.float() * torch.tensor(1.0 / QMAX[fmt], dtype=torch.float32)
    return torch.where(amax >= TINY, s, torch.zeros_like(s))


def inverse(scale):
    return torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))


def random_cache(pages, hkv, page, D, fmt, gen, std=1.0):
    """Codes [pages, hkv, page, D] and scales [pages, hkv] of random values (CPU)."""
    x = torch.randn(pages, hkv, page, D, generator=gen) * std
    s = page_scale(x.abs().amax((2, 3)), fmt)
    return encode(x * inverse(s)[:, :, None, None], fmt), s


def packed_v(codes):
    """Logical value codes [pages, hkv, page, D] in the cache's layout [.., page/4, D, 4]."""
    p, h, page, D = codes.shape
    raw = codes.view(torch.uint8).view(p, h, page // 4, 4, D).transpose(3, 4).contiguous()
    return raw.view(codes.dtype)


def unpacked_v(v):
    p, h, g, D, _ = v.shape
    raw = v.view(torch.uint8).transpose(3, 4).contiguous().view(p, h, 4 * g, D)
    return raw.view(v.dtype)


def block_tables(lens, page, gen, extra=3, junk=-1):
    """Random distinct pages for each sequence; entries past a length hold `junk`."""
    counts = [-(-n // page) for n in lens]
    perm = torch.randperm(sum(counts) + extra, generator=gen).tolist()
    t = torch.full((len(lens), max(1, max(counts))), junk, dtype=torch.int32)
    at = 0
    for n, c in enumerate(counts):
        t[n, :c] = torch.tensor(perm[at:at + c], dtype=torch.int32)
        at += c
    return t, sum(counts) + extra


def cumulative(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)


def append_ref(codes, scales, x, tables, ctx, new, page, fmt):
    """The append of include/gdn.h on logical codes, in place, token range by token range; fp32
    arithmetic as stated there (the codes are to come out equal, bit for bit)."""
    t0 = 0
    for n, (c, m) in enumerate(zip(ctx, new)):
        p = c // page
        while m and p * page < c + m:
            lo, hi = max(p * page, c), min((p + 1) * page, c + m)
            pid = int(tables[n, p])
            for h in range(codes.shape[1]):
                rows = x[t0 + lo - c:t0 + hi - c, h].float()
                good = torch.isfinite(rows)
                amax = torch.where(good, rows.abs(), torch.zeros_like(rows)).max()
                held = scales[pid, h].clone() if lo > p * page else torch.tensor(0.0)
                s = torch.maximum(held, page_scale(amax, fmt))
                inv = inverse(s)
                old = codes[pid, h, :lo - p * page]
                if old.numel():
                    codes[pid, h, :lo - p * page] = encode(values(old) * (held * inv), fmt)
                y = torch.where(good, rows * inv, torch.zeros_like(rows))
                y = torch.where(torch.isinf(rows) & (s > 0), rows, y)
                codes[pid, h, lo - p * page:hi - p * page] = encode(y, fmt)
                scales[pid, h] = s
            p += 1
        t0 += m


def attention_ref(q, codes_k, scale_k, codes_v, scale_v, tables, lens, new, page, scale, window):
    """fp64 attention; also sum p |v| of every output and the largest |score| sum of every row."""
    T, hq, D = q.shape
    hkv = codes_k.shape[1]
    G = hq // hkv
    out = torch.zeros(T, hq, D, dtype=torch.float64)
    mag = torch.zeros(T, hq, D, dtype=torch.float64)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    t = 0
    for n, (L, m) in enumerate(zip(lens, new)):
        if L:
            ids = tables[n, :-(-L // page)].long()
            k = (values(pick(codes_k, ids)).double() * scale_k[ids].double()[..., None, None])
            v = (values(pick(codes_v, ids)).double() * scale_v[ids].double()[..., None, None])
            k = k.transpose(0, 1).flatten(1, 2)[:, :L]
            v = v.transpose(0, 1).flatten(1, 2)[:, :L]
        for i in range(m):
            at = L - m + i
            j0 = max(0, at - window + 1) if window else 0
            if L and at >= 0:
                for h in range(hkv):
                    qq = q[t, h * G:(h + 1) * G].double()
                    x = qq @ k[h, j0:at + 1].T * scale
                    p = torch.softmax(x, -1)
                    out[t, h * G:(h + 1) * G] = p @ v[h, j0:at + 1]
                    mag[t, h * G:(h + 1) * G] = p @ v[h, j0:at + 1].abs()
                    lse[t, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            t += 1
    return out, lse, mag
