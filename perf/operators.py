"""Cases that time and check the operators of an attention layer next to the recurrent ones.

A stack of gated-delta-rule layers usually has a softmax-attention layer every few layers.  Its
serving and training operators are measured here:

  rope       q and k normalised per head (RMS) and rotated by position, one pass
  rope_grad  the gradients of that pass: of q, k and both norm weights
  cache      new keys and values quantised to 8 bits into a paged cache (one scale for each page
             and head), then every page that was written read back
  attention  queries (one token or a few drafted ones per sequence) over that cache

``run`` computes an operator in its plain form, elementary torch operations in 32 bits, or,
where ``own`` is set, through the package's entry points.  ``exact`` computes it from its
definition in 64 bits.  Lengths of sequences are part of a case (drawn from its ``mix``), values
come from the seed.
"""
import math
import random

import torch

own = False

EPS = 1e-6
TINY = 2.0 ** -100          # a page whose values are all below this is stored as zeros
QMAX = {"int8": 127.0, "e4m3": 448.0}
IO = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- the cases

def _rope(name, kind, T, hq, hkv, D, R, io="bf16", style="half", gate=False, offset=0.0):
    return {"name": name, "kind": kind, "T": T, "hq": hq, "hkv": hkv, "D": D, "R": R, "io": io,
            "style": style, "gate": gate, "offset": offset, "max_pos": 32768}


def _cache(name, N, new, ctx, hkv, D, page, fmt="int8", io="bf16", mix=1):
    return {"name": name, "kind": "cache", "N": N, "new": new, "ctx": ctx, "hkv": hkv, "D": D,
            "page": page, "fmt": fmt, "io": io, "mix": mix}


def _attn(name, N, kv, q, hq, hkv, D, page, fmt="int8", io="bf16", window=0, spread="even",
          mix=1):
    return {"name": name, "kind": "attention", "N": N, "kv": kv, "q": q, "hq": hq, "hkv": hkv,
            "D": D, "page": page, "fmt": fmt, "io": io, "window": window, "spread": spread,
            "mix": mix}


def listed():
    return [
        # a decode step of a small batch: latency; gated queries (q | gate per head), the first
        # quarter of the head rotated, weights stored around zero
        _rope("rope step 24", "rope", 24, 16, 2, 256, 64, gate=True, offset=1.0),
        # a prefill chunk, the whole head rotated
        _rope("rope prefill 16384", "rope", 16384, 32, 8, 128, 128),
        # a training step's backward
        _rope("rope grad 8192", "rope_grad", 8192, 16, 2, 256, 64, gate=True, offset=1.0),
        # a small odd fp32 run, neighbouring pairs rotated
        _rope("rope grad fp32 1531", "rope_grad", 1531, 6, 3, 64, 32, "f32", "pairs"),
        # one token appended to each of 96 requests (a step of a serving batch)
        _cache("cache step 96", 96, 1, 6000, 2, 256, 64, mix=11),
        # packed prompts, some continuing a part-filled page
        _cache("cache prefill 7x8192", 7, 8192, 777, 8, 128, 64, mix=12),
        # small pages, 8-bit floating point, fp32 inputs, odd head count
        _cache("cache e4m3 fp32", 5, 700, 300, 3, 64, 16, "e4m3", "f32", mix=13),
        # one request, a short context: latency
        _attn("attention 1x1500", 1, 1500, 1, 16, 2, 256, 64, mix=21),
        # a serving batch of mixed lengths, padding rows (length 0) among them
        _attn("attention 32x8192 ragged", 32, 8192, 1, 32, 8, 128, 64, spread="ragged", mix=22),
        # long contexts
        _attn("attention 64x65536", 64, 65536, 1, 32, 4, 128, 128, mix=23),
        # drafted tokens being verified: up to five per request
        _attn("attention draft 24x20000", 24, 20000, 5, 32, 4, 128, 32, "e4m3", mix=24),
        # a sliding window, small pages, fp32 inputs, odd group
        _attn("attention window fp32", 9, 5000, 3, 9, 3, 64, 16, "e4m3", "f32", window=1000,
              spread="ragged", mix=25),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "rope_grad", "cache", "cache", "attention", "attention"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    D = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8, 12, 16])
    if kind in ("rope", "rope_grad"):
        hq = min(hkv * group, 32)
        most = 16384 * 40 * 128 // ((hq + hkv) * D * (2 if io == "f32" else 1))
        T = _log(rng, 1, min(16384, most))
        R = rng.choice([r for r in (32, 48, 64, 96, 128, 256) if r <= D])
        c = _rope("", kind, T, hq, hkv, D, R, io, rng.choice(["half", "half", "pairs"]),
                  rng.random() < 0.5, rng.choice([0.0, 1.0]))
    elif kind == "cache":
        N = _log(rng, 1, 96)
        step = rng.random() < 0.4
        new = 1 if step else max(2, min(8192, 7 * 8192 * 8 * 128 // (2 * N * hkv * D)))
        new = new if step else _log(rng, 2, new)
        c = _cache("", N, new, _log(rng, 1, 6000), hkv, D, rng.choice([16, 32, 64, 128]),
                   rng.choice(["int8", "e4m3"]), io, rng.randrange(1 << 30))
    else:
        N = _log(rng, 1, 64)
        most = 32 * 65536 * 4 * 128 // (N * hkv * D)
        kv = _log(rng, 1, min(65536, most))
        c = _attn("", N, kv, rng.choice([1, 1, 1, 2, 4, 7]), hkv * group, hkv, D,
                  rng.choice([16, 32, 64, 128]), rng.choice(["int8", "e4m3"]), io,
                  rng.choice([0, 0, 0, max(1, kv // 3)]), rng.choice(["even", "ragged"]),
                  rng.randrange(1 << 30))
    c.pop("name")
    return c


def _lengths(case):
    """The sequences' lengths, from the case alone: (context before, new tokens) for the cache,
    (whole length, queries) for the attention."""
    r = random.Random(case["mix"])
    a, b = [], []
    for _ in range(case["N"]):
        if case["kind"] == "cache":
            a.append(r.randint(0, case["ctx"]))
            b.append(1 if case["new"] == 1 else r.randint(case["new"] // 2, case["new"]))
        else:
            q = r.randint(1, case["q"])
            if case["spread"] == "even":
                n = r.randint(3 * case["kv"] // 4, case["kv"])
            elif r.random() < 0.06:
                n = 0
            else:
                n = _log(r, 1, case["kv"])
            a.append(n if n == 0 else max(n, q))
            b.append(q)
    return a, b


def _itemsize(case):
    return 2 if case["io"] == "bf16" else 4


def work(case):
    e = _itemsize(case)
    if case["kind"] in ("rope", "rope_grad"):
        rows, T = case["T"] * (case["hq"] + case["hkv"]), case["T"]
        n = rows * case["D"]
        more = min(T, case["max_pos"]) * case["R"] * 4 + T * 4
        if case["kind"] == "rope":
            return {"bytes": 2 * n * e + more, "flops": 7 * n}
        return {"bytes": 3 * n * e + more, "flops": 14 * n}
    a, b = _lengths(case)
    hkv, D, page = case["hkv"], case["D"], case["page"]
    if case["kind"] == "cache":
        wrote = sum(b) * hkv * D * 2
        back = sum(c % page + n for c, n in zip(a, b)) * hkv * D * 2
        return {"bytes": wrote * (e + 1) + back * (1 + e), "flops": 3 * wrote + back}
    read = flops = 0
    for n, q in zip(a, b):
        if n:
            seen = min(n, case["window"] + q - 1) if case["window"] else n
            read += seen
            flops += 4 * seen * q * case["hq"] * D
    scales = read // page * hkv * 8
    return {"bytes": read * hkv * D * 2 + scales + 2 * sum(b) * case["hq"] * D * e,
            "flops": flops}


# ------------------------------------------------------------------------------ the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _store(x, fmt):
    """Codes (one byte each) and scales of pages x [pages, hkv, page, D]."""
    amax = x.abs().amax((2, 3))
    scale = torch.where(amax >= TINY, amax * (1.0 / QMAX[fmt]), torch.zeros_like(amax))
    y = x * torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))[:, :, None, None]
    y = y.clamp_(-QMAX[fmt], QMAX[fmt])
    codes = y.round_().to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), scale


def _interleaved(v):
    """The value cache's layout: four tokens' codes of a channel next to each other."""
    P, h, page, D = v.shape
    return v.view(P, h, page // 4, 4, D).transpose(3, 4).contiguous()


def _tables(lens, page, gen):
    """A block table (unused entries -1) over a pool whose pages are handed out at random; the
    pool's last page belongs to no sequence."""
    counts = torch.tensor([-(-n // page) for n in lens])
    total = int(counts.sum())
    table = torch.full((len(lens), max(1, int(counts.max()))), -1, dtype=torch.int32)
    seed = int(torch.randint(1 << 30, (1,), device="cuda", generator=gen))
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed))
    table[torch.arange(table.shape[1])[None] < counts[:, None]] = perm.to(torch.int32)
    return table.cuda(), total + 1


def _cumulative(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = _gen(seed)
    D, hkv, io = case["D"], case["hkv"], IO[case["io"]]
    s = {"case": dict(case)}
    if case["kind"] in ("rope", "rope_grad"):
        T, hq, R = case["T"], case["hq"], case["R"]
        # one projection holds q (and its gate, head by head), k and v
        wide = hq * D * (2 if case["gate"] else 1)
        proj = _randn(gen, T, wide + 2 * hkv * D).to(io)
        q = proj[:, :wide].view(T, hq, -1)[:, :, :D]
        k = proj[:, wide:wide + hkv * D].view(T, hkv, D)
        f = 1e6 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
        ang = torch.arange(case["max_pos"], device="cuda", dtype=torch.float64)[:, None] * f
        start = seed * 7919 % case["max_pos"]
        s.update(q=q, k=k, table=torch.cat([ang.cos(), ang.sin()], 1).float(),
                 pos=((torch.arange(T, device="cuda") + start) % case["max_pos"]).int(),
                 wq=1.0 - case["offset"] + 0.1 * _randn(gen, D),
                 wk=1.0 - case["offset"] + 0.1 * _randn(gen, D))
        if case["kind"] == "rope_grad":
            s.update(dqo=_randn(gen, T, hq, D).to(io), dko=_randn(gen, T, hkv, D).to(io))
        return s
    fmt, page = case["fmt"], case["page"]
    a, b = _lengths(case)
    whole = [x + y for x, y in zip(a, b)] if case["kind"] == "cache" else a
    table, pages = _tables(whole, page, gen)
    k, ks = _store(_randn(gen, pages, hkv, page, D), fmt)
    v_plain, vs = _store(_randn(gen, pages, hkv, page, D) * 0.5, fmt)
    kind = torch.int8 if fmt == "int8" else torch.float8_e4m3fn
    s.update(table=table, k=k.view(kind), v_plain=v_plain, v=_interleaved(v_plain).view(kind),
             k_scale=ks, v_scale=vs, cu=_cumulative(b))
    T = sum(b)
    if case["kind"] == "cache":
        lens = torch.tensor(a, dtype=torch.int32)
        s.update(ctx=lens.cuda(), start=(lens // page * page).cuda(), tokens=T,
                 new_k=_randn(gen, T, hkv, D).to(io),
                 new_v=(_randn(gen, T, 3 * hkv * D) * 0.5).to(io)[:, 2 * hkv * D:]
                 .view(T, hkv, D))
        back = [x % page + y for x, y in zip(a, b)]
        s.update(cu_back=_cumulative(back), back=sum(back))
    else:
        s.update(lens=torch.tensor(a, dtype=torch.int32, device="cuda"), most_kv=max(a),
                 most_q=max(b), scale=1.0 / math.sqrt(D),
                 q=(1.5 * _randn(gen, T, case["hq"], D)).to(io))
    return s


# ------------------------------------------------------------------------------ plain forms

def _rotate(y, pos, table, R, style, sign=1.0):
    c, n = table[pos.long(), None, :R // 2], sign * table[pos.long(), None, R // 2:]
    if style == "half":
        y1, y2 = y[..., :R // 2], y[..., R // 2:R]
        return torch.cat([y1 * c - y2 * n, y2 * c + y1 * n, y[..., R:]], -1)
    y1, y2 = y[..., 0:R:2], y[..., 1:R:2]
    return torch.cat([torch.stack([y1 * c - y2 * n, y2 * c + y1 * n], -1).flatten(-2),
                      y[..., R:]], -1)


def _plain_rope(s):
    c = s["case"]

    def one(x, w):
        xf = x.float()
        y = xf * torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS) * (w + c["offset"])
        return _rotate(y, s["pos"], s["table"], c["R"], c["style"]).to(x.dtype)

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def _plain_rope_grad(s):
    c = s["case"]

    def one(x, w, do):
        xf = x.float()
        r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
        n = xf * r
        dy = _rotate(do.float(), s["pos"], s["table"], c["R"], c["style"], -1.0)
        dn = dy * (w + c["offset"])
        dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
        return dx.to(x.dtype), (dy * n).sum((0, 1))

    dq, dwq = one(s["q"], s["wq"], s["dqo"])
    dk, dwk = one(s["k"], s["wk"], s["dko"])
    return dq, dk, dwq, dwk


def _values(codes, fmt):
    return codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float()


def _codes(y, fmt):
    y = y.clamp(-QMAX[fmt], QMAX[fmt])
    y = y.round().to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)
    return y.view(torch.uint8)


def _plain_cache(s):
    c = s["case"]
    page, fmt, io = c["page"], c["fmt"], IO[c["io"]]
    table, ctx, cu = s["table"].long(), s["ctx"].long(), s["cu"].long()
    N, null = ctx.numel(), s["k_scale"].shape[0] - 1
    new = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(N, device="cuda"), new, output_size=s["tokens"])
    pos = ctx[seq] + torch.arange(s["tokens"], device="cuda") - cu[seq]
    pid, slot = table[seq, pos // page], pos % page
    # the part-filled page that a sequence continues, if any (the pool's spare page if not)
    held = (ctx % page > 0) & (new > 0)
    first = table.gather(1, (ctx // page).clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    first = torch.where(held, first, null)
    kept = torch.arange(page, device="cuda") < (ctx % page)[:, None]

    def append(codes, scale, x):
        xf = x.float()
        amax = torch.zeros_like(scale).scatter_reduce_(
            0, pid[:, None].expand(-1, scale.shape[1]), xf.abs().amax(-1), "amax")
        cand = torch.where(amax >= TINY, amax * (1.0 / QMAX[fmt]), torch.zeros_like(amax))
        held_scale = torch.zeros_like(scale)
        held_scale[first] = scale[first] * held[:, None]
        touched = torch.zeros_like(scale, dtype=torch.bool)
        touched[pid] = True
        now = torch.where(touched, torch.maximum(held_scale, cand), scale)
        inv = torch.where(now > 0, 1.0 / now, torch.zeros_like(now))
        old = codes[first]
        ratio = (held_scale * inv)[first][:, :, None, None]
        codes[first] = torch.where((kept & held[:, None])[:, None, :, None],
                                   _codes(_values(old, fmt) * ratio, fmt), old)
        codes[pid, :, slot] = _codes(xf * inv[pid][:, :, None], fmt)
        scale.copy_(now)

    append(s["k"].view(torch.uint8), s["k_scale"], s["new_k"])
    append(s["v_plain"], s["v_scale"], s["new_v"])
    cb, start = s["cu_back"].long(), s["start"].long()
    seq = torch.repeat_interleave(torch.arange(N, device="cuda"), cb[1:] - cb[:-1],
                                  output_size=s["back"])
    pos = start[seq] + torch.arange(s["back"], device="cuda") - cb[seq]
    pid, slot = table[seq, pos // page], pos % page

    def read(codes, scale):
        return (_values(codes[pid, :, slot], fmt) * scale[pid][:, :, None]).to(io)

    return (read(s["k"].view(torch.uint8), s["k_scale"]), read(s["v_plain"], s["v_scale"]),
            s["k_scale"], s["v_scale"])


def _plain_attention(s):
    c = s["case"]
    page, fmt, hkv, hq, D = c["page"], c["fmt"], c["hkv"], c["hq"], c["D"]
    G, Q = hq // hkv, s["most_q"]
    cu, lens = s["cu"].long(), s["lens"].long()
    N, T = lens.numel(), s["q"].shape[0]
    new = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(N, device="cuda"), new, output_size=T)
    off = torch.arange(T, device="cuda") - cu[seq]
    pages = s["table"].long().clamp(min=0)

    def gathered(codes, scale):  # [N, hkv, keys, D]
        x = _values(codes[pages], fmt) * scale[pages][..., None, None]
        return x.transpose(1, 2).flatten(2, 3)

    qp = torch.zeros(N, Q, hq, D, device="cuda")
    qp[seq, off] = s["q"].float()
    qp = qp.view(N, Q, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(N, hkv, Q * G, D)
    x = torch.matmul(qp, gathered(s["k"].view(torch.uint8), s["k_scale"]).transpose(2, 3))
    x *= s["scale"]
    at = (lens - new)[:, None] + torch.arange(Q, device="cuda")             # a query's position
    key = torch.arange(x.shape[-1], device="cuda")
    seen = (key <= at[..., None]) & (key < lens[:, None, None])
    if c["window"]:
        seen &= key > at[..., None] - c["window"]
    x.masked_fill_(~seen.repeat_interleave(G, 1)[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, gathered(s["v_plain"], s["v_scale"]))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + torch.log(total))[..., 0]

    def rows(y):
        return y.view(N, hkv, Q, G, -1).permute(0, 2, 1, 3, 4).reshape(N, Q, hq, -1)[seq, off]

    return rows(o).to(s["q"].dtype), rows(lse[..., None])[..., 0]


def _own(s):
    from gated_delta_rule_07_gb300 import gdn
    c = s["case"]
    if c["kind"] in ("rope", "rope_grad"):
        more = {"eps": EPS, "weight_offset": c["offset"], "style": c["style"]}
        if c["kind"] == "rope":
            return gdn.qk_norm_rope(s["q"], s["k"], s["pos"], s["table"], s["wq"], s["wk"],
                                    **more)
        return gdn.qk_norm_rope_backward(s["q"], s["k"], s["pos"], s["table"], s["wq"], s["wk"],
                                         s["dqo"], s["dko"], **more)
    if "cache" not in s:  # the handle of the cache's buffers, which a program makes once
        s["cache"] = gdn.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    cache = s["cache"]
    if c["kind"] == "cache":
        gdn.kv_append(cache, s["new_k"], s["new_v"], s["table"], s["ctx"], s["cu"])
        k, v = gdn.kv_read(cache, s["table"], s["start"], s["cu_back"], s["back"], IO[c["io"]])
        return k, v, cache.k_scale, cache.v_scale
    return gdn.kv_attention(cache, s["q"], s["table"], s["lens"], s["cu"], scale=s["scale"],
                            window=c["window"])


def run(state):
    if own:
        return _own(state)
    plain = {"rope": _plain_rope, "rope_grad": _plain_rope_grad, "cache": _plain_cache,
             "attention": _plain_attention}
    return plain[state["case"]["kind"]](state)


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_turned(c, s, x, back):
    """Rows of x times the rotation matrix of each position (or its transpose), as complex
    numbers."""
    R = c["R"]
    t = s["table"].double()[s["pos"].long()][:, None]
    turn = torch.complex(t[..., :R // 2], -t[..., R // 2:] if back else t[..., R // 2:])
    if c["style"] == "half":
        z = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * turn
        head = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(x[..., :R].reshape(*x.shape[:-1], R // 2, 2)) * turn
        head = torch.view_as_real(z).reshape(*x.shape[:-1], R)
    return torch.cat([head, x[..., R:]], -1)


def _exact_rope(c, s):
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x = x.double()
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["D"] + EPS)
        out.append(_exact_turned(c, s, y * (w.double() + c["offset"]), False))
    return tuple(out)


def _exact_rope_grad(c, s):
    dxs, dws = [], []
    for x, w, do in ((s["q"], s["wq"], s["dqo"]), (s["k"], s["wk"], s["dko"])):
        x, w = x.double(), w.double() + c["offset"]
        dy = _exact_turned(c, s, do.double(), True)
        ms = (x * x).sum(-1, keepdim=True) / c["D"] + EPS
        dws.append((dy * x / torch.sqrt(ms)).sum(0).sum(0))
        along = (dy * w * x).sum(-1, keepdim=True)
        dxs.append(dy * w / torch.sqrt(ms) - x * along / (c["D"] * ms * torch.sqrt(ms)))
    return (*dxs, *dws)


def _exact_cache(c, s):
    page, fmt, top = c["page"], c["fmt"], QMAX[c["fmt"]]
    a, b = _lengths(c)
    table = s["table"].tolist()

    def grid(y):
        y = y.clamp(-top, top)
        return y.round() if fmt == "int8" else y.float().to(torch.float8_e4m3fn).double()

    result = []
    for codes, scales, x in ((s["k"].view(torch.uint8), s["k_scale"], s["new_k"]),
                             (s["v_plain"], s["v_scale"], s["new_v"])):
        scales, x, parts, t0 = scales.double(), x.double(), [], 0
        for n, (ctx, new) in enumerate(zip(a, b)):
            p = ctx // page
            while p * page < ctx + new:
                lo, hi = max(p * page, ctx), min((p + 1) * page, ctx + new)
                fresh = x[t0 + lo - ctx:t0 + hi - ctx]                      # [tokens, hkv, D]
                pid, n_old = table[n][p], lo - p * page
                scale = fresh.abs().amax((0, 2)) / top
                old = _values(codes[pid, :, :n_old], fmt).double().transpose(0, 1)
                if n_old:
                    was = scales[pid]
                    scale = torch.maximum(scale, was)
                    old = grid(old * (was / scale)[None, :, None])
                scales[pid] = scale
                both = torch.cat([old, grid(fresh / scale[None, :, None])])
                parts.append(both * scale[None, :, None])
                p += 1
            t0 += new
        result += [torch.cat(parts), scales]
    return result[0], result[2], result[1], result[3]


def _exact_attention(c, s):
    page, fmt, G = c["page"], c["fmt"], c["hq"] // c["hkv"]
    a, b = _lengths(c)
    outs, lses, t0 = [], [], 0
    for n, (length, new) in enumerate(zip(a, b)):
        q = s["q"][t0:t0 + new].double()
        t0 += new
        if length == 0:
            outs.append(torch.zeros_like(q))
            lses.append(torch.full(q.shape[:2], -math.inf, device="cuda", dtype=q.dtype))
            continue
        ids = s["table"][n, :-(-length // page)].long()

        def whole(codes, scale):  # [hkv, keys, D]
            x = _values(codes[ids], fmt).double() * scale[ids].double()[..., None, None]
            return x.transpose(0, 1).flatten(1, 2)[:, :length]

        k = whole(s["k"].view(torch.uint8), s["k_scale"])
        v = whole(s["v_plain"], s["v_scale"])
        x = torch.einsum("ihgd,hkd->ihgk", q.view(new, -1, G, c["D"]), k) * s["scale"]
        at = length - new + torch.arange(new, device="cuda")
        gap = at[:, None] - torch.arange(length, device="cuda")
        hide = (gap < 0) | (gap >= c["window"]) if c["window"] else gap < 0
        x = x.masked_fill(hide[:, None, None], -math.inf)
        lses.append(torch.logsumexp(x, -1).flatten(1))
        outs.append(torch.einsum("ihgk,hkd->ihgd", torch.softmax(x, -1), v).flatten(1, 2))
    return torch.cat(outs), torch.cat(lses)


def exact(case, seed):
    s = prepare(case, seed)
    definition = {"rope": _exact_rope, "rope_grad": _exact_rope_grad, "cache": _exact_cache,
                  "attention": _exact_attention}
    return definition[case["kind"]](case, s)
