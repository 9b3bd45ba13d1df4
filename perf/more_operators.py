"""Cases that time and check linear attention with a decay for each head, and 8-bit checkpoints.

Linear attention whose state decays by a constant of the head is the plain relative of the gated
delta rule (no gates, no correction of what a key held before): per value head,

    h_t = e^g h_{t-1} + k_t v_t^T,        o_t = h_t^T q_t,        g = log_decay[head] <= 0.

Stacks mix both, and train and serve them over the same packed rows and pools of states:

  prompt      packed sequences in chunks, with the states that they start from and leave
  grad        the gradients of that pass: of q, k, v and the starting states, from activations as
              they are or from their 8-bit checkpoints
  step        one token of each request over a pool of state slots
  checkpoint  activations held in 8 bits from the forward to the backward pass (one scale for each
              head's row of a token), opened again

``run`` computes an operator in its plain form, elementary torch operations in 32 bits, or,
where ``own`` is set, through the package's entry points.  ``exact`` computes it from its
definition in 64 bits, token after token.  Lengths of sequences are part of a case (drawn from its
``mix``), values come from the seed.
"""
import math
import random

import torch

own = False

C = 256                     # chunk of the plain form
TINY = 2.0 ** -100          # a row whose values are all below this is held as zeros
QMAX = {"int8": 127.0, "e4m3": 448.0}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
IO = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- the cases

def _pass(name, kind, N, L, hk, hv, K, V, io="bf16", spread="even", carry=True, held="",
          wide=False, mix=1):
    """N sequences of up to L tokens.  carry: they continue from states (and gradients of the
    states that they leave come back); held: the backward reads 8-bit checkpoints of this format;
    wide: q, k and v are slices of one projection."""
    return {"name": name, "kind": kind, "N": N, "L": L, "hk": hk, "hv": hv, "K": K, "V": V,
            "io": io, "spread": spread, "carry": carry, "held": held, "wide": wide, "mix": mix}


def _step(name, B, slots, hk, hv, K, V, io="bf16", pad=0):
    return {"name": name, "kind": "step", "B": B, "slots": slots, "hk": hk, "hv": hv, "K": K,
            "V": V, "io": io, "pad": pad}


def _checkpoint(name, T, hk, hv, K, V, fmt="int8", io="bf16", wide=False):
    return {"name": name, "kind": "checkpoint", "T": T, "hk": hk, "hv": hv, "K": K, "V": V,
            "fmt": fmt, "io": io, "wide": wide}


def listed():
    return [
        # one long document, the workload that the recurrent layers are benchmarked on
        _pass("prompt 65536", "prompt", 1, 65536, 16, 32, 128, 128, spread="whole", carry=False),
        # packed prompts of mixed lengths, continuing from states, read from one projection
        _pass("prompts 8x16384 ragged", "prompt", 8, 16384, 16, 32, 128, 128, spread="ragged",
              wide=True, mix=31),
        # one short chunk of a prompt: latency
        _pass("prompt 300", "prompt", 1, 300, 4, 4, 128, 128, spread="whole", mix=32),
        # fp32, an odd number of heads, key heads narrower than value heads
        _pass("prompts fp32 5x900", "prompt", 5, 900, 3, 6, 64, 128, "f32", mix=33),
        # a training step over packed documents, activations kept as they are
        _pass("grad 16384", "grad", 1, 16384, 16, 32, 128, 128, spread="whole", carry=False),
        # the same kind of step from 8-bit checkpoints, no shared heads, states carried between steps
        _pass("grad 8x4096 from int8", "grad", 8, 4096, 8, 8, 128, 128, held="int8", mix=34),
        # small fp32 gradients, ragged, from checkpoints in 8-bit floating point
        _pass("grad fp32 4x500 from e4m3", "grad", 4, 500, 2, 6, 128, 64, "f32", "ragged",
              held="e4m3", mix=35),
        # a serving batch's step over its pool of states (512 MiB, as the recurrent layers' step)
        _step("step 256", 256, 256, 16, 32, 128, 128),
        # a few requests, with padding rows: latency
        _step("step 5 fp32", 5, 40, 2, 6, 64, 128, "f32", pad=2),
        # q, k and v of a training step held in 8 bits and opened again
        _checkpoint("checkpoint 32768", 32768, 16, 32, 128, 128),
        # a small odd one: 8-bit floating point, fp32 activations, slices of a projection
        _checkpoint("checkpoint e4m3 fp32 777", 777, 3, 9, 64, 128, "e4m3", "f32", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["prompt", "prompt", "grad", "grad", "step", "checkpoint"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    K, V = rng.choice([(128, 128), (128, 128), (128, 128), (64, 64), (128, 64), (64, 128)])
    hk = rng.choice([1, 2, 3, 4, 8, 16])
    hv = hk * rng.choice([g for g in (1, 1, 2, 3, 4) if g * hk <= 32])
    if kind == "step":
        B = _log(rng, 1, 256)
        c = _step("", B, B + rng.choice([0, 3, 17]), hk, hv, K, V, io, rng.choice([0, 0, B // 4]))
    elif kind == "checkpoint":
        c = _checkpoint("", _log(rng, 1, 32768 // (2 if io == "f32" else 1)), hk, hv, K, V,
                        rng.choice(["int8", "e4m3"]), io, rng.random() < 0.5)
    else:
        most = 65536 if kind == "prompt" else 16384
        if io == "f32":
            most //= 8
        N = _log(rng, 1, 16)
        c = _pass("", kind, N, _log(rng, 1, most // N), hk, hv, K, V, io,
                  rng.choice(["even", "ragged"]), rng.random() < 0.6,
                  rng.choice(["", "int8", "e4m3"]) if kind == "grad" else "",
                  rng.random() < 0.4, rng.randrange(1 << 30))
    c.pop("name")
    return c


def _lengths(case):
    r = random.Random(case["mix"])
    lens = []
    for _ in range(case["N"]):
        if case["spread"] == "whole":
            n = case["L"]
        elif case["spread"] == "even":
            n = r.randint(max(1, 3 * case["L"] // 4), case["L"])
        else:
            n = 0 if r.random() < 0.06 else _log(r, 1, case["L"])
        lens.append(n)
    if sum(lens) == 0:
        lens[0] = case["L"]
    return lens


def _itemsize(case):
    return 2 if case["io"] == "bf16" else 4


def work(case):
    e, hk, hv, K, V = _itemsize(case), case["hk"], case["hv"], case["K"], case["V"]
    state = hv * K * V * 4
    if case["kind"] == "step":
        rows = case["B"] - case["pad"]
        return {"bytes": rows * (2 * state + (2 * hk * K + 2 * hv * V) * e),
                "flops": rows * hv * K * V * 4}
    keys, values = 2 * hk * K, hv * V            # elements a token
    if case["kind"] == "checkpoint":
        n, rows = case["T"] * (keys + values), case["T"] * (2 * hk + hv)
        return {"bytes": 2 * n * e + 2 * (n + 4 * rows), "flops": 4 * n}
    T, N = sum(_lengths(case)), case["N"]
    ends = (2 if case["carry"] else 1) * N * state
    if case["kind"] == "prompt":
        return {"bytes": T * (keys + 2 * values) * e + ends, "flops": 4 * T * hv * K * V}
    read = (keys + values) * (1 if case["held"] else e) + values * e
    if case["held"]:
        read += 4 * (2 * hk + hv)
    return {"bytes": T * (read + (keys + values) * e) + (3 if case["carry"] else 1) * N * state,
            "flops": 10 * T * hv * K * V}


# ------------------------------------------------------------------------------ the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _qkv(case, T, gen):
    """q, k [T, hk, K] and v [T, hv, V]: rows of their own, or slices of one projection's rows (an
    output gate stands behind them there)."""
    io, hk, hv, K, V = IO[case["io"]], case["hk"], case["hv"], case["K"], case["V"]
    if not case.get("wide"):
        return ((_randn(gen, T, hk, K) * K ** -0.5).to(io), _randn(gen, T, hk, K).to(io),
                _randn(gen, T, hv, V).to(io))
    p = _randn(gen, T, 2 * hk * K + 2 * hv * V)
    p[:, :hk * K] *= K ** -0.5
    q, k, v, _ = p.to(io).split([hk * K, hk * K, hv * V, hv * V], 1)
    return q.view(T, hk, K), k.view(T, hk, K), v.view(T, hv, V)


def _store(x, fmt):
    """Codes of the rows of x, and each row's scale."""
    xf = x.float()
    amax = xf.abs().amax(-1)
    scale = torch.where(amax >= TINY, amax * (1.0 / QMAX[fmt]), torch.zeros_like(amax))
    y = xf * torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))[..., None]
    y = y.clamp_(-QMAX[fmt], QMAX[fmt])
    return (y.round_().to(torch.int8) if fmt == "int8" else y.to(CODES[fmt])), scale


def prepare(case, seed):
    gen, io = _gen(seed), IO[case["io"]]
    hk, hv, K, V = case["hk"], case["hv"], case["K"], case["V"]
    s = {"case": dict(case)}
    # half-lives from under a token to a thousand tokens, as fixed slopes spread them over heads
    s["g"] = -torch.exp(torch.rand(hv, device="cuda", generator=gen) * math.log(1000.0)
                        + math.log(7e-4))
    if case["kind"] == "step":
        B, S = case["B"], case["slots"]
        s["q"], s["k"], s["v"] = _qkv(case, B, gen)
        s["state"] = _randn(gen, S, hv, K, V)
        order = torch.rand(S, device="cuda", generator=gen).argsort()[:B]
        order[:case["pad"]] = -1
        s["slot"] = order[torch.rand(B, device="cuda", generator=gen).argsort()].int()
        return s
    if case["kind"] == "checkpoint":
        s["q"], s["k"], s["v"] = _qkv(case, case["T"], gen)
        return s
    lens = _lengths(case)
    T, cu = sum(lens), [0]
    for n in lens:
        cu.append(cu[-1] + n)
    s.update(cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), T=T, most=max(lens))
    s["q"], s["k"], s["v"] = _qkv(case, T, gen)
    s["h0"] = _randn(gen, case["N"], hv, K, V) if case["carry"] else None
    if case["kind"] == "grad":
        # a mean over the tokens' losses makes these small
        s["dout"] = (_randn(gen, T, hv, V) * 1e-5).to(io)
        s["dh"] = _randn(gen, case["N"], hv, K, V) * 1e-5 if case["carry"] else None
        if case["held"]:
            s["held"] = [_store(s.pop(n), case["held"]) for n in ("q", "k", "v")]
    return s


# ------------------------------------------------------------------------------ plain forms

def _open(codes, scale, io):
    return (codes.float() * scale[..., None]).to(io)


def _activations(s):
    if "held" in s:
        return [_open(*h, IO[s["case"]["io"]]) for h in s["held"]]
    return s["q"], s["k"], s["v"]


class _Rows:
    """Packed rows [T, heads, D] laid out as [N, hv, chunks, C, D] in fp32, and back."""

    def __init__(self, s):
        c, cu = s["case"], s["cu"].long()
        self.N, self.hv, self.nc = c["N"], c["hv"], max(1, -(-s["most"] // C))
        self.lens = cu[1:] - cu[:-1]
        self.seq = torch.repeat_interleave(torch.arange(self.N, device="cuda"), self.lens,
                                           output_size=s["T"])
        self.off = torch.arange(s["T"], device="cuda") - cu[self.seq]
        at = torch.arange(self.nc * C, device="cuda")
        self.left = (self.lens[:, None] - 1 - at).view(self.N, 1, self.nc, C)  # tokens behind it
        g = s["g"].double()[:, None]
        i = torch.arange(C, device="cuda")
        self.grown = torch.exp(g * (i + 1)).float()[:, None, :, None]
        self.to_end = torch.exp(g * (C - 1 - i)).float()[:, None, :, None]
        gap = i[:, None] - i
        self.within = torch.where(gap >= 0, torch.exp(g[..., None] * gap.clamp(min=0)), 0.0)
        self.within = self.within.float()[:, None]
        j = torch.arange(self.nc, device="cuda")
        before = j[:, None] - 1 - j
        self.between = torch.where(before >= 0, torch.exp(g[..., None] * C * before.clamp(min=0)),
                                   0.0).float()
        self.from_start = torch.exp(g * C * j).float()[None, :, :, None, None]
        self.at_end = torch.where(self.left >= 0, torch.exp(
            g[None, :, None] * self.left.clamp(min=0)), 0.0).float()[..., None]
        self.since = torch.exp(g * (at + 1)).float().view(1, self.hv, self.nc, C, 1)
        self.whole = torch.exp(g * self.lens).t().float()[..., None, None]

    def take(self, x):
        y = torch.zeros(self.N, self.nc * C, x.shape[1], x.shape[2], device="cuda")
        y[self.seq, self.off] = x.float()
        y = y.transpose(1, 2).reshape(self.N, x.shape[1], self.nc, C, x.shape[2])
        return y.repeat_interleave(self.hv // x.shape[1], 1)

    def give(self, y, heads=None):
        y = y.reshape(self.N, self.hv, self.nc * C, y.shape[-1])
        if heads and heads != self.hv:
            y = y.view(self.N, heads, self.hv // heads, *y.shape[2:]).sum(2)
        return y.transpose(1, 2)[self.seq, self.off]

    def entering(self, k, v, h0):
        """The state that enters each chunk."""
        add = torch.matmul((k * self.to_end).transpose(3, 4), v)
        h = torch.einsum("hcd,nhdkv->nhckv", self.between, add)
        return h if h0 is None else h + self.from_start * h0[:, :, None]


def _plain_prompt(s):
    r, (q, k, v) = _Rows(s), _activations(s)
    io = q.dtype
    q, k, v = r.take(q), r.take(k), r.take(v)
    out = torch.matmul(torch.matmul(q, k.transpose(3, 4)) * r.within, v)
    out += torch.matmul(q * r.grown, r.entering(k, v, s["h0"]))
    last = torch.matmul((k * r.at_end).flatten(2, 3).transpose(2, 3), v.flatten(2, 3))
    if s["h0"] is not None:
        last = last + r.whole * s["h0"]
    return r.give(out).to(io), last


def _plain_grad(s):
    r, (q, k, v) = _Rows(s), _activations(s)
    io, hk = q.dtype, q.shape[1]
    q, k, v, do = r.take(q), r.take(k), r.take(v), r.take(s["dout"])
    p = torch.matmul(q, k.transpose(3, 4)) * r.within
    dp = torch.matmul(do, v.transpose(3, 4)) * r.within
    h = r.entering(k, v, s["h0"])
    dq = torch.matmul(dp, k) + torch.matmul(do * r.grown, h.transpose(3, 4))
    # the gradient of the state that leaves each chunk, from the chunks behind it
    d = torch.einsum("hdc,nhdkv->nhckv", r.between,
                     torch.matmul((q * r.grown).transpose(3, 4), do))
    dk = torch.matmul(dp.transpose(3, 4), q) + torch.matmul(v * r.to_end, d.transpose(3, 4))
    dv = torch.matmul(p.transpose(3, 4), do) + torch.matmul(k * r.to_end, d)
    dh0 = torch.matmul((q * r.since).flatten(2, 3).transpose(2, 3), do.flatten(2, 3))
    if s["dh"] is not None:
        dk += torch.matmul(v * r.at_end, s["dh"][:, :, None].transpose(3, 4))
        dv += torch.matmul(k * r.at_end, s["dh"][:, :, None])
        dh0 = dh0 + r.whole * s["dh"]
    return r.give(dq, hk).to(io), r.give(dk, hk).to(io), r.give(dv).to(io), dh0


def _plain_step(s):
    G = s["case"]["hv"] // s["case"]["hk"]
    slot, state = s["slot"].long(), s["state"]
    live = (slot >= 0)[:, None, None]
    at = slot.clamp(min=0)
    q, k = (s[n].float().repeat_interleave(G, 1) for n in ("q", "k"))
    h = state[at] * torch.exp(s["g"])[:, None, None] + k[..., None] * s["v"].float()[:, :, None]
    out = torch.where(live, (h * q[..., None]).sum(2), 0.0)
    # (a padding row writes nothing: its rows go to a spare slot)
    spare = torch.cat([state, torch.empty_like(state[:1])])
    spare[torch.where(slot >= 0, slot, state.shape[0])] = h
    state.copy_(spare[:-1])
    return out.to(s["v"].dtype), state


def _plain_checkpoint(s):
    held = [_store(s[n], s["case"]["fmt"]) for n in ("q", "k", "v")]
    return [_open(*h, IO[s["case"]["io"]]) for h in held] + [h[1] for h in held]


def _own(s):
    from gated_delta_rule_07_gb300 import gdn
    c = s["case"]
    if c["kind"] == "prompt":
        return gdn.linear_attention(s["q"], s["k"], s["v"], s["g"], s["h0"], s["cu"])
    if c["kind"] == "step":
        out = gdn.linear_attention_decode(s["q"], s["k"], s["v"], s["g"], s["slot"], s["state"])
        return out, s["state"]
    if c["kind"] == "checkpoint":
        held = gdn.checkpoint_pack(s["q"], s["k"], s["v"], dtype=CODES[c["fmt"]])
        return [*gdn.checkpoint_open(*held), *(h.scale for h in held)]
    if "held" in s:
        q, k, v = (gdn.Checkpoint(*h, IO[c["io"]]) for h in s["held"])
    else:
        q, k, v = s["q"], s["k"], s["v"]
    return gdn.linear_attention_backward(q, k, v, s["g"], s["dout"], s["h0"], s["dh"], s["cu"])


def run(state):
    if own:
        return _own(state)
    plain = {"prompt": _plain_prompt, "grad": _plain_grad, "step": _plain_step,
             "checkpoint": _plain_checkpoint}
    return plain[state["case"]["kind"]](state)


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_heads(s, n, lo, hi, x):
    """Rows lo .. hi of x in 64 bits, one for each value head."""
    y = x[lo:hi].double()
    return y.repeat_interleave(s["case"]["hv"] // y.shape[1], 1)


def _exact_prompt(c, s):
    decay, outs, ends, t0 = torch.exp(s["g"].double())[:, None, None], [], [], 0
    for n, length in enumerate(_lengths(c)):
        q, k, v = (_exact_heads(s, n, t0, t0 + length, s[x]) for x in ("q", "k", "v"))
        t0 += length
        h = torch.zeros(c["hv"], c["K"], c["V"], dtype=torch.float64, device="cuda")
        if s["h0"] is not None:
            h += s["h0"][n]
        out = torch.empty(length, c["hv"], 1, c["V"], dtype=torch.float64, device="cuda")
        q, k, v = q[:, :, None], k[..., None], v[:, :, None]
        for t in range(length):
            h.mul_(decay).addcmul_(k[t], v[t])
            torch.bmm(q[t], h, out=out[t])
        outs.append(out[:, :, 0])
        ends.append(h)
    return torch.cat(outs), torch.stack(ends)


def _exact_grad(c, s):
    decay, t0, hk = torch.exp(s["g"].double())[:, None, None], 0, c["hk"]
    acts = _activations(s)
    all_q, all_k, all_v, all_h = [], [], [], []
    for n, length in enumerate(_lengths(c)):
        q, k, v, do = (_exact_heads(s, n, t0, t0 + length, x) for x in (*acts, s["dout"]))
        t0 += length
        h = torch.zeros(c["hv"], c["K"], c["V"], dtype=torch.float64, device="cuda")
        d = torch.zeros_like(h)
        if s["h0"] is not None:
            h += s["h0"][n]
            d += s["dh"][n]
        dq, dk, dv = (torch.empty_like(x)[..., None] for x in (q, k, v))
        q4, k4, v4, do4 = q[..., None], k[..., None], v[..., None], do[..., None]
        kt, vt, dot = k[:, :, None], v[:, :, None], do[:, :, None]
        for t in range(length):
            h.mul_(decay).addcmul_(k4[t], vt[t])
            torch.bmm(h, do4[t], out=dq[t])
        for t in range(length - 1, -1, -1):   # d: the gradient of the state after token t
            d.addcmul_(q4[t], dot[t])
            torch.bmm(d, v4[t], out=dk[t])
            dv[t] = torch.bmm(kt[t], d).transpose(1, 2)
            d.mul_(decay)
        all_q.append(dq[..., 0].unflatten(1, (hk, -1)).sum(2))
        all_k.append(dk[..., 0].unflatten(1, (hk, -1)).sum(2))
        all_v.append(dv[..., 0])
        all_h.append(d)
    return torch.cat(all_q), torch.cat(all_k), torch.cat(all_v), torch.stack(all_h)


def _exact_step(c, s):
    G, decay = c["hv"] // c["hk"], torch.exp(s["g"].double())[:, None, None]
    state = s["state"].double()
    out = torch.zeros(c["B"], c["hv"], c["V"], dtype=torch.float64, device="cuda")
    for b, slot in enumerate(s["slot"].tolist()):
        if slot >= 0:
            q, k = (s[x][b].double().repeat_interleave(G, 0) for x in ("q", "k"))
            state[slot] = decay * state[slot] + torch.einsum("hk,hv->hkv", k, s["v"][b].double())
            out[b] = torch.einsum("hk,hkv->hv", q, state[slot])
    return out, state


def _exact_checkpoint(c, s):
    # which code a value takes is decided in fp32 by definition (a quotient next to a border has no
    # other answer); what the code stands for is exact
    values, scales = [], []
    top = torch.tensor(QMAX[c["fmt"]], device="cuda")
    for name in ("q", "k", "v"):
        scale = s[name].float().abs().max(-1, keepdim=True).values * top.reciprocal()
        scale = scale.masked_fill(scale * top < TINY, 0.0)
        y = (s[name].float() * scale.reciprocal().masked_fill(scale == 0, 0.0)).clip(-top, top)
        y = y.to(CODES["e4m3"]) if c["fmt"] == "e4m3" else y.double().round()
        values.append(y.double() * scale.double())
        scales.append(scale[..., 0].double())
    return values + scales


def exact(case, seed):
    # token after token takes about 50 us a token and pass over the sequence
    if case["kind"] in ("prompt", "grad"):
        passes = 1 if case["kind"] == "prompt" else 3
        if passes * sum(_lengths(case)) > 200000:
            return None
    s = prepare(case, seed)
    definition = {"prompt": _exact_prompt, "grad": _exact_grad, "step": _exact_step,
                  "checkpoint": _exact_checkpoint}
    return definition[case["kind"]](case, s)
