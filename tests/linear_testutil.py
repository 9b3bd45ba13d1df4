"""Linear attention with a decay for each head and the 8-bit checkpoints in plain fp64 forms, for the
tests.  Sums over pairs of tokens, straight from o_t = sum_{s <= t} a^(t - s) (q_t . k_s) v_s + a^(t + 1)
q_t h0 and its derivatives; any device."""
import torch

QMAX = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def cumulative(lens, device="cuda"):
    c = torch.zeros(len(lens) + 1, dtype=torch.int32)
    c[1:] = torch.tensor(lens).cumsum(0)
    return c.to(device)


def _power(g, steps):
    """a^steps [hv, ...] for steps >= 0, 0 below; a^0 = 1 whatever a is."""
    g = g.double().view(-1, *([1] * steps.dim()))
    s = steps.double()
    return torch.where(s > 0, torch.exp(g * s.clamp(min=1.0)), (s == 0).double())


def _heads(x, hv):
    return x.double().transpose(0, 1).repeat_interleave(hv // x.shape[1], 0)  # [hv, L, D]


def forward(q, k, v, g, h0, lens):
    """out [T, hv, V], h_final [N, hv, K, V]."""
    hv, outs, ends, t0 = v.shape[1], [], [], 0
    for n, L in enumerate(lens):
        Q, Kk, Vv = (_heads(x[t0:t0 + L], hv) for x in (q, k, v))
        t0 += L
        i = torch.arange(L, device=q.device)
        o = (Q @ Kk.transpose(1, 2) * _power(g, i[:, None] - i)) @ Vv
        h = (Kk * _power(g, L - 1 - i)[..., None]).transpose(1, 2) @ Vv
        if h0 is not None:
            o = o + _power(g, i + 1)[..., None] * (Q @ h0[n].double())
            h = h + _power(g, torch.tensor(L, device=q.device))[:, None, None] * h0[n].double()
        outs.append(o.transpose(0, 1))
        ends.append(h)
    return torch.cat(outs), torch.stack(ends)


def backward(q, k, v, g, do, h0, dh, lens):
    """dq, dk [T, hk, K], dv [T, hv, V], dh0 [N, hv, K, V]."""
    hk, hv, res, t0 = q.shape[1], v.shape[1], [[], [], [], []], 0
    for n, L in enumerate(lens):
        Q, Kk, Vv, Do = (_heads(x[t0:t0 + L], hv) for x in (q, k, v, do))
        t0 += L
        i = torch.arange(L, device=q.device)
        w = _power(g, i[:, None] - i)
        P, dP = Q @ Kk.transpose(1, 2) * w, Do @ Vv.transpose(1, 2) * w
        since, left = _power(g, i + 1)[..., None], _power(g, L - 1 - i)[..., None]
        dq, dk, dv = dP @ Kk, dP.transpose(1, 2) @ Q, P.transpose(1, 2) @ Do
        d0 = (Q * since).transpose(1, 2) @ Do
        if h0 is not None:
            dq = dq + since * (Do @ h0[n].double().transpose(1, 2))
        if dh is not None:
            D = dh[n].double()
            dk = dk + left * (Vv @ D.transpose(1, 2))
            dv = dv + left * (Kk @ D)
            d0 = d0 + _power(g, torch.tensor(L, device=q.device))[:, None, None] * D
        group = lambda x: x.view(hk, hv // hk, L, x.shape[-1]).sum(1).transpose(0, 1)  # noqa: E731
        for r, x in zip(res, (group(dq), group(dk), dv.transpose(0, 1), d0)):
            r.append(x)
    return (*(torch.cat(r) for r in res[:3]), torch.stack(res[3]))


def magnitudes(f, *args):
    """The same sums over absolute values: what roundings inside them are relative to."""
    return f(*(a.abs() if isinstance(a, torch.Tensor) and a.dim() > 1 else a for a in args))


def inner_error(tokens, tensor_cores):
    """What a pass's arithmetic may be off, relative to the sum of its terms' magnitudes.

    fp32: a term is one of at most tokens + 128 added one after another (2^-24 each), times a power of
    the decay whose exponent, x, is off by x 2^-23 (and x e^-x < 1).
    Tensor cores: besides, three operands rounded to fp16 (2^-11 each: the weighted products, the state,
    the weighted sources)."""
    return (tokens + 136) * 2.0 ** -24 + (3 * 2.0 ** -11 if tensor_cores else 0.0)


def assert_close(got, want, magnitude, inner, what=""):
    """Off by the output's rounding, and `inner` of the terms' magnitudes."""
    assert got.shape == want.shape, (got.shape, want.shape)
    g = got.double()
    assert torch.isfinite(g).all(), what
    bound = HALF_STEP[got.dtype] * want.abs() + inner * magnitude * (1 + 2.0 ** -7) + 1e-37
    worst = ((g - want).abs() / bound).max() if g.numel() else torch.tensor(0.0)
    assert worst <= 1.0, f"{what}: {float(worst):.2f} of the bound"


def checkpoint(x, dtype):
    """codes (as fp64 values) and scales of the rows of x, in the definition's fp32."""
    xf = x.float()
    fine = torch.where(torch.isfinite(xf), xf, torch.zeros_like(xf))
    amax = fine.abs().amax(-1)
    top = torch.tensor(QMAX[dtype], device=x.device)
    scale = torch.where(amax >= 2.0 ** -100, amax * (1 / top), torch.zeros_like(amax))
    inv = torch.where(scale > 0, 1 / scale, torch.zeros_like(scale))
    y = fine * inv[..., None]
    y = torch.where(torch.isinf(xf), torch.copysign(top, xf), y).clamp(-top, top)
    y = y.round() if dtype is torch.int8 else y.to(dtype).float()
    return y.double(), scale
