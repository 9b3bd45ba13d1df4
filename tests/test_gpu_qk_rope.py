"""GPU: query/key norms with the rotation (gdn_qk_norm_rope) and their gradients against fp64.

Tolerances, from the arithmetic (u = 2^-24).  Forward, per element on the scale |a| + |b| of its
pair after norm and weight: the mean square is a sum of at most 13 roundings deep (8 in a lane, 5
shuffles), so r is off by at most 6.5 u + 2 u of rsqrt + 2 u of the mean and eps; weight and norm
add 3 u, the rotation 3 u: 17 u, bounded by 2^-19.  bf16 (8 significant
bits) adds half an ulp of the result, at most 2^-8 of it.
Backward, per element on the scale of the terms it sums: three such factors and another sum over
the row: bounded by 2^-18; bf16 adds 2^-8 of the result.  Weight gradients sum tokens x heads
terms in at most ~(rows of a warp + 320 CTA steps) roundings: 2^-14 of the sum of magnitudes.
"""
import pytest
import torch

import attention_testutil as at

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_rule_07_gb300 import build
    build.build()
    from gated_delta_rule_07_gb300 import gdn as mod
    assert torch.cuda.is_available()
    return mod


def make(T, hq, hkv, D, R, io, gate=False, seed=0, max_pos=4096, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    wide = hq * D * (2 if gate else 1)
    proj = (torch.randn(T, wide + 2 * hkv * D, generator=gen) * std).to(io)
    q = proj[:, :wide].view(T, hq, -1)[:, :, :D]
    k = proj[:, wide:wide + hkv * D].view(T, hkv, D)
    pos = torch.randint(0, max_pos, (T,), generator=gen).int()
    w = 1 + 0.2 * torch.randn(2, D, generator=gen)
    do = torch.randn(T, hq + hkv, D, generator=gen).to(io)
    return proj, q, k, pos, at.table(max_pos, R), w[0], w[1], do[:, :hq].contiguous(), \
        do[:, hq:].contiguous()


def on_gpu(proj, q, k):
    """The same slices of the projection, on the GPU (strides kept)."""
    g = proj.cuda()
    return [g.as_strided(x.shape, x.stride(), x.storage_offset()) for x in (q, k)]


def close(got, ref, mag, rel, io, what):
    got = got.double().cpu()
    tol = rel * mag + (2.0 ** -8 * ref.abs() if io == torch.bfloat16 else 0)
    bad = (got - ref).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), float(((got - ref).abs() - tol).max()))


CASES = [(1, 1, 1, 64, 64), (3, 16, 2, 256, 64), (37, 6, 3, 64, 32), (5, 7, 1, 128, 96),
         (129, 4, 4, 128, 128), (33, 5, 2, 256, 256), (2500, 32, 8, 128, 128), (17, 3, 1, 64, 0),
         (11, 2, 5, 128, 48), (3000, 9, 3, 256, 16)]


@pytest.mark.parametrize("io", at.IOS, ids=at.IO_IDS)
@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("T,hq,hkv,D,R", CASES)
def test_forward_and_gradients(gdn, T, hq, hkv, D, R, style, io):
    offset, gate = (1.0, True) if D == 256 else (0.0, False)
    proj, q, k, pos, tab, wq, wk, dqo, dko = make(T, hq, hkv, D, R, io, gate, seed=T + D)
    wq, wk = wq - offset, wk - offset
    gq, gk = on_gpu(proj, q, k)
    args = (gq, gk, pos.cuda(), tab.cuda(), wq.cuda(), wk.cuda())
    kw = dict(eps=1e-6, weight_offset=offset, style=style, check_status=True)
    outs = gdn.qk_norm_rope(*args, **kw)
    grads = gdn.qk_norm_rope_backward(*args, dqo.cuda(), dko.cuda(), **kw)
    for i, (x, w, do) in enumerate(((q, wq, dqo), (k, wk, dko))):
        ref, mag = at.rope(x, pos, tab, w, 1e-6, offset, style)
        close(outs[i], ref, mag, 2.0 ** -19, io, ("out", i))
        dx, dw, dx_mag, dw_mag = at.rope_grad(x, pos, tab, w, 1e-6, offset, style, do)
        close(grads[i], dx, dx_mag, 2.0 ** -18, io, ("dx", i))
        close(grads[2 + i], dw, dw_mag, 2.0 ** -14, torch.float32, ("dw", i))


def test_without_weights(gdn):
    proj, q, k, pos, tab, *_ = make(9, 4, 2, 128, 64, torch.float32)
    gq, gk = on_gpu(proj, q, k)
    out = gdn.qk_norm_rope(gq, gk, pos.cuda(), tab.cuda())
    for x, o in ((q, out[0]), (k, out[1])):
        ref, mag = at.rope(x, pos, tab, None, 1e-6, 0.0, "half")
        close(o, ref, mag, 2.0 ** -19, torch.float32, "no weights")


def test_small_and_large_rows(gdn):
    """Rows of zeros (r = 1 / sqrt(eps)) and rows near the ends of the fp32 range of squares."""
    proj, q, k, pos, tab, wq, wk, *_ = make(6, 2, 2, 64, 64, torch.float32)
    factor = torch.tensor([0.0, 1e-20, 1e-3, 1e3, 1e17, 1.0])
    proj.mul_(factor[:, None])
    gq, gk = on_gpu(proj, q, k)
    out = gdn.qk_norm_rope(gq, gk, pos.cuda(), tab.cuda(), wq.cuda(), wk.cuda(),
                           check_status=True)
    for x, w, o in ((q, wq, out[0]), (k, wk, out[1])):
        ref, mag = at.rope(x, pos, tab, w, 1e-6, 0.0, "half")
        close(o, ref, mag, 2.0 ** -19, torch.float32, "rows")


def test_bad_positions_are_reported_and_skipped(gdn):
    proj, q, k, pos, tab, wq, wk, dqo, dko = make(8, 2, 1, 128, 64, torch.bfloat16, max_pos=100)
    pos[2], pos[5] = 100, -1
    gq, gk = on_gpu(proj, q, k)
    args = (gq, gk, pos.cuda(), tab.cuda(), wq.cuda(), wk.cuda())
    p = gdn.QkRopeProblem(8, 2, 1, 128, 64, 0, gdn.GDN_BF16, 100, 1e-6, 0.0, *gq.stride()[:2],
                          *gk.stride()[:2])
    qo, ko = torch.full_like(dqo.cuda(), 7.0), torch.full_like(dko.cuda(), 7.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_qk_norm_rope(p, *args, qo, ko, st)
    assert gdn.gdn_device_status(st) == 6
    good = [0, 1, 3, 4, 6, 7]
    assert bool((qo[[2, 5]] == 7).all()) and bool((ko[[2, 5]] == 7).all())
    ref, mag = at.rope(q[good], pos[good], tab, wq, 1e-6, 0.0, "half")
    close(qo[good], ref, mag, 2.0 ** -19, torch.bfloat16, "good rows")
    grads = gdn.qk_norm_rope_backward(*args, dqo.cuda(), dko.cuda())
    _, dw, _, dw_mag = at.rope_grad(q[good], pos[good], tab, wq, 1e-6, 0.0, "half", dqo[good])
    close(grads[2], dw, dw_mag, 2.0 ** -14, torch.float32, "dw of the good rows")


def test_gradients_repeat_bit_for_bit(gdn):
    proj, q, k, pos, tab, wq, wk, dqo, dko = make(3001, 5, 2, 128, 128, torch.bfloat16)
    gq, gk = on_gpu(proj, q, k)
    args = (gq, gk, pos.cuda(), tab.cuda(), wq.cuda(), wk.cuda(), dqo.cuda(), dko.cuda())
    first = gdn.qk_norm_rope_backward(*args)
    for _ in range(3):
        again = gdn.qk_norm_rope_backward(*args)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_no_tokens(gdn):
    e = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    tab = at.table(16, 64).cuda()
    w = torch.ones(128, device="cuda")
    q, k = gdn.qk_norm_rope(e, e, pos, tab, w, w)
    assert q.shape == (0, 4, 128) and k.shape == (0, 4, 128)
    dq, dk, dwq, dwk = gdn.qk_norm_rope_backward(e, e, pos, tab, w, w, e, e)
    assert dq.shape == (0, 4, 128) and not dwq.any() and not dwk.any()


def test_on_another_stream(gdn):
    proj, q, k, pos, tab, wq, wk, *_ = make(700, 8, 2, 128, 128, torch.bfloat16)
    gq, gk = on_gpu(proj, q, k)
    args = (gq, gk, pos.cuda(), tab.cuda(), wq.cuda(), wk.cuda())
    want = gdn.qk_norm_rope(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = gdn.qk_norm_rope(*args, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    do = (torch.randn_like(want[0]), torch.randn_like(want[1]))
    want = gdn.qk_norm_rope_backward(*args, *do)
    s.wait_stream(torch.cuda.current_stream())
    got = gdn.qk_norm_rope_backward(*args, *do, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("io", at.IOS, ids=at.IO_IDS)
@pytest.mark.parametrize("hq,hkv,D", [(3, 1, 64), (5, 6, 64), (3, 1, 128), (2, 1, 256)])
def test_no_eps(gdn, hq, hkv, D, io):
    """eps = 0 with numbers of heads that do not fill a warp's rows."""
    proj, q, k, pos, tab, wq, wk, dqo, dko = make(70, hq, hkv, D, 32, io, seed=D + hq)
    gq, gk = on_gpu(proj, q, k)
    args = (gq, gk, pos.cuda(), tab.cuda(), wq.cuda(), wk.cuda())
    outs = gdn.qk_norm_rope(*args, eps=0.0, check_status=True)
    grads = gdn.qk_norm_rope_backward(*args, dqo.cuda(), dko.cuda(), eps=0.0, check_status=True)
    for i, (x, w, do) in enumerate(((q, wq, dqo), (k, wk, dko))):
        ref, mag = at.rope(x, pos, tab, w, 0.0, 0.0, "half")
        close(outs[i], ref, mag, 2.0 ** -19, io, ("out", i))
        dx, dw, dx_mag, dw_mag = at.rope_grad(x, pos, tab, w, 0.0, 0.0, "half", do)
        assert torch.isfinite(grads[i].float()).all() and torch.isfinite(grads[2 + i]).all()
        close(grads[i], dx, dx_mag, 2.0 ** -18, io, ("dx", i))
        close(grads[2 + i], dw, dw_mag, 2.0 ** -14, torch.float32, ("dw", i))
