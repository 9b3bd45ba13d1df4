"""GPU: linear attention with a decay for each head (prompts, gradients, single tokens) against plain
fp64 forms."""
import pytest
import torch

import linear_testutil as lt

pytestmark = pytest.mark.gpu
BF16, F32, INF = torch.bfloat16, torch.float32, float("inf")


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_rule_07_gb300 import build
    build.build()
    from gated_delta_rule_07_gb300 import gdn as mod
    assert torch.cuda.is_available()
    return mod


def decays(hv, gen):
    """Slow and fast heads, one that forgets nothing and one that forgets at every token."""
    g = -torch.exp(torch.rand(hv, generator=gen) * 7.2 - 7.2)
    special = [0.0, -INF, -30.0, -1e-4]
    for i in range(min(hv // 2, len(special))):
        g[2 * i + 1] = special[i]
    return g.cuda()


class Case:
    """Inputs on the GPU.  scale: sizes of q, k, v, dout and the states."""

    def __init__(self, lens, hk, hv, K, V, io=BF16, carry=True, wide=False, seed=0,
                 scale=(0.1, 1.0, 1.0, 1e-4)):
        gen = torch.Generator().manual_seed(seed)
        rand = lambda *n: torch.randn(*n, generator=gen)  # noqa: E731
        T, N = sum(lens), len(lens)
        self.lens, self.io, self.shape = lens, io, (hk, hv, K, V)
        # (rows behind the last sequence, which the table leaves out, where `tail` is set)
        if wide:  # one projection: a gap between the heads' parts, and a gate behind
            p = rand(T, 2 * hk * (K + 16) + hv * V * 2).to(io).cuda()
            q, k, v, _ = p.split([hk * (K + 16), hk * (K + 16), hv * V, hv * V], 1)
            self.q = q.view(T, hk, K + 16)[..., :K] if T else q.reshape(T, hk, K + 16)[..., :K]
            self.k = k.view(T, hk, K + 16)[..., 16:] if T else k.reshape(T, hk, K + 16)[..., 16:]
            self.v = v.view(T, hv, V)
        else:
            self.q, self.k = ((rand(T, hk, K) * s).to(io).cuda() for s in scale[:2])
            self.v = (rand(T, hv, V) * scale[2]).to(io).cuda()
        self.g = decays(hv, gen)
        self.cu = lt.cumulative(lens)
        self.do = (rand(T, hv, V) * scale[3]).to(io).cuda()
        s = scale[1] * scale[2]
        self.h0 = (rand(N, hv, K, V) * s).cuda() if carry else None
        self.dh = (rand(N, hv, K, V) * scale[0] * scale[3]).cuda() if carry else None
        self.cores = io is BF16

    def forward(self, gdn, **kw):
        return gdn.linear_attention(self.q, self.k, self.v, self.g, self.h0, self.cu,
                                    check_status=True, **kw)

    def backward(self, gdn, **kw):
        return gdn.linear_attention_backward(self.q, self.k, self.v, self.g, self.do, self.h0,
                                             self.dh, self.cu, check_status=True, **kw)

    def check_forward(self, got):
        args = self.q, self.k, self.v, self.g, self.h0, self.lens
        want, size = lt.forward(*args), lt.magnitudes(lt.forward, *args)
        most = max(self.lens)
        lt.assert_close(got[0], want[0], size[0], lt.inner_error(most, self.cores), "out")
        lt.assert_close(got[1], want[1], size[1], lt.inner_error(most, False), "h_final")

    def check_backward(self, got):
        args = self.q, self.k, self.v, self.g, self.do, self.h0, self.dh, self.lens
        want, size = lt.backward(*args), lt.magnitudes(lt.backward, *args)
        most = max(self.lens)
        for i, name in enumerate(("dq", "dk", "dv", "dh0")):
            lt.assert_close(got[i], want[i], size[i], lt.inner_error(most, self.cores and i < 3),
                            name)


SHAPES = [  # lengths, hk, hv
    ([1], 1, 1), ([64], 1, 2), ([65], 2, 2), ([128, 129, 127], 2, 4), ([300, 0, 1, 77, 0], 2, 6),
    ([0, 0, 5], 3, 3), ([1100, 3, 600], 1, 4), ([2300], 1, 3)]


@pytest.mark.parametrize("io,K,V", [(BF16, 128, 128), (F32, 128, 128), (BF16, 64, 128),
                                    (F32, 128, 64), (BF16, 64, 64), (F32, 64, 64),
                                    (BF16, 128, 64)])
@pytest.mark.parametrize("lens,hk,hv", SHAPES)
def test_prompts(gdn, lens, hk, hv, io, K, V):
    c = Case(lens, hk, hv, K, V, io, carry=len(lens) != 1, seed=len(lens) + hv)
    c.check_forward(c.forward(gdn))


@pytest.mark.parametrize("io,K,V", [(BF16, 128, 128), (F32, 128, 128), (BF16, 64, 128),
                                    (F32, 128, 64), (BF16, 64, 64), (F32, 64, 64),
                                    (BF16, 128, 64)])
@pytest.mark.parametrize("lens,hk,hv", SHAPES)
def test_gradients(gdn, lens, hk, hv, io, K, V):
    c = Case(lens, hk, hv, K, V, io, carry=len(lens) != 1, seed=10 + len(lens) + hv)
    c.check_backward(c.backward(gdn))


@pytest.mark.parametrize("hk,hv", [(4, 12), (12, 12)])
@pytest.mark.parametrize("io,K,V", [(BF16, 128, 128), (F32, 128, 128), (BF16, 64, 128),
                                    (BF16, 128, 64), (BF16, 64, 64)])
def test_walks_of_several_chunks(gdn, io, K, V, hk, hv):
    """So many tokens and heads that a segment is several chunks, and its last one a part of one."""
    c = Case([4000, 33, 2111], hk, hv, K, V, io, seed=hk)
    c.check_forward(c.forward(gdn))
    c.check_backward(c.backward(gdn))


@pytest.mark.parametrize("io", [BF16, F32])
def test_slices_of_one_projection(gdn, io):
    c = Case([130, 61], 2, 4, 128, 128, io, wide=True, seed=3)
    assert not c.q.is_contiguous() and not c.v.is_contiguous()
    c.check_forward(c.forward(gdn))
    c.check_backward(c.backward(gdn))


@pytest.mark.parametrize("scale", [(1e4, 1e4, 1e4, 1e-12), (1e-9, 1e3, 1e-9, 1e6),
                                   (1e-3, 1e-15, 1e12, 1e-3)])
def test_sizes_far_from_one(gdn, scale):
    """bf16 has fp32's range, and what the tensor cores are given has to bear it."""
    c = Case([200, 90], 1, 2, 128, 128, scale=scale, seed=7)
    c.check_forward(c.forward(gdn))
    c.check_backward(c.backward(gdn))


def test_rows_of_very_different_sizes(gdn):
    """One token's key a million times the others', in the middle of a chunk: the others' own outputs
    keep their accuracy relative to the terms that they see."""
    c = Case([256], 1, 2, 128, 128, carry=False, seed=8)
    c.k[100] *= 2.0 ** 12
    c.v[30] *= 2.0 ** 12
    c.check_forward(c.forward(gdn))
    c.check_backward(c.backward(gdn))


@pytest.mark.parametrize("io", [BF16, F32])
def test_rows_behind_the_last_sequence_are_left(gdn, io):
    c = Case([100, 50, 30], 1, 2, 128, 128, io, seed=5)
    p, lens = _problem(gdn, c, 2), [100, 50]
    cu = lt.cumulative(lens)
    # what stands there may be anything
    for x in (c.q, c.k, c.v, c.do):
        x[150:] = float("nan")
    for n in range(2):
        out = torch.full_like(c.v, 7.0)
        last = torch.empty(2, 2, 128, 128, device="cuda")
        ws = torch.full((gdn.gdn_linear_attention_workspace_size(p),), 255, dtype=torch.uint8,
                        device="cuda")
        gdn.gdn_linear_attention(p, c.q, c.k, c.v, c.g, c.h0[:2].contiguous(), cu, out, last, ws)
        assert (out[150:] == 7).all()
    cut = [x[:150] for x in (c.q, c.k, c.v, c.do)]
    args = (*cut[:3], c.g, c.h0[:2], lens)
    want, size = lt.forward(*args), lt.magnitudes(lt.forward, *args)
    lt.assert_close(out[:150], want[0], size[0], lt.inner_error(100, c.cores))
    lt.assert_close(last, want[1], size[1], lt.inner_error(100, False))
    grads = [torch.full_like(x, 7.0) for x in (c.q, c.k, c.v)]
    dh0 = torch.empty_like(last)
    ws = torch.full((gdn.gdn_linear_attention_backward_workspace_size(p),), 255, dtype=torch.uint8,
                    device="cuda")
    gdn.gdn_linear_attention_backward(p, c.q, c.k, c.v, None, c.g, c.h0[:2].contiguous(), cu, c.do,
                                      c.dh[:2].contiguous(), *grads, dh0, ws)
    args = (*cut[:3], c.g, cut[3], c.h0[:2], c.dh[:2], lens)
    want, size = lt.backward(*args), lt.magnitudes(lt.backward, *args)
    for i, x in enumerate((*grads, dh0)):
        if i < 3:
            assert (x[150:] == 7).all()
            x = x[:150]
        lt.assert_close(x, want[i], size[i], lt.inner_error(100, c.cores and i < 3))


def _problem(gdn, c, N):
    T, (hk, hv, K, V) = c.q.shape[0], c.shape
    return gdn.LinearProblem(T, N, hk, hv, K, V, gdn._IO[c.io], *c.q.stride()[:2], *c.k.stride()[:2],
                             *c.v.stride()[:2])


@pytest.mark.parametrize("io", [BF16, F32])
def test_a_neighbours_infinities_stay_its_own(gdn, io):
    """Sequences that share a chunk's rows: what is not finite in one leaves the others alone."""
    c = Case([40, 30, 50], 1, 2, 128, 128, io, seed=6)
    for x, bad in ((c.q, INF), (c.k, float("nan")), (c.v, -INF), (c.do, float("nan"))):
        x[40:70] = bad
    out, last = c.forward(gdn)
    grads = c.backward(gdn)
    for n, rows in ((0, slice(0, 40)), (2, slice(70, 120))):
        cut = [x[rows] for x in (c.q, c.k, c.v, c.do)]
        h0, dh, L = c.h0[n:n + 1], c.dh[n:n + 1], [rows.stop - rows.start]
        args = (*cut[:3], c.g, h0, L)
        want, size = lt.forward(*args), lt.magnitudes(lt.forward, *args)
        lt.assert_close(out[rows], want[0], size[0], lt.inner_error(50, c.cores), "out")
        lt.assert_close(last[n:n + 1], want[1], size[1], lt.inner_error(50, False), "h_final")
        args = (*cut[:3], c.g, cut[3], h0, dh, L)
        want, size = lt.backward(*args), lt.magnitudes(lt.backward, *args)
        for i in range(4):
            x = grads[i][rows] if i < 3 else grads[i][n:n + 1]
            lt.assert_close(x, want[i], size[i], lt.inner_error(50, c.cores and i < 3), str(i))


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("which,bad", [("k", INF), ("v", -INF), ("v", float("nan")), ("q", INF)])
def test_what_is_not_finite_stays_behind(gdn, io, which, bad):
    """A value that is not finite leaves the outputs alone that lie 128 tokens before it or more.  (As many
    heads as SMs, so that a segment has several chunks.)"""
    c = Case([1000], 1, 152, 128, 128, io, seed=13)
    x = getattr(c, which)
    x[700, -1, 5] = bad
    out, _ = c.forward(gdn)
    cut = 700 - 127
    args = (c.q[:cut], c.k[:cut], c.v[:cut], c.g, c.h0, [cut])
    want, size = lt.forward(*args), lt.magnitudes(lt.forward, *args)
    lt.assert_close(out[:cut], want[0], size[0], lt.inner_error(cut, c.cores), "out")
    assert not torch.isfinite(out[700, -1]).all()


@pytest.mark.parametrize("io", [BF16, F32])
def test_what_passes_the_range_is_not_finite(gdn, io):
    """Products beyond fp32's range are not lost without a sign of it (each output here is 2^150 or more)."""
    q, v = torch.full((300, 1, 128), 2.0 ** 50, dtype=io, device="cuda"), None
    v = q.repeat(1, 2, 1)
    g = torch.tensor([0.0, -0.1], device="cuda")
    out, _ = gdn.linear_attention(q, q, v, g, check_status=True)
    assert not torch.isfinite(out).any()
    for x in gdn.linear_attention_backward(q, q, v, g, v, check_status=True)[:3]:
        assert not torch.isfinite(x).any()


@pytest.mark.parametrize("io,K,V", [(BF16, 128, 128), (F32, 64, 128)])
def test_pieces_continue(gdn, io, K, V):
    """A sequence in one call, and in pieces that carry its state (which may be updated in place)."""
    c = Case([517], 2, 4, K, V, io, seed=9)
    whole = c.forward(gdn)
    state, outs = c.h0.clone(), []
    p = _problem(gdn, c, 1)
    for b, e in ((0, 1), (1, 130), (130, 389), (389, 517)):
        out = torch.empty_like(c.v[b:e])
        p.total_tokens = e - b
        ws = torch.empty(gdn.gdn_linear_attention_workspace_size(p), dtype=torch.uint8, device="cuda")
        gdn.gdn_linear_attention(p, c.q[b:e], c.k[b:e], c.v[b:e], c.g, state, None, out, state, ws)
        outs.append(out)
    c.check_forward((torch.cat(outs), state))
    c.check_forward(whole)


@pytest.mark.parametrize("bad", ["table falls", "starts late", "ends late", "decay above 0",
                                 "decay NaN"])
@pytest.mark.parametrize("io", [BF16, F32])
def test_bad_tables_and_decays_write_nothing(gdn, bad, io):
    c = Case([100, 50, 30], 1, 2, 128, 128, io, seed=5)
    if bad == "table falls":
        c.cu[2] = 90
    elif bad == "starts late":
        c.cu[0] = 1
    elif bad == "ends late":
        c.cu[3] = 181
    else:
        c.g[1] = 0.01 if bad == "decay above 0" else float("nan")
    p, st = _problem(gdn, c, 3), torch.zeros(1, dtype=torch.int32, device="cuda")
    out, last = torch.full_like(c.v, 7.0), torch.full_like(c.h0, 7.0)
    ws = torch.empty(gdn.gdn_linear_attention_backward_workspace_size(p), dtype=torch.uint8,
                     device="cuda")
    gdn.gdn_linear_attention(p, c.q, c.k, c.v, c.g, c.h0, c.cu, out, last, ws, dev_status=st)
    assert gdn.gdn_device_status(st) == 6
    grads = [torch.full_like(x, 7.0) for x in (c.q, c.k, c.v, c.h0)]
    gdn.gdn_linear_attention_backward(p, c.q, c.k, c.v, None, c.g, c.h0, c.cu, c.do, c.dh, *grads,
                                      ws, dev_status=st)
    assert gdn.gdn_device_status(st) == 6
    assert all((x == 7).all() for x in (out, last, *grads))
    with pytest.raises(gdn.GdnError, match="DEVICE_INPUT"):
        c.forward(gdn)


@pytest.mark.parametrize("io", [BF16, F32])
def test_many_sequences(gdn, io):
    """More than the blocks look at themselves; and a bad table among so many."""
    gen = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 5, (700,), generator=gen).tolist()
    lens[350] = 300
    c = Case(lens, 1, 2, 64, 64, io, seed=4)
    c.check_forward(c.forward(gdn))
    c.check_backward(c.backward(gdn))
    c.cu[600] = c.cu[-1] + 1
    p, st = _problem(gdn, c, 700), torch.zeros(1, dtype=torch.int32, device="cuda")
    out, last = torch.full_like(c.v, 7.0), torch.full_like(c.h0, 7.0)
    ws = torch.full((gdn.gdn_linear_attention_workspace_size(p),), 255, dtype=torch.uint8, device="cuda")
    gdn.gdn_linear_attention(p, c.q, c.k, c.v, c.g, c.h0, c.cu, out, last, ws, dev_status=st)
    assert gdn.gdn_device_status(st) == 6
    assert (out == 7).all() and (last == 7).all()


def test_no_tokens(gdn):
    for io in (BF16, F32):
        c = Case([0, 0], 1, 2, 128, 64, io, seed=1)
        out, last = c.forward(gdn)
        assert out.shape == (0, 2, 64) and torch.equal(last, c.h0)
        dq, dk, dv, dh0 = c.backward(gdn)
        assert dq.shape == (0, 1, 128) and torch.equal(dh0, c.dh)
        c.h0 = c.dh = None
        assert (c.forward(gdn)[1] == 0).all() and (c.backward(gdn)[3] == 0).all()


@pytest.mark.parametrize("io,K,V", [(BF16, 128, 128), (F32, 64, 64)])
def test_the_same_bits_again_and_in_a_graph(gdn, io, K, V):
    c = Case([700, 33, 140], 2, 6, K, V, io, seed=12)
    first = [*c.forward(gdn), *c.backward(gdn)]
    call = lambda: [  # noqa: E731
        *gdn.linear_attention(c.q, c.k, c.v, c.g, c.h0, c.cu),
        *gdn.linear_attention_backward(c.q, c.k, c.v, c.g, c.do, c.h0, c.dh, c.cu)]
    assert all(torch.equal(a, b) for a, b in zip(first, call()))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = call()
    c2 = Case([700, 33, 140], 2, 6, K, V, io, seed=13)
    for name in ("q", "k", "v", "do", "h0", "dh", "g"):
        getattr(c, name).copy_(getattr(c2, name))
    graph.replay()
    again = [*c2.forward(gdn), *c2.backward(gdn)]
    assert all(torch.equal(a, b) for a, b in zip(again, kept))


def test_a_graph_with_another_table(gdn):
    """A padded batch: the table of a captured call changes between replays."""
    c = Case([200, 56], 1, 2, 128, 128, seed=14)
    out = None
    with torch.cuda.stream(torch.cuda.Stream()):
        gdn.linear_attention(c.q, c.k, c.v, c.g, c.h0, c.cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, last = gdn.linear_attention(c.q, c.k, c.v, c.g, c.h0, c.cu)
    for lens in ([1, 200], [0, 256], [130, 0]):
        c.cu.copy_(lt.cumulative(lens))
        graph.replay()
        T = sum(lens)
        c.lens = lens
        args = c.q[:T], c.k[:T], c.v[:T], c.g, c.h0, lens
        want, size = lt.forward(*args), lt.magnitudes(lt.forward, *args)
        lt.assert_close(out[:T], want[0], size[0], lt.inner_error(256, c.cores))
        lt.assert_close(last, want[1], size[1], lt.inner_error(256, False))


# ------------------------------------------------------------------------------- single tokens

@pytest.mark.parametrize("io,K,V", [(BF16, 128, 128), (F32, 64, 128), (BF16, 128, 64),
                                    (F32, 64, 64)])
@pytest.mark.parametrize("B,hk,hv,wide", [(1, 1, 1, False), (5, 2, 6, True), (37, 4, 4, False)])
def test_steps(gdn, B, hk, hv, wide, io, K, V):
    c = Case([B], hk, hv, K, V, io, wide=wide, seed=B)
    gen = torch.Generator().manual_seed(B)
    state = torch.randn(B + 3, hv, K, V, generator=gen).cuda()
    slot = torch.randperm(B + 3, generator=gen)[:B].int().cuda()
    if B > 4:
        slot[[0, 3]] = -1
    before = state.clone()
    out = gdn.linear_attention_decode(c.q, c.k, c.v, c.g, slot, state, check_status=True)
    used = set()
    for b, s in enumerate(slot.tolist()):
        if s < 0:
            assert (out[b] == 0).all()
            continue
        used.add(s)
        args = c.q[b:b + 1], c.k[b:b + 1], c.v[b:b + 1], c.g, before[s:s + 1], [1]
        want, size = lt.forward(*args), lt.magnitudes(lt.forward, *args)
        # (fp32: K products and a joint of their sums)
        lt.assert_close(out[b:b + 1], want[0], size[0], lt.inner_error(1, False))
        lt.assert_close(state[s:s + 1], want[1], size[1], 4 * 2.0 ** -24)
    for s in set(range(B + 3)) - used:
        assert torch.equal(state[s], before[s])


def test_steps_skip_bad_slots(gdn):
    c = Case([6], 1, 2, 64, 64, F32, seed=2)
    state = torch.randn(4, 2, 64, 64, generator=torch.Generator().manual_seed(1)).cuda()
    before = state.clone()
    slot = torch.tensor([1, 4, 2, 2, -1, 0], dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(c.v, 7.0)
    p = _problem(gdn, c, 1)
    gdn.gdn_linear_attention_decode(p, 4, c.q, c.k, c.v, c.g, slot, state, out, st)
    assert gdn.gdn_device_status(st) == 6
    assert (out[1:4] == 7).all() and (out[4] == 0).all()
    assert torch.equal(state[2:], before[2:])
    for b, s in ((0, 1), (5, 0)):
        want = lt.forward(c.q[b:b + 1], c.k[b:b + 1], c.v[b:b + 1], c.g, before[s:s + 1], [1])
        assert torch.allclose(out[b:b + 1].double(), want[0], rtol=1e-5, atol=1e-5)
        assert torch.allclose(state[s:s + 1].double(), want[1], rtol=1e-5, atol=1e-5)
    # a head whose decay cannot be is skipped, the others are not
    c.g[1] = float("nan")
    state.copy_(before)
    out.fill_(7.0)
    slot = torch.tensor([0, 1, 2, 3, -1, -1], dtype=torch.int32, device="cuda")
    gdn.gdn_linear_attention_decode(p, 4, c.q, c.k, c.v, c.g, slot, state, out, st)
    assert gdn.gdn_device_status(st) == 6
    assert (out[:4, 1] == 7).all() and torch.equal(state[:, 1], before[:, 1])
    assert not torch.equal(state[:, 0], before[:, 0])


@pytest.mark.parametrize("io", [BF16, F32])
def test_steps_continue_a_prompt(gdn, io):
    """A prompt, then single tokens; against one call over all of it."""
    c = Case([90], 2, 4, 128, 128, io, seed=4)
    state = torch.empty(3, 4, 128, 128, device="cuda")
    out, last = gdn.linear_attention(c.q[:70], c.k[:70], c.v[:70], c.g, c.h0)
    state[2] = last[0]
    outs = [out]
    slot = torch.tensor([2], dtype=torch.int32, device="cuda")
    for t in range(70, 90):
        outs.append(gdn.linear_attention_decode(c.q[t:t + 1], c.k[t:t + 1], c.v[t:t + 1], c.g, slot,
                                                state))
    c.check_forward((torch.cat(outs), state[2:]))


def test_offsets_past_32_bits(gdn):
    """A pool of states larger than 2^31 elements, and its last slot."""
    slots, hv = 1100, 130
    c = Case([1], 1, hv, 128, 128, seed=3)
    state = torch.empty(slots, hv, 128, 128, device="cuda")
    assert state.numel() > 2 ** 31
    state[-1].normal_()
    before = state[-1:].clone()
    slot = torch.tensor([slots - 1], dtype=torch.int32, device="cuda")
    out = gdn.linear_attention_decode(c.q, c.k, c.v, c.g, slot, state, check_status=True)
    args = c.q, c.k, c.v, c.g, before, [1]
    want, size = lt.forward(*args), lt.magnitudes(lt.forward, *args)
    lt.assert_close(out, want[0], size[0], lt.inner_error(1, False))
    lt.assert_close(state[-1:], want[1], size[1], 4 * 2.0 ** -24)


@pytest.mark.parametrize("io,T", [(BF16, 530000), (F32, 530000)])
def test_rows_past_32_bits(gdn, io, T):
    """Values and outputs of more than 2^31 elements: the last sequence's rows and gradients."""
    hv, L = 32, 500
    gen = torch.Generator("cuda").manual_seed(5)
    rand = lambda *n: torch.randn(*n, device="cuda", generator=gen, dtype=io)  # noqa: E731
    q, k, v, do = rand(T, 2, 128), rand(T, 2, 128), rand(T, hv, 128), rand(T, hv, 128)
    assert v.numel() > 2 ** 31
    g = decays(hv, torch.Generator().manual_seed(1))
    cu = torch.tensor([0, T - L, T], dtype=torch.int32, device="cuda")
    cut = [x[T - L:] for x in (q, k, v, do)]
    out, last = gdn.linear_attention(q, k, v, g, None, cu, check_status=True)
    args = (*cut[:3], g, None, [L])
    want, size = lt.forward(*args), lt.magnitudes(lt.forward, *args)
    lt.assert_close(out[T - L:], want[0], size[0], lt.inner_error(L, io is BF16), "out")
    lt.assert_close(last[1:], want[1], size[1], lt.inner_error(L, False), "h_final")
    del out
    grads = gdn.linear_attention_backward(q, k, v, g, do, None, None, cu, check_status=True)
    args = (*cut[:3], g, cut[3], None, None, [L])
    want, size = lt.backward(*args), lt.magnitudes(lt.backward, *args)
    for i, name in enumerate(("dq", "dk", "dv")):
        lt.assert_close(grads[i][T - L:], want[i], size[i], lt.inner_error(L, io is BF16), name)


# ------------------------------------------------------------------------------- what is refused

def test_refusals_of_gpu_tensors(gdn):
    c = Case([20, 10], 2, 4, 128, 128, seed=2)
    ok = dict(q=c.q, k=c.k, v=c.v, g=c.g, h0=c.h0, cu=c.cu)
    call = lambda **kw: (lambda a: gdn.linear_attention(  # noqa: E731
        a["q"], a["k"], a["v"], a["g"], a["h0"], a["cu"]))({**ok, **kw})
    call()
    for kw in (dict(k=c.k[:10]), dict(k=c.k[:, :1]), dict(v=c.v[:10]), dict(v=c.v.float()),
               dict(v=c.v[:, :3]), dict(q=c.q.transpose(1, 2)), dict(g=c.g[:3]),
               dict(g=c.g.double()), dict(h0=c.h0[:1]), dict(h0=c.h0.transpose(2, 3)),
               dict(cu=c.cu[:1]), dict(cu=c.cu.long()), dict(cu=c.cu.cpu()), dict(cu=c.cu[:2]),
               dict(q=c.q[..., :96], k=c.k[..., :96]), dict(q=c.q.half()),
               dict(q=torch.empty(30, 2, 132, device="cuda").to(BF16)[..., 4:])):
        with pytest.raises(gdn.GdnError):
            call(**kw)
    with pytest.raises(gdn.GdnError):
        gdn.linear_attention_backward(c.q, c.k, c.v, c.g, c.do.transpose(0, 1), c.h0, c.dh, c.cu)
    with pytest.raises(gdn.GdnError):
        gdn.linear_attention_backward(c.q, c.k, c.v, c.g, c.do, c.h0, c.dh[:1], c.cu)
    with pytest.raises(gdn.GdnError, match="WORKSPACE"):
        gdn.linear_attention(c.q, c.k, c.v, c.g, workspace=torch.empty(
            64, dtype=torch.uint8, device="cuda"))
    state = torch.zeros(4, 4, 128, 128, device="cuda")
    slot = torch.zeros(30, dtype=torch.int32, device="cuda")
    for kw in (dict(slot=slot[:3]), dict(slot=slot.long()), dict(state=state[:, :3]),
               dict(state=state.transpose(2, 3)), dict(state=state.half())):
        a = {**dict(slot=slot, state=state), **kw}
        with pytest.raises(gdn.GdnError):
            gdn.linear_attention_decode(c.q, c.k, c.v, c.g, a["slot"], a["state"])
