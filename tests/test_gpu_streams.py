"""GPU: calls on another stream than torch's current one, while the current one has work pending.

The caller orders the streams for the inputs; what a call allocates or clears inside is its own to
order.  Each test leaves a long spin on the current stream (or on the call's), so that memory which
changes hands too early is seen: by a status word that still holds junk, by outputs that another
tensor's late fill lands in, by temporaries that are filled while the call still uses them.
"""
import pytest
import torch

import attention_testutil as at

pytestmark = pytest.mark.gpu

SPIN = 100_000_000  # clock cycles, about 50 ms


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_rule_07_gb300 import build
    build.build()
    from gated_delta_rule_07_gb300 import gdn as mod
    assert torch.cuda.is_available()
    return mod


class Layer:
    """Inputs of every call of the attention layer, and the calls as functions of them."""

    def __init__(self, gdn, seed=0):
        gen = torch.Generator().manual_seed(seed)
        T, hq, hkv, D, page, held = 37, 8, 2, 128, 16, 21
        rand = lambda *n: torch.randn(*n, generator=gen).bfloat16().cuda()  # noqa: E731
        self.gdn, self.T, self.held = gdn, T, held
        self.q, self.k, self.v = rand(T, hq, D), rand(T, hkv, D), rand(T, hkv, D)
        self.do = rand(T, hq, D), rand(T, hkv, D)
        self.pos = torch.arange(T, dtype=torch.int32).cuda()
        self.tab = at.table(64, 64).cuda()
        self.w = torch.ones(D).cuda()
        self.table = torch.tensor([[3, 0, 2, 5]], dtype=torch.int32).cuda()
        self.start = torch.tensor([held], dtype=torch.int32).cuda()
        self.whole = self.start + T
        kc, ks = at.random_cache(6, hkv, page, D, torch.int8, gen)
        vc, vs = at.random_cache(6, hkv, page, D, torch.int8, gen)
        self.stored = kc.cuda(), at.packed_v(vc).cuda(), ks.cuda(), vs.cuda()
        self.fresh()
        torch.cuda.synchronize()

    def fresh(self):
        self.cache = self.gdn.KVCache(*(t.clone() for t in self.stored))

    def calls(self):
        g = self.gdn
        return {
            "qk_norm_rope": lambda q=None, **kw: g.qk_norm_rope(
                self.q if q is None else q, self.k, self.pos, self.tab, self.w, self.w, **kw),
            "qk_norm_rope_backward": lambda q=None, **kw: g.qk_norm_rope_backward(
                self.q if q is None else q, self.k, self.pos, self.tab, self.w, self.w, *self.do,
                **kw),
            "kv_append": lambda q=None, **kw: g.kv_append(
                self.cache, self.k, self.v, self.table, self.start, **kw),
            "kv_read": lambda q=None, **kw: g.kv_read(
                self.cache, self.table, self.start, None, self.T, **kw),
            "kv_attention": lambda q=None, **kw: g.kv_attention(
                self.cache, self.q if q is None else q, self.table, self.whole, **kw),
        }

    def results(self, out):
        return list(out) if out is not None else [t.clone() for t in (
            self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale)]


class Recurrent:
    """The same for the recurrent layers' calls."""

    def __init__(self, gdn, seed=0):
        gen = torch.Generator().manual_seed(seed)
        T, hk, hv, D, N = 200, 2, 4, 128, 3
        rand = lambda *n: torch.randn(*n, generator=gen).bfloat16().cuda()  # noqa: E731
        self.gdn, self.heads = gdn, (hk, hv, D, D)
        self.q, self.v, self.do = rand(T, hk, D) / 11, rand(T, hv, D), rand(T, hv, D)
        self.k = rand(T, hk, D)
        self.k = (self.k.float() / self.k.float().norm(dim=-1, keepdim=True)).bfloat16()
        self.g = -torch.rand(T, hv, generator=gen).cuda()
        self.beta = torch.rand(T, hv, generator=gen).cuda()
        self.cu = at.cumulative([70, 1, 129]).cuda()
        self.x = rand(T, 2 * hk * D + hv * D)
        self.conv, self.ab = torch.randn(self.x.shape[1], 4, generator=gen).cuda(), rand(T, hv)
        self.log, self.bias = torch.zeros(hv).cuda(), torch.zeros(hv).cuda()
        self.h0 = torch.randn(N, hv, D, D, generator=gen).cuda()
        self.slot = torch.tensor([2, -1, 0], dtype=torch.int32).cuda()
        self.fresh()
        torch.cuda.synchronize()

    def fresh(self):
        self.state = self.h0.clone()

    def calls(self):
        g = self.gdn
        rows = self.q[:3], self.k[:3], self.v[:3], self.g[:3], self.beta[:3]
        return {
            "forward": lambda q=None, **kw: g.forward(
                self.q if q is None else q, self.k, self.v, self.g, self.beta, self.h0, self.cu,
                P=2, **kw),
            "backward": lambda q=None, **kw: g.backward(
                self.q if q is None else q, self.k, self.v, self.g, self.beta, self.do,
                cu_seqlens=self.cu, **kw),
            "prologue": lambda q=None, **kw: g.prologue(
                self.x, self.conv, self.ab, self.ab, self.log, self.bias, *self.heads, None,
                self.cu, **kw),
            "decode": lambda q=None, **kw: (g.decode(
                rows[0] if q is None else q[:3], *rows[1:], self.slot, self.state, **kw),
                self.state),
        }

    def results(self, out):
        return [t.clone() for t in out]


NAMES = ["qk_norm_rope", "qk_norm_rope_backward", "kv_append", "kv_read", "kv_attention"]
MORE = ["forward", "backward", "prologue", "decode"]


def layer_of(gdn, name):
    return Recurrent(gdn) if name in MORE else Layer(gdn)


def same(got, want):
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def small_junk():
    """Blocks of the size of a status word that hold an error code, back in the current stream's
    pool."""
    held = [torch.full((1,), 6, dtype=torch.int32, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("name", NAMES + MORE)
def test_status_word_with_work_pending(gdn, name):
    """The status word is cleared on the call's stream, not behind the current one's work."""
    layer = layer_of(gdn, name)
    want = layer.results(layer.calls()[name]())
    torch.cuda.synchronize()
    layer.fresh()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        small_junk()
        torch.cuda._sleep(SPIN)
        out = layer.calls()[name](check_status=True, stream=stream)
        torch.cuda.synchronize()
        if name not in ("kv_append", "decode") or stream is s:  # (those change what they read)
            same(layer.results(out), want)


def test_recorded_error_is_not_wiped(gdn):
    """With the current stream about to clear memory, an error of the call is still reported."""
    layer = Layer(gdn)
    layer.table[0, 1] = 77  # outside the pool
    layer.pos[3] = -1
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for name in NAMES:
        torch.cuda._sleep(SPIN)
        with pytest.raises(gdn.GdnError) as e:
            layer.calls()[name](check_status=True, stream=s)
        assert e.value.status == 6, name
        torch.cuda.synchronize()


@pytest.mark.parametrize("name", [n for n in NAMES + MORE if n != "kv_append"])
def test_outputs_do_not_take_memory_in_use(gdn, name):
    """Memory that the current stream will still write, freed before the call, is not its output."""
    layer = layer_of(gdn, name)
    want = layer.results(layer.calls()[name]())
    layer.fresh()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(SPIN)
    junk = [torch.empty_like(t) for t in want for _ in range(4)]
    for t in junk:
        t.view(torch.uint8).fill_(0x7f)
    del junk
    out = layer.calls()[name](stream=s)
    torch.cuda.synchronize()
    same(layer.results(out), want)


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", NAMES + MORE)
def test_memory_is_held_until_the_call_is_done(gdn, name, handle):
    """Inputs and temporaries that the host lets go of while the call still waits for its turn are
    not filled by later tensors of the current stream."""
    layer = layer_of(gdn, name)
    want = layer.results(layer.calls()[name]())
    layer.fresh()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    before = torch.cuda.memory_reserved()
    q = layer.q.clone()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(SPIN)
    out = layer.calls()[name](q=q, stream=s.cuda_stream if handle else s)
    del q
    later = []
    for n in (layer.q.numel() * 2, 1 << 20, 2 << 20, 4 << 20):  # (workspaces: a few MB, some more)
        later += [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(4)]
    for n in (16 << 20, 64 << 20, 160 << 20):
        later.append(torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    same(layer.results(out), want)
    assert torch.cuda.memory_reserved() - before < 1 << 30


def test_default_stream_handle(gdn):
    """Handle 0 is the legacy default stream."""
    layer = Layer(gdn)
    want = layer.results(layer.calls()["kv_attention"]())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        out = layer.calls()["kv_attention"](stream=0)
    torch.cuda.synchronize()
    same(layer.results(out), want)


def test_refusals_on_a_stream_are_the_same(gdn):
    layer = Layer(gdn)
    s = torch.cuda.Stream()
    for kw in ({}, {"stream": s}, {"check_status": True}, {"stream": s, "check_status": True}):
        with pytest.raises(gdn.GdnError) as e:
            gdn.kv_attention(layer.cache, layer.q.half(), layer.table, layer.whole, **kw)
        assert e.value.status == 2
        with pytest.raises(gdn.GdnError) as e:
            gdn.kv_attention(layer.cache, layer.q[0], layer.table, layer.whole, **kw)
        assert e.value.status == 1
        with pytest.raises(gdn.GdnError) as e:
            gdn.qk_norm_rope_backward(layer.q.half(), layer.k, layer.pos, layer.tab, layer.w,
                                      layer.w, *layer.do, **kw)
        assert e.value.status == 2
