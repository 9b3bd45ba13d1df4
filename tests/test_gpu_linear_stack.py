"""GPU: linear attention's calls run together (examples/linear_stack.py), under autograd, on named streams
with work pending, and what the torch binding refuses of them."""
import importlib.util
import os

import pytest
import torch

import linear_testutil as lt

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
SPIN = 100_000_000  # clock cycles, about 50 ms
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "linear_stack.py")


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_rule_07_gb300 import build
    build.build()
    from gated_delta_rule_07_gb300 import gdn as mod
    assert torch.cuda.is_available()
    return mod


@pytest.fixture(scope="module")
def stack(gdn):
    spec = importlib.util.spec_from_file_location("linear_stack", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_steps_agree_with_one_call(stack):
    """The same tokens one at a time and all at once: they differ in roundings alone, a few bf16 ones
    (2^-8) a layer and the fp16 ones of the tensor cores.  A wrong state or slot makes them differ by
    their size."""
    steps, whole = stack.serve()
    assert torch.isfinite(steps.float()).all()
    assert (steps.float() - whole.float()).norm() / whole.float().norm() < 0.05


def test_prompt_in_pieces(stack):
    gen = torch.Generator("cuda").manual_seed(9)
    x = torch.randn(2, 300, stack.HIDDEN, device="cuda", generator=gen).bfloat16()

    def run(cuts):
        s, at, out = stack.Stack(2), [0, 0], None
        for cut in cuts:
            rows = torch.cat([x[n, at[n]:at[n] + cut[n]] for n in range(2)])
            out = s.extend(rows, cut)
            at = [a + c for a, c in zip(at, cut)]
        return torch.stack([out[cuts[-1][0] - 1], out[-1]]).float()

    a, b = run([[290, 41]]), run([[130, 0], [127, 1], [33, 40]])
    assert (a - b).norm() / a.norm() < 0.05


@pytest.mark.parametrize("hold", [None, torch.int8, torch.float8_e4m3fn])
def test_gradients_of_the_operator_under_autograd(stack, gdn, hold):
    gen = torch.Generator().manual_seed(2)
    rand = lambda *n: torch.randn(*n, generator=gen).to(BF16).cuda()  # noqa: E731
    lens, hk, hv = [140, 3, 60], 2, 4
    T = sum(lens)
    q, k, v = (t.requires_grad_() for t in (rand(T, hk, 128), rand(T, hk, 128), rand(T, hv, 128)))
    h0 = torch.randn(3, hv, 128, 128, generator=gen).cuda().requires_grad_()
    g, cu = stack.slopes(hv), lt.cumulative(lens)
    do, dh = rand(T, hv, 128), torch.randn(3, hv, 128, 128, generator=gen).cuda()
    out, last = stack.LinearAttention.apply(q, k, v, g, h0, cu, hold)
    got = torch.autograd.grad([out, last], [q, k, v, h0], [do, dh])
    at = (q, k, v) if hold is None else gdn.checkpoint_open(
        *gdn.checkpoint_pack(q.detach(), k.detach(), v.detach(), dtype=hold))
    args = *(t.detach() for t in at), g, do, h0.detach(), dh, lens
    want, size = lt.backward(*args), lt.magnitudes(lt.backward, *args)
    for i in range(4):
        lt.assert_close(got[i], want[i], size[i], lt.inner_error(140, i < 3), str(i))


def test_gradients_of_the_stack(stack):
    """From 8-bit checkpoints they differ by what the checkpoints do: half a step of a row's 127 is
    2^-8 of its largest value, a few times its typical one's rounding."""
    loss, kept = stack.gradients()
    again, held = stack.gradients(hold=torch.int8)
    assert torch.equal(loss, again)
    for a, b in zip(kept, held):
        assert torch.isfinite(a.float()).all() and a.float().norm() > 0
        assert (a.float() - b.float()).norm() / a.float().norm() < 0.05


def test_captured_training_step(stack, gdn):
    """Forward and backward captured together, replayed on other inputs."""
    gen = torch.Generator().manual_seed(4)
    rand = lambda *n: torch.randn(*n, generator=gen).to(BF16).cuda()  # noqa: E731
    ins = [rand(300, 2, 128), rand(300, 2, 128), rand(300, 4, 128), rand(300, 4, 128)]
    more = [rand(*t.shape) for t in ins]
    g, cu = stack.slopes(4), lt.cumulative([200, 100])

    def call(q, k, v, do):
        held = gdn.checkpoint_pack(q, k, v)
        return [*gdn.linear_attention(q, k, v, g, None, cu),
                *gdn.linear_attention_backward(*held, g, do, None, None, cu)]

    with torch.cuda.stream(torch.cuda.Stream()):
        call(*ins)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = call(*ins)
    for a, b in zip(ins, more):
        a.copy_(b)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(kept, call(*more)))


# ------------------------------------------------------------------------------- streams

class Calls:
    def __init__(self, gdn, seed=0):
        gen = torch.Generator().manual_seed(seed)
        rand = lambda *n: torch.randn(*n, generator=gen).to(BF16).cuda()  # noqa: E731
        T, hk, hv, D = 300, 2, 4, 128
        self.gdn = gdn
        self.q, self.k, self.v, self.do = rand(T, hk, D), rand(T, hk, D), rand(T, hv, D), rand(T, hv, D)
        self.g = -torch.rand(hv, generator=gen).cuda()
        self.cu = lt.cumulative([170, 1, 129])
        self.h0 = torch.randn(3, hv, D, D, generator=gen).cuda()
        self.slot = torch.tensor([2, -1, 0], dtype=torch.int32).cuda()
        self.held = gdn.checkpoint_pack(self.q, self.k, self.v)
        self.fresh()
        torch.cuda.synchronize()

    def fresh(self):
        self.state = self.h0.clone()

    def __call__(self, name, q=None, **kw):
        g, q = self.gdn, self.q if q is None else q
        if name == "forward":
            return g.linear_attention(q, self.k, self.v, self.g, self.h0, self.cu, **kw)
        if name == "backward":
            return g.linear_attention_backward(q, self.k, self.v, self.g, self.do, self.h0, self.h0,
                                               self.cu, **kw)
        if name == "backward of checkpoints":
            return g.linear_attention_backward(*self.held, self.g, self.do, self.h0, None, self.cu, **kw)
        if name == "decode":
            return g.linear_attention_decode(q[:3], self.k[:3], self.v[:3], self.g, self.slot,
                                             self.state, **kw), self.state
        if name == "pack":
            return [t for c in g.checkpoint_pack(q, self.k, **kw) for t in (c.codes, c.scale)]
        kw.pop("check_status", None)
        return g.checkpoint_open(*self.held, **kw)


NAMES = ["forward", "backward", "backward of checkpoints", "decode", "pack", "open"]


def same(got, want):
    assert len(got) == len(want)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_named_streams_with_work_pending(gdn, name):
    calls = Calls(gdn)
    want = [t.clone() for t in calls(name)]
    for as_handle in (False, True):
        calls.fresh()
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        torch.cuda._sleep(SPIN)       # memory that the current stream will still write is not an output
        junk = [torch.empty_like(t) for t in want for _ in range(4)]
        junk += [torch.empty(1, dtype=torch.int32, device="cuda") for _ in range(8)]
        for t in junk:
            t.view(torch.uint8).fill_(0x7f)
        del junk
        out = calls(name, check_status=True, stream=s.cuda_stream if as_handle else s)
        torch.cuda.synchronize()
        same(out, want)


@pytest.mark.parametrize("name", NAMES)
def test_memory_is_held_until_the_call_is_done(gdn, name):
    calls = Calls(gdn)
    want = [t.clone() for t in calls(name)]
    calls.fresh()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    q = calls.q.clone()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(SPIN)
    out = calls(name, q=q, stream=s)
    del q
    later = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")
             for n in (calls.q.numel() * 2, 1 << 20, 2 << 20, 4 << 20, 16 << 20, 64 << 20)
             for _ in range(3)]
    torch.cuda.synchronize()
    same(out, want)
    del later


def test_two_calls_at_once(gdn):
    """Two streams, each with its own inputs, at the same time."""
    a, b = Calls(gdn, 1), Calls(gdn, 2)
    want = [[t.clone() for t in c(n)] for c in (a, b) for n in ("forward", "backward")]
    torch.cuda.synchronize()
    streams, got = (torch.cuda.Stream(), torch.cuda.Stream()), []
    for _ in range(3):
        got = [c(n, stream=s) for c, s in zip((a, b), streams) for n in ("forward", "backward")]
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        same(x, y)


# ------------------------------------------------------------------------------- refusals

def test_broadcast_rows(gdn):
    """Rows that are all heads' or all tokens' (strides of zero) are the same as their copies."""
    c = Calls(gdn)
    for q, k, v in ((c.q[:, :1].expand(-1, 2, -1), c.k, c.v), (c.q, c.k[:1].expand(300, -1, -1), c.v),
                    (c.q, c.k, c.v[:, 2:3].expand(-1, 4, -1))):
        got = gdn.linear_attention(q, k, v, c.g, c.h0, c.cu)
        args = q, k, v, c.g, c.h0, [170, 1, 129]
        want, size = lt.forward(*args), lt.magnitudes(lt.forward, *args)
        lt.assert_close(got[0], want[0], size[0], lt.inner_error(170, True))
        lt.assert_close(got[1], want[1], size[1], lt.inner_error(170, False))
        got = gdn.linear_attention_backward(q, k, v, c.g, c.do, c.h0, None, c.cu)
        args = q, k, v, c.g, c.do, c.h0, None, [170, 1, 129]
        want, size = lt.backward(*args), lt.magnitudes(lt.backward, *args)
        for i in range(4):
            lt.assert_close(got[i], want[i], size[i], lt.inner_error(170, i < 3))


def test_strides_of_a_dimension_of_one_row_mean_nothing(gdn):
    c = Calls(gdn)
    odd = lambda t: t.as_strided(t.shape, (3, 5, 1))  # noqa: E731  (one token, one head)
    q, k, v = (odd(t[:1, :1].contiguous()) for t in (c.q, c.k, c.v))
    g, h0 = c.g[:1], c.h0[:1, :1].contiguous()
    args = q, k, v, g, h0, [1]
    want, size = lt.forward(*args), lt.magnitudes(lt.forward, *args)
    out, last = gdn.linear_attention(q, k, v, g, h0)
    lt.assert_close(out, want[0], size[0], lt.inner_error(1, True))
    lt.assert_close(last, want[1], size[1], lt.inner_error(1, False))
    held, = gdn.checkpoint_pack(q)
    assert torch.equal(held.codes, gdn.checkpoint_pack(q.contiguous())[0].codes)


def test_workspace_of_another_kind(gdn):
    c = Calls(gdn)
    for bad in (torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(64, 64, device="cuda").t()):
        with pytest.raises(gdn.GdnError):
            gdn.linear_attention(c.q, c.k, c.v, c.g, workspace=bad)
    big = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    want = c("forward")
    same(c("forward", workspace=big), want)
    same(c("backward", workspace=big), c("backward"))
