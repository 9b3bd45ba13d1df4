"""Linear attention and the 8-bit checkpoints on the host: what they refuse (before any CUDA work, so
without a GPU), and the fp64 forms that the GPU tests compare with."""
import pytest
import torch

import linear_testutil as lt


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_rule_07_gb300 import build
    build.build()
    from gated_delta_rule_07_gb300 import gdn as mod
    return mod


FAKE = 1 << 20  # never dereferenced: validation fails first


def problem(gdn, **kw):
    d = dict(total_tokens=300, num_seqs=1, hk=2, hv=4, k_dim=128, v_dim=128, io_dtype=0,
             q_token_stride=256, q_head_stride=128, k_token_stride=256, k_head_stride=128,
             v_token_stride=512, v_head_stride=128)
    d.update(kw)
    return gdn.LinearProblem(**d)


def forward(gdn, p, ws=1 << 40, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, h0=None, cu=None, out=FAKE, last=FAKE, work=FAKE)
    a.update(kw)
    return gdn._lib.gdn_linear_attention(p, a["q"], a["k"], a["v"], a["g"], a["h0"], a["cu"],
                                         a["out"], a["last"], a["work"], ws, None, None)


def backward(gdn, p, ws=1 << 40, saved=None, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, h0=None, cu=None, do=FAKE, dh=None, dq=FAKE, dk=FAKE,
             dv=FAKE, dh0=FAKE, work=FAKE)
    a.update(kw)
    return gdn._lib.gdn_linear_attention_backward(
        p, a["q"], a["k"], a["v"], saved, a["g"], a["h0"], a["cu"], a["do"], a["dh"], a["dq"],
        a["dk"], a["dv"], a["dh0"], a["work"], ws, None, None)


def decode(gdn, p, slots=8, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, slot=FAKE, state=FAKE, out=FAKE)
    a.update(kw)
    return gdn._lib.gdn_linear_attention_decode(p, slots, a["q"], a["k"], a["v"], a["g"], a["slot"],
                                                a["state"], a["out"], None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(total_tokens=-1), 1), (dict(num_seqs=0), 1), (dict(hk=0), 1), (dict(hk=3), 1),
    (dict(hv=0), 1), (dict(k_dim=0), 1), (dict(q_token_stride=4), 1), (dict(k_head_stride=-128), 1),
    (dict(v_token_stride=513), 1), (dict(io_dtype=1, v_head_stride=130), 1), (dict(k_dim=96), 2),
    (dict(v_dim=256), 2), (dict(io_dtype=2), 2), (dict(hv=70000, hk=70000), 2)])
def test_refuses(gdn, kw, status):
    p = problem(gdn, **kw)
    assert gdn.gdn_check_linear_problem(p) == status
    assert forward(gdn, p) == backward(gdn, p) == decode(gdn, p) == status
    assert gdn.gdn_linear_attention_workspace_size(p) == 0
    assert gdn.gdn_linear_attention_backward_workspace_size(p) == 0


def test_refuses_pointers(gdn):
    p = problem(gdn)
    assert gdn.gdn_check_linear_problem(p) == 0
    for name in ("q", "k", "v", "g", "out"):
        assert forward(gdn, p, **{name: None}) == 1, name
    for name in ("q", "k", "v", "out", "h0", "last"):
        assert forward(gdn, p, **{name: FAKE + 8}) == 1, name
    for name in ("q", "k", "v", "g", "do", "dq", "dk", "dv"):
        assert backward(gdn, p, **{name: None}) == 1, name
    for name in ("q", "k", "v", "do", "h0", "dh", "dq", "dk", "dv", "dh0"):
        assert backward(gdn, p, **{name: FAKE + 4}) == 1, name
    for name in ("q", "k", "v", "g", "slot", "state", "out"):
        assert decode(gdn, p, **{name: None}) == 1, name
    for name in ("q", "k", "v", "state", "out"):
        assert decode(gdn, p, **{name: FAKE + 8}) == 1, name
    assert decode(gdn, p, slots=0) == 1
    # several sequences need their table
    many = problem(gdn, num_seqs=2)
    assert forward(gdn, many) == backward(gdn, many) == 1
    # 8-bit activations stand in place of the others
    held = gdn.LinearSaved(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0)
    assert backward(gdn, p, saved=held) == 1
    none = dict(q=None, k=None, v=None)
    assert backward(gdn, p, saved=gdn.LinearSaved(FAKE, FAKE, None, FAKE, FAKE, FAKE, 0),
                    **none) == 1
    assert backward(gdn, p, saved=gdn.LinearSaved(FAKE, FAKE, FAKE, FAKE, None, FAKE, 0),
                    **none) == 1
    assert backward(gdn, p, saved=gdn.LinearSaved(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2),
                    **none) == 2


def test_refuses_workspaces(gdn):
    p = problem(gdn)
    need = gdn.gdn_linear_attention_workspace_size(p)
    more = gdn.gdn_linear_attention_backward_workspace_size(p)
    most = gdn.gdn_linear_attention_backward_workspace_size(p, True)
    assert need > 0 and 2 * need <= more < most
    for ws, at in ((need - 1, FAKE), (1 << 40, None), (1 << 40, FAKE + 4)):
        assert forward(gdn, p, ws=ws, work=at) == 3
    assert backward(gdn, p, ws=more - 1) == 3
    held = gdn.LinearSaved(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0)
    assert backward(gdn, p, ws=most - 1, saved=held, q=None, k=None, v=None) == 3


@pytest.mark.parametrize("kw,status", [
    (dict(total_tokens=-1), 1), (dict(heads=0), 1), (dict(head_dim=0), 1), (dict(x=None), 1),
    (dict(codes=None), 1), (dict(scale=None), 1), (dict(x=FAKE + 8), 1), (dict(codes=FAKE + 8), 1),
    (dict(token_stride=257), 1), (dict(head_stride=-128), 1), (dict(head_dim=96), 2),
    (dict(io_dtype=2), 2), (dict(total_tokens=1 << 30, heads=4), 2)])
def test_checkpoint_refuses(gdn, kw, status):
    d = dict(x=FAKE, codes=FAKE, scale=FAKE, total_tokens=5, token_stride=256, head_stride=128,
             heads=2, head_dim=128, io_dtype=0)
    L, one = gdn._lib, gdn.CheckpointDesc * 1
    bad = one(gdn.CheckpointDesc(**{**d, **kw}))
    assert L.gdn_checkpoint_pack(bad, 1, 0, None, None) == status
    assert L.gdn_checkpoint_open(bad, 1, 0, None) == status
    good = one(gdn.CheckpointDesc(**d))
    for count, fmt, want in ((0, 0, 1), (9, 0, 2), (1, 2, 2)):
        assert L.gdn_checkpoint_pack(good, count, fmt, None, None) == want
        assert L.gdn_checkpoint_open(good, count, fmt, None) == want
    assert L.gdn_checkpoint_pack(None, 1, 0, None, None) == 1


def test_python_refuses_before_any_cuda_work(gdn):
    x, g = torch.zeros(3, 2, 128).bfloat16(), torch.zeros(2)
    calls = [lambda: gdn.linear_attention(x, x, x, g),                    # not on the GPU
             lambda: gdn.linear_attention(x.half(), x, x, g),
             lambda: gdn.linear_attention(x[0], x, x, g),
             lambda: gdn.linear_attention_backward(x, x, x, g, x),
             lambda: gdn.linear_attention_decode(x, x, x, g, torch.zeros(3, dtype=torch.int32),
                                                 torch.zeros(3, 2, 128, 128)),
             lambda: gdn.checkpoint_pack(x),
             lambda: gdn.checkpoint_pack(),
             lambda: gdn.checkpoint_open(),
             lambda: gdn.checkpoint_pack(x, dtype=torch.uint8),
             lambda: gdn.Checkpoint(x.to(torch.int8), torch.zeros(3, 2)),  # not on the GPU
             lambda: gdn.Checkpoint(x, torch.zeros(3, 2))]
    for i, call in enumerate(calls):
        with pytest.raises(gdn.GdnError):
            call()


@pytest.mark.parametrize("lens,carry", [([5, 0, 3], True), ([7], False)])
def test_fp64_gradients_against_differences(lens, carry):
    gen = torch.Generator().manual_seed(4)
    rand = lambda *n: torch.randn(*n, generator=gen, dtype=torch.float64)  # noqa: E731
    T, N, hk, hv, K, V = sum(lens), len(lens), 1, 2, 3, 2
    q, k, v, do = rand(T, hk, K), rand(T, hk, K), rand(T, hv, V), rand(T, hv, V)
    g = torch.tensor([-0.3, 0.0], dtype=torch.float64)
    h0, dh = (rand(N, hv, K, V), rand(N, hv, K, V)) if carry else (None, None)
    got = lt.backward(q, k, v, g, do, h0, dh, lens)

    def value(q, k, v, h0):
        o, h = lt.forward(q, k, v, g, h0, lens)
        return (o * do).sum() + ((h * dh).sum() if carry else 0.0)

    args, eps = [q, k, v, h0], 1e-6
    for i, x in enumerate(args):
        if x is None:
            continue
        for j in range(x.numel()):
            ends = []
            for s in (eps, -eps):
                y = x.clone()
                y.view(-1)[j] += s
                ends.append(value(*(y if n == i else a for n, a in enumerate(args))))
            assert abs((ends[0] - ends[1]) / (2 * eps) - got[i].reshape(-1)[j]) < 1e-7


def test_fp64_form_is_the_recurrence():
    gen = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(6, 1, 3, generator=gen, dtype=torch.float64) for _ in range(3))
    h0 = torch.randn(1, 1, 3, 3, generator=gen, dtype=torch.float64)
    for decay in (-0.7, 0.0, float("-inf")):
        g = torch.tensor([decay], dtype=torch.float64)
        out, last = lt.forward(q, k, v, g, h0, [6])
        h = h0[0, 0]
        for t in range(6):
            h = torch.exp(g[0]) * h + torch.outer(k[t, 0], v[t, 0])
            assert torch.allclose(out[t, 0], h.T @ q[t, 0], atol=1e-13, rtol=0)
        assert torch.allclose(last[0, 0], h, atol=1e-13, rtol=0)


@pytest.mark.parametrize("saved", [False, True])
def test_a_workspace_size_is_one_problems(gdn, saved):
    """Over lengths at which the number of segments goes up and down: a call wants the size that it was
    asked for, and one byte less is refused."""
    held = gdn.LinearSaved(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0) if saved else None
    rows = dict(q=None, k=None, v=None) if saved else {}
    for tokens in (1, 127, 129, 1000, 4991, 4992, 4993, 20000, 70001):
        for kw in (dict(), dict(num_seqs=3), dict(q_head_stride=0), dict(io_dtype=1)):
            p = problem(gdn, total_tokens=tokens, **kw)
            cu = FAKE if p.num_seqs > 1 else None
            need = gdn.gdn_linear_attention_workspace_size(p)
            assert need >= p.num_seqs * 4 * 128 * 128 * 4 and forward(gdn, p, ws=need - 1, cu=cu) == 3
            need = gdn.gdn_linear_attention_backward_workspace_size(p, saved)
            assert backward(gdn, p, ws=need - 1, saved=held, cu=cu, **rows) == 3


def test_checkpoint_scales_are_aligned_as_floats(gdn):
    c = gdn.CheckpointDesc(x=FAKE, codes=FAKE, scale=FAKE + 2, total_tokens=5, token_stride=256,
                           head_stride=128, heads=2, head_dim=128, io_dtype=0)
    one = (gdn.CheckpointDesc * 1)(c)
    assert gdn._lib.gdn_checkpoint_pack(one, 1, 0, None, None) == 1
    assert gdn._lib.gdn_checkpoint_open(one, 1, 0, None) == 1
