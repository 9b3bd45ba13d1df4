"""GPU: linear attention where its tensor-core kernels hand over between heads and scale their operands:
many short sequences of shared key heads, rows of very different sizes, values at the ends of bf16's
range, and states that have to keep every bit."""
import pytest
import torch

import linear_testutil as lt

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_rule_07_gb300 import build
    build.build()
    from gated_delta_rule_07_gb300 import gdn as mod
    assert torch.cuda.is_available()
    return mod


def rand(gen, *shape, io=BF16):
    return torch.randn(*shape, generator=gen).to(io).cuda()


@pytest.mark.parametrize("hk,hv", [(1, 4), (2, 6), (4, 8)])
@pytest.mark.parametrize("K,V", [(128, 128), (64, 128)])
def test_many_sequences_of_one_chunk_with_shared_key_heads(gdn, hk, hv, K, V):
    """Every segment is one chunk, walked for a key head's value heads one after another; the states
    that they start from differ by powers of two up to 2^20 from head to head."""
    gen = torch.Generator().manual_seed(hv + K)
    lens = torch.randint(0, 129, (120,), generator=gen).tolist()
    lens[7], lens[8] = 128, 1
    T, N, cu = sum(lens), len(lens), lt.cumulative(lens)
    q, k, v, do = rand(gen, T, hk, K), rand(gen, T, hk, K), rand(gen, T, hv, V), rand(gen, T, hv, V)
    g = -torch.rand(hv, generator=gen).cuda() * 0.2
    sizes = torch.exp2(torch.randint(0, 21, (N, hv, 1, 1), generator=gen).float())
    h0, dh = ((torch.randn(N, hv, K, V, generator=gen) * sizes).cuda() for _ in range(2))
    first = gdn.linear_attention_backward(q, k, v, g, do, h0, dh, cu, check_status=True)
    args = q, k, v, g, do, h0, dh, lens
    want, size = lt.backward(*args), lt.magnitudes(lt.backward, *args)
    for i, name in enumerate(("dq", "dk", "dv", "dh0")):
        lt.assert_close(first[i], want[i], size[i], lt.inner_error(128, i < 3), name)
    for _ in range(20):
        again = gdn.linear_attention_backward(q, k, v, g, do, h0, dh, cu)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# ------------------------------------------------------------------------------- sizes of the operands

def close(got, want, size, tokens, what=""):
    lt.assert_close(got, want, size, lt.inner_error(tokens, True), what)


@pytest.mark.parametrize("times", [2.0 ** 30, 2.0 ** 60])
@pytest.mark.parametrize("hk,hv", [(2, 2), (1, 3)])
def test_gradients_of_a_token_keep_their_own_accuracy(gdn, hk, hv, times):
    """One token's dout (v, k) far above the others': dq (dk, dv) of the others have the accuracy that
    they have without it, for each is made of its own token's dout (v, k) and of the other tensors."""
    gen = torch.Generator().manual_seed(hv)
    T, lens, cu = 300, [300], lt.cumulative([300])
    q, k, v, do = (rand(gen, T, h, 128) for h in (hk, hk, hv, hv))
    g = -torch.rand(hv, generator=gen).cuda() * 0.1
    h0, dh = (torch.randn(1, hv, 128, 128, generator=gen).cuda() for _ in range(2))
    for i, name in enumerate(("do", "v", "k")):
        x = dict(q=q, k=k, v=v, do=do)
        x[name] = x[name].clone()
        x[name][100] *= times
        args = x["q"], x["k"], x["v"], g, x["do"], h0, dh
        got = gdn.linear_attention_backward(*args, cu, check_status=True)
        close(got[i], lt.backward(*args, lens)[i], lt.magnitudes(lt.backward, *args, lens)[i], 300, name)


@pytest.mark.parametrize("small,large", [(2.0 ** -100, 2.0 ** 40), (2.0 ** -120, 2.0 ** 50)])
def test_small_rows_against_large_ones(gdn, small, large):
    """q (dout) so small that its fp16 form needs more than a power of two that fp32 holds beside the
    others'; what comes out is of ordinary size."""
    gen = torch.Generator().manual_seed(3)
    T, lens, cu = 300, [170, 130], lt.cumulative([170, 130])
    q, k, v, do = (rand(gen, T, h, 128) for h in (1, 1, 2, 2))
    g = torch.tensor([-0.3, -0.01], device="cuda")
    h0, dh = (torch.randn(2, 2, 128, 128, generator=gen).cuda() for _ in range(2))
    args = q * small, k * large, v * large, g, h0 * large ** 2
    out, last = gdn.linear_attention(*args, cu, check_status=True)
    want, size = lt.forward(*args, lens), lt.magnitudes(lt.forward, *args, lens)
    close(out, want[0], size[0], 170, "out")
    args = q * large, k * large, v * large, g, do * small, h0 * large ** 2, dh * large * small
    got = gdn.linear_attention_backward(*args, cu, check_status=True)
    want, size = lt.backward(*args, lens), lt.magnitudes(lt.backward, *args, lens)
    for i, name in enumerate(("dq", "dk", "dv")):
        close(got[i], want[i], size[i], 170, name)


@pytest.mark.parametrize("start", ["token", "h0"])
def test_states_beside_the_largest_keys_and_values(gdn, start):
    """A state of 2^110 beside a key of 2^70 and a value of 2^70 of different tokens: what would be their
    product is beyond fp32, but nothing is that is computed.  152 heads, so that the chunks are of one
    segment; one has values."""
    T, hv = 400, 152
    q, k = (torch.zeros(T, 1, 128, device="cuda", dtype=BF16) for _ in range(2))
    v = torch.zeros(T, hv, 128, device="cuda", dtype=BF16)
    h0 = torch.zeros(1, hv, 128, 128, device="cuda")
    if start == "token":
        k[10, 0, 0], v[10, -1, 0] = 2.0 ** 70, 2.0 ** 40
    else:
        k[10, 0, 1], v[10, -1, 1] = 2.0 ** 70, 2.0 ** -40
        h0[0, -1, 0, 0] = 2.0 ** 110
    k[11, 0, 2], v[11, -1, 2] = 1.0, 2.0 ** 70
    q[128:, 0, 0] = 2.0 ** -25
    out, last = gdn.linear_attention(q, k, v, torch.zeros(hv, device="cuda"), h0, check_status=True)
    assert last[0, -1, 0, 0] == 2.0 ** 110
    want = torch.zeros_like(out)
    want[128:, -1, 0] = 2.0 ** 85
    # (powers of two: nothing is rounded that is not below what the range allows, 2^79 here)
    assert ((out.double() - want.double()).abs() <= 2.0 ** 79).all()


def test_sums_beside_the_largest_keys_and_values(gdn):
    """The same where what is beyond the range is the scale of the chunks' growth: a key of 2^78 and a value
    of 2^77 of different tokens, and products of no more than 2^125."""
    T, hv = 400, 152
    q, k = (torch.zeros(T, 1, 128, device="cuda", dtype=BF16) for _ in range(2))
    v = torch.zeros(T, hv, 128, device="cuda", dtype=BF16)
    k[10, 0, 0], v[10, -1, 0] = 2.0 ** 78, 2.0 ** 47
    k[11, 0, 2], v[11, -1, 2] = 2.0 ** -20, 2.0 ** 77
    q[128:, 0, 0] = 2.0 ** -40
    out, last = gdn.linear_attention(q, k, v, torch.zeros(hv, device="cuda"), check_status=True)
    assert last[0, -1, 0, 0] == 2.0 ** 125
    want = torch.zeros_like(out)
    want[128:, -1, 0] = 2.0 ** 85
    assert ((out.double() - want.double()).abs() <= 2.0 ** 79).all()


def test_a_state_that_forgets_its_start(gdn):
    """A start of 2^100, and keys times values of 2^-27: by the time that the start has decayed below them,
    the state is what thousands of tokens have gathered, and its bound has to be too.  Every element is
    the same, so the definition is a geometric sum."""
    T, hv, d = 70000, 152, 0.85 ** (1 / 128)
    x = (2 - 2.0 ** -7) * 2.0 ** -14
    q = torch.ones(T, 1, 128, device="cuda", dtype=BF16)
    k = torch.full_like(q, x)
    v = torch.full((T, hv, 64), x / 2, device="cuda", dtype=BF16)
    g = torch.full((hv,), d, device="cuda").log()
    h0 = torch.full((1, hv, 128, 64), 2.0 ** 100, device="cuda")
    out, last = gdn.linear_attention(q, k, v, g, h0, check_status=True)
    t = torch.arange(T, device="cuda", dtype=torch.float64) + 1
    a = g[0].double()
    want = 128 * (torch.exp(a * t) * 2.0 ** 100 + x * x / 2 * torch.expm1(a * t) / torch.expm1(a))
    off = (out[:, [0, 76, 151]].double() / want[:, None, None] - 1).abs().amax((1, 2))
    # (a bf16 rounding, three fp16 ones, and the powers: t log2(a) of up to 130 is off by 2^-24 of it, twice)
    assert off.max() <= 2.0 ** -8 + 3 * 2.0 ** -11 + 130 * 2.0 ** -23


# ------------------------------------------------------------------------------- states to the last bit

@pytest.mark.parametrize("where", ["h_final", "dh0"])
def test_states_keep_every_bit_of_their_terms(gdn, where):
    """Each element of the state is one product, of a token whose key is one feature, and the tokens
    behind it (before it, for dh0) have none, however far the state decays on its way.  Whatever its
    weight is, all elements of a row share it, so their ratios to v (dout) agree to the roundings of one
    weighting, a decay a tile of 64 tokens, and a decay a segment: 12 of 2^-24 at most, each way, with
    the row's own scale.  (A part of the weighted rows left out is up to 2^-18.)"""
    gen = torch.Generator().manual_seed(1)
    T, hv = 384, 4
    g = torch.tensor([-0.01, -0.07, -0.1, -0.13], device="cuda")   # 2^-3 to 2^-48 over 256 tokens
    one, x = torch.zeros(T, 1, 128, device="cuda", dtype=BF16), rand(gen, T, hv, 128)
    rows = slice(0, 128) if where == "h_final" else slice(256, 384)
    one[rows, 0] = torch.eye(128, device="cuda", dtype=BF16)
    x[x == 0] = 1.0
    if where == "h_final":
        got = gdn.linear_attention(one, one, x, g, check_status=True)[1][0]
        steps = 383.0 - torch.arange(128, device="cuda", dtype=torch.float64)
    else:
        got = gdn.linear_attention_backward(one, one, x, g, x, check_status=True)[3][0]
        steps = 257.0 + torch.arange(128, device="cuda", dtype=torch.float64)
    ratio = got.double() / x[rows].double().transpose(0, 1)              # [hv, K, V]
    want = torch.exp(g.double()[:, None] * steps)
    assert ((ratio.mean(-1) / want - 1).abs() <= 60 * 2.0 ** -22).all()  # (the powers' own error)
    assert ((ratio / ratio.mean(-1, keepdim=True) - 1).abs() <= 24 * 2.0 ** -24).all()


@pytest.mark.parametrize("size", [1.0, 2.0 ** 60])
@pytest.mark.parametrize("hk,hv", [(2, 2), (1, 3)])
def test_rows_of_zeros(gdn, hk, hv, size):
    """Masked tokens: their rows of q, or of dout, are zeros, and so are their outputs and their dq; the
    tokens beside them are as they are, whatever the keys and values are."""
    gen = torch.Generator().manual_seed(4)
    T, lens, cu = 330, [200, 130], lt.cumulative([200, 130])
    q, k, v, do = (rand(gen, T, h, 128) for h in (hk, hk, hv, hv))
    masked = torch.rand(T, generator=gen).cuda() < 0.5
    masked[:40] = True
    q[masked], do[masked] = 0.0, 0.0
    g = -torch.rand(hv, generator=gen).cuda() * 0.1
    args = q / size, k * size, v * size, g, None
    out, _ = gdn.linear_attention(*args, cu, check_status=True)
    assert (out[masked] == 0).all()
    close(out, lt.forward(*args, lens)[0], lt.magnitudes(lt.forward, *args, lens)[0], 200, "out")
    args = q, k * size, v * size, g, do / size, None, None
    got = gdn.linear_attention_backward(*args, cu, check_status=True)
    want, sizes = lt.backward(*args, lens), lt.magnitudes(lt.backward, *args, lens)
    assert (got[0][masked] == 0).all()
    for i, name in enumerate(("dq", "dk", "dv")):
        close(got[i], want[i], sizes[i], 200, name)
