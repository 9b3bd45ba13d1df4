"""GPU: activations held in 8 bits, opened again, and read by the backward passes."""
import pytest
import torch

import linear_testutil as lt

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
FORMATS = [torch.int8, torch.float8_e4m3fn]


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_rule_07_gb300 import build
    build.build()
    from gated_delta_rule_07_gb300 import gdn as mod
    assert torch.cuda.is_available()
    return mod


def check(c, x, dtype):
    codes, scale = lt.checkpoint(x, dtype)
    assert c.dtype is x.dtype and c.shape == x.shape
    assert torch.equal(c.scale, scale)
    got = c.codes.double() if dtype is torch.int8 else c.codes.float().double()
    assert torch.equal(got, codes)
    return codes, scale


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("T,H,D", [(1, 1, 64), (3, 5, 128), (129, 2, 256), (1000, 7, 64),
                                   (511, 32, 128)])
def test_codes_and_values(gdn, T, H, D, dtype, io):
    x = (torch.randn(T, H, D, generator=torch.Generator().manual_seed(T)) * 3).to(io).cuda()
    x *= torch.exp2(torch.arange(T * H, device="cuda") % 60 - 30).view(T, H, 1).to(io)
    held, = gdn.checkpoint_pack(x, dtype=dtype, check_status=True)
    codes, scale = check(held, x, dtype)
    back, = gdn.checkpoint_open(held)
    # the product of a code and its scale, exact in 64 bits, rounded once in fp32 and once more
    assert torch.equal(back, (codes.float() * scale[..., None]).to(io))
    step = 0.5 * scale.double()[..., None] if dtype is torch.int8 else \
        (x.double().abs() * 2.0 ** -4).maximum(scale.double()[..., None] * 2.0 ** -10)
    assert ((back.double() - x.double()).abs() <= step * (1 + 2.0 ** -20) +
            back.double().abs() * lt.HALF_STEP[io] + 2.0 ** -22 * x.double().abs()).all()


def test_offsets_past_32_bits(gdn):
    """More than 2^31 elements, in a slice of rows as long again: the last rows."""
    x = torch.empty(530000, 2, 32, 128, dtype=BF16, device="cuda")[:, 1]
    assert x.numel() > 2 ** 31
    x[-100:].normal_()
    x[:-100] = 1.0
    held, = gdn.checkpoint_pack(x, check_status=True)
    codes, scale = lt.checkpoint(x[-100:], torch.int8)
    assert torch.equal(held.scale[-100:], scale) and torch.equal(held.codes[-100:].double(), codes)
    assert torch.equal(held.scale[:-100], torch.full_like(held.scale[:-100], 1 / torch.tensor(127.)))
    back, = gdn.checkpoint_open(held)
    assert torch.equal(back[-100:], (codes.float() * scale[..., None]).to(BF16))


@pytest.mark.parametrize("dtype", FORMATS)
def test_several_tensors_and_slices(gdn, dtype):
    gen = torch.Generator().manual_seed(1)
    p = torch.randn(77, 4 * 144, generator=gen).to(BF16).cuda()
    q = p[:, :288].view(77, 2, 144)[..., 16:]           # heads with a gap between them
    k = torch.randn(13, 3, 256, generator=gen).cuda()   # other dtypes and sizes in the same call
    v = torch.randn(1, 1, 64, generator=gen).to(BF16).cuda()
    e = torch.empty(0, 4, 128, device="cuda")
    tensors = q, k, e, v, k[:, 1:2], k[5:6], q[::3], v
    held = gdn.checkpoint_pack(*tensors, dtype=dtype)
    for c, x in zip(held, tensors):
        codes, scale = check(c, x, dtype)
    back = gdn.checkpoint_open(*held)
    for c, x, y in zip(held, tensors, back):
        assert y.is_contiguous() and y.dtype is x.dtype and y.shape == x.shape
        assert torch.equal(y, gdn.checkpoint_open(c)[0])


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("dtype", FORMATS)
def test_rows_at_the_edges(gdn, dtype, io):
    """Zeros, values below the least scale, and values that are not finite."""
    inf, nan = float("inf"), float("nan")
    x = torch.randn(9, 2, 128, generator=torch.Generator().manual_seed(3)).to(io).cuda()
    x[0] = 0.0
    x[1] = 2.0 ** -101
    x[2] = 2.0 ** -100
    x[3, :, 5], x[3, :, 6], x[3, :, 100] = inf, -inf, nan
    x[4] = inf
    x[5] = nan
    x[6] = torch.finfo(io).max
    x[7, 0] = -0.0
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    held, = gdn.checkpoint_pack(x, dtype=dtype)
    check(held, x, dtype)
    assert torch.isfinite(gdn.checkpoint_open(held)[0].float()).all()
    with pytest.raises(gdn.GdnError, match="DEVICE_RANGE"):
        gdn.checkpoint_pack(x, dtype=dtype, check_status=True)
    gdn.checkpoint_pack(x[6:], dtype=dtype, check_status=True)
    assert int(st) == 0


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("io,K,V,hk,hv", [(BF16, 128, 128, 2, 2), (BF16, 128, 128, 1, 3),
                                          (BF16, 64, 128, 2, 4), (F32, 128, 64, 1, 2)])
def test_linear_attention_backward_reads_them(gdn, dtype, io, K, V, hk, hv):
    """The gradients at the values that the checkpoints stand for, to the bit those of the call that is
    given these values."""
    gen = torch.Generator().manual_seed(K + hv)
    lens = [150, 0, 259]
    rand = lambda *n: torch.randn(*n, generator=gen).to(io).cuda()  # noqa: E731
    T = sum(lens)
    q, k, v, do = rand(T, hk, K), rand(T, hk, K), rand(T, hv, V), rand(T, hv, V)
    g = -torch.rand(hv, generator=gen).cuda()
    h0, dh = (torch.randn(3, hv, K, V, generator=gen).cuda() for _ in range(2))
    held = gdn.checkpoint_pack(q, k, v, dtype=dtype)
    got = gdn.linear_attention_backward(*held, g, do, h0, dh, lt.cumulative(lens),
                                        check_status=True)
    opened = gdn.checkpoint_open(*held)
    want = gdn.linear_attention_backward(*opened, g, do, h0, dh, lt.cumulative(lens))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    args = *opened, g, do, h0, dh, lens
    exact, size = lt.backward(*args), lt.magnitudes(lt.backward, *args)
    for i in range(4):
        cores = io is BF16 and i < 3
        lt.assert_close(got[i], exact[i], size[i], lt.inner_error(259, cores))


def test_the_delta_rules_backward_reads_them(gdn):
    gen = torch.Generator().manual_seed(5)
    T, hk, hv = 100, 1, 2
    q, k = (torch.nn.functional.normalize(torch.randn(T, hk, 128, generator=gen), dim=-1)
            .to(BF16).cuda() for _ in range(2))
    v, do = (torch.randn(T, hv, 128, generator=gen).to(BF16).cuda() for _ in range(2))
    g, beta = -torch.rand(T, hv, generator=gen).cuda(), torch.rand(T, hv, generator=gen).cuda()
    held = gdn.checkpoint_pack(q, k, v)
    got = gdn.backward(*held, g, beta, do)
    want = gdn.backward(*gdn.checkpoint_open(*held), g, beta, do)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = gdn.backward(*held, g, beta, do, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_refusals(gdn):
    x = torch.zeros(3, 2, 128, device="cuda").to(BF16)
    c, d = gdn.checkpoint_pack(x, x)
    e, = gdn.checkpoint_pack(x, dtype=torch.float8_e4m3fn)
    f, = gdn.checkpoint_pack(x.float())
    g, do = torch.zeros(2, device="cuda"), x
    for q, k, v in ((c, d, x), (c, d, e), (c, d, f)):
        with pytest.raises(gdn.GdnError):
            gdn.linear_attention_backward(q, k, v, g, do)
    for bad in ((x[0],), (x.half(),), (x[..., :96],), (x.cpu(),), (x.transpose(1, 2),), (x,) * 9,
                (torch.zeros(3, 2, 132, device="cuda")[..., 2:130],)):
        with pytest.raises(gdn.GdnError):
            gdn.checkpoint_pack(*bad)
    for codes, scale in ((c.codes[:2], c.scale), (c.codes, c.scale.double()),
                         (c.codes.transpose(0, 1), c.scale.t()), (c.codes.cpu(), c.scale),
                         (c.codes.view(torch.uint8), c.scale)):
        with pytest.raises(gdn.GdnError):
            gdn.Checkpoint(codes, scale)
    with pytest.raises(gdn.GdnError):
        gdn.checkpoint_open(c, e)


@pytest.mark.parametrize("dtype", FORMATS)
def test_a_part_of_the_tokens(gdn, dtype):
    """Codes and scales of some tokens are a checkpoint of these, wherever they start."""
    gen = torch.Generator().manual_seed(9)
    q, k, v, do = (torch.randn(200, 3, 128, generator=gen).to(BF16).cuda() for _ in range(4))
    g = -torch.rand(3, generator=gen).cuda()
    held = gdn.checkpoint_pack(q, k, v, dtype=dtype)
    for b, e in ((1, 200), (50, 133), (199, 200)):
        part = [gdn.Checkpoint(c.codes[b:e], c.scale[b:e], c.dtype) for c in held]
        opened = gdn.checkpoint_open(*part)
        for x, y in zip(opened, gdn.checkpoint_open(*held)):
            assert torch.equal(x, y[b:e])
        got = gdn.linear_attention_backward(*part, g, do[b:e].contiguous(), check_status=True)
        want = gdn.linear_attention_backward(*opened, g, do[b:e].contiguous())
        assert all(torch.equal(x, y) for x, y in zip(got, want))
