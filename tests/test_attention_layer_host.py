"""The softmax-attention layers' operators on the host: what they refuse (before any CUDA work, so
without a GPU), and the fp64 forms that the GPU tests compare with."""

import os
import subprocess
import sys

import pytest
import torch

import attention_testutil as at


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_rule_07_gb300 import build
    build.build()
    from gated_delta_rule_07_gb300 import gdn as mod
    return mod


FAKE = 1 << 20  # never dereferenced: validation fails first


def rope_problem(gdn, **kw):
    d = dict(total_tokens=8, hq=4, hkv=2, head_dim=128, rotary_dim=64, style=0, io_dtype=0,
             max_positions=16, eps=1e-6, weight_offset=0.0, q_token_stride=512,
             q_head_stride=128, k_token_stride=256, k_head_stride=128)
    d.update(kw)
    return gdn.QkRopeProblem(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(total_tokens=-1), 1), (dict(hq=0), 1), (dict(hkv=0), 1), (dict(max_positions=0), 1),
    (dict(rotary_dim=144), 1), (dict(rotary_dim=-16), 1), (dict(style=2), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(q_token_stride=4), 1),
    (dict(k_head_stride=12), 1), (dict(q_head_stride=-128), 1), (dict(head_dim=96), 2),
    (dict(rotary_dim=40), 2), (dict(io_dtype=3), 2), (dict(hq=70000), 2)])
def test_rope_refuses(gdn, kw, status):
    p = rope_problem(gdn, **kw)
    L = gdn._lib
    assert L.gdn_qk_norm_rope(p, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, None,
                              None) == status
    assert L.gdn_qk_norm_rope_backward(p, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, FAKE,
                                       FAKE, FAKE, FAKE, FAKE, 1 << 30, None, None) == status
    assert gdn.gdn_qk_norm_rope_backward_workspace_size(p) == 0


def test_rope_refuses_pointers(gdn):
    p, L = rope_problem(gdn), gdn._lib
    good = [FAKE, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, None, None]
    for i, bad in ((0, None), (1, None), (2, None), (3, None), (6, None), (7, None),
                   (0, FAKE + 2), (1, FAKE + 8), (3, FAKE + 4), (4, FAKE + 4), (6, FAKE + 8)):
        args = list(good)
        args[i] = bad
        assert L.gdn_qk_norm_rope(p, *args) == 1, (i, bad)
    assert L.gdn_qk_norm_rope(None, *good) == 1
    grad = [FAKE, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE]
    for i in (0, 1, 2, 3, 6, 7, 8, 9, 10, 11):
        args = list(grad)
        args[i] = None
        assert L.gdn_qk_norm_rope_backward(p, *args, FAKE, 1 << 30, None, None) == 1, i
    need = gdn.gdn_qk_norm_rope_backward_workspace_size(p)
    assert need > 0
    for ws, size in ((None, need), (FAKE, need - 1), (FAKE + 4, need)):
        assert L.gdn_qk_norm_rope_backward(p, *grad, ws, size, None, None) == 3


def cache_desc(gdn, **kw):
    d = dict(k_codes=FAKE, v_codes=FAKE, k_scale=FAKE, v_scale=FAKE, num_pages=4, page_size=64,
             hkv=2, head_dim=128, format=0)
    d.update(kw)
    return gdn.KvCacheDesc(**d)


def kv_problem(gdn, **kw):
    d = dict(total_tokens=8, num_seqs=2, max_pages=2, hq=4, io_dtype=0, k_token_stride=256,
             k_head_stride=128, v_token_stride=256, v_head_stride=128, q_token_stride=512,
             q_head_stride=128)
    d.update(kw)
    return gdn.KvProblem(**d)


def kv_calls(gdn, c, p, cu=FAKE, scale=1.0, window=0):
    L = gdn._lib
    return (L.gdn_kv_append(c, p, FAKE, FAKE, FAKE, FAKE, cu, None, None),
            L.gdn_kv_read(c, p, FAKE, FAKE, cu, FAKE, FAKE, None, None),
            L.gdn_kv_attention(c, p, FAKE, FAKE, FAKE, cu, scale, window, FAKE, None, FAKE,
                               1 << 40, None, None))


@pytest.mark.parametrize("c,p,status", [
    (dict(k_codes=None), {}, 1), (dict(v_codes=FAKE + 8), {}, 1), (dict(k_scale=None), {}, 1),
    (dict(v_scale=None), {}, 1), (dict(num_pages=0), {}, 1), (dict(hkv=0), {}, 1),
    (dict(page_size=48), {}, 2), (dict(page_size=256), {}, 2), (dict(head_dim=96), {}, 2),
    (dict(format=2), {}, 2), ({}, dict(total_tokens=-1), 1), ({}, dict(num_seqs=0), 1),
    ({}, dict(max_pages=0), 1), ({}, dict(io_dtype=2), 2), ({}, dict(max_pages=1 << 26), 2)])
def test_cache_calls_refuse(gdn, c, p, status):
    c, p = cache_desc(gdn, **c), kv_problem(gdn, **p)
    assert kv_calls(gdn, c, p) == (status,) * 3
    assert gdn.gdn_kv_attention_workspace_size(c, p) == 0


def test_cache_calls_refuse_arguments(gdn):
    c, p, L = cache_desc(gdn), kv_problem(gdn), gdn._lib
    assert kv_calls(gdn, None, p) == (1,) * 3 and kv_calls(gdn, c, None) == (1,) * 3
    assert kv_calls(gdn, c, p, cu=None) == (1,) * 3      # eight rows of two sequences
    assert kv_calls(gdn, c, p, window=-1)[2] == 1
    assert kv_calls(gdn, c, kv_problem(gdn, hq=3))[2] == 1
    assert kv_calls(gdn, c, kv_problem(gdn, q_head_stride=4))[2] == 1
    assert kv_calls(gdn, c, kv_problem(gdn, k_token_stride=4))[0] == 1
    assert kv_calls(gdn, c, kv_problem(gdn, v_head_stride=-128))[0] == 1
    append = [FAKE, FAKE, FAKE, FAKE]
    for i, bad in ((0, None), (1, None), (2, None), (3, None), (0, FAKE + 8), (1, FAKE + 2)):
        args = list(append)
        args[i] = bad
        assert L.gdn_kv_append(c, p, *args, FAKE, None, None) == 1
    for args in ((None, FAKE, FAKE, FAKE, FAKE), (FAKE, FAKE, FAKE, None, FAKE),
                 (FAKE, FAKE, FAKE, FAKE, FAKE + 8)):
        assert L.gdn_kv_read(c, p, *args, None, None) == 1
    for q, table, lens, out in ((None, FAKE, FAKE, FAKE), (FAKE, None, FAKE, FAKE),
                                (FAKE, FAKE, None, FAKE), (FAKE, FAKE, FAKE, None),
                                (FAKE + 4, FAKE, FAKE, FAKE)):
        assert L.gdn_kv_attention(c, p, q, table, lens, FAKE, 1.0, 0, out, None, FAKE, 1 << 40,
                                  None, None) == 1


def test_binding_refuses(gdn):
    """Shapes, dtypes, strides and devices are checked before a pointer is passed on."""
    b, f = torch.bfloat16, torch.float32
    q, k = torch.zeros(3, 4, 128, dtype=b), torch.zeros(3, 2, 128, dtype=b)
    pos, tab = torch.zeros(3, dtype=torch.int32), torch.zeros(8, 64)
    w = torch.ones(128)
    for args, status in (((q, k, pos, tab, w, w), 1),                      # on the CPU
                         ((q.half(), k.half(), pos, tab, w, w), 2),
                         ((q, k.float(), pos, tab, w, w), 1),
                         ((q, k[:2], pos, tab, w, w), 1),
                         ((q, k, pos.long(), tab, w, w), 1),
                         ((q, k, pos, tab.double(), w, w), 1),
                         ((q, k, pos, tab, w[:64], w), 1),
                         ((q.transpose(1, 2), k, pos, tab, w, w), 1)):
        with pytest.raises(gdn.GdnError) as e:
            gdn.qk_norm_rope(*args)
        assert e.value.status == status
    with pytest.raises(gdn.GdnError):
        gdn.qk_norm_rope(q, k, pos, tab, w, w, style="spiral")
    with pytest.raises(gdn.GdnError):
        gdn.qk_norm_rope_backward(q, k, pos, tab, w, w, torch.zeros(1, dtype=b).expand(3, 4, 128),
                                  k)
    kc = torch.zeros(2, 1, 16, 64, dtype=torch.int8)
    vc = torch.zeros(2, 1, 4, 64, 4, dtype=torch.int8)
    s = torch.zeros(2, 1)
    for args, status in (((kc, vc, s, s), 1), ((kc, kc, s, s), 1), ((kc, vc, s, s.double()), 1),
                         ((kc.to(torch.uint8), vc, s, s), 2), ((kc, vc, s[:1], s), 1),
                         ((kc[:, :, ::2], vc, s, s), 1)):
        with pytest.raises(gdn.GdnError) as e:
            gdn.KVCache(*args)
        assert e.value.status == status


def test_gradient_against_differences():
    """The fp64 gradient formula that the kernel is held to, against central differences of the
    fp64 forward: step h = 1e-5 leaves h^2 of the third derivative (inputs and weights of order 1:
    below 1e-8) plus rounding 1e-16 / h = 1e-11 a term."""
    for style, R in (("half", 32), ("pairs", 48)):
        gen = torch.Generator().manual_seed(R)
        q, do = (torch.randn(2, 2, 64, generator=gen, dtype=torch.float64) for _ in range(2))
        w = 1 + 0.2 * torch.randn(64, generator=gen, dtype=torch.float64)
        pos, tab = torch.tensor([3, 41]), at.table(64, R)
        dx, dw, _, _ = at.rope_grad(q, pos, tab, w, 1e-6, 0.5, style, do)
        x, h = q.double(), 1e-5

        def loss(x, w):
            return float((at.rope(x, pos, tab, w, 1e-6, 0.5, style)[0] * do.double()).sum())

        for e in range(0, x.numel(), 17):
            d = torch.zeros(x.numel(), dtype=torch.float64)
            d[e] = h
            d = d.view(x.shape)
            assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * h) - float(dx.flatten()[e])) < 1e-6
        for e in range(0, 64, 5):
            d = torch.zeros(64, dtype=torch.float64)
            d[e] = h
            assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * h) - float(dw[e])) < 1e-6


def test_values_layout_roundtrip():
    gen = torch.Generator().manual_seed(0)
    codes = torch.randint(-127, 128, (3, 2, 32, 64), generator=gen).to(torch.int8)
    v = at.packed_v(codes)
    assert v.shape == (3, 2, 8, 64, 4) and v.is_contiguous()
    assert int(v[1, 1, 5, 7, 2]) == int(codes[1, 1, 5 * 4 + 2, 7])
    assert torch.equal(at.unpacked_v(v), codes)


def test_workspace_for_refuses(gdn):
    """kv_attention_workspace refuses as the call itself does."""
    class Cache:
        desc = cache_desc(gdn)
    table = torch.zeros(2, 2, dtype=torch.int32)
    for q, t, status in ((torch.zeros(8, 4, 128, dtype=torch.float16), table, 2),
                         (torch.zeros(8, 512, dtype=torch.bfloat16), table, 1),
                         (torch.zeros(8, 4, 128, dtype=torch.bfloat16), table[0], 1)):
        with pytest.raises(gdn.GdnError) as e:
            gdn.kv_attention_workspace(Cache, q, t)
        assert e.value.status == status


class OnGpu:
    """Looks like a tensor on some GPU; there is nothing behind it."""

    def __init__(self, shape, dtype, index):
        self.shape, self.dtype, self.device = shape, dtype, torch.device("cuda", index)
        self.is_cuda = True

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE


def test_cache_buffers_on_one_gpu(gdn):
    def cache(*index):
        return gdn.KVCache(*(OnGpu(s, d, i) for s, d, i in zip(
            ((2, 1, 16, 64), (2, 1, 4, 64, 4), (2, 1), (2, 1)),
            (torch.int8, torch.int8, torch.float32, torch.float32), index)))
    c = cache(1, 1, 1, 1)
    assert c._handle.device == 1 and c.desc.num_pages == 2 and c.desc.k_codes == FAKE
    for index in ((0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1), (1, 0, 0, 0)):
        with pytest.raises(gdn.GdnError) as e:
            cache(*index)
        assert e.value.status == 1 and "cuda:1" in str(e.value)


def test_cache_keeps_its_buffers(gdn):
    """The calls go by the buffers' addresses: assigning another tensor is refused."""
    c = gdn.KVCache(*(OnGpu(s, d, 0) for s, d in (
        ((2, 1, 16, 64), torch.int8), ((2, 1, 4, 64, 4), torch.int8), ((2, 1), torch.float32),
        ((2, 1), torch.float32))))
    for name in ("k", "v", "k_scale", "v_scale", "buffers"):
        with pytest.raises(AttributeError):
            setattr(c, name, None)
    assert c.buffers == (c.k, c.v, c.k_scale, c.v_scale)


def test_strides_of_single_rows_do_not_count(gdn):
    """The stride of a dimension of one row says nothing, so it is not held to 16 bytes."""
    for kw, ok in ((dict(total_tokens=1, q_token_stride=1001, k_token_stride=-3), True),
                   (dict(total_tokens=0, q_token_stride=1001), True),
                   (dict(hq=1, q_head_stride=7), True), (dict(hkv=1, k_head_stride=7), True),
                   (dict(total_tokens=2, q_token_stride=1001), False),
                   (dict(hq=1, k_head_stride=7), False)):
        got = gdn.gdn_qk_norm_rope_backward_workspace_size(rope_problem(gdn, **kw))
        assert (got > 0) == ok, kw
    for c, kw, ok in (({}, dict(total_tokens=1, q_token_stride=1001), True),
                      (dict(hkv=1), dict(hq=1, q_head_stride=7), True),
                      ({}, dict(total_tokens=2, q_token_stride=1001), False),
                      (dict(hkv=1), dict(hq=2, q_head_stride=7), False)):
        got = gdn.gdn_kv_attention_workspace_size(cache_desc(gdn, **c), kv_problem(gdn, **kw))
        assert (got > 0) == ok, kw


def test_recurrent_calls_do_without_the_binding(gdn):
    """A missing (or unloadable) torch binding leaves the module's other calls usable; the attention
    layer's calls say what is missing."""
    code = """
import torch
from gated_delta_rule_07_gb300 import build
build.TORCH_LIB = {path!r}
from gated_delta_rule_07_gb300 import gdn
assert gdn.gdn_workspace_size(gdn.make_problem(64, 1, 1, 1, 128, 128)) > 0
for _ in range(2):
    try:
        gdn.qk_norm_rope(torch.zeros(1, 1, 64), torch.zeros(1, 1, 64), None, None)
        raise SystemExit("loaded")
    except ImportError as e:
        assert build.TORCH_LIB in str(e), e
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for path in ("/nowhere/_gdn_torch.so", os.path.abspath(__file__)):
        subprocess.run([sys.executable, "-c", code.format(path=path)], check=True, cwd=root)


def test_binding_of_another_torch_is_stale(gdn, monkeypatch, tmp_path):
    """A binding is built again for another torch or Python, whatever the sources' times."""
    from gated_delta_rule_07_gb300 import build
    assert not build._binding_stale() and not build._library_stale()
    with open(build.TORCH_FOR) as f:
        assert f.read() == build.torch_build() and torch.__version__ in build.torch_build()
    other = tmp_path / "for"
    other.write_text(build.torch_build().replace(torch.__version__, "1.0"))
    monkeypatch.setattr(build, "TORCH_FOR", str(other))
    assert build._binding_stale() and not build._library_stale()
    monkeypatch.setattr(build, "TORCH_FOR", str(tmp_path / "none"))
    assert build._binding_stale()


def test_stream_of_another_gpu_is_refused(gdn):
    """A stream that torch would leave aside, because the tensors are on another GPU."""
    class Stream:
        cuda_stream, device = FAKE, torch.device("cuda", 1)
    on = OnGpu((2, 2), torch.float32, 1)
    assert gdn._side_stream(Stream, (None, on)) is Stream
    with pytest.raises(gdn.GdnError) as e:
        gdn._side_stream(Stream, (None, OnGpu((2, 2), torch.float32, 0), on))
    assert e.value.status == 1 and "cuda:1" in str(e.value) and "cuda:0" in str(e.value)
