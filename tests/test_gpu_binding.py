"""GPU: what the torch binding of the attention layer's calls refuses of GPU tensors.

Every case starts from arguments that are right and changes one property; the refusal comes before
any launch, and its message has to name the property.
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


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def ints(*shape):
    return zeros(*shape, dtype=torch.int32)


def kv_calls(gdn, cache):
    """The cache's calls on right arguments: two sequences, four rows."""
    k, q = zeros(4, 2, 64), zeros(4, 6, 64)
    table, lens, cu = ints(2, 3), ints(2), at.cumulative([1, 3]).cuda()
    return {
        "kv_append": dict(cache=cache, k=k, v=k.clone(), block_table=table, ctx_lens=lens,
                          cu_seqlens=cu),
        "kv_read": dict(cache=cache, block_table=table, start=lens, cu_seqlens=cu, tokens=4),
        "kv_attention": dict(cache=cache, q=q, block_table=table, kv_lens=lens, cu_seqlens=cu),
    }


def refused(gdn, call, kw, status, *words):
    with pytest.raises(gdn.GdnError) as e:
        call(**kw)
    assert e.value.status == status, str(e.value)
    for w in words:
        assert w in str(e.value), (w, str(e.value))


def test_tensors_of_another_gpu(gdn):
    """The cache's GPU is compared with the tensors' (set to another here: there is one GPU)."""
    cache = gdn.KVCache.empty(4, 2, 16, 64)
    cache._handle.device = cache.k.device.index + 1
    for name, kw in kv_calls(gdn, cache).items():
        refused(gdn, getattr(gdn, name), kw, 1, "cuda:0", "cuda:1")


def odd(t):
    """The same rows with strides that no 16-byte load could follow where a dimension is one."""
    wide = torch.zeros(t.numel() + 4096, dtype=t.dtype, device=t.device)
    strides = [1001 if n == 1 else s for n, s in zip(t.shape[:2], t.stride())] + [1]
    got = wide.as_strided(t.shape, strides)
    return got.copy_(t)


@pytest.mark.parametrize("io", at.IOS, ids=at.IO_IDS)
@pytest.mark.parametrize("T,heads", [(1, 4), (5, 1), (1, 1)])
def test_single_rows_of_any_stride(gdn, T, heads, io):
    """One token, or one head: the results are those of contiguous tensors."""
    gen = torch.Generator("cuda").manual_seed(T + heads)
    q, k, v, dq, dk = (torch.randn(T, heads, 64, device="cuda", generator=gen).to(io)
                       for _ in range(5))
    pos, tab, w = torch.arange(T, device="cuda").int(), at.table(16, 32).cuda(), torch.ones(64).cuda()
    for call, more in ((gdn.qk_norm_rope, ()), (gdn.qk_norm_rope_backward, (dq, dk))):
        want = call(q, k, pos, tab, w, w, *more)
        got = call(odd(q), odd(k), pos, tab, w, w, *more)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    table, held = ints(1, 1), ints(1)
    outs = []
    for f in (lambda t: t, odd):
        cache = gdn.KVCache.empty(1, heads, 16, 64)
        gdn.kv_append(cache, f(k), f(v), table, held, check_status=True)
        outs.append([*gdn.kv_read(cache, table, None, None, T),
                     *gdn.kv_attention(cache, f(q), table, held + T, check_status=True)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def rope_args():
    T, D = 5, 64
    return dict(q=zeros(T, 4, D), k=zeros(T, 2, D), positions=ints(T),
                cos_sin=zeros(8, 32, dtype=torch.float32),
                q_weight=zeros(D, dtype=torch.float32), k_weight=zeros(D, dtype=torch.float32))


def skewed(t):
    """The same values with another order of strides."""
    return t.transpose(0, -1).contiguous().transpose(0, -1)


ROPE_CHANGES = [
    ("q", lambda t: t.float(), 1, "k is"), ("q", lambda t: t.half(), 2, "dtype"),
    ("q", lambda t: t[0], 1, "q is"), ("q", skewed, 1, "last dimension"),
    ("q", lambda t: t[:4], 1, "go together"), ("q", lambda t: t.cpu(), 1, "q is"),
    ("k", lambda t: t.float(), 1, "k is"), ("k", lambda t: t[:4], 1, "go together"),
    ("k", lambda t: t[..., :32], 1, "go together"), ("k", lambda t: t.cpu(), 1, "k is"),
    ("k", lambda t: None, 1, "k is to be a tensor"),
    ("positions", lambda t: t.long(), 1, "positions"), ("positions", lambda t: t[:4], 1, "positions"),
    ("positions", lambda t: t.cpu(), 1, "positions"),
    ("positions", lambda t: ints(10)[::2], 1, "positions"),
    ("cos_sin", lambda t: t.double(), 1, "cos_sin"), ("cos_sin", lambda t: t[0], 1, "cos_sin"),
    ("cos_sin", skewed, 1, "cos_sin"), ("cos_sin", lambda t: t.cpu(), 1, "cos_sin"),
    ("q_weight", lambda t: t[:32], 1, "q_weight"), ("k_weight", lambda t: t.bfloat16(), 1, "k_weight"),
    ("k_weight", lambda t: t.cpu(), 1, "k_weight"),
]


@pytest.mark.parametrize("name,change,status,word", ROPE_CHANGES)
def test_norms_refuse(gdn, name, change, status, word):
    kw = rope_args()
    kw[name] = change(kw[name])
    refused(gdn, gdn.qk_norm_rope, kw, status, word)
    kw.update(dq_out=zeros(5, 4, 64), dk_out=zeros(5, 2, 64))
    refused(gdn, gdn.qk_norm_rope_backward, kw, status, word)


@pytest.mark.parametrize("name,change,status,word", [
    ("dq_out", lambda t: t.float(), 1, "dq_out"), ("dq_out", lambda t: t[:4], 1, "dq_out"),
    ("dk_out", lambda t: zeros(5, 4, 64), 1, "dk_out"), ("dk_out", skewed, 1, "dk_out"),
    ("dk_out", lambda t: t.cpu(), 1, "dk_out"),
    ("dq_out", lambda t: t[:, :1].expand(5, 4, 64), 1, "dq_out"),
    ("workspace", lambda t: zeros(16), 3, "qk_norm_rope_backward"),
    ("workspace", lambda t: torch.zeros(1 << 20), 1, "workspace"),
    ("workspace", lambda t: zeros(1 << 20, 2)[:, 0], 1, "workspace")])
def test_gradients_refuse(gdn, name, change, status, word):
    kw = dict(rope_args(), dq_out=zeros(5, 4, 64), dk_out=zeros(5, 2, 64))
    kw[name] = change(kw.get(name))
    refused(gdn, gdn.qk_norm_rope_backward, kw, status, word)


KV_CHANGES = [
    ("kv_append", "k", lambda t: t.half(), 2, "dtype"), ("kv_append", "k", lambda t: t.float(), 1, "v is"),
    ("kv_append", "k", lambda t: t[:, :1], 1, "k does not fit"),
    ("kv_append", "v", lambda t: t[..., :32], 1, "v does not fit"),
    ("kv_append", "v", lambda t: t[:3], 1, "numbers of tokens"),
    ("kv_append", "v", lambda t: t.cpu(), 1, "v is"), ("kv_append", "v", lambda t: t.float(), 1, "v is"),
    ("kv_append", "ctx_lens", lambda t: t.long(), 1, "lengths"),
    ("kv_append", "ctx_lens", lambda t: ints(3), 1, "lengths"),
    ("kv_append", "ctx_lens", lambda t: None, 1, "kv_append"),
    ("kv_append", "cu_seqlens", lambda t: ints(2), 1, "cu_seqlens"),
    ("kv_append", "cu_seqlens", lambda t: None, 1, "kv_append"),   # four rows of two sequences
    ("kv_append", "block_table", skewed, 1, "block_table"),
    ("kv_append", "block_table", lambda t: t[0], 1, "block_table"),
    ("kv_read", "block_table", lambda t: t.long(), 1, "block_table"),
    ("kv_read", "block_table", lambda t: t.cpu(), 1, "block_table"),
    ("kv_read", "start", lambda t: ints(1), 1, "lengths"),
    ("kv_read", "cu_seqlens", lambda t: t.cpu(), 1, "cu_seqlens"),
    ("kv_read", "tokens", lambda t: -1, 1, "kv_read"),
    ("kv_attention", "q", lambda t: t[..., :32], 1, "q does not fit"),
    ("kv_attention", "q", lambda t: t[:, :5], 1, "kv_attention"),      # five heads over two
    ("kv_attention", "q", lambda t: t.half(), 2, "dtype"), ("kv_attention", "q", skewed, 1, "q is"),
    ("kv_attention", "q", lambda t: t.cpu(), 1, "q is"),
    ("kv_attention", "kv_lens", lambda t: t.float(), 1, "lengths"),
    ("kv_attention", "kv_lens", lambda t: ints(1), 1, "lengths"),
    ("kv_attention", "kv_lens", lambda t: None, 1, "kv_attention"),
    ("kv_attention", "cu_seqlens", lambda t: ints(4), 1, "cu_seqlens"),
    ("kv_attention", "block_table", lambda t: ints(2, 6)[:, ::2], 1, "block_table"),
    ("kv_attention", "window", lambda t: -1, 1, "window"),
    ("kv_attention", "window", lambda t: 1 << 31, 1, "window"),
    ("kv_attention", "workspace", lambda t: zeros(16), 3, "kv_attention"),
    ("kv_attention", "workspace", lambda t: torch.zeros(1 << 26), 1, "workspace"),
]


@pytest.mark.parametrize("call,name,change,status,word", KV_CHANGES)
def test_cache_calls_refuse(gdn, call, name, change, status, word):
    kw = kv_calls(gdn, gdn.KVCache.empty(4, 2, 16, 64))[call]
    kw[name] = change(kw.get(name))
    refused(gdn, getattr(gdn, call), kw, status, word)


@pytest.mark.parametrize("i,change,status,word", [
    (0, lambda t: t.to(torch.uint8), 2, "dtype"), (0, lambda t: t[0], 1, "k is to be"),
    (0, lambda t: zeros(2, 1, 16, 128, dtype=torch.int8)[..., ::2], 1, "k is"),
    (1, lambda t: t.view(2, 1, 16, 64), 1, "v is"),
    (1, lambda t: t.view(torch.float8_e4m3fn), 1, "v is"), (1, lambda t: t.cpu(), 1, "v is"),
    (2, lambda t: t.double(), 1, "k_scale"), (2, lambda t: t[:1], 1, "k_scale"),
    (3, lambda t: t[0], 1, "v_scale"), (3, lambda t: t.cpu(), 1, "v_scale")])
def test_cache_buffers_refused(gdn, i, change, status, word):
    buffers = [zeros(2, 1, 16, 64, dtype=torch.int8), zeros(2, 1, 4, 64, 4, dtype=torch.int8),
               zeros(2, 1, dtype=torch.float32), zeros(2, 1, dtype=torch.float32)]
    gdn.KVCache(*buffers)
    buffers[i] = change(buffers[i])
    with pytest.raises(gdn.GdnError) as e:
        gdn.KVCache(*buffers)
    assert e.value.status == status and word in str(e.value)
