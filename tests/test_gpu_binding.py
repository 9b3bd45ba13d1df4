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
