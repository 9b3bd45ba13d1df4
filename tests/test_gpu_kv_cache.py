"""GPU: the 8-bit paged cache, written (gdn_kv_append) and read back (gdn_kv_read).

The append's arithmetic is stated operation by operation in include/gdn.h, so codes and scales are
compared for equality with a plain form of it; values read back are code * scale, one rounding.
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


class Pool:
    """A cache on the GPU and its logical copy on the CPU."""

    def __init__(self, gdn, pages, hkv, page, D, fmt, gen):
        self.kc, self.ks = at.random_cache(pages, hkv, page, D, fmt, gen)
        self.vc, self.vs = at.random_cache(pages, hkv, page, D, fmt, gen, 0.3)
        self.page, self.fmt = page, fmt
        self.cache = gdn.KVCache(self.kc.cuda(), at.packed_v(self.vc).cuda(), self.ks.cuda(),
                                 self.vs.cuda())

    def append(self, gdn, k, v, tables, ctx, new, cu="packed", **kw):
        at.append_ref(self.kc, self.ks, k, tables, ctx, new, self.page, self.fmt)
        at.append_ref(self.vc, self.vs, v, tables, ctx, new, self.page, self.fmt)
        cu = at.cumulative(new).cuda() if cu == "packed" else cu
        gdn.kv_append(self.cache, k.cuda(), v.cuda(), tables.cuda(),
                      torch.tensor(ctx, dtype=torch.int32).cuda(), cu, **kw)

    def check(self, tables, lens):
        """Every token of every sequence has the plain form's code, and the scales agree."""
        for got, codes in ((self.cache.k, self.kc), (at.unpacked_v(self.cache.v), self.vc)):
            got, codes = at.values(got).cpu(), at.values(codes)
            for n, L in enumerate(lens):
                for p in range(-(-L // self.page)):
                    t = min(self.page, L - p * self.page)
                    pid = int(tables[n, p])
                    assert torch.equal(got[pid, :, :t], codes[pid, :, :t]), (n, p)
        assert torch.equal(self.cache.k_scale.cpu(), self.ks)
        assert torch.equal(self.cache.v_scale.cpu(), self.vs)


def draws(gen, T, hkv, D, io, std=1.0):
    return [(torch.randn(T, hkv, D, generator=gen) * std).to(io) for _ in range(2)]


SHAPES = [(1, 64, 16), (3, 128, 64), (2, 256, 128), (5, 128, 32), (1, 256, 16)]


@pytest.mark.parametrize("io", at.IOS, ids=at.IO_IDS)
@pytest.mark.parametrize("fmt", at.FORMATS, ids=at.FORMAT_IDS)
@pytest.mark.parametrize("hkv,D,page", SHAPES)
def test_append_matches_plain_form(gdn, hkv, D, page, fmt, io):
    """Packed prompts of odd lengths: empty ones, ones inside a page, ones that end on its edge,
    ones that continue a part-filled page (whose values here are larger and smaller than the
    new ones, so that its scale grows or stays)."""
    gen = torch.Generator().manual_seed(D + page + hkv)
    ctx = [0, 5, page, page - 1, 2 * page + 3, 7, 0, page + page // 2]
    new = [1, 0, page, 1, 3 * page - 3, 2, 2 * page + 5, page // 2]
    lens = [a + b for a, b in zip(ctx, new)]
    tables, pages = at.block_tables(lens, page, gen)
    pool = Pool(gdn, pages, hkv, page, D, fmt, gen)
    k, v = draws(gen, sum(new), hkv, D, io, 1.3)
    pool.append(gdn, k, v, tables, ctx, new, check_status=True)
    pool.check(tables, lens)


@pytest.mark.parametrize("hkv", [22, 41])
@pytest.mark.parametrize("fmt", at.FORMATS, ids=at.FORMAT_IDS)
def test_many_heads_and_pages(gdn, hkv, fmt):
    """Enough pages and heads that a CTA takes several heads of a page (22: two for the append; 41:
    four, and two for the read back), the last of them fewer; one value in some heads is not
    finite."""
    gen = torch.Generator().manual_seed(hkv)
    page, D = 16, 64
    ctx, new = [3, 0, 40], [700, 1, 1400]
    lens = [a + b for a, b in zip(ctx, new)]
    tables, pages = at.block_tables(lens, page, gen)
    pool = Pool(gdn, pages, hkv, page, D, fmt, gen)
    k, v = draws(gen, sum(new), hkv, D, torch.bfloat16)
    k[100, 1, 5], k[1500, hkv - 1, 63], v[700, 2, 0] = float("inf"), float("nan"), -float("inf")
    pool.append(gdn, k, v, tables, ctx, new)
    pool.check(tables, lens)
    got = gdn.kv_read(pool.cache, tables.cuda(), None, at.cumulative(lens).cuda(), sum(lens),
                      torch.float32)
    for out, codes, scales in zip(got, (pool.kc, pool.vc), (pool.ks, pool.vs)):
        values = at.values(codes).float()
        for n, first in enumerate(at.cumulative(lens)[:-1].tolist()):
            pos = torch.arange(lens[n])
            pid = tables[n].long()[pos // page]
            want = values[pid, :, pos % page] * scales[pid][:, :, None]
            assert torch.equal(out[first:first + lens[n]].cpu(), want)


@pytest.mark.parametrize("fmt", at.FORMATS, ids=at.FORMAT_IDS)
def test_token_by_token(gdn, fmt):
    """Seventy single tokens of growing size for each of five sequences, without cu_seqlens: pages
    fill, and their earlier codes follow the scale each time."""
    gen = torch.Generator().manual_seed(3)
    page, hkv, D, N = 32, 2, 128, 5
    ctx = [0, 3, 31, 32, 40]
    tables, pages = at.block_tables([c + 70 for c in ctx], page, gen)
    pool = Pool(gdn, pages, hkv, page, D, fmt, gen)
    for i in range(70):
        k, v = draws(gen, N, hkv, D, torch.bfloat16, 0.5 + 0.03 * (i % 40))
        pool.append(gdn, k, v, tables, [c + i for c in ctx], [1] * N, cu=None)
    pool.check(tables, [c + 70 for c in ctx])


def test_strided_inputs(gdn):
    """Keys and values as slices of one projection."""
    gen = torch.Generator().manual_seed(5)
    hkv, D, page, T = 3, 128, 16, 45
    tables, pages = at.block_tables([T], page, gen)
    pool = Pool(gdn, pages, hkv, page, D, torch.int8, gen)
    proj = torch.randn(T, 2 * hkv * D + 64, generator=gen).bfloat16().cuda()
    k = proj[:, 32:32 + hkv * D].view(T, hkv, D)
    v = proj[:, 64 + hkv * D:].view(T, hkv, D)
    at.append_ref(pool.kc, pool.ks, k.cpu(), tables, [0], [T], page, torch.int8)
    at.append_ref(pool.vc, pool.vs, v.cpu(), tables, [0], [T], page, torch.int8)
    gdn.kv_append(pool.cache, k, v, tables.cuda(), torch.zeros(1, dtype=torch.int32).cuda())
    pool.check(tables, [T])


@pytest.mark.parametrize("fmt", at.FORMATS, ids=at.FORMAT_IDS)
@pytest.mark.parametrize("io", at.IOS, ids=at.IO_IDS)
def test_zero_tiny_and_non_finite_values(gdn, io, fmt):
    """Pages of zeros and of values below 2^-100 get scale 0 (a later token wakes such a page);
    infinities take the largest code, NaN 0, and both are reported."""
    gen = torch.Generator().manual_seed(7)
    page, hkv, D = 16, 1, 64
    tables, pages = at.block_tables([18, 18, 18, 18], page, gen)
    pool = Pool(gdn, pages, hkv, page, D, fmt, gen)
    k, v = draws(gen, 72, hkv, D, io)
    k[:16], v[18:34] = 0, 1e-32
    k[16:18] = 0
    pool.append(gdn, k, v, tables, [0] * 4, [18] * 4, check_status=True)
    pool.check(tables, [18] * 4)
    assert float(pool.cache.k_scale[int(tables[0, 0]), 0]) == 0.0
    assert float(pool.cache.v_scale[int(tables[1, 0]), 0]) == 0.0
    k, v = draws(gen, 4, hkv, D, io)
    k[1, 0, 5], k[1, 0, 6], v[2, 0, 0] = float("inf"), -float("inf"), float("nan")
    k[3, 0] = float("inf")  # nothing finite in a page that holds values
    with pytest.raises(gdn.GdnError) as e:
        pool.append(gdn, k, v, tables, [18] * 4, [1] * 4, check_status=True)
    assert e.value.status == 7
    pool.check(tables, [19] * 4)


def test_stale_scale_of_a_reused_page_is_ignored(gdn):
    gen = torch.Generator().manual_seed(9)
    tables, pages = at.block_tables([10], 16, gen)
    pool = Pool(gdn, pages, 2, 16, 64, torch.int8, gen)
    pool.cache.k_scale.fill_(1e6)
    pool.cache.v_scale.fill_(float("nan"))
    pool.ks.fill_(1e6)
    pool.vs.fill_(float("nan"))
    k, v = draws(gen, 10, 2, 64, torch.float32)
    pool.append(gdn, k, v, tables, [0], [10])
    pid = int(tables[0, 0])
    assert torch.equal(pool.cache.v_scale[pid].cpu(), pool.vs[pid])
    assert torch.equal(pool.cache.k_scale[pid].cpu(), pool.ks[pid])


@pytest.mark.parametrize("io", at.IOS, ids=at.IO_IDS)
@pytest.mark.parametrize("fmt", at.FORMATS, ids=at.FORMAT_IDS)
@pytest.mark.parametrize("hkv,D,page", SHAPES)
def test_read_back(gdn, hkv, D, page, fmt, io):
    gen = torch.Generator().manual_seed(D * hkv + page)
    start = [0, 3, page - 1, page, 0, 2 * page + 1]
    count = [1, 2 * page, 2, page, 0, page - 3]
    tables, pages = at.block_tables([a + b for a, b in zip(start, count)], page, gen)
    pool = Pool(gdn, pages, hkv, page, D, fmt, gen)
    k, v = gdn.kv_read(pool.cache, tables.cuda(), torch.tensor(start, dtype=torch.int32).cuda(),
                       at.cumulative(count).cuda(), sum(count), io, check_status=True)
    for got, codes, scales in ((k, pool.kc, pool.ks), (v, pool.vc, pool.vs)):
        want = []
        for n, (a, c) in enumerate(zip(start, count)):
            for pos in range(a, a + c):
                pid = int(tables[n, pos // page])
                want.append(at.values(codes[pid, :, pos % page]) * scales[pid][:, None])
        assert torch.equal(got.cpu(), torch.stack(want).to(io))


def test_every_code_reads_back(gdn):
    """All 256 codes (e4m3's two NaN codes aside), keys and values."""
    for fmt in at.FORMATS:
        codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(1, 1, 4, 64)
        codes = codes.repeat(1, 1, 4, 1).contiguous().view(fmt)
        one = torch.full((1, 1), 0.5)
        cache = gdn.KVCache(codes.cuda(), at.packed_v(codes).cuda(), one.cuda(), one.cuda())
        k, v = gdn.kv_read(cache, torch.zeros(1, 1, dtype=torch.int32).cuda(), None, None, 16,
                           torch.float32)
        want = at.values(codes)[0, 0] * 0.5
        ok = ~torch.isnan(want)
        for got in (k, v):
            assert torch.equal(got[:, 0].cpu()[ok], want[ok])


def test_bad_tables_are_reported_and_skipped(gdn):
    """A length past the table, a page outside the pool, a negative length: those sequences leave
    the cache as it was; the others are written."""
    gen = torch.Generator().manual_seed(11)
    page = 16
    tables, pages = at.block_tables([32] * 5, page, gen)
    pool = Pool(gdn, pages, 1, page, 64, torch.int8, gen)
    before = [x.clone() for x in (pool.cache.k, pool.cache.v, pool.cache.k_scale)]
    k, v = draws(gen, 5 * 8, 1, 64, torch.bfloat16)
    bad = tables.clone()
    bad[1, 0], bad[4, 0] = pages, -5
    ctx = [4, 4, 30, -1, 4]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = gdn.KvProblem(40, 5, 2, 0, gdn.GDN_BF16, 64, 64, 64, 64, 0, 0)
    gdn.gdn_kv_append(pool.cache.desc, p, k.cuda(), v.cuda(), bad.cuda(),
                      torch.tensor(ctx, dtype=torch.int32).cuda(),
                      at.cumulative([8] * 5).cuda(), st)
    assert gdn.gdn_device_status(st) == 6
    for n in range(1, 5):
        for pid in tables[n].tolist():
            for x, y in zip(before, (pool.cache.k, pool.cache.v, pool.cache.k_scale)):
                assert torch.equal(x[pid].view(torch.uint8), y[pid].view(torch.uint8)), n
    at.append_ref(pool.kc, pool.ks, k[:8], tables[:1], [4], [8], page, torch.int8)
    assert torch.equal(pool.cache.k[int(tables[0, 0]), :, :12].cpu(),
                       pool.kc[int(tables[0, 0]), :, :12])
    # a table of rows that does not ascend reaches no row outside [0, T)
    cu = torch.tensor([0, 8, 60, 24, 32, 40], dtype=torch.int32).cuda()
    gdn.gdn_kv_append(pool.cache.desc, p, k.cuda(), v.cuda(), tables.cuda(),
                      torch.zeros(5, dtype=torch.int32).cuda(), cu, st)
    assert gdn.gdn_device_status(st) == 6


def test_many_short_sequences(gdn):
    """More sequences than one search step covers, most of them empty."""
    gen = torch.Generator().manual_seed(13)
    page, N = 16, 1500
    new = [int(x) for x in torch.randint(0, 4, (N,), generator=gen)]
    ctx = [int(x) for x in torch.randint(0, 20, (N,), generator=gen)]
    lens = [a + b for a, b in zip(ctx, new)]
    tables, pages = at.block_tables(lens, page, gen)
    pool = Pool(gdn, pages, 1, page, 64, torch.int8, gen)
    k, v = draws(gen, sum(new), 1, 64, torch.bfloat16)
    pool.append(gdn, k, v, tables, ctx, new, check_status=True)
    pool.check(tables, lens)


def test_offsets_past_32_bits(gdn):
    """Pages whose bytes lie beyond 2^32 in both halves of the cache."""
    page, hkv, D = 128, 8, 256
    pages = (1 << 32) // (page * hkv * D) + 3
    cache = gdn.KVCache.empty(pages, hkv, page, D)
    gen = torch.Generator().manual_seed(17)
    k, v = draws(gen, 130, hkv, D, torch.bfloat16)
    tables = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32)
    gdn.kv_append(cache, k.cuda(), v.cuda(), tables.cuda(),
                  torch.zeros(1, dtype=torch.int32).cuda(), check_status=True)
    small_k, ks = torch.zeros(2, hkv, page, D, dtype=torch.int8), torch.zeros(2, hkv)
    small_v, vs = small_k.clone(), ks.clone()
    order = torch.tensor([[1, 0]])
    at.append_ref(small_k, ks, k, order, [0], [130], page, torch.int8)
    at.append_ref(small_v, vs, v, order, [0], [130], page, torch.int8)
    gk, gv = gdn.kv_read(cache, tables.cuda(), None, None, 130, torch.float32, check_status=True)
    for got, codes, s in ((gk, small_k, ks), (gv, small_v, vs)):
        want = torch.cat([at.values(codes[1]) * s[1][:, None, None],
                          (at.values(codes[0]) * s[0][:, None, None])[:, :2]], 1)
        assert torch.equal(got.cpu(), want.transpose(0, 1))


def test_no_tokens(gdn):
    cache = gdn.KVCache.empty(2, 1, 16, 64)
    e = torch.empty(0, 1, 64, device="cuda")
    t = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    gdn.kv_append(cache, e, e, t, torch.zeros(1, dtype=torch.int32, device="cuda"))
    k, v = gdn.kv_read(cache, t, None, None, 0)
    assert k.shape == (0, 1, 64) and v.shape == (0, 1, 64)
