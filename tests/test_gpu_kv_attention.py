"""GPU: attention over the 8-bit paged cache (gdn_kv_attention) against fp64.

Tolerances, from the arithmetic.  A score is a sum of D exact products accumulated in fp32 (a
product of the inputs and the code is exact in the operands used; fp32 inputs are split in two):
rounding errors of at most 2^-23 of the running sum add up like a walk, sqrt(D) 2^-23 sum |q k|
scale, below 2^-14 for the inputs here (D <= 256, sum |q k| scale < 20).  A weight's relative error
is that of exp: the score's error plus 2^-21.  bf16: weights are rounded to fp16 (2^-11 each), so
out is off by at most (2^-11 + 2^-14 + ..) sum p |v| and half an ulp of 8 significant bits,
2^-8 |out|; fp16's smallest step,
2^-24, is 2^-32 of a row's largest weight, so every key may add half that of the largest value: the
bound is 2^-10 sum p |v| + 2^-8 |out| + 2^-33 keys max |v|.  fp32: 2^-13 sum p |v| (twice the score's bound).  lse: the score's
bound, 2^-13 with the sum's and log's.
"""
import itertools
import math

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


def check(out, lse, ref, io, what="", floor=0.0):
    o, l, mag = ref
    out, lse = out.double().cpu(), lse.double().cpu()
    if io == torch.bfloat16:
        tol = 2.0 ** -10 * mag + 2.0 ** -8 * o.abs() + floor
    else:
        tol = 2.0 ** -13 * mag
    err = (out - o).abs()
    assert not torch.isnan(out).any(), what
    assert bool((err <= tol).all()), (what, float((err - tol).max()), int((err > tol).sum()))
    empty = torch.isinf(l)
    assert torch.equal(torch.isinf(lse), empty) and bool((lse[empty] < 0).all()), what
    assert bool(((lse - l).abs()[~empty] <= 2.0 ** -13 * l.abs().clamp(min=1)[~empty]).all()), what


class Problem:
    def __init__(self, gdn, lens, new, hq, hkv, D, page, fmt, io, seed=0, std_q=1.2, junk=-1):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.new, self.page, self.io = lens, new, page, io
        self.tables, pages = at.block_tables(lens, page, gen, junk=junk)
        self.kc, self.ks = at.random_cache(pages, hkv, page, D, fmt, gen)
        self.vc, self.vs = at.random_cache(pages, hkv, page, D, fmt, gen, 0.4)
        self.q = (std_q * torch.randn(sum(new), hq, D, generator=gen)).to(io)
        self.gdn, self.D = gdn, D
        self.load()

    def load(self):
        self.cache = self.gdn.KVCache(self.kc.cuda(), at.packed_v(self.vc).cuda(), self.ks.cuda(),
                                      self.vs.cuda())

    def run(self, window=0, cu="packed", q=None, **kw):
        cu = at.cumulative(self.new).cuda() if cu == "packed" else cu
        kw.setdefault("check_status", True)
        return self.gdn.kv_attention(self.cache, self.q.cuda() if q is None else q,
                                     self.tables.cuda(),
                                     torch.tensor(self.lens, dtype=torch.int32).cuda(), cu,
                                     window=window, **kw)

    def ref(self, window=0, scale=None):
        return at.attention_ref(self.q, self.kc, self.ks, self.vc, self.vs, self.tables,
                                self.lens, self.new, self.page,
                                self.D ** -0.5 if scale is None else scale, window)


def edge_lengths(page):
    return [0, 1, 2, 15, 16, 17, page - 1, page, page + 1, 3 * page + 5, 31, 33, 64, 65, 777]


@pytest.mark.parametrize("io", at.IOS, ids=at.IO_IDS)
@pytest.mark.parametrize("fmt", at.FORMATS, ids=at.FORMAT_IDS)
@pytest.mark.parametrize("hq,hkv,D,page", [(8, 1, 128, 64), (3, 3, 64, 16), (16, 2, 256, 64),
                                           (12, 1, 128, 32), (16, 1, 64, 128), (14, 2, 256, 16),
                                           (20, 1, 128, 16), (40, 1, 256, 32), (10, 2, 64, 32)])
def test_one_query_per_sequence(gdn, hq, hkv, D, page, fmt, io):
    lens = edge_lengths(page)
    p = Problem(gdn, lens, [1] * len(lens), hq, hkv, D, page, fmt, io, seed=hq + D)
    check(*p.run(), p.ref(), io)
    check(*p.run(cu=None), p.ref(), io)


@pytest.mark.parametrize("io", at.IOS, ids=at.IO_IDS)
@pytest.mark.parametrize("fmt", at.FORMATS, ids=at.FORMAT_IDS)
@pytest.mark.parametrize("window", [0, 1, 7, 100])
@pytest.mark.parametrize("hq,hkv,D,page", [(8, 2, 128, 64), (7, 1, 64, 16), (4, 4, 256, 32)])
def test_several_queries_and_windows(gdn, hq, hkv, D, page, window, fmt, io):
    """Drafted tokens: each row has its own last key; rows before the first key (more rows than
    tokens) are empty; sequences without rows take no part."""
    lens = [0, 1, 3, 40, 129, 300, 64, 16, 500]
    new = [2, 3, 3, 5, 1, 9, 0, 16, 33]
    p = Problem(gdn, lens, new, hq, hkv, D, page, fmt, io, seed=window + D)
    check(*p.run(window), p.ref(window), io)


@pytest.mark.parametrize("fmt", at.FORMATS, ids=at.FORMAT_IDS)
@pytest.mark.parametrize("group,D", [(4, 128), (5, 64), (4, 256)])
def test_some_sequences_with_many_rows(gdn, group, D, fmt):
    """Few rows on average (so the few-rows kernel), many in some sequences: several row tiles."""
    new = [1, 9, 1, 1, 2, 17, 1, 1, 1]
    lens = [700, 33, 1, 0, 64, 2000, 128, 16, 15]
    p = Problem(gdn, lens, new, 2 * group, 2, D, 32, fmt, torch.bfloat16, seed=group + D)
    check(*p.run(), p.ref(), torch.bfloat16)


@pytest.mark.parametrize("io", at.IOS, ids=at.IO_IDS)
def test_long_sequences_are_split_and_joined(gdn, io):
    """One long sequence among short ones: work split over its length and joined."""
    lens, new = [20011, 5, 3000, 1], [1, 1, 2, 1]
    for hq, hkv, D, page, fmt in ((8, 1, 128, 64, torch.int8), (4, 2, 64, 16, at.FORMATS[1]),
                                  (16, 2, 256, 128, torch.int8), (12, 1, 128, 32, at.FORMATS[1]),
                                  (40, 2, 64, 64, torch.int8), (64, 1, 128, 16, torch.int8)):
        p = Problem(gdn, lens, new, hq, hkv, D, page, fmt, io, seed=D)
        check(*p.run(), p.ref(), io, (hq, D))


def test_many_sequences(gdn):
    gen = torch.Generator().manual_seed(1)
    lens = [int(x) for x in torch.randint(0, 90, (700,), generator=gen)]
    new = [int(x) for x in torch.randint(0, 3, (700,), generator=gen)]
    lens = [max(a, b) if a else 0 for a, b in zip(lens, new)]
    p = Problem(gdn, lens, new, 4, 2, 64, 16, torch.int8, torch.bfloat16)
    check(*p.run(), p.ref(), torch.bfloat16)


@pytest.mark.parametrize("hq", [6, 32])  # few rows, and many (another kernel)
@pytest.mark.parametrize("fmt", at.FORMATS, ids=at.FORMAT_IDS)
def test_bytes_past_the_length_do_not_count(gdn, fmt, hq):
    """Unused slots of a last page hold every byte there is (e4m3's NaN codes too), unused table
    entries any number, unused pages' scales NaN: the result does not change by a bit."""
    lens, new, page = [1, 18, 45, 64, 0], [1, 1, 3, 1, 1], 32
    p = Problem(gdn, lens, new, hq, 2, 128, page, fmt, torch.bfloat16, seed=4)
    want = p.run()
    check(*want, p.ref(), torch.bfloat16)
    used = set()
    for n, L in enumerate(lens):
        for i in range(-(-L // page)):
            pid = int(p.tables[n, i])
            used.add(pid)
            t = min(page, L - i * page)
            for codes in (p.kc, p.vc):
                raw = codes.view(torch.uint8)
                fill = torch.tensor([0x7f, 0xff, 0x80, 0x7e], dtype=torch.uint8).repeat(32)
                raw[pid, :, t:] = fill[:128]
    for pid in range(p.ks.shape[0]):
        if pid not in used:
            p.ks[pid] = float("nan")
            p.vs[pid] = float("inf")
    for junk in (-1, 10 ** 9, -2 ** 31):
        for n, L in enumerate(lens):
            p.tables[n, -(-L // page):] = junk
        p.load()
        got = p.run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_many_rows(gdn):
    """More rows than one row tile holds, of one sequence and of several; the maximum of a row
    moves late (large keys at the end) and early; odd counts."""
    for hq, hkv, D, page, new, lens in ((64, 1, 128, 32, [3, 1], [700, 129]),
                                        (24, 2, 64, 16, [11, 40], [300, 77]),
                                        (7, 1, 128, 128, [100], [515]),
                                        (10, 1, 64, 64, [64, 0, 1], [64, 10, 2])):
        for fmt in at.FORMATS:
            for window in (0, 50):
                p = Problem(gdn, lens, new, hq, hkv, D, page, fmt, torch.bfloat16, seed=hq)
                late = p.tables[0, (lens[0] - 1) // page]
                p.ks[late] *= 8
                p.load()
                floor = 2.0 ** -33 * max(lens) * float(p.vs.max()) * at.QMAX[fmt]
                check(*p.run(window), p.ref(window), torch.bfloat16, (hq, D, fmt, window), floor)


def test_scales_of_very_different_pages(gdn):
    """Pages whose value scales differ by up to 2^80 and key scales by 2^6, a page of zeros among
    them, with the weight on the page of small values: the sum keeps its relative accuracy."""
    for fmt, io, hq in itertools.product(at.FORMATS, at.IOS, (2, 12)):
        p = Problem(gdn, [16 * 6], [1], hq, 1, 128, 16, fmt, io, seed=8, std_q=0.3)
        ids = p.tables[0].long()
        p.vs[ids, 0] *= torch.tensor([1.0, 2.0 ** -40, 2.0 ** 40, 2.0 ** -14, 0.0, 1.0])
        p.ks[ids, 0] *= torch.tensor([1.0, 64.0, 0.01, 1.0, 1.0, 0.0])
        p.load()
        check(*p.run(), p.ref(), io, (fmt, io))
    # all the weight on the small page
    p = Problem(gdn, [32], [1], 1, 1, 64, 16, torch.int8, torch.bfloat16, seed=9)
    ids = p.tables[0].long()
    p.kc[ids[0]], p.kc[ids[1]] = 1, -1
    p.ks[ids] = 40.0 / 64
    p.q[:] = 1.0
    p.vs[ids, 0] = torch.tensor([2.0 ** -60, 1.0])
    p.load()
    check(*p.run(), p.ref(), torch.bfloat16, "weight on the small page")


@pytest.mark.parametrize("io", at.IOS, ids=at.IO_IDS)
def test_large_and_small_queries(gdn, io):
    """Queries far outside the fp16 range (their scores brought back by `scale`), tiny ones and
    zeros."""
    p = Problem(gdn, [70, 70, 70], [1, 1, 1], 4, 2, 128, 32, torch.int8, io, seed=10)
    p.q[0] *= 2.0 ** 60
    check(*(x[:1] for x in p.run(scale=2.0 ** -62)),
          tuple(x[:1] for x in p.ref(scale=2.0 ** -62)), io)
    p.q[0], p.q[1] = 0, p.q[1] * 2.0 ** -40
    check(*p.run(), p.ref(), io)


def test_strided_queries(gdn):
    """Queries as the first half of each head of a gated projection."""
    p = Problem(gdn, [100, 33], [1, 2], 8, 2, 128, 64, torch.int8, torch.bfloat16, seed=12)
    wide = torch.randn(3, 8, 256).bfloat16().cuda()
    wide[:, :, :128] = p.q.cuda()
    check(*p.run(q=wide[:, :, :128]), p.ref(), torch.bfloat16)


def test_shared_pages(gdn):
    """Two sequences whose tables share a prefix."""
    p = Problem(gdn, [100, 120], [1, 1], 4, 2, 64, 16, torch.int8, torch.bfloat16, seed=13)
    p.tables[1, :6] = p.tables[0, :6]
    check(*p.run(), p.ref(), torch.bfloat16)


def test_bad_lengths_and_pages_are_reported(gdn):
    p = Problem(gdn, [40, 40, 40], [1, 1, 1], 4, 2, 64, 16, torch.int8, torch.bfloat16, seed=14)
    ref = p.ref()
    tables = p.tables.clone()
    p.lens = [40, 49, 40]          # past the table's 3 pages
    with pytest.raises(gdn.GdnError) as e:
        p.run()
    assert e.value.status == 6
    got = p.run(check_status=False)
    for i in (0, 2):
        check(got[0][i:i + 1], got[1][i:i + 1], tuple(x[i:i + 1] for x in ref), torch.bfloat16)
    p.lens = [40, 40, 40]
    p.tables[2, 1] = p.ks.shape[0]  # outside the pool: its keys are left out
    with pytest.raises(gdn.GdnError) as e:
        p.run()
    assert e.value.status == 6
    got = p.run(check_status=False)
    p.tables = tables
    for i in (0, 1):
        check(got[0][i:i + 1], got[1][i:i + 1], tuple(x[i:i + 1] for x in ref), torch.bfloat16)
    assert not torch.isnan(got[0]).any()


def test_repeats_bit_for_bit_and_on_another_stream(gdn):
    p = Problem(gdn, [9000, 3, 1200], [2, 1, 1], 16, 2, 128, 64, torch.int8, torch.bfloat16)
    want = p.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for kw in ({}, {}, {"stream": s}):
        got = p.run(**kw)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_one_workspace_for_many_calls(gdn):
    """A workspace kept by the caller, filled with other calls' contents and with junk."""
    p = Problem(gdn, [5000, 100], [1, 1], 8, 1, 128, 64, torch.int8, torch.bfloat16, seed=20)
    o = Problem(gdn, [50, 4000], [3, 1], 8, 1, 128, 64, torch.int8, torch.bfloat16, seed=21)
    want, other = p.run(), o.run()
    ws = torch.full((64 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(p.run(workspace=ws)[0], want[0])
        assert torch.equal(o.run(workspace=ws)[0], other[0])


def test_offsets_past_32_bits(gdn):
    """Pages beyond 2^32 bytes of a large cache give what the same pages of a small one give."""
    page, hkv, D = 128, 8, 256
    pages = (1 << 32) // (page * hkv * D) + 3
    p = Problem(gdn, [300], [1], 16, hkv, D, page, torch.int8, torch.bfloat16, seed=22)
    want = p.run()
    ids = p.tables[0].long()
    big = gdn.KVCache.empty(pages, hkv, page, D)
    far = torch.tensor([pages - 1, 0, pages - 2])
    big.k[far.cuda()], big.v[far.cuda()] = p.cache.k[ids.cuda()], p.cache.v[ids.cuda()]
    big.k_scale[far.cuda()] = p.cache.k_scale[ids.cuda()]
    big.v_scale[far.cuda()] = p.cache.v_scale[ids.cuda()]
    p.cache, p.tables = big, far.int()[None]
    got = p.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_graph_capture(gdn):
    """A captured call replays on new contents of the same buffers."""
    p = Problem(gdn, [600, 40], [1, 1], 8, 2, 128, 64, torch.int8, torch.bfloat16, seed=23)
    q, tables = p.q.cuda(), p.tables.cuda()
    lens = torch.tensor(p.lens, dtype=torch.int32).cuda()
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    gdn.kv_attention(p.cache, q, tables, lens, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = gdn.kv_attention(p.cache, q, tables, lens, workspace=ws)
    for new_lens in ([600, 40], [1, 33], [311, 0]):
        lens.copy_(torch.tensor(new_lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        p.lens = new_lens
        check(out, lse, p.ref(), torch.bfloat16, new_lens)


def test_append_then_attend_matches_unquantised(gdn):
    """The whole path: appended prompts and single tokens, then attention, against fp64 attention
    over what the cache reads back."""
    gen = torch.Generator().manual_seed(30)
    hq, hkv, D, page = 8, 2, 128, 32
    lens = [70, 5]
    cache = gdn.KVCache.empty(8, hkv, page, D)
    tables = torch.tensor([[3, 1, 7], [2, 0, 5]], dtype=torch.int32).cuda()
    k, v = [torch.randn(75, hkv, D, generator=gen).bfloat16().cuda() for _ in range(2)]
    gdn.kv_append(cache, k, v, tables, torch.zeros(2, dtype=torch.int32).cuda(),
                  at.cumulative(lens).cuda(), check_status=True)
    for step in range(3):
        held = torch.tensor(lens, dtype=torch.int32).cuda()
        k, v = [torch.randn(2, hkv, D, generator=gen).bfloat16().cuda() for _ in range(2)]
        q = torch.randn(2, hq, D, generator=gen).bfloat16().cuda()
        gdn.kv_append(cache, k, v, tables, held, check_status=True)
        out, lse = gdn.kv_attention(cache, q, tables, held + 1, check_status=True)
        lens = [n + 1 for n in lens]
        kk, vv = gdn.kv_read(cache, tables, None, at.cumulative(lens).cuda(), sum(lens),
                             torch.float32)
        at0 = 0
        for n, L in enumerate(lens):
            kn, vn = kk[at0:at0 + L].double().cpu(), vv[at0:at0 + L].double().cpu()
            at0 += L
            x = torch.einsum("hgd,jhd->hgj", q[n].double().cpu().view(hkv, hq // hkv, D), kn)
            w = torch.softmax(x / math.sqrt(D), -1)
            want = torch.einsum("hgj,jhd->hgd", w, vn).reshape(hq, D)
            mag = torch.einsum("hgj,jhd->hgd", w, vn.abs()).reshape(hq, D)
            err = (out[n].double().cpu() - want).abs()
            assert bool((err <= 2.0 ** -10 * mag + 2.0 ** -8 * want.abs()).all())


# Rows a kv head of the two kernels for bf16 and D <= 128 (more than sixteen: the one on tcgen05, with
# items of 32 or 64 rows); fp32 has one.
ROWS = [2, 24, 40]


def check_range(out, lse, ref, io, lens, p, fmt, what=""):
    """As `check`, with the floor that fp16's smallest step leaves: a weight off by 2^-25 where the
    row's largest (page scales included) is 2^8 at least, so 2^-33 of the largest value a key."""
    floor = 2.0 ** -33 * max(lens) * float(p.vs.max()) * at.QMAX[fmt]
    o, l, mag = ref
    check(out, lse, (o, l, mag + 2.0 ** 13 * floor if io == torch.float32 else mag), io, what, floor)


@pytest.mark.parametrize("io", at.IOS, ids=at.IO_IDS)
@pytest.mark.parametrize("fmt", at.FORMATS, ids=at.FORMAT_IDS)
@pytest.mark.parametrize("rows", ROWS)
def test_many_keys_of_any_value_scale(gdn, rows, fmt, io):
    """Twenty thousand keys of nearly the same score, with value scales from the smallest that an
    append writes (2^-100 over the largest code) to large ones, and all of them zero."""
    least = 2.0 ** -100 / at.QMAX[fmt]
    p = Problem(gdn, [20000], [1], rows, 1, 64, 128, fmt, io, seed=40 + rows, std_q=0.01)
    for scale in (least, 2.0 ** -60, 2.0 ** 60, 2.0 ** 110, 0.0):
        p.vs[:] = scale
        p.load()
        check_range(*p.run(), p.ref(), io, p.lens, p, fmt, scale)


@pytest.mark.parametrize("io", at.IOS, ids=at.IO_IDS)
@pytest.mark.parametrize("fmt", at.FORMATS, ids=at.FORMAT_IDS)
@pytest.mark.parametrize("rows", ROWS)
def test_small_scales_and_late_scores(gdn, rows, fmt, io):
    """The smallest value scales, and scores that rise by 2^6, where the reference stays."""
    p = Problem(gdn, [1200], [1], rows, 1, 64, 16, fmt, io, seed=50 + rows)
    ids = p.tables[0].long()
    p.q[:] = 1.0
    p.kc.view(torch.uint8)[:] = at.encode(torch.ones(1), fmt).view(torch.uint8)
    p.ks[ids, 0] = 0.0
    p.ks[ids[8:], 0] = 4.2 / 64 ** 0.5  # 64 products of 1 and 1, scaled by 64^-1/2: 4.2 = 6 ln 2
    p.vs[:] = 2.0 ** -100 / at.QMAX[fmt]
    p.load()
    check_range(*p.run(), p.ref(), io, p.lens, p, fmt)


@pytest.mark.parametrize("io", at.IOS, ids=at.IO_IDS)
@pytest.mark.parametrize("fmt", at.FORMATS, ids=at.FORMAT_IDS)
@pytest.mark.parametrize("rows", ROWS)
def test_pages_of_zeros_among_others(gdn, rows, fmt, io):
    """Pages of value scale 0 (their codes are not zeros here) first, last, and among pages of large
    and of small scales: they take their share of the weights and give nothing."""
    for lens in ([1000, 30], [5000, 16]):
        p = Problem(gdn, lens, [1, 1], rows, 1, 64, 16, fmt, io, seed=60 + rows, std_q=0.3)
        drawn = p.vs.clone()
        for scale in (2.0 ** 60, 1.0, 2.0 ** -60):
            for zeros in (slice(0, 20), slice(20, None), slice(0, None, 2), slice(1, None, 2)):
                p.vs[:] = drawn * scale
                p.vs[p.tables[0].long()[zeros]] = 0.0
                p.load()
                check_range(*p.run(), p.ref(), io, p.lens, p, fmt, (lens, scale, zeros))


@pytest.mark.parametrize("io", at.IOS, ids=at.IO_IDS)
@pytest.mark.parametrize("fmt", at.FORMATS, ids=at.FORMAT_IDS)
@pytest.mark.parametrize("rows", ROWS)
def test_value_scales_far_apart(gdn, rows, fmt, io):
    """Page scales spread over 2^90, in random, falling and rising order: the largest pages make the
    output, every page its part of the sum."""
    gen = torch.Generator().manual_seed(rows)
    p = Problem(gdn, [9000, 700], [1, 1], rows, 1, 64, 32, fmt, io, seed=70 + rows)
    drawn = p.vs.clone()
    exponents = 90 * torch.rand(p.vs.shape, generator=gen) - 45
    ids = p.tables[0].long()
    for order in (None, True, False):
        e = exponents.clone()
        if order is not None:
            e[ids] = exponents[ids].sort(0, descending=order).values
        p.vs = drawn * torch.exp2(e)
        p.load()
        check_range(*p.run(), p.ref(), io, p.lens, p, fmt, order)


@pytest.mark.parametrize("io", at.IOS, ids=at.IO_IDS)
@pytest.mark.parametrize("fmt", at.FORMATS, ids=at.FORMAT_IDS)
@pytest.mark.parametrize("rows", ROWS)
def test_one_large_query_element(gdn, rows, fmt, io):
    """A channel of the queries 2^20 times as large as the others, where the keys are zero: the
    scores come from the others alone.  (An element off by 2^-39 of the largest is off by 2^-19 of
    its own size here, below the score's rounding in the bounds above.)"""
    p = Problem(gdn, [300, 17], [1, 1], rows, 1, 128, 32, fmt, io, seed=80 + rows)
    p.q[:, :, 5] = 2.0 ** 20
    p.kc.view(torch.uint8)[..., 5] = 0
    p.load()
    check(*p.run(), p.ref(), io)


# The many-row kernel's own code for what the tests above show of the other: MANY are rows of a kv
# head that take it, with items of 32 and of 64 rows.
MANY = ROWS[1:]


def kernels_of(call):
    """Names of the kernels that call() launches."""
    act = torch.profiler.ProfilerActivity
    names = []
    for _ in range(2):  # (the first profile of a process may come back empty)
        with torch.profiler.profile(activities=[act.CPU, act.CUDA]) as prof:
            call()
            torch.cuda.synchronize()
        names = [e.name for e in prof.events()]
    return names


def test_which_kernel_runs(gdn):
    """ROWS reach the kernels that their comment says."""
    for io in at.IOS:
        for rows in ROWS:
            p = Problem(gdn, [100], [1], rows, 1, 128, 32, torch.int8, io)
            names = " ".join(kernels_of(p.run))
            many = io == torch.bfloat16 and rows in MANY
            assert ("kv_attention_tc_kernel" in names) == many, (io, rows, names)
            assert ("kv_attention_kernel" in names) == (not many), (io, rows, names)
            if many:
                size = {24: "32>", 40: "64>"}[rows]
                assert f"kv_attention_tc_kernel<128, false, {size}" in names, names


@pytest.mark.parametrize("fmt", at.FORMATS, ids=at.FORMAT_IDS)
@pytest.mark.parametrize("rows", MANY)
def test_many_rows_scales_of_very_different_pages(gdn, rows, fmt):
    """As test_scales_of_very_different_pages, for the many-row kernel."""
    p = Problem(gdn, [16 * 6, 16 * 9 + 3], [1, 1], rows, 1, 128, 16, fmt, torch.bfloat16, seed=8,
                std_q=0.3)
    for n in (0, 1):
        ids = p.tables[n].long()
        p.vs[ids[:6], 0] *= torch.tensor([1.0, 2.0 ** -40, 2.0 ** 40, 2.0 ** -14, 0.0, 1.0])
        p.ks[ids[:6], 0] *= torch.tensor([1.0, 64.0, 0.01, 1.0, 1.0, 0.0])
    p.load()
    check_range(*p.run(), p.ref(), torch.bfloat16, p.lens, p, fmt)


@pytest.mark.parametrize("rows", MANY)
def test_many_rows_repeat_bit_for_bit(gdn, rows):
    """Items cut between CTAs and several items a CTA, again and on another stream."""
    for lens in ([9000, 3, 1200], [70, 300, 5] * 100):
        p = Problem(gdn, lens, [1] * len(lens), 2 * rows, 2, 128, 64, torch.int8, torch.bfloat16)
        want = p.run()
        check(*want, p.ref(), torch.bfloat16)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        for kw in ({}, {}, {"stream": s}):
            got = p.run(**kw)
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("rows", MANY)
def test_many_rows_of_many_sequences(gdn, rows):
    """More sequences than the many-row kernel has threads, some without rows, some without keys."""
    gen = torch.Generator().manual_seed(rows)
    lens = [int(x) for x in torch.randint(0, 200, (1300,), generator=gen)]
    new = [int(x) for x in torch.randint(0, 3, (1300,), generator=gen)]
    new[0] = 5
    p = Problem(gdn, lens, new, rows, 1, 64, 16, torch.int8, torch.bfloat16, seed=rows)
    check(*p.run(), p.ref(), torch.bfloat16)


@pytest.mark.parametrize("rows", MANY)
def test_many_rows_bad_lengths_and_pages(gdn, rows):
    """As test_bad_lengths_and_pages_are_reported, for the many-row kernel: the keys of a page outside
    the pool are left out, the row's other keys count."""
    p = Problem(gdn, [40, 340, 40], [1, 1, 1], rows, 1, 64, 16, torch.int8, torch.bfloat16, seed=14)
    ref = p.ref()
    p.lens = [40, 401, 40]          # past the table's 22 pages
    with pytest.raises(gdn.GdnError) as e:
        p.run()
    assert e.value.status == 6
    got = p.run(check_status=False)
    for i in (0, 2):
        check(got[0][i:i + 1], got[1][i:i + 1], tuple(x[i:i + 1] for x in ref), torch.bfloat16)
    p.lens = [40, 340, 40]
    for bad in (p.ks.shape[0], -7, 2 ** 31 - 1):
        tables = p.tables.clone()
        p.tables[1, 3] = bad
        with pytest.raises(gdn.GdnError) as e:
            p.run()
        assert e.value.status == 6
        got = p.run(check_status=False)
        p.tables = tables
        for i in (0, 2):
            check(got[0][i:i + 1], got[1][i:i + 1], tuple(x[i:i + 1] for x in ref), torch.bfloat16)
        # the same sequence without the sixteen keys of that page
        less = Problem(gdn, [324], [1], rows, 1, 64, 16, torch.int8, torch.bfloat16)
        less.tables = torch.cat([tables[1, :3], tables[1, 4:]])[None]
        less.q, less.kc, less.ks, less.vc, less.vs = p.q[1:2], p.kc, p.ks, p.vc, p.vs
        check(got[0][1:2], got[1][1:2], less.ref(), torch.bfloat16)


@pytest.mark.parametrize("rows", MANY)
def test_many_rows_large_and_small_queries(gdn, rows):
    p = Problem(gdn, [70, 300, 70], [1, 1, 1], rows, 1, 128, 32, torch.int8, torch.bfloat16, seed=10)
    p.q[0] *= 2.0 ** 60
    check(*(x[:1] for x in p.run(scale=2.0 ** -62)),
          tuple(x[:1] for x in p.ref(scale=2.0 ** -62)), torch.bfloat16)
    p.q[0], p.q[1] = 0, p.q[1] * 2.0 ** -40
    check(*p.run(), p.ref(), torch.bfloat16)


@pytest.mark.parametrize("rows", MANY)
def test_many_rows_one_workspace_for_many_calls(gdn, rows):
    p = Problem(gdn, [5000, 100], [1, 1], rows, 1, 128, 64, torch.int8, torch.bfloat16, seed=20)
    o = Problem(gdn, [50, 4000], [1, 1], rows, 1, 128, 64, torch.int8, torch.bfloat16, seed=21)
    want, other = p.run(), o.run()
    check(*want, p.ref(), torch.bfloat16)
    ws = torch.full((128 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(p.run(workspace=ws)[0], want[0])
        assert torch.equal(o.run(workspace=ws)[0], other[0])


def test_many_rows_offsets_past_32_bits(gdn):
    page, hkv, D = 128, 8, 128
    pages = (1 << 32) // (page * hkv * D) + 3
    p = Problem(gdn, [300], [1], 24 * hkv, hkv, D, page, torch.int8, torch.bfloat16, seed=22)
    want = p.run()
    check(*want, p.ref(), torch.bfloat16)
    ids = p.tables[0].long()
    big = gdn.KVCache.empty(pages, hkv, page, D)
    far = torch.tensor([pages - 1, 0, pages - 2])
    big.k[far.cuda()], big.v[far.cuda()] = p.cache.k[ids.cuda()], p.cache.v[ids.cuda()]
    big.k_scale[far.cuda()] = p.cache.k_scale[ids.cuda()]
    big.v_scale[far.cuda()] = p.cache.v_scale[ids.cuda()]
    p.cache, p.tables = big, far.int()[None]
    got = p.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("rows", MANY)
def test_many_rows_graph_capture(gdn, rows):
    p = Problem(gdn, [600, 40], [1, 1], rows, 1, 128, 64, torch.int8, torch.bfloat16, seed=23)
    q, tables = p.q.cuda(), p.tables.cuda()
    lens = torch.tensor(p.lens, dtype=torch.int32).cuda()
    ws = gdn.kv_attention_workspace(p.cache, q, tables)
    gdn.kv_attention(p.cache, q, tables, lens, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = gdn.kv_attention(p.cache, q, tables, lens, workspace=ws)
    for new_lens in ([600, 40], [1, 33], [311, 0]):
        lens.copy_(torch.tensor(new_lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        p.lens = new_lens
        check(out, lse, p.ref(), torch.bfloat16, new_lens)
