"""Ends of the rotation and cache calls' ranges on the GPU: offsets that do not fit, values that are not
finite, scales and scores of any size, long sums, small rows, empty batches, the calls among other work."""
import math

import pytest
import torch

import cache_bounds
from cache_util import Problem, angles, check_attention, quantise, unpack, values
from packed_varlen_attention_cu_gb300 import api
from test_gpu_cache import attend, i32, on_gpu, word

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ offsets that decrease or leave the tensor
# Rows of a sequence whose offsets do so are left out and status 301 tells of it.

def rows_that_fit(cu, t):
    """(sequence, index in it) of every row that belongs to a sequence inside the tensor; None elsewhere."""
    own = [None] * t
    for b in range(len(cu) - 1):
        if 0 <= cu[b] <= cu[b + 1] <= t:
            for r in range(cu[b], cu[b + 1]):
                own[r] = (b, r - cu[b])
    return own


OFFSETS = [[0, 2, 9], [0, 5, 3], [0, -3, 4], [0, 2, 1], [2, 5, 5], [-1, 2, 4], [0, 2 ** 31 - 1, -2 ** 31]]


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("cu", OFFSETS)
def test_append_leaves_out_sequences_whose_offsets_do_not_fit(cu, int4):
    p = Problem([40, 40], [2, 2], 4, 2, 64, 16, int4, garbage=1.0)
    cache, status, t = on_gpu(p), word(), 4
    before = [x.clone() for x in (cache.k, cache.v)]
    q, k, v = (x.contiguous().cuda() for x in (p.q, p.k_new, p.v_new))
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    table = angles(64, 64).cuda()
    args = (k, v, p.table.cuda(), i32([40, 40]))
    api.cache_append(cache, *args, cu_new=i32(cu), table=table, q=q, q_out=qo, k_out=ko, status=status)
    assert api.cache_status(status) == 301
    slots = set()
    for r, own in enumerate(rows_that_fit(cu, t)):
        left_out = bool((qo[r] == 7).all()) and bool((ko[r] == 7).all())
        assert left_out == (own is None)
        if own is not None:
            pos = 40 - (cu[own[0] + 1] - cu[own[0]]) + own[1]
            slots.add((int(p.table[own[0], pos // 16]), pos % 16))
    for x, old in zip((cache.k, cache.v), before):
        changed = (x != old).any(-1).any(1).cpu()  # [page, slot]
        assert {tuple(c) for c in changed.nonzero().tolist()} == slots
    # without a status word the same rows are left out
    again, qo2 = on_gpu(p), torch.full_like(q, 7.0)
    api.cache_append(again, *args, cu_new=i32(cu), table=table, q=q, q_out=qo2)
    assert torch.equal(again.k, cache.k) and torch.equal(again.v, cache.v) and torch.equal(qo2, qo)


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("cu", OFFSETS)
def test_read_leaves_out_sequences_whose_offsets_do_not_fit(cu, int4):
    p = Problem([40, 40], [2, 2], 4, 2, 64, 16, int4)
    ko, vo = (torch.full((4, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    status = word()
    api.cache_read(on_gpu(p), p.table.cuda(), i32(cu), ko, vo, starts=i32([3, 17]), status=status)
    assert api.cache_status(status) == 301
    for r, own in enumerate(rows_that_fit(cu, 4)):
        for x, o in (("k", ko), ("v", vo)):
            want = torch.full((2, 64), 7.0) if own is None else p.cached(x, own[0])[(3, 17)[own[0]] + own[1]].float()
            assert torch.equal(o[r].cpu(), want.bfloat16())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cu", OFFSETS)
def test_rotation_leaves_out_documents_whose_offsets_do_not_fit(cu, dtype):
    x = torch.randn((4, 2, 64)).to(dtype).cuda()
    table = angles(8, 64).cuda()
    out, want, status = torch.full_like(x, 7.0), torch.full_like(x, 7.0), word()
    api.rope(x, None, table, out, None, cu_seqlens=i32(cu), status=status)
    assert api.cache_status(status) == 301
    own = rows_that_fit(cu, 4)
    pos = [-1 if o is None else o[1] for o in own]
    api.rope(x, None, table, want, None, positions=i32(pos))  # (rows of no document: outside the table)
    assert torch.equal(out, want)


def test_one_bad_offset_among_thousands():
    n = 5000
    cu = torch.arange(n + 1, dtype=torch.int32)
    cu[3333] = n + 7
    x = torch.randn((n, 1, 64)).bfloat16().cuda()
    out, status = torch.full_like(x, 7.0), word()
    api.rope(x, None, angles(4, 64).cuda(), out, None, cu_seqlens=cu.cuda(), status=status)
    assert api.cache_status(status) == 301
    cache = api.KVCache.alloc(1, 1, 64, 16)
    k = torch.empty((n, 1, 64), dtype=torch.bfloat16, device="cuda")
    table, lens = torch.zeros((n, 1), dtype=torch.int32, device="cuda"), torch.ones(n, dtype=torch.int32, device="cuda")
    status = word()
    api.cache_read(cache, table, cu.cuda(), k, torch.empty_like(k), status=status)
    assert api.cache_status(status) == 301
    status = word()
    api.cache_append(cache, x, x, table, lens, cu_new=cu.cuda(), status=status)
    assert api.cache_status(status) == 301
    status = word()  # offsets that fit, the first rows and the last ones of no sequence
    api.rope(x, None, angles(4, 64).cuda(), out, None, cu_seqlens=torch.arange(5, n - 5, dtype=torch.int32).cuda(), status=status)
    assert api.cache_status(status) == 0


def test_a_long_pack_with_a_document_past_its_end():
    """Runs of 32 rows a warp in the read-back; the last document says that it goes on behind the tensor."""
    n, cu = 100000, [0, 40000, 80001, 100001]
    x = torch.randn((n, 1, 64)).bfloat16().cuda()
    pages = torch.arange(80001 // 64 + 1, dtype=torch.int32, device="cuda")[None].expand(3, -1).contiguous()
    cache = api.KVCache.alloc(pages.shape[1], 1, 64, 64)
    api.cache_append(cache, x[:80001], x[:80001], pages[:1], i32([80001]), cu_new=i32([0, 80001]))
    ko, vo, status = torch.full_like(x, 7.0), torch.full_like(x, 7.0), word()
    api.cache_read(cache, pages, i32(cu), ko, vo, status=status)
    assert api.cache_status(status) == 301
    assert torch.equal(ko[:40000], x[:40000]) and torch.equal(vo[40000:80001], x[:40001]) and bool((ko[80001:] == 7).all())
    out, status = torch.full_like(x, 7.0), word()
    api.rope(x, None, angles(50000, 64).cuda(), out, None, cu_seqlens=i32(cu), status=status)
    assert api.cache_status(status) == 301
    assert bool((out[80001:] == 7).all()) and bool((out[:80001] != 7).flatten(1).any(1).all())


# ------------------------------------------------------------------ infinities and NaN that a token sees

def poison(p, b, j, what, where, h, dim):
    """A NaN or infinity in the key or the value (all dims of it with dim None) of token j, kv head h."""
    page, slot = int(p.table[b, j // p.page]), j % p.page
    if p.int4:
        groups = slice(None) if dim is None else dim // 64
        getattr(p, where + "_scales")[page, h, slot, groups] = what
    else:
        getattr(p, where)[page, h, slot, slice(None) if dim is None else dim] = what


# one context that every piece of the line cuts, and a batch of whole ones
SHAPES = [([4033], 32, 8, 128), ([4032], 32, 8, 128), ([700, 64, 65, 1] * 150, 4, 2, 64)]


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("lens,hq,hkv,d", SHAPES)
@pytest.mark.parametrize("at", ["last", "first", "middle", "page"])
def test_a_nan_key_that_is_seen_reaches_its_rows(int4, lens, hq, hkv, d, at):
    p = Problem(lens, [1] * len(lens), hq, hkv, d, 16, int4)
    clean = attend(p, cu=False, fp32=True)
    hit = torch.zeros((p.tokens, hq), dtype=torch.bool)
    for b in range(0, len(lens), 3):
        h = b % hkv if len(lens) > 1 else slice(None, None, 2)
        n = lens[b]
        j = {"last": [n - 1], "first": [0], "middle": [n // 2], "page": list(range(n // 2 // 16 * 16, min(n // 2 // 16 * 16 + 16, n)))}[at]
        for x in j:
            poison(p, b, x, math.nan, "k", h, None)
        hit.view(p.tokens, hkv, -1)[b, h] = True
    out, lse = attend(p, cu=False, fp32=True)
    hit = hit.cuda()
    assert bool(torch.isnan(out[hit]).all()) and bool(torch.isnan(lse.t()[hit]).all())
    assert torch.equal(out[~hit], clean[0][~hit]) and torch.equal(lse.t()[~hit], clean[1].t()[~hit])


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("lens,hq,hkv,d", SHAPES)
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("tiny", [False, True])
def test_a_value_that_is_not_finite_reaches_its_dim(int4, lens, hq, hkv, d, what, tiny):
    """Of a bf16 cache the dim, of a 4-bit cache the group of 64; LSE and the other dims stay.
    tiny: the first key outweighs all others, whose weights underflow."""
    p = Problem(lens, [1] * len(lens), hq, hkv, d, 16, int4)
    if tiny:
        if int4:
            p.q.mul_(40)
        else:
            for b in range(len(lens)):
                p.k[p.table[b, 0].long(), :, 0] *= 60
    clean = attend(p, cu=False, fp32=True)
    hit = torch.zeros((p.tokens, d), dtype=torch.bool)
    for b in range(0, len(lens), 3):
        poison(p, b, lens[b] - 1, what, "v", slice(None), d - 3)
        hit[b, slice(d - 64, d) if int4 else d - 3] = True
    out, lse = attend(p, cu=False, fp32=True)
    hit = hit.cuda()[:, None].expand(out.shape)
    assert not bool(torch.isfinite(out[hit]).any())
    assert torch.equal(out[~hit], clean[0][~hit]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("lens,hq,hkv,d", SHAPES)
def test_infinite_keys(lens, hq, hkv, d):
    """A score of -inf is a weight of 0; a score of +inf makes the row NaN, as the formula does."""
    p = Problem(lens, [1] * len(lens), hq, hkv, d, 16)
    p.q = p.q.contiguous()
    p.q[..., 5] = p.q[..., 5].abs() + 0.5
    without = {b: lens[b] // 2 for b in range(0, len(lens), 3) if lens[b] > 1}
    for b, j in without.items():
        poison(p, b, j, -math.inf, "k", slice(None), 5)
    p.rows["k"] = p.k.double()
    out, lse = attend(p, cu=False, fp32=True)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    for b in list(without)[:2]:
        k, v = p.cached("k", b), p.cached("v", b)
        keep = torch.arange(lens[b]) != without[b]
        s = torch.einsum("hgd,lhd->hgl", p.q[b].double().unflatten(0, (hkv, -1)), k[keep]) * d ** -0.5
        o = torch.einsum("hgl,lhd->hgd", s.softmax(-1), v[keep]).flatten(0, 1)
        # weights of 16 bits and scores good to 2e-5 (128 products of magnitude 10 in all, a last bit each)
        assert float((out[b].double().cpu() - o).abs().max()) <= 4e-5 * float(v[keep].abs().max())
        assert float((lse[:, b].double().cpu() - torch.logsumexp(s, -1).flatten()).abs().max()) <= 2e-5
    for b, j in without.items():
        poison(p, b, j, math.inf, "k", slice(None), 5)
    out, lse = attend(p, cu=False, fp32=True)
    hit = torch.zeros(p.tokens, dtype=torch.bool)
    hit[list(without)] = True
    assert bool(torch.isnan(out[hit.cuda()]).all()) and bool(torch.isfinite(out[~hit.cuda()]).all())
    assert bool(torch.isnan(lse[:, hit.cuda()]).all()) and bool(torch.isfinite(lse[:, ~hit.cuda()]).all())


@pytest.mark.parametrize("int4", [False, True])
def test_rows_that_see_nothing_of_a_piece_stay_finite(int4):
    """Drafts under a short window: pieces that hold no key of a row are not poisoned."""
    p = Problem([4000], [16], 8, 2, 64, 16, int4)
    check_attention(p, *attend(p, window=5), p.attend(5))


# ------------------------------------------------------------------ scales and scores of any size

@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("scale", [1e-45, 1e-40, 1e-38, 1e-30])
def test_tiny_scales_weigh_equally(int4, scale):
    """Scores that are 0 for fp32's weights: the result is the average, LSE the logarithm of the count."""
    p = Problem([4033, 20, 1], [1, 2, 1], 8, 2, 128, 16, int4)
    out, lse = attend(p, scale=scale, fp32=True)
    for b, (n, m) in enumerate(zip(p.lens, p.news)):
        v = p.cached("v", b)
        for i in range(m):
            c, r = n - m + i + 1, int(p.cu[b]) + i
            mean = v[:c].mean(0).repeat_interleave(4, 0)
            # equal weights of 1: sums of at most 4033 values below 6, each addition half a step of a sum below 2^15 / n
            assert float((out[r].double().cpu() - mean).abs().max()) <= 1e-4
            assert float((lse[:, r].double().cpu() - math.log(c)).abs().max()) <= 2e-6


# scale, and what the queries are multiplied by: the scores' magnitude is the product of both
@pytest.mark.parametrize("int4,scale,size", [(False, 1e38, 1e-38), (False, 1e30, 1.0), (False, 1.0, 1e12), (False, 1e-10, 1e30),
                                             (True, 1e17, 1.0), (True, 1.0, 1e12), (True, 1e-10, 1e18), (True, 1e15, 1e-14)])
def test_huge_scales_and_scores(int4, scale, size):
    """Where the scores are further apart than fp32's weights reach, the largest key takes all the weight; else the formula."""
    p = Problem([300, 4033], [1, 1], 4, 2, 64, 16, int4, seed=3)
    p.q = (p.q.double() * size).bfloat16()
    out, lse = attend(p, scale=scale, fp32=True, cu=False, q=p.q.contiguous().cuda())
    for b in range(2):
        k, v = p.cached("k", b), p.cached("v", b)
        s = torch.einsum("hgd,lhd->hgl", p.q[b].double().unflatten(0, (2, 2)), k) * float(torch.tensor(scale, dtype=torch.float32))
        want, ll = torch.einsum("hgl,lhd->hgd", s.softmax(-1), v).flatten(0, 1), torch.logsumexp(s, -1).flatten()
        # small scores: 64 products of magnitude 40 in all, a last bit each (size 1e-38: of a subnormal number, 1.4e-45
        # times 1e38): 64 * 40 * 2^-23 = 3e-4 of a weight, times values below 5; large ones: the best two are further
        # apart than their rounding
        top = s.topk(2, -1).values
        clear = ((top[..., 0] - top[..., 1]) > 100) if scale * size > 1e3 else torch.ones(2, 2, dtype=torch.bool)
        assert int(clear.sum()) >= 3
        off = (out[b].double().cpu() - want).abs().amax(-1)
        assert bool((off[clear.flatten()] <= 2e-3).all()), off
        assert bool(((lse[:, b].double().cpu() - ll).abs() <= 1e-3 + 1e-4 * ll.abs()).all())


# ------------------------------------------------------------------ long sums, precision of an fp32 result

@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("d,hq,hkv,lens,news,window", [
    (128, 8, 2, [20000, 1, 777, 9000] + [50] * 30, [1] * 34, 0),
    (64, 8, 2, [20000, 1, 777, 9000] + [50] * 30, [1] * 34, 0),
    (128, 32, 8, [1000, 4033], [1, 1], 0),
    (64, 14, 2, [300, 2500, 17], [4, 6, 1], 0),
    (128, 6, 1, [300, 2500, 17], [16, 3, 1], 200),
    (64, 4, 4, [64, 16, 5000], [1, 1, 2], 0)])
def test_fp32_results(int4, d, hq, hkv, lens, news, window):
    p = Problem(lens, news, hq, hkv, d, 16, int4, seed=len(lens))
    out, lse = attend(p, window=window, fp32=True)
    cache_bounds.check(out, lse, cache_bounds.attend(p, window))
    # a bf16 result is the same sums, rounded once
    short, same = attend(p, window=window)
    assert torch.equal(short, out.bfloat16()) and torch.equal(same, lse)


@pytest.mark.parametrize("int4", [False, True])
def test_partials_of_disjoint_caches_merge_in_fp32(int4):
    d, hq, hkv = 128, 8, 2
    p = Problem([1600, 64], [1, 1], hq, hkv, d, 16, int4)
    cache, q = on_gpu(p), p.q.contiguous().cuda()

    def over(table, lens):
        out, lse = torch.empty((2, hq, d), device="cuda"), torch.empty((hq, 2), device="cuda")
        api.cache_attn(cache, q, table.contiguous().cuda(), i32(lens), out, lse, api.alloc_cache_workspace(2, hq, hkv, d))
        return out, lse
    a, la = over(p.table[:, :2], [32, 32])
    b, lb = over(p.table[:, 2:], [1568, 32])
    out, lse = torch.empty_like(a), torch.empty_like(la)
    api.merge_partials(a, la, b, lb, out, lse)
    cache_bounds.check(out, lse, cache_bounds.attend(p))


@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** -15, 2.0 ** 22])
def test_sizes_of_values_in_4_bits(size):
    """The header's range of values (the largest of these are below 2^24), fp32 results."""
    p = Problem([3000, 300, 17], [1, 2, 1], 8, 2, 128, 16, True, v_spread=size, garbage=0.0)
    check = attend(p, fp32=True)
    cache_bounds.check(*check, cache_bounds.attend(p))


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 8])
def test_4_bits_by_rows_a_head(rows, window):
    """Up to four rows share the columns of two key tiles, with one maximum for both; more do not."""
    p = Problem([2100, 65, 16, 1], [1, 1, 1, 1], 2 * rows, 2, 128, 32, True, seed=rows)
    cache_bounds.check(*attend(p, window=window, fp32=True), cache_bounds.attend(p, window))


@pytest.mark.parametrize("int4", [False, True])
def test_long_sums_of_values_with_a_mean(int4):
    """64 contexts of 131072 tokens, so that a warp sums tens of thousands of keys in one place, weights
    near 1 and values of mean 1.  The weights' 16 bits and the scores' errors average out over so many
    keys (below 1e-6); what is left is 2048 additions of fp32 a warp with errors of either sign, at most half
    a step of a sum that grows to its end: 2^-24 * sqrt(2048 / 3) / sqrt(3) = 9e-7 expected, 2^-17 is eight times
    that.  (A bias of half a last bit an addition would be 2048 / 2 * 2^-24 = 6e-5.)"""
    d, hkv, page, ctx, batch = 128, 8, 64, 131072, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    shape = (ctx // page, hkv, page)
    if int4:
        k, v = (torch.randint(0, 256, shape + (d // 2,), generator=g, dtype=torch.uint8, device="cuda") for _ in "kv")
        ks, vs = (torch.empty(shape + (d // 64, 2), dtype=torch.bfloat16, device="cuda") for _ in "kv")
        for s, mean in ((ks, 0.0), (vs, 1.0)):
            s[..., 0] = torch.rand(shape + (2,), generator=g, device="cuda") * 0.05 + 0.1
            s[..., 1] = mean - 7.5 * s[..., 0].float()
        cache = api.KVCache(k, v, ks, vs)

        def rows(h, x, s):
            sc = s[:, h].double()
            code = unpack(x[:, h].cpu()).cuda().double().unflatten(-1, (2, 64))
            return (sc[..., 1:] + code * sc[..., :1]).flatten(-2).flatten(0, 1)
    else:
        k = torch.randn(shape + (d,), generator=g, device="cuda").bfloat16()
        v = (torch.rand(shape + (d,), generator=g, device="cuda") * 1.5 + 0.25).bfloat16()
        ks = vs = None
        cache = api.KVCache(k, v)

        def rows(h, x, s):
            return x[:, h].flatten(0, 1).double()
    table = torch.stack([torch.randperm(ctx // page, generator=g, device="cuda") for _ in range(batch)]).int()
    q = (torch.randn((1, 4 * hkv, d), generator=g, device="cuda") * 0.3).bfloat16().expand(batch, -1, -1).contiguous()
    out, lse = torch.empty((batch, 4 * hkv, d), device="cuda"), torch.empty((4 * hkv, batch), device="cuda")
    api.cache_attn(cache, q, table, i32([ctx] * batch), out, lse, api.alloc_cache_workspace(batch, 4 * hkv, hkv, d))
    for h in range(hkv):
        kk, vv = rows(h, k, ks), rows(h, v, vs)
        s = q[0, 4 * h:4 * h + 4].double() @ kk.t() * d ** -0.5
        want = s.softmax(-1) @ vv
        off = (out[:, 4 * h:4 * h + 4].double() - want) / want
        assert float(off.abs().max()) <= 2 ** -17, (float(off.abs().max()), float(off.mean()))
        assert float((lse[4 * h:4 * h + 4].double() - torch.logsumexp(s, -1)[:, None]).abs().max()) <= 1e-5


# ------------------------------------------------------------------ 4-bit rows of small magnitude

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("top", [2.0 ** -60, 2.0 ** -99, 2.0 ** -101, 2.0 ** -120, 2.0 ** -125, 2.0 ** -128, 2.0 ** -130])
def test_codes_of_small_groups_are_the_nearest(d, top):
    """Scales down to bf16's smallest subnormal number, 2^-133: every code is round((x - low) / scale)."""
    g = torch.Generator().manual_seed(0)
    rows = (torch.randn((40, 1, d), generator=g) * top).bfloat16()
    rows[0, 0, :] = 0
    rows[1, 0, ::2], rows[1, 0, 1::2] = 2.0 ** -133, 0
    low, high = (f(rows.double().unflatten(-1, (-1, 64)), -1) for f in (torch.amin, torch.amax))
    scale = ((high - low) / 15).float().bfloat16().double()
    x = rows.double().unflatten(-1, (-1, 64))
    ratio = (x - low[..., None]) / torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
    code = torch.where(scale[..., None] > 0, ratio.round().clamp(0, 15), torch.zeros_like(x)).flatten(-2)
    # (a quotient next to a border may go either way: reciprocal and product round, 2 * 2^-24 of at most 15)
    clear = ((ratio - ratio.floor() - 0.5).abs() > 2.0 ** -18).flatten(-2)
    cache = api.KVCache.alloc(3, 1, d, 16, api.CACHE_INT4)
    dev, table, ends = rows.cuda(), i32([[2, 0, 1]]), i32([0, 40])
    api.cache_append(cache, dev, dev, table, ends[1:], cu_new=ends)
    j = torch.arange(40)
    at = (torch.tensor([2, 0, 1])[j // 16], slice(None), j % 16)
    for held, pair in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
        got = unpack(held.cpu()[at])
        assert torch.equal(got[clear], code.long()[clear]) and bool(((got - code).abs() <= 1).all())
        assert torch.equal(pair.cpu()[at].double(), torch.stack((scale, low), -1))
    ko, vo = torch.empty_like(dev), torch.empty_like(dev)
    api.cache_read(cache, table, ends, ko, vo)
    want = values(got, scale.float(), low.float()).float().bfloat16()
    assert torch.equal(ko.cpu(), want) and torch.equal(vo.cpu(), want)


def test_codes_of_ordinary_groups_did_not_change():
    rows = torch.randn((64, 2, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    cache = api.KVCache.alloc(1, 2, 128, 64, api.CACHE_INT4)
    api.cache_append(cache, rows.cuda(), rows.cuda(), i32([[0]]), i32([64]), cu_new=i32([0, 64]))
    assert torch.equal(unpack(cache.k[0].transpose(0, 1).cpu()), quantise(rows)[0])


# ------------------------------------------------------------------ nothing to do

@pytest.mark.parametrize("sequences", [0, 3])
def test_an_empty_batch(sequences):
    """No new token in the whole batch: every call returns and writes nothing."""
    cache = api.KVCache.alloc(2, 2, 64, 16)
    kv, qs = (torch.empty((0, h, 64), dtype=torch.bfloat16, device="cuda") for h in (2, 4))
    table, lens = torch.zeros((sequences, 2), dtype=torch.int32, device="cuda"), i32([5] * sequences)
    cu, status = i32([0] * (sequences + 1)), word()
    ang = angles(8, 64).cuda()
    api.cache_append(cache, kv, kv, table, lens, cu_new=cu, table=ang, q=qs, q_out=qs, k_out=kv, status=status)
    api.cache_append(cache, kv, kv, table, lens, cu_new=cu, status=status)
    api.rope(qs, kv, ang, qs, kv, cu_seqlens=cu, status=status)
    api.cache_read(cache, table, cu, kv, kv, status=status)
    lse = torch.empty((4, 0), device="cuda")
    api.cache_attn(cache, qs, table, lens, qs, lse, api.alloc_cache_workspace(sequences, 4, 2, 64), cu_new=cu, status=status)
    assert api.cache_status(status) == 0 and not bool(cache.k.any()) and not bool(cache.v.any())


# ------------------------------------------------------------------ the calls among other work of a stream

def test_captured_behind_a_copy_and_across_streams():
    """The lengths and rows come by a copy right before the calls, the attention runs on another
    stream behind an event: eagerly, captured, and replayed with other inputs."""
    p = Problem([700, 33, 64], [1, 1, 1], 8, 2, 64, 16, garbage=0.0)
    cache, table, ang = on_gpu(p), p.table.cuda(), angles(800, 64).cuda()
    src = torch.randn((3, 12, 64), device="cuda").bfloat16()
    wide, lens = torch.zeros_like(src), i32([0, 0, 0])
    src_lens, qr = i32(p.lens), torch.empty((3, 8, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(qr), torch.empty((8, 3), device="cuda")
    ws, side = api.alloc_cache_workspace(3, 8, 2, 64), torch.cuda.Stream()

    def step():
        wide.copy_(src)
        lens.copy_(src_lens)
        api.cache_append(cache, wide[:, 8:10], wide[:, 10:], table, lens, table=ang, q=wide[:, :8], q_out=qr)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            api.cache_attn(cache, qr, table, lens, out, lse, ws)
            lens.zero_()
        torch.cuda.current_stream().wait_stream(side)
        wide.zero_()
    main = torch.cuda.Stream()
    with torch.cuda.stream(main):
        step()
    torch.cuda.synchronize()
    want = out.clone(), lse.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        step()
    out.zero_(), lse.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    src.normal_()
    src_lens.copy_(i32([650, 20, 1]))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    got = out.clone(), lse.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(out, got[0]) and torch.equal(lse, got[1]) and not torch.equal(got[0], want[0])


def test_without_torchs_private_stream_function(monkeypatch):
    """The calls go to the current stream also where torch has no function for its bare handle."""
    p = Problem([50, 7], [1, 1], 4, 2, 64, 16)
    want = attend(p)
    monkeypatch.setattr(api, "_raw_stream", None)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert api._queue(None, 0) == side.cuda_stream
        got = attend(p)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
