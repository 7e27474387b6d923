"""The paged cache on the GPU: append, read-back and attention, alone and as a model
uses them together, against the definitions in 64 bits."""
import math

import pytest
import torch

from cache_util import U16, Problem, angles, check_attention, pack, quantise, rotate, unpack, values
from packed_varlen_attention_cu_gb300 import api
from packed_varlen_attention_cu_gb300 import workloads as W
from packed_varlen_attention_cu_gb300._lib import PvaError

pytestmark = pytest.mark.gpu


def on_gpu(p):
    return api.KVCache(p.k.cuda(), p.v.cuda(), *(None if s is None else s.cuda() for s in (p.k_scales, p.v_scales)))


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def attend(p, cache=None, window=0, scale=0.0, fp32=False, cu=True, status=None, table=None, q=None, max_new=None):
    cache = cache or on_gpu(p)
    q = (p.wide.cuda()[:, :p.hq] if p.wide is not None else p.q.contiguous().cuda()) if q is None else q
    out = torch.full((p.tokens, p.hq, p.d), math.nan, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
    lse = torch.full((p.hq, p.tokens), math.nan, device="cuda")
    max_new = max(p.news + [1]) if max_new is None else max_new
    ws = api.alloc_cache_workspace(len(p.lens), p.hq, p.hkv, p.d, max_new)
    ws.fill_(255)  # what a workspace holds does not matter
    api.cache_attn(cache, q, (p.table if table is None else table).cuda(), i32(p.lens), out, lse, ws,
                   cu_new=p.cu.cuda() if cu else None, max_new=max_new, window=window, softmax_scale=scale,
                   status=status)
    return out, lse


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("d,rot,inter,page", [(128, 128, False, 16), (128, 64, True, 64), (64, 64, True, 32),
                                              (64, 32, False, 256), (128, 0, False, 16)])
@pytest.mark.parametrize("strided", [False, True])
def test_append(int4, d, rot, inter, page, strided):
    lens, news = [40, 1, 0, 300, 17, 16], [40, 1, 0, 33, 1, 16]
    p = Problem(lens, news, 5, 3, d, page, int4, seed=d + rot, spare_rows=2, garbage=9.0, strided=True)
    t = p.tokens - 2
    cache, status = on_gpu(p), word()
    before = [x.clone() for x in (cache.k, cache.v)]
    wide = p.wide.cuda()
    q, k, v = wide[:, :5], wide[:, 5:8], wide[:, 8:]
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    table = angles(300, rot)
    qo, ko = torch.full((t + 2, 5, d), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((t + 2, 3, d), 7.0, dtype=torch.bfloat16, device="cuda")
    api.cache_append(cache, k, v, p.table.cuda(), i32(lens), cu_new=p.cu.cuda(), table=table.cuda() if rot else None,
                     q=q, q_out=qo, k_out=ko, interleaved=inter, status=status)
    assert api.cache_status(status) == 0
    pos = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, news)])
    seq = torch.cat([torch.full((m,), b) for b, m in enumerate(news)])
    for x, o in ((p.q, qo), (p.k_new, ko)):
        y, mag = rotate(x[:t], table, pos, inter) if rot else (x[:t].double(), torch.zeros(1))
        assert bool(((o[:t].double().cpu() - y).abs() <= U16 * y.abs() + 2 ** -22 * mag).all())
        assert bool((o[t:] == 7).all())
    # what the cache holds of the new tokens: the rotated bf16 keys and the values, or their codes
    at = (p.table[seq, pos // page].long(), slice(None), pos % page)
    for x, rows, old in (("k", ko[:t].cpu(), before[0]), ("v", p.v_new[:t], before[1])):
        held = getattr(cache, x).cpu()
        if int4:
            code, scale, low = quantise(rows)
            assert torch.equal(unpack(held[at]), code)
            assert torch.equal(getattr(cache, x + "_scales").cpu()[at].float(), torch.stack((scale, low), -1))
            # a value is at most half a step off, and the top one 15 roundings of the scale
            s = scale.double()[..., None].expand(*scale.shape, 64).flatten(-2)
            assert bool(((values(code, scale, low) - rows.double()).abs() <= s * (0.5 + 15 * U16) * 1.0001).all())
        else:
            assert torch.equal(held[at], rows)
        keep = old.cpu()
        keep[at] = held[at]
        assert torch.equal(keep, held)  # nothing else was touched


def test_append_without_offsets_and_without_queries():
    p = Problem([5, 33, 64], [1, 1, 1], 4, 2, 64, 16, garbage=0.0)
    a, b = on_gpu(p), on_gpu(p)
    table = angles(64, 64).cuda()
    k, v = p.k_new.contiguous().cuda(), p.v_new.contiguous().cuda()
    api.cache_append(a, k, v, p.table.cuda(), i32(p.lens), cu_new=p.cu.cuda(), table=table)
    api.cache_append(b, k, v, p.table.cuda(), i32(p.lens), table=table)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and not torch.equal(a.k.cpu(), p.k)


def test_queries_in_place():
    p = Problem([9, 20], [3, 2], 4, 2, 128, 16, garbage=0.0, strided=True)
    wide, table = p.wide.cuda(), angles(20, 128).cuda()
    args = (wide[:, 4:6], wide[:, 6:], p.table.cuda(), i32(p.lens))
    out = torch.empty((5, 4, 128), dtype=torch.bfloat16, device="cuda")
    api.cache_append(on_gpu(p), *args, cu_new=p.cu.cuda(), table=table, q=wide[:, :4], q_out=out)
    api.cache_append(on_gpu(p), *args, cu_new=p.cu.cuda(), table=table, q=wide[:, :4], q_out=wide[:, :4])
    assert torch.equal(wide[:, :4], out)


@pytest.mark.parametrize("d", [64, 128])
def test_append_of_extreme_rows(d):
    """Constant groups, infinities, NaN, the type's largest and smallest values, in 4 bits."""
    big = float(torch.finfo(torch.bfloat16).max)
    rows = torch.zeros((8, 1, d), dtype=torch.bfloat16)
    rows[1] = 3.25
    rows[2, 0, ::2] = big
    rows[2, 0, 1::2] = -big
    rows[3, 0, 5] = math.inf
    rows[4, 0, 6] = -math.inf
    rows[5, 0, 7] = math.nan
    rows[6, 0, 8] = 1e-40
    rows[7, 0, 9] = -1e-38
    cache = api.KVCache.alloc(1, 1, d, 16, api.CACHE_INT4)
    dev = rows.cuda()
    api.cache_append(cache, dev, dev, i32([[0]]), i32([8]), cu_new=i32([0, 8]))
    ko, vo = torch.empty_like(dev), torch.empty_like(dev)
    api.cache_read(cache, i32([[0]]), i32([0, 8]), ko, vo)
    got = ko[:, 0].float().cpu()
    assert torch.equal(ko.view(torch.int16), vo.view(torch.int16))
    assert bool((got[0] == 0).all()) and bool((got[1] == 3.25).all())
    # the range overflows to infinity, as that of an infinity does: the group reads back as NaN
    for r in (2, 3, 4, 5):
        assert bool(torch.isnan(got[r, :64]).all())
    for r in (3, 4, 5):
        assert bool((got[r, 64:] == 0).all())
    assert bool((got[6].abs() <= 2e-40).all()) and bool((got[7].abs() <= 2e-38).all())


@pytest.mark.parametrize("int4", [False, True])
def test_append_skips_bad_pages_and_tells(int4):
    p = Problem([20, 20, 20, 20], [20, 20, 20, 20], 2, 2, 64, 16, int4, garbage=1.0)
    table = p.table.clone()
    table[0, 0], table[1, 1], table[2, 0] = -1, p.k.shape[0], -2 ** 31
    cache, status = on_gpu(p), word()
    before = cache.k.clone()
    q = p.q.contiguous().cuda()
    qo = torch.zeros_like(q)
    api.cache_append(cache, p.k_new.contiguous().cuda(), p.v_new.contiguous().cuda(), table.cuda(), i32(p.lens),
                     cu_new=p.cu.cuda(), q=q, q_out=qo, status=status)
    assert api.cache_status(status) == 300
    assert torch.equal(qo, q)
    changed = (cache.k != before).flatten(1).any(1).cpu()
    named = torch.zeros(p.k.shape[0], dtype=torch.bool)
    named[table[(table >= 0) & (table < p.k.shape[0])].long()] = True
    assert torch.equal(changed, named)


def test_append_lengths_that_do_not_fit():
    """More new tokens than the length counts, lengths past the table, past the angles."""
    p = Problem([16, 16, 16], [4, 4, 4], 2, 2, 64, 16, garbage=1.0)
    k, v = p.k_new.contiguous().cuda(), p.v_new.contiguous().cuda()
    for lens, code in (([2, 16, 16], 301), ([16, 18, 16], 300), ([-2 ** 31, 16, 16], 301)):
        cache, status = on_gpu(p), word()
        api.cache_append(cache, k, v, p.table.cuda(), i32(lens), cu_new=p.cu.cuda(), status=status)
        assert api.cache_status(status) == code
    cache, status = on_gpu(p), word()
    before = cache.k.clone()
    api.cache_append(cache, k, v, p.table.cuda(), i32(p.lens), cu_new=p.cu.cuda(), table=angles(13, 64).cuda(), status=status)
    assert api.cache_status(status) == 303
    slots = (cache.k != before).any(-1).any(1).cpu()  # [page, slot]
    assert not bool(slots[:, 13:].any()) and int(slots[:, 12].sum()) == 3


# ------------------------------------------------------------------ read

@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("d,hkv,page", [(128, 3, 16), (64, 1, 64), (64, 8, 1024), (128, 2, 32)])
def test_read(int4, d, hkv, page):
    lens = [70, 0, 1, 300, 16]
    p = Problem(lens, lens, hkv, hkv, d, page, int4, seed=d)
    cache, status = on_gpu(p), word()
    starts, counts = [3, 0, 0, 299, 16], [60, 0, 1, 1, 0]
    cu = torch.tensor([0] + counts).cumsum(0).int().cuda()
    t = int(cu[-1])
    ko, vo = (torch.full((t + 2, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    api.cache_read(cache, p.table.cuda(), cu, ko, vo, starts=i32(starts), status=status)
    assert api.cache_status(status) == 0
    for x, o in (("k", ko), ("v", vo)):
        want = torch.cat([p.cached(x, b)[s:s + n] for b, (s, n) in enumerate(zip(starts, counts))])
        assert torch.equal(o[:t].cpu(), want.float().bfloat16()) and bool((o[t:] == 7).all())
    api.cache_read(cache, p.table.cuda(), p.cu.cuda(), ko2 := torch.empty((sum(lens), hkv, d), dtype=torch.bfloat16, device="cuda"), torch.empty_like(ko2))
    want = torch.cat([p.cached("k", b) for b in range(len(lens))])
    assert torch.equal(ko2.cpu(), want.float().bfloat16())


def test_read_leaves_out_what_has_no_page():
    p = Problem([40, 40], [40, 40], 1, 1, 64, 16)
    table = p.table.clone()
    table[0, 1] = -1
    status = word()
    ko, vo = (torch.full((80, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    api.cache_read(on_gpu(p), table.cuda(), p.cu.cuda(), ko, vo, status=status)
    assert api.cache_status(status) == 300
    assert bool((ko[16:32] == 7).all()) and bool((ko[:16] != 7).any())
    status = word()
    api.cache_read(on_gpu(p), p.table.cuda(), p.cu.cuda(), ko, vo, starts=i32([2 ** 31 - 10, -5]), status=status)
    assert api.cache_status(status) == 300


# ------------------------------------------------------------------ attention

LENS = [1, 0, 2, 15, 16, 17, 63, 64, 65, 127, 129, 500, 1000]


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (7, 1), (14, 2), (32, 8), (16, 1), (40, 1), (9, 3)])
def test_single_tokens(int4, d, hq, hkv):
    p = Problem(LENS, [1] * len(LENS), hq, hkv, d, 16, int4, seed=hq)
    # a sequence without any cached token gives an empty row
    q = Problem([n for n in LENS if n], [1] * (len(LENS) - 1), hq, hkv, d, 16, int4, seed=hq)
    check_attention(q, *attend(q, cu=False), q.attend())
    out, lse = attend(p, cu=False)
    assert bool((out[1] == 0).all()) and bool(torch.isneginf(lse[:, 1]).all())
    assert bool(torch.isfinite(out).all())


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("d,hq,hkv,page", [(128, 8, 2, 16), (64, 14, 2, 64), (128, 4, 4, 32), (64, 6, 1, 1024)])
@pytest.mark.parametrize("window", [0, 1, 5, 64, 100])
def test_drafts(int4, d, hq, hkv, page, window):
    lens = [1, 3, 0, 16, 20, 64, 130, 257, 700, 33]
    news = [1, 3, 0, 1, 5, 8, 2, 16, 7, 0]
    p = Problem(lens, news, hq, hkv, d, page, int4, seed=window, spare_rows=3, strided=True)
    status = word()
    out, lse = attend(p, window=window, status=status)
    assert api.cache_status(status) == 0
    check_attention(p, out, lse, p.attend(window))
    assert bool(torch.isnan(out[p.tokens - 3:]).all()) and bool(torch.isnan(lse[:, p.tokens - 3:]).all())


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("new", [17, 40, 150])
def test_more_new_tokens(int4, new):
    """Chunks of a prompt: many query rows for a sequence, some of them without any context."""
    lens, news = [new, new + 200, 300, 1], [new, new, 1, 1]
    p = Problem(lens, news, 8, 2, 64, 16, int4, seed=new)
    check_attention(p, *attend(p), p.attend())
    # an upper bound of the new tokens that is not one costs speed alone
    a, b = attend(p), attend(p, max_new=1)
    check_attention(p, *b, p.attend())
    assert torch.isfinite(a[0]).all()


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_long_contexts_and_a_mixed_batch(int4, d):
    lens = [20000, 1, 777, 9000] + [50] * 30
    p = Problem(lens, [1] * len(lens), 8, 2, d, 64, int4)
    check_attention(p, *attend(p, cu=False), p.attend())


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("spread", [8.0, 1e-3])
def test_peaked_and_flat_scores(int4, spread):
    p = Problem([3000, 100], [2, 1], 8, 2, 128, 16, int4, spread=spread)
    check_attention(p, *attend(p), p.attend())


def test_scale_and_fp32_output():
    p = Problem([400, 77], [1, 3], 8, 2, 128, 16)
    check_attention(p, *attend(p, scale=0.3), p.attend(scale=0.3))
    a, la = attend(p, fp32=True)
    b, lb = attend(p)
    assert torch.equal(a.bfloat16(), b) and torch.equal(la, lb)
    check_attention(p, a, la, p.attend())


def test_fp32_output_keeps_the_weights():
    """A bf16 cache's weights go into the products with 16 bits: each is off by 2^-17 of itself at
    most, so an fp32 output is off by 2^-17 of the sum of |weight * value| and the scores' own error
    (a score of these sizes: below 128 products of fp32, 2e-6 in all; the values are below 6)."""
    p = Problem([400, 77, 3000], [1, 3, 1], 8, 2, 128, 16)
    out, _ = attend(p, fp32=True)
    o, _, _, _ = p.attend()
    assert float((out.double().cpu() - o).abs().max()) <= (2 ** -17 + 2 * 4e-6) * 6


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("v_spread", [1e-6, 1e6])
@pytest.mark.parametrize("spread", [1e-4, 1.0, 30.0])
def test_small_and_large_values(int4, v_spread, spread):
    p = Problem([300, 17, 1], [1, 2, 1], 8, 2, 128, 16, int4, spread=spread, v_spread=v_spread)
    if spread == 30.0:
        p.q.mul_(1 / 30)
    check_attention(p, *attend(p), p.attend())


@pytest.mark.parametrize("int4", [False, True])
def test_thousands_of_sequences(int4):
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 40, (2500,), generator=g).tolist()
    news = [min(n, int(x)) for n, x in zip(lens, torch.randint(0, 3, (2500,), generator=g))]
    p = Problem(lens, news, 2, 1, 64, 16, int4, spare_rows=1)
    check_attention(p, *attend(p), p.attend())


def test_a_cache_without_pages():
    """Empty sequences need no page: an empty cache and a table without columns are fine."""
    cache = api.KVCache(*(torch.zeros((0, 2, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv"))
    q = torch.randn((3, 4, 64), device="cuda").bfloat16()
    out, lse = torch.ones_like(q), torch.ones((4, 3), device="cuda")
    ws, status = api.alloc_cache_workspace(3, 4, 2, 64), word()
    table = torch.zeros((3, 0), dtype=torch.int32, device="cuda")
    api.cache_attn(cache, q, table, i32([0, 0, 0]), out, lse, ws, cu_new=i32([0, 0, 0, 0]), status=status)
    assert api.cache_status(status) == 0 and bool((out == 1).all()) and bool((lse == 1).all())
    # tokens without a page: nothing to read, and told
    api.cache_attn(cache, q, table, i32([5, 1, 3]), out, lse, ws, status=status)
    assert api.cache_status(status) == 300 and bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    status = word()
    api.cache_append(cache, k, k, table, i32([5, 1, 3]), status=status)
    assert api.cache_status(status) == 300
    status = word()
    api.cache_read(cache, table, i32([0, 1, 2, 3]), k, torch.empty_like(k), status=status)
    assert api.cache_status(status) == 300


@pytest.mark.parametrize("int4", [False, True])
def test_lengths_written_just_before(int4):
    """Kernels that change the lengths run right before each call, without a wait in between."""
    lens = [37, 700, 5, 64]
    p = Problem(lens, [1] * 4, 8, 2, 64, 16, int4)
    cache, table, q = on_gpu(p), p.table.cuda(), p.q.contiguous().cuda()
    dev = i32([0] * 4)
    ws = api.alloc_cache_workspace(4, 8, 2, 64)
    outs = []
    for cut in (0, 1, 4, 0, 3):
        dev.copy_(i32(lens))
        dev.sub_(cut)
        out, lse = torch.empty_like(q), torch.empty((8, 4), device="cuda")
        api.cache_attn(cache, q, table, dev, out, lse, ws)
        dev.zero_()
        outs.append((cut, out, lse))
    for cut, out, lse in outs:
        p.lens = [n - cut for n in lens]
        check_attention(p, out, lse, p.attend())


def test_one_row_larger_than_all_others():
    """A running maximum that rises at the last key, and one that stands at the first."""
    for at in (0, 999, 500):
        p = Problem([1000], [1], 4, 2, 64, 16, garbage=math.inf)
        k = p.cached("k", 0)
        page, slot = p.table[0, at // 16].long(), at % 16
        p.k[page, :, slot] = p.k[page, :, slot] * 60
        p.rows["k"] = p.k.double()
        check_attention(p, *attend(p, cu=False), p.attend())
        assert k.shape[0] == 1000


@pytest.mark.parametrize("garbage", [math.nan, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("int4", [False, True])
def test_slots_of_no_token_do_not_matter(garbage, int4):
    p = Problem([1, 17, 50, 95], [1, 1, 1, 1], 8, 2, 64, 32, int4, garbage=garbage)
    check_attention(p, *attend(p), p.attend())


@pytest.mark.parametrize("int4", [False, True])
def test_keys_before_a_window_do_not_matter(int4):
    p = Problem([300, 95], [1, 1], 8, 2, 64, 32, int4)
    want = p.attend(window=40)
    for b, n in enumerate(p.lens):
        for j in range(n - 40):
            at = (int(p.table[b, j // 32]), slice(None), j % 32)
            for x in "kv":
                (getattr(p, x + "_scales") if int4 else getattr(p, x))[at] = math.nan
    check_attention(p, *attend(p, window=40), want)


@pytest.mark.parametrize("int4", [False, True])
def test_missing_pages_are_left_out_and_told(int4):
    p = Problem([100, 100, 40, 64], [1, 2, 1, 1], 8, 2, 64, 16, int4)
    p.table[0, 2], p.table[1, 0], p.table[2] = -1, -7, -1
    status = word()
    out, lse = attend(p, status=status)
    assert api.cache_status(status) == 300
    check_attention(p, out, lse, p.attend())
    bad = p.table.clone()
    bad[bad < 0] = p.k.shape[0]
    again = attend(p, table=bad)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("int4", [False, True])
def test_padded_batch(int4):
    """Rows of no sequence (length 0, no pages) in a batch of single tokens: no failure, nothing
    appended or rotated for them, empty results; the others as without them."""
    lens = [33, 0, 7, 0, 0, 100]
    p = Problem(lens, [int(n > 0) for n in lens], 8, 2, 64, 16, int4)
    cache, status = on_gpu(p), word()
    t = len(lens)
    q, k = (torch.randn((t, h, 64), device="cuda").bfloat16() for h in (8, 2))
    qo = torch.full_like(q, 7.0)
    table = torch.full((t, 7), -1, dtype=torch.int32)
    table[:, :p.table.shape[1]] = p.table
    held = [x.clone() for x in (cache.k, cache.v)]
    api.cache_append(cache, k, k, table.cuda(), i32(lens), table=angles(100, 64).cuda(), q=q, q_out=qo, status=status)
    out, lse = torch.full_like(q, 7.0), torch.full((8, t), 7.0, device="cuda")
    api.cache_attn(cache, qo, table.cuda(), i32(lens), out, lse, api.alloc_cache_workspace(t, 8, 2, 64), status=status)
    assert api.cache_status(status) == 0
    none = torch.tensor([n == 0 for n in lens], device="cuda")
    assert bool((qo[none] == 7).all()) and bool((qo[~none] != 7).any(-1).all())
    assert bool((out[none] == 0).all()) and bool(torch.isneginf(lse[:, none]).all())
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse[:, ~none]).all())
    changed = [(a.view(torch.uint8) != b.view(torch.uint8)).flatten(1).any(1).sum().item()
               for a, b in zip((cache.k, cache.v), held)]  # by their bits: slots of no token are NaN
    assert max(changed) <= 3


def test_long_sums_of_codes_have_no_bias():
    """64 contexts of 131072 tokens, so that whole contexts are summed in one place, with equal
    weights (queries of 0, weights exactly 1): the result is an average of random values, three
    hundred times smaller than they are.  At most 64 products' sums stand between two corrections of
    the codes' middle; each may lose a last bit (2^-23) of a sum that is below 15 scales a weight."""
    d, hkv, page, ctx, batch = 128, 8, 64, 131072, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    shape = (ctx // page, hkv, page)
    cache = api.KVCache(*(torch.randint(0, 256, shape + (d // 2,), generator=g, dtype=torch.uint8, device="cuda") for _ in "kv"),
                        *(torch.empty(shape + (d // 64, 2), dtype=torch.bfloat16, device="cuda") for _ in "kv"))
    for s in (cache.k_scales, cache.v_scales):
        s[..., 0] = torch.rand(shape + (2,), generator=g, device="cuda") * 0.2 + 0.3
        s[..., 1] = -7.5 * s[..., 0].float()
    table = torch.stack([torch.randperm(ctx // page, generator=g, device="cuda") for _ in range(batch)]).int()
    q = torch.zeros((batch, 4 * hkv, d), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty((batch, 4 * hkv, d), device="cuda"), torch.empty((4 * hkv, batch), device="cuda")
    ws = api.alloc_cache_workspace(batch, 4 * hkv, hkv, d)
    api.cache_attn(cache, q, table, i32([ctx] * batch), out, lse, ws)
    total = torch.zeros((hkv, d), dtype=torch.float64, device="cuda")
    for h in range(hkv):
        sc = cache.v_scales[:, h].double()
        code = unpack(cache.v[:, h].cpu()).cuda().double().unflatten(-1, (2, 64))
        total[h] = (sc[..., 1:] + code * sc[..., :1]).flatten(-2).sum((0, 1))
    mean = (total / ctx).repeat_interleave(4, 0)
    assert float((out.double() - mean).abs().max()) <= 64 * 2 ** -23 * 15 * 0.5 + 1e-6
    assert float((lse.double() - math.log(ctx)).abs().max()) <= 1e-5


@pytest.mark.parametrize("int4", [False, True])
def test_strided_page_table_and_shared_pages(int4):
    """A table with rows further apart than they are long; two sequences over the same pages."""
    p = Problem([100, 70, 100], [1, 1, 1], 8, 2, 64, 16, int4)
    p.table[2] = p.table[0]
    wide = torch.full((3, 40), 7777, dtype=torch.int32)
    wide[:, 5:5 + p.table.shape[1]] = p.table
    table = wide.cuda()[:, 5:5 + p.table.shape[1]]
    check_attention(p, *attend(p, table=table), p.attend())
    ko = torch.empty((270, 2, 64), dtype=torch.bfloat16, device="cuda")
    api.cache_read(on_gpu(p), table, i32([0, 100, 170, 270]), ko, torch.empty_like(ko))
    assert torch.equal(ko.cpu(), torch.cat([p.cached("k", b) for b in range(3)]).float().bfloat16())
    with pytest.raises(ValueError):
        attend(p, table=wide.cuda().t())


def test_misaligned_tensors_are_refused():
    p = Problem([20], [1], 4, 2, 64, 16)
    odd = torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(1, 4, 64)
    with pytest.raises(PvaError):
        attend(p, q=odd)
    flat = torch.zeros((3, 4 * 64 + 4), dtype=torch.bfloat16, device="cuda")
    rows = flat[:, :256].view(3, 4, 64)  # rows 8 bytes off every other time
    out = torch.empty((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(PvaError):
        api.rope(rows, None, angles(3, 64).cuda(), out, None)


def test_lengths_that_do_not_fit_are_told():
    p = Problem([40, 40], [2, 2], 4, 2, 64, 16)
    cache = on_gpu(p)
    for lens, news, code in (([40, 100], [2, 2], 300), ([40, 1], [2, 2], 301), ([-5, 40], [2, 2], 301)):
        status = word()
        p.lens, p.news = lens, news
        out, lse = attend(p, cache=cache, status=status)
        assert api.cache_status(status) == code
        good = 0 if lens[0] == 40 else 1
        rows = slice(2 * good, 2 * good + 2)
        assert bool(torch.isfinite(out[rows].float()).all()) and bool(torch.isfinite(lse[:, rows]).all())
    # offsets that leave the tensor or decrease: those sequences are left out
    for cu in ([0, 2, 9], [0, 5, 3], [0, -3, 4], [3, 1, 4]):
        status = word()
        p.lens, p.news, p.cu = [40, 40], [2, 2], torch.tensor(cu, dtype=torch.int32)
        attend(p, cache=cache, status=status)
        assert api.cache_status(status) == 301


def test_cache_past_32_bit_offsets():
    """Pages that lie more than 2^32 bytes, and more than 2^31 elements, into the cache."""
    d, hkv, page = 128, 8, 64
    pages = (1 << 31) // (hkv * page * d) + 600
    cache = api.KVCache(*(torch.empty((pages, hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in "kv"))
    p = Problem([700], [1], 8, 8, d, page, seed=5)
    far = pages - 1 - torch.arange(p.table.shape[1])
    for x in "kv":
        getattr(cache, x)[far.cuda()] = getattr(p, x)[p.table[0].long()].cuda()
    table = far[None].int()
    check_attention(p, *attend(p, cache=cache, table=table), p.attend())
    k = torch.randn((1, hkv, d)).bfloat16().cuda()
    api.cache_append(cache, k, k, table.cuda(), i32([700]))
    assert torch.equal(cache.k[far[-1], :, 699 % page], k[0])
    ko = torch.empty((700, hkv, d), dtype=torch.bfloat16, device="cuda")
    api.cache_read(cache, table.cuda(), i32([0, 700]), ko, torch.empty_like(ko))
    assert torch.equal(ko[:699].cpu(), p.cached("k", 0)[:699].bfloat16()) and torch.equal(ko[699], k[0])


@pytest.mark.parametrize("int4", [False, True])
def test_same_result_every_time(int4):
    p = Problem([5000, 3, 800, 2100], [1, 4, 2, 1], 8, 2, 128, 16, int4)
    cache = on_gpu(p)
    a = attend(p, cache)
    for _ in range(5):
        b = attend(p, cache)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_and_replayed_with_growing_lengths():
    """One captured decoding step serves every later token: lengths are read on the device."""
    hq, hkv, d, page, steps = 8, 2, 64, 16, 40
    cache = api.KVCache.alloc(8, hkv, d, page, api.CACHE_BF16)
    table = i32([[3, 1, 5, 7], [2, 0, 6, 4]])
    lens = i32([1, 15])
    ang = angles(64, d).cuda()
    wide = torch.zeros((2, hq + 2 * hkv, d), dtype=torch.bfloat16, device="cuda")
    q, k, v = wide[:, :hq], wide[:, hq:hq + hkv], wide[:, hq + hkv:]
    qr, out = (torch.empty((2, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse = torch.empty((hq, 2), device="cuda")
    ws = api.alloc_cache_workspace(2, hq, hkv, d)

    def step():
        api.cache_append(cache, k, v, table, lens, table=ang, q=q, q_out=qr)
        api.cache_attn(cache, qr, table, lens, out, lse, ws)
        lens.add_(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    cache.k.zero_(), cache.v.zero_()
    lens.copy_(i32([1, 15]))
    g = torch.Generator().manual_seed(0)
    ks, vs = [[], []], [[], []]
    for b, n in ((0, 0), (1, 14)):
        ks[b] += [torch.zeros(hkv, d).double()] * n
        vs[b] += [torch.zeros(hkv, d).double()] * n
    for _ in range(steps):
        x = torch.randn(wide.shape, generator=g).bfloat16()
        wide.copy_(x)
        graph.replay()
        for b in range(2):
            n = len(ks[b])
            kr, _ = rotate(x[b:b + 1, hq:hq + hkv], ang.cpu(), torch.tensor([n]), False)
            qq, _ = rotate(x[b:b + 1, :hq], ang.cpu(), torch.tensor([n]), False)
            ks[b].append(kr[0].float().bfloat16().double())
            vs[b].append(x[b, hq + hkv:].double())
            kk, vv = torch.stack(ks[b]), torch.stack(vs[b])
            s = torch.einsum("hgd,lhd->hgl", qq[0].float().bfloat16().double().unflatten(0, (hkv, -1)), kk) / d ** 0.5
            pr = s.softmax(-1)
            o = torch.einsum("hgl,lhd->hgd", pr, vv)
            big = torch.einsum("hgl,lhd->hgd", pr, vv.abs())
            # a rotated bf16 key or query may round to the neighbour of the 64-bit one: 2^-7 of one
            # product of a score at a 2^-16 chance; 1e-3 of the magnitude covers a few of them
            e = U16 * (o.abs() + big) + 1e-3 * big.amax(-1, keepdim=True)
            assert bool(((out[b].double().cpu().unflatten(0, (hkv, -1)) - o).abs() <= e).all())


def test_other_stream_and_two_workspaces_at_once():
    p = Problem([3000, 40, 900], [1, 1, 1], 8, 2, 64, 16)
    want = attend(p, cu=False)
    cache, table, lens = on_gpu(p), p.table.cuda(), i32(p.lens)
    q = p.q.contiguous().cuda()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(q) for _ in streams]
    lses = [torch.empty((8, 3), device="cuda") for _ in streams]
    spaces = [api.alloc_cache_workspace(3, 8, 2, 64) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, o, l, w in zip(streams, outs, lses, spaces):
            api.cache_attn(cache, q, table, lens, o, l, w, stream=s)
    torch.cuda.synchronize()
    for o, l in zip(outs, lses):
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (64, 14, 2)])
@pytest.mark.parametrize("window", [0, 50])
def test_prompts_then_tokens(d, hq, hkv, window):
    """Prompts go into the cache and through attn_fwd as a pack; the same attention over the
    cache agrees; a second chunk runs both ways (read back + attn_fwd over slices, and over the
    cache); then single tokens."""
    page, lens = 32, [70, 1, 200, 33]
    g = torch.Generator().manual_seed(d)
    table = torch.arange(40, dtype=torch.int32, device="cuda").flip(0).view(4, 10).contiguous()
    cache = api.KVCache.alloc(40, hkv, d, page)
    ang = angles(320, d).cuda()
    history = torch.zeros((4, 320, hq + 2 * hkv, d), dtype=torch.bfloat16)
    status = word()

    def chunk(before, news):
        """Append news[b] tokens to each sequence; (rotated q, cu, total lengths)."""
        after = [a + n for a, n in zip(before, news)]
        rows = []
        for b, (a, n) in enumerate(zip(before, news)):
            history[b, a:a + n] = torch.randn((n, hq + 2 * hkv, d), generator=g).bfloat16()
            rows.append(history[b, a:a + n])
        wide = torch.cat(rows).cuda()
        cu = torch.tensor([0] + news).cumsum(0).int().cuda()
        qr, kr = torch.empty_like(wide[:, :hq].contiguous()), torch.empty_like(wide[:, hq:hq + hkv].contiguous())
        api.cache_append(cache, wide[:, hq:hq + hkv], wide[:, hq + hkv:], table, i32(after), cu_new=cu, table=ang,
                         q=wide[:, :hq], q_out=qr, k_out=kr, status=status)
        return qr, kr, wide[:, hq + hkv:].contiguous(), cu, after

    def reference(qr, cu, after, news):
        """64 bits, from what the calls rotated."""
        full = api.KVCache(cache.k, cache.v)
        n = sum(after)
        kk, vv = (torch.empty((n, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
        api.cache_read(full, table, torch.tensor([0] + after).cumsum(0).int().cuda(), kk, vv)
        outs, errs, at = [], [], 0
        for b, (l, m) in enumerate(zip(after, news)):
            k, v = kk[at:at + l].double(), vv[at:at + l].double()
            at += l
            pos, j = torch.arange(l - m, l, device="cuda")[:, None], torch.arange(l, device="cuda")[None]
            ok = (j <= pos) & (j > pos - window if window else j >= 0)
            s = torch.einsum("mhgd,lhd->hgml", qr[int(cu[b]):int(cu[b]) + m].double().unflatten(1, (hkv, -1)), k) * d ** -0.5
            pr = s.masked_fill(~ok, -math.inf).softmax(-1)
            o = torch.einsum("hgml,lhd->mhgd", pr, v).flatten(1, 2)
            outs.append(o)
            errs.append(U16 * (o.abs() + torch.einsum("hgml,lhd->mhgd", pr, v.abs()).flatten(1, 2)) + 1e-5)
        return torch.cat(outs), torch.cat(errs)

    def over_cache(qr, cu, after, news):
        out = torch.empty_like(qr)
        lse = torch.empty((hq, qr.shape[0]), device="cuda")
        ws = api.alloc_cache_workspace(4, hq, hkv, d, max(news))
        api.cache_attn(cache, qr, table, i32(after), out, lse, ws, cu_new=cu, max_new=max(news), window=window, status=status)
        return out, lse

    # 1. prompts
    qr, kr, v, cu, after = chunk([0] * 4, lens)
    t = qr.shape[0]
    kind = W.MASK_SLIDING_WINDOW if window else W.MASK_CAUSAL
    pa = api.PackedAttention(cu, api.make_mask(kind, t, t, window=window), hq, hkv, head_dim=d)
    pa.plan()
    o1, l1 = pa.forward(qr, kr, v)
    o2, l2 = over_cache(qr, cu, after, lens)
    ref, err = reference(qr, cu, after, lens)
    assert bool(((o1.double() - ref).abs() <= err).all()) and bool(((o2.double() - ref).abs() <= err).all())
    assert float((l1 - l2).abs().max()) < 1e-4
    # 2. a second chunk of each prompt over its cached context
    news = [30, 64, 1, 17]
    qr, kr, v, cu, total = chunk(after, news)
    n = sum(total)
    kk, vv = (torch.empty((n, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    cua = torch.tensor([0] + total).cumsum(0).int()
    api.cache_read(cache, table, cua.cuda(), kk, vv, status=status)
    rows = [[int(cu[b]), news[b], total[b] - news[b], int(cua[b]), total[b], 0, api.SLICE_CAUSAL, window] for b in range(4)]
    mask = api.make_mask(W.MASK_SLICES, qr.shape[0], n, slices=torch.tensor(rows).numpy())
    params = api.make_params(hq, hkv, c_tile=api.default_c_tile(d))
    wl = api.alloc_worklist(0, mask, params)
    api.build_worklist(None, mask, params, wl)
    o1 = torch.empty_like(qr)
    l1 = torch.empty((hq, qr.shape[0]), device="cuda")
    api.attn_fwd(qr, kk, vv, None, mask, params, wl, o1, l1)
    o2, l2 = over_cache(qr, cu, total, news)
    ref, err = reference(qr, cu, total, news)
    assert bool(((o1.double() - ref).abs() <= err).all()) and bool(((o2.double() - ref).abs() <= err).all())
    assert float((l1 - l2).abs().max()) < 1e-4
    # 3. tokens
    for _ in range(3):
        qr, kr, v, cu, total = chunk(total, [1] * 4)
        o2, _ = over_cache(qr, cu, total, [1] * 4)
        ref, err = reference(qr, cu, total, [1] * 4)
        assert bool(((o2.double() - ref).abs() <= err).all())
    assert api.cache_status(status) == 0


def test_partials_of_a_shared_prompt_merge():
    """Answers that share a prompt: attention over the prompt's pages and over each answer's own
    rows, merged by merge_partials, is the attention over both."""
    d, hq, hkv, page = 64, 8, 2, 16
    p = Problem([96, 40, 25], [0, 1, 1], hq, hkv, d, page, garbage=0.0)
    cache, q = on_gpu(p), p.q.contiguous().cuda()
    both = torch.full((2, 9), -1, dtype=torch.int32)
    for i, b in enumerate((1, 2)):
        both[i, :6] = p.table[0, :6]
        both[i, 6:9] = p.table[b, :3]

    def over(table, lens):
        out, lse = torch.empty((2, hq, d), device="cuda"), torch.empty((hq, 2), device="cuda")
        ws = api.alloc_cache_workspace(2, hq, hkv, d)
        api.cache_attn(cache, q, table.cuda(), i32(lens), out, lse, ws)
        return out, lse
    whole, wl = over(both, [136, 121])
    a, la = over(p.table[:1, :6].expand(2, 6).contiguous(), [96, 96])
    b, lb = over(p.table[1:, :3].contiguous(), [40, 25])
    out, lse = torch.empty_like(a), torch.empty_like(la)
    api.merge_partials(a, la, b, lb, out, lse)
    # each side's weights are rounded to bf16 once: values are below 5 here
    assert float((out - whole).abs().max()) <= 2 * U16 * 5 and float((lse - wl).abs().max()) <= 1e-5


def test_calls_on_wrong_tensors_are_refused():
    p = Problem([20], [1], 4, 2, 64, 16)
    cache = on_gpu(p)
    q, out, lse = p.q.contiguous().cuda(), torch.empty((1, 4, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((4, 1), device="cuda")
    ws = api.alloc_cache_workspace(1, 4, 2, 64)
    args = dict(page_table=p.table.cuda(), kv_lens=i32([20]), out=out, lse=lse, workspace=ws)

    def call(**kw):
        api.cache_attn(cache, kw.pop("q", q), **{**args, **kw})
    call()
    for kw in (dict(q=q.float()), dict(out=out.half()), dict(out=out[:, :2]), dict(lse=lse.double()), dict(lse=lse.t()),
               dict(kv_lens=i32([20]).long()), dict(kv_lens=i32([])), dict(page_table=p.table), dict(page_table=p.table.cuda()[0]),
               dict(cu_new=i32([0])), dict(q=q.cpu()), dict(q=q.transpose(0, 1))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(PvaError):
        call(workspace=ws[:0])
    with pytest.raises(PvaError):
        call(max_new=0)
    k = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        api.cache_append(cache, k, k[:, :1], args["page_table"], args["kv_lens"])
    with pytest.raises(ValueError):
        api.cache_append(cache, k, k, args["page_table"], args["kv_lens"], q=q)
    with pytest.raises(ValueError):
        api.cache_read(cache, args["page_table"], i32([0, 1]), k, k.float())
    assert pack(unpack(torch.arange(32, dtype=torch.uint8))).tolist() == list(range(32))
