"""Rotation of packs (and its gradient) on the GPU against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from cache_util import U16, U32, angles, rotate
from packed_varlen_attention_cu_gb300 import api
from packed_varlen_attention_cu_gb300 import workloads as W

pytestmark = pytest.mark.gpu


def bound(y, mag, dtype):
    """Two products and a sum in fp32, one rounding to the type."""
    e = 2 * U32 * mag + U32 * y.abs()
    return e * 1.01 + (U16 * y.abs() if dtype == torch.bfloat16 else 0) + 1e-38


def close(got, y, mag, dtype):
    off = (got.double().cpu() - y).abs()
    assert bool((off <= bound(y, mag, dtype)).all()), float((off / bound(y, mag, dtype)).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (128, 16), (64, 64), (64, 32), (64, 48), (128, 112)])
@pytest.mark.parametrize("inverse", [False, True])
def test_documents(dtype, inter, d, rot, inverse):
    lens = [1, 0, 37, 5, 0, 130, 1]
    cu = torch.tensor([0] + lens).cumsum(0).int()
    t, hq, hkv = int(cu[-1]) + 3, 7, 2  # three rows belong to no document
    g = torch.Generator().manual_seed(d + rot)
    x = torch.randn((t, hq + hkv, d), generator=g).to(dtype)
    table = angles(130, rot)
    pos = torch.cat([torch.arange(n) for n in lens])
    dev = x.cuda()
    q, k = dev[:, :hq], dev[:, hq:]  # strided
    qo, ko = torch.full((t, hq, d), 7.0, dtype=dtype, device="cuda"), torch.full((t, hkv, d), 7.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.rope(q, k, table.cuda(), qo, ko, cu_seqlens=cu.cuda(), interleaved=inter, inverse=inverse, status=status)
    y, mag = rotate(x[:t - 3], table, pos, inter, inverse)
    close(qo[:t - 3], y[:, :hq], mag[:, :hq], dtype)
    close(ko[:t - 3], y[:, hq:], mag[:, hq:], dtype)
    assert bool((qo[t - 3:] == 7).all()) and bool((ko[t - 3:] == 7).all())
    assert api.cache_status(status) == 0
    # in place, in the strided tensor itself
    api.rope(q, k, table.cuda(), q, k, cu_seqlens=cu.cuda(), interleaved=inter, inverse=inverse)
    assert torch.equal(q[:t - 3], qo[:t - 3]) and torch.equal(k[:t - 3], ko[:t - 3])
    assert torch.equal(dev[t - 3:].cpu(), x[t - 3:])


@pytest.mark.parametrize("hq,hkv", [(1, 0), (0, 1), (4, 4), (32, 8), (33, 1)])
@pytest.mark.parametrize("t", [1, 2, 300])
def test_heads_and_row_numbers(hq, hkv, t):
    d = 64
    g = torch.Generator().manual_seed(t)
    q, k = (torch.randn((t, h, d), generator=g).bfloat16() for h in (hq, hkv))
    table = angles(t, d)
    qd, kd = (x.cuda() if x.shape[1] else None for x in (q, k))
    qo, ko = (None if x is None else torch.empty_like(x) for x in (qd, kd))
    api.rope(qd, kd, table.cuda(), qo, ko)
    for x, o in ((q, qo), (k, ko)):
        if o is not None:
            close(o, *rotate(x, table, torch.arange(t), False), torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hq,hkv", [(3, 1), (4, 4), (5, 4), (9, 4), (12, 4)])  # 1 to 4 passes of heads
@pytest.mark.parametrize("d", [64, 128])
def test_many_tokens_of_few_heads(dtype, hq, hkv, d):
    t = 9001
    g = torch.Generator().manual_seed(hq)
    q, k = (torch.randn((t, h, d), generator=g).to(dtype) for h in (hq, hkv))
    table = angles(t, d)
    qd, kd = q.cuda(), k.cuda()
    api.rope(qd, kd, table.cuda(), qd, kd)
    for x, o in ((q, qd), (k, kd)):
        close(o, *rotate(x, table, torch.arange(t), False), dtype)
    # the same rows into a cache: bit for bit the rotated ones
    if dtype == torch.bfloat16:
        pages = torch.arange((t + 63) // 64, dtype=torch.int32, device="cuda").view(1, -1)
        cache = api.KVCache.alloc(num_pages=pages.numel(), num_kv_heads=hkv, head_dim=d, page_size=64)
        ends, qo = torch.tensor([0, t], dtype=torch.int32, device="cuda"), torch.empty_like(qd)
        api.cache_append(cache, k.cuda(), k.cuda(), pages, ends[1:], cu_new=ends, table=table.cuda(), q=q.cuda(), q_out=qo)
        ko, vo = torch.empty_like(kd), torch.empty_like(kd)
        api.cache_read(cache, pages, ends, ko, vo)
        assert torch.equal(qo, qd) and torch.equal(ko, kd) and torch.equal(vo, k.cuda())


def test_positions_of_a_zigzag_shard():
    cu = W.cu_seqlens_of([70, 5, 300, 129, 1, 200])
    t, hq, d = int(cu[-1]), 3, 128
    pos = torch.cat([torch.arange(int(n)) for n in np.diff(cu)])
    x = torch.randn((t, hq, d), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    table = angles(300, d).cuda()
    cud = torch.from_numpy(cu).cuda()
    whole = torch.empty_like(x)
    api.rope(x, None, table, whole, None, cu_seqlens=cud)
    n = api.zigzag_shard_len(cu, 2, 1)
    gmap = torch.empty(n, dtype=torch.int32, device="cuda")
    api.zigzag_shard(cud, 2, 1, gmap)
    part, out, want = (torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    api.gather_rows(x, gmap, part)
    api.rope(part, None, table, out, None, positions=pos.cuda()[gmap.long()].int())
    api.gather_rows(whole, gmap, want)
    assert torch.equal(out, want)


def test_position_outside_the_table_is_left_out_and_told():
    t, d = 6, 64
    x = torch.randn((t, 2, d)).bfloat16().cuda()
    table = angles(4, d).cuda()
    out = torch.full_like(x, 5.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.tensor([0, 3, 4, -1, 2 ** 31 - 1, 1], dtype=torch.int32, device="cuda")
    api.rope(x, None, table, out, None, positions=pos, status=status)
    assert api.cache_status(status) == 303
    assert bool((out[2:5] == 5).all())
    y, mag = rotate(x.cpu()[[0, 1, 5]], table.cpu(), torch.tensor([0, 3, 1]), False)
    close(out[[0, 1, 5]], y, mag, torch.bfloat16)


@pytest.mark.parametrize("inter", [False, True])
def test_gradient_against_the_formula_and_differences(inter):
    """The loss is sum(w * rope(x)): its gradient is the turn back of w, and differences of
    the fp32 forward agree with it (the map is linear: any step gives the slope; a step of
    1 keeps the rounding of the two sums, 2^-24 a term over their magnitude, below it)."""
    t, h, d = 5, 2, 64
    g = torch.Generator().manual_seed(1)
    x, w, e = (torch.randn((t, h, d), generator=g) for _ in range(3))
    table = angles(t, d)
    xd = x.double().requires_grad_()
    r = d // 2
    c, s = table.double()[:, None].unbind(-1)
    a, b = (xd[..., 0::2], xd[..., 1::2]) if inter else (xd[..., :r], xd[..., r:])
    ya, yb = a * c - b * s, b * c + a * s
    wa, wb = (w[..., 0::2], w[..., 1::2]) if inter else (w[..., :r], w[..., r:])
    (ya * wa + yb * wb).sum().backward()
    grad = torch.empty((t, h, d), device="cuda")
    api.rope(w.cuda(), None, table.cuda(), grad, None, interleaved=inter, inverse=True)
    _, mag = rotate(w, table, torch.arange(t), inter, True)
    close(grad, xd.grad, mag, torch.float32)

    def loss(z):
        y = torch.empty((t, h, d), device="cuda")
        api.rope(z.cuda(), None, table.cuda(), y, None, interleaved=inter)
        return float((y.double().cpu() * w.double()).sum())
    slope = loss(x + e) - loss(x)
    step = ((x + e).double() - x.double())
    want = float((grad.double().cpu() * step).sum())
    terms = float((w.abs() * (2 * x.abs() + e.abs())).sum()) * 2  # |y| is at most 2 |x| here
    assert abs(slope - want) <= 4 * U32 * terms


def test_many_documents_and_a_large_pack():
    """One token a document, and offsets past 2^31 bytes."""
    n = 70001
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    x = torch.randn((n, 1, 64), device="cuda").bfloat16()
    out = torch.empty_like(x)
    api.rope(x, None, angles(1, 64).cuda(), out, None, cu_seqlens=cu)
    assert torch.equal(out, x)  # position 0 turns by nothing
    t, h, d = 140000, 64, 128
    x = torch.empty((t, h, d), dtype=torch.bfloat16, device="cuda").normal_()
    table = angles(t, d)
    out = torch.empty_like(x)
    api.rope(x, None, table.cuda(), out, None)
    for r in (0, 65535, 131072, t - 1):
        y, mag = rotate(x[r:r + 1].cpu(), table, torch.tensor([r]), False)
        close(out[r:r + 1], y, mag, torch.bfloat16)
