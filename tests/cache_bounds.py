"""64-bit results of the attention over a cache, with the error that its kernels' arithmetic
allows in a 2-norm sense: tight enough that a lost tile of keys, or weights of 8 bits, show."""
from __future__ import annotations

import math

import torch

U24, LAST = 2.0 ** -24, 2.0 ** -23  # half a step of fp32; what a sum rounded towards 0 loses at most


def spread_of_groups(p, x, b):
    """(middle, scale) of every dim's group, float64 [n, hkv, d] (4 bits)."""
    j = torch.arange(p.lens[b])
    pair = getattr(p, x + "_scales")[p.table[b, j // p.page].long(), :, j % p.page].double()
    scale, low = pair.unbind(-1)
    return tuple(z[..., None].expand(*z.shape, 64).flatten(-2) for z in (low + 7.5 * scale, scale))


def weigh8(w, scale, v, mid):
    """sum of weight * v with weight * scale as one bf16 number against (v - mid) / scale."""
    ws = (w[..., None] * scale).float().bfloat16().double()
    return (ws * (v - mid) / scale + w[..., None] * mid).sum(-2)


def attend(p, window=0, drop=None, eight=False):
    """(out, lse, E of out, E of lse), float64.  drop = (sequence, first key): 16 keys left out;
    eight: 4-bit weights rounded to 8 bits (both to show that the bounds notice).

    E of out, an element's expected error where all of a kernel's roundings are as large as they can be:
      - weights as two bf16 numbers: 2^-17 of each, independently, times the value (4 bits: the value
        off its group's middle, which goes another way);
      - a score's products and sums in fp32, a k16 product rounded towards 0 each: d / 16 + 4 last bits
        of the sum of magnitudes (4 bits: of |q| (|low| + code * scale)); 2^-22 of the exponential;
      - bf16: tiles of 16 keys summed from 0 by two products, sqrt(keys / 16) roundings of fp32, 16 for the joins;
      - 4 bits: 128 products between two corrections, each losing half a last bit on the average of a
        sum that grows to its end: 128 / 4 last bits of 7.5 scales; 16 roundings for the joins."""
    hq, hkv, d = p.hq, p.hkv, p.d
    out = torch.zeros((p.tokens, hq, d), dtype=torch.float64)
    e_out = torch.zeros_like(out)
    lse = torch.zeros((hq, p.tokens), dtype=torch.float64)
    e_lse = torch.zeros_like(lse)
    for b, (n, m) in enumerate(zip(p.lens, p.news)):
        a, k, v = int(p.cu[b]), p.cached("k", b), p.cached("v", b)
        kmag, mid, scale = k.abs(), torch.zeros_like(v), torch.ones_like(v)
        if p.int4:
            kmid, kscale = spread_of_groups(p, "k", b)
            low = kmid - 7.5 * kscale
            kmag = low.abs() + (k - low)
            mid, scale = spread_of_groups(p, "v", b)
        for i in range(m):
            pos = n - m + i
            j = torch.arange(max(0, pos - window + 1) if window else 0, pos + 1)
            if drop is not None and drop[0] == b:
                j = j[(j < drop[1]) | (j >= drop[1] + 16)]
            q = p.q[a + i].double().unflatten(0, (hkv, hq // hkv))
            s = torch.einsum("hgd,lhd->hgl", q, k[j]) * d ** -0.5
            mag = torch.einsum("hgd,lhd->hgl", q.abs(), kmag[j]) * d ** -0.5
            ll = torch.logsumexp(s, -1)
            w = (s - ll[..., None]).exp()
            vj, mj, sj = (x[j].transpose(0, 1)[:, None] for x in (v, mid, scale))  # [hkv, 1, keys, d]
            o = weigh8(w, sj, vj, mj) if eight else (w[..., None] * vj).sum(-2)
            ds = mag.amax(-1) * (d / 16 + 4) * LAST + 2.0 ** -22 + 4 * U24 * ll.abs()
            square = ((w ** 2)[..., None] * vj ** 2).sum(-2).sqrt()
            e = 2.0 ** -17 * ((w ** 2)[..., None] * (vj - mj) ** 2).sum(-2).sqrt() + ds[..., None] * square
            if p.int4:
                e = e + 32 * LAST * 7.5 * (w[..., None] * sj).sum(-2) + 16 * U24 * (w[..., None] * vj.abs()).sum(-2)
            else:
                e = e + (2 * LAST + (math.sqrt(len(j) / 16) + 16) * U24) * (w[..., None] * vj.abs()).sum(-2)
            out[a + i], e_out[a + i] = o.flatten(0, 1), e.flatten(0, 1)
            lse[:, a + i], e_lse[:, a + i] = ll.flatten(), ds.flatten()
    return out, lse, e_out, e_lse


def check(got, lse, ref):
    """An fp32 result against `attend`: every row's error in the 2-norm, every element's up to 8 times E."""
    o, l, e, le = ref
    off = (got.double().cpu() - o).abs()
    rows = off.norm(dim=-1) / e.norm(dim=-1)
    assert bool((rows <= 1).all()), f"a row's error is {float(rows.max()):.3g} of its bound"
    assert bool((off <= 8 * e).all()), f"an element's error is {float((off / e).max()):.3g} of what is expected"
    lo = (lse.double().cpu() - l).abs() / le
    assert bool((lo <= 1).all()), f"lse: {float(lo.max()):.3g} of its bound"
