"""Plain 64-bit forms of the rotation and cache calls, and problems for them."""
from __future__ import annotations

import math

import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24  # half a step of bf16 and of fp32, relative to the value


def angles(max_pos, rot, base=10000.0):
    """fp32 table [max_pos, rot / 2, 2] on the CPU."""
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return torch.stack((a.cos(), a.sin()), -1).float()


def rotate(x, table, pos, inter, inverse=False):
    """(rotated x, sum of the magnitudes of its two products), float64 [tokens, heads, d]."""
    x = x.double()
    r = 2 * table.shape[1]
    c, s = table.double()[pos.long()][:, None].unbind(-1)
    if inverse:
        s = -s
    ia, ib = (slice(0, r, 2), slice(1, r, 2)) if inter else (slice(0, r // 2), slice(r // 2, r))
    a, b = x[..., ia], x[..., ib]
    y, mag = x.clone(), torch.zeros_like(x)
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia], mag[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return y, mag


def quantise(rows):
    """bf16 rows [..., d] -> (codes int64 [..., d], scale, low float32 [..., d / 64]), in fp32 as the format says."""
    d = rows.shape[-1]
    x = rows.float().unflatten(-1, (d // 64, 64))
    low, high = x.amin(-1), x.amax(-1)
    scale = ((high - low) * torch.tensor(1.0 / 15.0, dtype=torch.float32)).bfloat16().float()
    inv = torch.where(scale == 0, torch.zeros_like(scale), torch.ones_like(scale) / scale)
    code = ((x - low[..., None]) * inv[..., None]).round().clamp(0, 15)
    return code.flatten(-2).long(), scale, low


def place(d, i):
    """(byte of the row, shift inside it) of dim i's code."""
    word, bit = (i // 8 % 8) * (d // 64) + i // 64, 4 * (i % 8 // 2) + 16 * (i % 2)
    return 4 * word + bit // 8, bit % 8


def unpack(packed):
    """uint8 rows [..., d / 2] -> codes int64 [..., d]."""
    d = 2 * packed.shape[-1]
    at = [place(d, i) for i in range(d)]
    by = packed.long()[..., torch.tensor([p for p, _ in at])]
    return (by >> torch.tensor([s for _, s in at])) & 15


def pack(codes):
    d = codes.shape[-1]
    out = torch.zeros(codes.shape[:-1] + (d // 2,), dtype=torch.uint8)
    for i in range(d):
        p, s = place(d, i)
        out[..., p] |= (codes[..., i] << s).to(torch.uint8)
    return out


def values(codes, scale, low):
    """float64 values of codes [..., d] with scale, low [..., d / 64]."""
    x = codes.double().unflatten(-1, (scale.shape[-1], 64))
    return (low.double()[..., None] + x * scale.double()[..., None]).flatten(-2)


class Problem:
    """A paged cache on the CPU with rows of every sequence in it, pages in random
    order, garbage (NaN) in every slot that belongs to no token."""

    def __init__(self, lens, news, hq, hkv, d, page, int4=False, seed=0, spare_rows=0, garbage=math.nan,
                 spread=1.0, strided=False, v_spread=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.news, self.hq, self.hkv, self.d, self.page, self.int4 = lens, news, hq, hkv, d, page, int4
        used = [-(-n // page) for n in lens]
        width, count = max(used + [1]), sum(used) + 2
        order = torch.randperm(count, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cu = torch.tensor([0] + news).cumsum(0).to(torch.int32)
        t = int(self.cu[-1]) + spare_rows
        self.tokens = t
        wide = torch.randn((t, hq + 2 * hkv, d), generator=g).mul(spread).bfloat16()
        self.wide = wide if strided else None
        self.q, self.k_new, self.v_new = wide[:, :hq], wide[:, hq:hq + hkv], wide[:, hq + hkv:]
        shape = (count, hkv, page)
        self.rows = {}
        for x in "kv":
            rows = torch.randn(shape + (d,), generator=g).mul(spread if x == "k" or v_spread is None else v_spread).bfloat16()
            mine = torch.zeros((count, page), dtype=torch.bool)
            for b, n in enumerate(lens):
                j = torch.arange(n)
                mine[self.table[b, j // page].long(), j % page] = True
            mine = mine[:, None, :, None].expand(shape + (1,))
            if int4:
                code, scale, low = quantise(rows)
                pair = torch.stack((scale, low), -1).bfloat16()
                pair[~mine[..., 0]] = garbage
                self.rows[x] = values(code, pair[..., 0].float(), pair[..., 1].float())
                setattr(self, x, pack(code))
                setattr(self, x + "_scales", pair)
            else:
                rows = torch.where(mine, rows, torch.tensor(garbage).bfloat16())
                self.rows[x] = rows.double()
                setattr(self, x, rows)
                setattr(self, x + "_scales", None)

    def cached(self, x, b, n=None):
        """Rows 0 .. n of sequence b, float64 [n, hkv, d]."""
        j = torch.arange(self.lens[b] if n is None else n)
        return self.rows[x][self.table[b, j // self.page].long(), :, j % self.page]

    def attend(self, window=0, scale=None, q=None):
        """(out, lse, bound of out's error in bf16, bound of lse's), float64; rows of no sequence are NaN."""
        hq, hkv, d = self.hq, self.hkv, self.d
        scale = d ** -0.5 if scale is None else scale
        q = (self.q if q is None else q).double()
        out = torch.full((self.tokens, hq, d), math.nan, dtype=torch.float64)
        err = torch.zeros_like(out)
        lse = torch.full((hq, self.tokens), math.nan, dtype=torch.float64)
        lerr = torch.zeros_like(lse)
        for b, (n, m) in enumerate(zip(self.lens, self.news)):
            a = int(self.cu[b])
            if m == 0:
                continue
            k, v = self.cached("k", b), self.cached("v", b)
            pos = torch.arange(n - m, n)[:, None]
            j = torch.arange(n)[None]
            ok = (j <= pos) & (j > pos - window if window else j >= 0)
            ok = ok & (self.table[b, j[0] // self.page] >= 0)[None]
            qq = q[a:a + m].unflatten(1, (hkv, hq // hkv))
            kk = torch.where(torch.isfinite(k), k, torch.zeros_like(k))  # slots of no token
            vv = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
            s = torch.einsum("mhgd,lhd->hgml", qq, kk) * scale
            mag = torch.einsum("mhgd,lhd->hgml", qq.abs(), kk.abs()) * scale
            s = s.masked_fill(~ok, -math.inf)
            ll = torch.logsumexp(s, -1)
            p = torch.where(ok, (s - ll.clamp(min=-1e300)[..., None]).exp(), torch.zeros_like(s))
            o = torch.einsum("hgml,lhd->mhgd", p, vv)
            pv = torch.einsum("hgml,lhd->mhgd", p, vv.abs())
            big = torch.einsum("hgml,lhd->mhgd", p, vv.abs().amax(-1, keepdim=True).expand_as(vv))
            # scores in fp32: d products and sums, 4-bit codes as 128 + code with the 128 taken off again
            # (that is at most 16 times the magnitude); two more roundings for scale and base 2
            ds = (torch.where(ok, mag, torch.zeros_like(mag)).amax(-1) * (d + 4) * 2 * U32 *
                  (16 if self.int4 else 1) + 2e-6)
            # the weights are rounded to bf16 once, the output once (fp32 output: not at all)
            e16 = U16 * (o.abs() + 2 * big if self.int4 else o.abs() + pv) + 2 * ds.permute(2, 0, 1)[..., None] * big
            out[a:a + m], err[a:a + m] = o.flatten(1, 2), e16.flatten(1, 2) + 1e-6 * big.flatten(1, 2) + 1e-30
            lse[:, a:a + m] = ll.flatten(0, 1)
            lerr[:, a:a + m] = (2 * ds + 4 * U32 * ll.abs().nan_to_num(0, 0, 0)).flatten(0, 1)
        return out, lse, err, lerr


def check_attention(p, out, lse, ref, label=""):
    o, l, e, le = ref
    out, lse = out.double().cpu(), lse.double().cpu()
    mine = ~torch.isnan(l)
    rows = mine.t()
    assert torch.equal(torch.isneginf(lse[mine]), torch.isneginf(l[mine])), f"{label}: empty rows differ"
    fin = torch.isfinite(l) & mine
    d = (lse - l).abs()
    assert bool((d[fin] <= le[fin]).all()), f"{label}: lse off by {(d[fin] / le[fin]).max():.3g} of its bound"
    assert bool(torch.isfinite(out[rows]).all()), f"{label}: not finite"
    off = (out - o).abs()[rows]
    assert bool((off <= e[rows]).all()), f"{label}: out off by {(off / e[rows]).max():.3g} of its bound"
