"""Cross attention on the GPU: packs of targets over packs of sources with the
gradients, and rows over a cached source, against the definitions in 64 bits.
The packs' tolerances are those of the method's target (see gpu_util and
test_gpu_bwd), the cache's bounds those of cache_util."""
import math

import numpy as np
import pytest
import torch

from cache_util import U16, U32, Problem, check_attention, pack, quantise, unpack, values
from gpu_util import compare, to_np
from packed_varlen_attention_cu_gb300 import api
from test_gpu_bwd import REL_L2, _check
from test_gpu_cache import i32, on_gpu, word

pytestmark = pytest.mark.gpu

# (rows of the target, keys of its source): short pairs that share tiles, pairs past a tile on one
# side, exact tiles, one row or key, and empty sides in all places
PAIRS = [(0, 5), (5, 9), (1, 1), (40, 100), (130, 40), (1, 300), (0, 17), (64, 0), (128, 128), (127, 1), (3, 127),
         (200, 385), (30, 20), (30, 30), (30, 40), (0, 0), (300, 0), (2, 2)]


class Pack:
    """Targets and sources on the CPU, and what attention gives for them in 64 bits."""

    def __init__(self, pairs, hq, hkv, d, seed=0, scale=0.0, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.pairs, self.hq, self.hkv, self.d = pairs, hq, hkv, d
        self.cu, self.ck = (torch.tensor([0] + [p[i] for p in pairs]).cumsum(0).to(torch.int32) for i in (0, 1))
        self.tq, self.tk = int(self.cu[-1]), int(self.ck[-1])
        self.q, self.dout = (torch.randn((self.tq, hq, d), generator=g).mul(spread).bfloat16() for _ in range(2))
        self.k, self.v = (torch.randn((self.tk, hkv, d), generator=g).mul(spread).bfloat16() for _ in range(2))
        self.scale = scale or d ** -0.5

    def forward(self, q=None, k=None, v=None):
        q, k, v = (x.double() if y is None else y for x, y in ((self.q, q), (self.k, k), (self.v, v)))
        out = torch.zeros((self.tq, self.hq, self.d), dtype=torch.float64)
        lse = torch.full((self.hq, self.tq), -math.inf, dtype=torch.float64)
        for a, e, c, f in zip(self.cu[:-1].tolist(), self.cu[1:].tolist(), self.ck[:-1].tolist(), self.ck[1:].tolist()):
            if e > a and f > c:
                s = torch.einsum("mhgd,lhd->hgml", q[a:e].unflatten(1, (self.hkv, -1)), k[c:f]) * self.scale
                ll = torch.logsumexp(s, -1)
                out[a:e] = torch.einsum("hgml,lhd->mhgd", (s - ll[..., None]).exp(), v[c:f]).flatten(1, 2)
                lse[:, a:e] = ll.flatten(0, 1)
        return out, lse

    def gradients(self):
        """The formulas of the header, from the forward's 64-bit results."""
        q, k, v, do = (x.double() for x in (self.q, self.k, self.v, self.dout))
        out, lse = self.forward()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        for a, e, c, f in zip(self.cu[:-1].tolist(), self.cu[1:].tolist(), self.ck[:-1].tolist(), self.ck[1:].tolist()):
            if e > a and f > c:
                qq, dd = (x[a:e].unflatten(1, (self.hkv, -1)) for x in (q, do))
                s = torch.einsum("mhgd,lhd->hgml", qq, k[c:f]) * self.scale
                p = (s - lse[:, a:e].unflatten(0, (self.hkv, -1))[..., None]).exp()
                dp = torch.einsum("mhgd,lhd->hgml", dd, v[c:f])
                delta = (do[a:e] * out[a:e]).sum(-1).t().unflatten(0, (self.hkv, -1))
                ds = p * (dp - delta[..., None]) * self.scale
                dq[a:e] = torch.einsum("hgml,lhd->mhgd", ds, k[c:f]).flatten(1, 2)
                dk[c:f] = torch.einsum("hgml,mhgd->lhd", ds, qq)
                dv[c:f] = torch.einsum("hgml,mhgd->lhd", p, dd)
        return dq, dk, dv


class Run:
    """The pack on the GPU: worklist, tensors, results filled with NaN."""

    def __init__(self, p, pack=1, dispatch=api.DISPATCH_DYNAMIC, fp32=False):
        self.p = p
        self.cu, self.ck = p.cu.cuda(), p.ck.cuda()
        self.q, self.k, self.v, self.dout = (x.cuda() for x in (p.q, p.k, p.v, p.dout))
        self.mask = api.make_mask(api.MASK_CROSS, p.tq, p.tk, cu_keys=self.ck)
        self.params = api.make_params(p.hq, p.hkv, c_tile=api.default_c_tile(p.d), dispatch=dispatch, pack_docs=pack)
        self.wl = api.alloc_worklist(len(p.pairs), self.mask, self.params)
        self.wl.fill_(255)
        self.out = torch.full(p.q.shape, math.nan, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
        self.lse = torch.full((p.hq, p.tq), math.nan, device="cuda")

    def build(self):
        api.build_worklist(self.cu, self.mask, self.params, self.wl)
        return self

    def forward(self):
        api.attn_fwd(self.q, self.k, self.v, self.cu, self.mask, self.params, self.wl, self.out, self.lse,
                     softmax_scale=self.p.scale)
        return self

    def backward(self, fp32=False):
        nd = len(self.p.pairs)
        plan = api.alloc_bwd_plan(nd, self.mask, self.params)
        plan.fill_(255)
        api.build_bwd_plan(self.wl, nd, self.mask, self.params, plan)
        kind = torch.float32 if fp32 else torch.bfloat16
        grads = [torch.full(x.shape, math.nan, dtype=kind, device="cuda") for x in (self.q, self.k, self.v)]
        api.attn_bwd(self.q, self.k, self.v, self.out, self.lse, self.dout, self.cu, nd, self.mask, self.params, self.wl, plan,
                     *grads, softmax_scale=self.p.scale)
        torch.cuda.synchronize()
        assert api.worklist_error(self.wl) == 0
        return grads

    def check(self, label=""):
        torch.cuda.synchronize()
        assert api.worklist_error(self.wl) == 0
        o, l = self.p.forward()
        compare(to_np(self.out), to_np(self.lse), o.numpy(), l.numpy(), label)
        return self


# ------------------------------------------------------------------ packs

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (6, 2), (7, 1)])
@pytest.mark.parametrize("pack", [0, 1])
@pytest.mark.parametrize("dispatch", [api.DISPATCH_DYNAMIC, api.DISPATCH_STATIC])
def test_forward(d, hq, hkv, pack, dispatch):
    r = Run(Pack(PAIRS, hq, hkv, d, seed=d + hq), pack, dispatch, fp32=hq == 6).build().forward().check(f"cross {d} {hq}/{hkv}")
    types = api.decode_worklist(r.wl)["slices"][:, 6]
    assert (types == 5).any() == bool(pack)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (6, 2), (7, 1)])
@pytest.mark.parametrize("pack", [0, 1])
def test_backward(d, hq, hkv, pack):
    p = Pack(PAIRS, hq, hkv, d, seed=3 * d + hq)
    got = Run(p, pack).build().forward().backward(fp32=hq == 6)
    _check([to_np(x) for x in got], [x.numpy() for x in p.gradients()], f"cross {d} {hq}/{hkv}")
    # rows without keys and keys without rows: exact zeros
    for (m, n), a, c in zip(PAIRS, p.cu.tolist(), p.ck.tolist()):
        if m == 0 or n == 0:
            assert not got[0][a:a + m].any() and not got[1][c:c + n].any() and not got[2][c:c + n].any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pack", [0, 1])
def test_sources_of_one_key_move_no_scores(d, pack):
    """With one key P is 1 and dS = P (dP - D) is 0, whatever dO and V are.  P is off by its LSE's and exponent's
    rounding, 2^-24 of numbers below 2^6 in base 2 and 2^-22, so by less than 2^-17, and as far is dS from 0, of |dP|;
    D from an O in bf16 would leave 2^-8 of it."""
    p = Pack([(1 + i % 50, 1) for i in range(40)], 4, 2, d, seed=d)
    got = Run(p, pack).build().forward().backward(fp32=True)
    dp = (p.dout.double().norm(dim=-1).max() * p.v.double().norm(dim=-1).max())
    assert (p.q.double().norm(dim=-1).max() * p.k.double().norm(dim=-1).max()) * p.scale * math.log2(math.e) < 2 ** 6
    one = p.scale * dp * 2.0 ** -17
    assert got[0].abs().max() <= one * p.k.abs().max().double()
    assert got[1].abs().max() <= one * p.q.abs().max().double() * 50 * 2  # a key's rows, and its two heads


def test_gradients_of_short_sources():
    """dS goes into the products as bf16 and the results leave as bf16: each rounding is 2^-8 of a number at most, evenly
    spread, so below 2^-8 / sqrt(3) in the mean, both together below 0.0032."""
    p = Pack([(1 + i % 30, 2 + i % 7) for i in range(200)], 4, 2, 128, seed=2)
    for g, r in zip(Run(p).build().forward().backward(), p.gradients()):
        assert (g.double().cpu() - r).norm() <= 0.0032 * r.norm()


def test_gradients_against_differences():
    """Along random directions, (f(x + h u) - f(x - h u)) / 2h of the 64-bit forward, f = sum(out * dout): h = 1e-5
    leaves h^2 of the third derivative and 1e-16 / h of rounding, both below 1e-9; the gradients' own error is REL_L2."""
    p = Pack([(37, 150), (4, 3), (130, 20)], 4, 2, 64, seed=5)
    got = Run(p).build().forward().backward(fp32=True)
    formula = p.gradients()
    g = torch.Generator().manual_seed(6)
    for i, (name, x) in enumerate((("q", p.q), ("k", p.k), ("v", p.v))):
        for _ in range(3):
            u = torch.randn(x.shape, generator=g, dtype=torch.float64)
            f = [(p.forward(**{name: x.double() + s * 1e-5 * u})[0] * p.dout.double()).sum() for s in (1, -1)]
            slope = (f[0] - f[1]) / 2e-5
            norm = formula[i].norm() * u.norm()
            assert abs((formula[i] * u).sum() - slope) <= 1e-6 * norm
            assert abs((got[i].double().cpu() * u).sum() - slope) <= REL_L2 * norm


def test_long_sides_and_many_heads():
    """Rows and keys of many tiles, more units than CTAs."""
    p = Pack([(700, 1300), (129, 2049), (1025, 64)], 16, 4, 128, seed=8, spread=1.5)
    r = Run(p).build().forward().check("long")
    _check([to_np(x) for x in r.backward()], [x.numpy() for x in p.gradients()], "long")


def test_short_pairs_share_tiles():
    p = Pack([(1 + i % 13, 2 + i % 29) for i in range(300)], 4, 2, 64, seed=9)
    a, b = (Run(p, pack, fp32=True).build().forward().check() for pack in (0, 1))
    ca, cb = api.worklist_counts(a.wl), api.worklist_counts(b.wl)
    assert ca["pairs_per_head"] == cb["pairs_per_head"] == sum(m * n for m, n in p.pairs)
    assert ca["tiles_per_head"] == 300 and cb["tiles_per_head"] < 60
    # whole groups: at most a tile on either side, none that the next pair would still fit into
    g = api.decode_worklist(b.wl)["slices"]
    assert (g[:, 1] <= 128).all() and (g[:, 4] <= 128).all()
    lens = {int(c): n for n, c in zip((n for _, n in p.pairs), p.ck.tolist())}
    rows = {int(c): m for m, c in zip((m for m, _ in p.pairs), p.ck.tolist())}
    for s, t in zip(g[:-1], g[1:]):
        assert s[1] + rows[int(t[3])] > 128 or s[4] + lens[int(t[3])] > 128


def test_one_side_without_tokens():
    p = Pack([(40, 0), (300, 0)], 4, 2, 64)
    r = Run(p).build().forward()
    torch.cuda.synchronize()
    assert not r.out.any() and bool(torch.isneginf(r.lse).all())
    assert not r.backward()[0].any()
    p = Pack([(0, 40), (0, 300)], 4, 2, 128)
    got = Run(p).build().forward().backward()
    assert not got[1].any() and not got[2].any()
    p = Pack([(0, 0)], 4, 2, 128)
    Run(p).build().forward().backward()
    p = Pack([], 4, 2, 128)
    Run(p).build().forward().backward()


@pytest.mark.parametrize("what", ["keys_total", "keys_first", "keys_order", "rows_total"])
def test_offsets_that_do_not_fit(what):
    p = Pack([(40, 50), (30, 60), (10, 70)], 4, 2, 64)
    r = Run(p)
    if what == "keys_total":
        r.ck[-1] += 1
    elif what == "keys_first":
        r.ck[0] = 1
    elif what == "keys_order":
        r.ck[1], r.ck[2] = 100, 90
    else:
        r.cu[-1] -= 1
    r.build().forward()
    torch.cuda.synchronize()
    assert api.worklist_error(r.wl) == 102
    assert bool(torch.isnan(r.out).all())  # nothing is written


def test_a_worklist_of_another_kind_is_refused():
    """The attention compares the kind that the worklist was built for with the call's mask."""
    p = Pack([(40, 40), (30, 30)], 4, 2, 64)
    r = Run(p).build()
    causal = api.make_mask(api.MASK_CAUSAL, p.tq, p.tk)
    api.attn_fwd(r.q, r.k, r.v, r.cu, causal, r.params, r.wl, r.out, r.lse)
    torch.cuda.synchronize()
    assert api.worklist_error(r.wl) == 102 and bool(torch.isnan(r.out).all())
    api.build_worklist(r.cu, causal, r.params, r.wl)
    r.forward()
    torch.cuda.synchronize()
    assert api.worklist_error(r.wl) == 102 and bool(torch.isnan(r.out).all())
    r.build().forward().check()


def test_a_worklist_of_another_kind_is_refused_by_the_backward():
    p = Pack([(40, 40), (30, 30)], 4, 2, 64)
    r = Run(p).build().forward()
    causal = api.make_mask(api.MASK_CAUSAL, p.tq, p.tk)
    for built, called in ((causal, r.mask), (r.mask, causal)):
        api.build_worklist(r.cu, built, r.params, r.wl)
        plan = api.alloc_bwd_plan(2, r.mask, r.params)
        api.build_bwd_plan(r.wl, 2, built, r.params, plan)
        dq, dk, dv = (torch.full(x.shape, math.nan, dtype=torch.bfloat16, device="cuda") for x in (r.q, r.k, r.v))
        api.attn_bwd(r.q, r.k, r.v, r.out, r.lse, r.dout, r.cu, 2, called, r.params, r.wl, plan, dq, dk, dv)
        torch.cuda.synchronize()
        assert api.worklist_error(r.wl) == 102 and bool(torch.isnan(dq).all())
    got = r.build().backward()
    _check([to_np(x) for x in got], [x.numpy() for x in p.gradients()], "after a refusal")


def test_refused_by_the_binding():
    p = Pack([(40, 50), (30, 60)], 4, 2, 64)
    r = Run(p)
    with pytest.raises(ValueError):
        api.build_worklist(r.cu[:2], r.mask, r.params, r.wl)
    with pytest.raises(ValueError):
        api.make_mask(api.MASK_CAUSAL, p.tq, p.tk, cu_keys=r.ck)
    with pytest.raises(ValueError):
        api.make_mask(api.MASK_CROSS, p.tq, p.tk, cu_keys=r.ck.long())


def test_sources_cut_in_two_are_joined_by_accumulation():
    p = Pack([(100, 300), (7, 20), (150, 129)], 4, 2, 128, seed=11)
    o_run = torch.full(p.q.shape, math.nan, device="cuda")
    l_run = torch.full((4, p.tq), -math.inf, device="cuda")
    cuts = [n // 3 for _, n in p.pairs]
    for first in (True, False):
        rows = [i for c, n, cut in zip(p.ck.tolist(), (n for _, n in p.pairs), cuts) for i in range(c, c + n) if (i - c < cut) == first]
        part = Pack([(m, cut if first else n - cut) for (m, n), cut in zip(p.pairs, cuts)], 4, 2, 128)
        part.q, part.k, part.v = p.q, p.k[rows], p.v[rows]
        r = Run(part).build()
        api.attn_fwd_accumulate(r.q, r.k, r.v, r.cu, r.mask, r.params, r.wl, o_run, l_run)
    torch.cuda.synchronize()
    o, l = p.forward()
    compare(to_np(o_run), to_np(l_run), o.numpy(), l.numpy(), "two parts")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pack", [0, 1])
def test_gradients_of_sources_cut_in_two(d, pack):
    """Each part's call gets the joined O and LSE, so its P sums to less than 1 and D = rowsum(dO O) is of all keys: dK and dV
    of a part are those of its keys, dQ adds up.  Parts of 1 to 128 keys and of more, in shared tiles and in their own."""
    p = Pack([(40, 120), (100, 300), (7, 20), (150, 129), (3, 2), (60, 256), (33, 500), (2, 12), (20, 30)], 4, 2, d, seed=11 + d)
    cuts = [60, 100, 10, 64, 1, 128, 1, 5, 29]
    o_run = torch.full(p.q.shape, math.nan, device="cuda")
    l_run = torch.full((4, p.tq), -math.inf, device="cuda")
    parts = []
    for first in (True, False):
        rows = [i for c, (_, n), cut in zip(p.ck.tolist(), p.pairs, cuts) for i in range(c, c + n) if (i - c < cut) == first]
        part = Pack([(m, cut if first else n - cut) for (m, n), cut in zip(p.pairs, cuts)], 4, 2, d)
        part.q, part.dout, part.k, part.v = p.q, p.dout, p.k[rows], p.v[rows]
        r = Run(part, pack).build()
        api.attn_fwd_accumulate(r.q, r.k, r.v, r.cu, r.mask, r.params, r.wl, o_run, l_run)
        parts.append((rows, part, r))
    whole, joined = p.gradients(), p.forward()
    total, norms = torch.zeros_like(whole[0]), 0
    for rows, part, r in parts:
        part.forward = lambda: joined  # (the formulas read O and LSE from here)
        r.out, r.lse = o_run.bfloat16(), l_run
        got = r.backward(fp32=True)
        want = part.gradients()
        _check([to_np(x) for x in got], [x.numpy() for x in want], f"part of {len(rows)} keys")
        assert (want[1] - whole[1][rows]).norm() < 1e-9 * whole[1].norm() and (want[2] - whole[2][rows]).norm() < 1e-9 * whole[2].norm()
        total += got[0].double().cpu()
        norms += want[0].norm()
    assert (total - whole[0]).norm() <= REL_L2 * norms


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shift", [6.0, 8.0, 10.0])
def test_keys_outside_the_call_count_where_they_weigh_little(d, shift):
    """A source's second part has scores lower by `shift` (weights of e^-6 to e^-10 beside the first part's) and values 1024
    times as large, so D of the first part's call is still moved by it."""
    p = Pack([(40, 60), (7, 20), (100, 128), (3, 2), (64, 100)], 4, 2, d, seed=21 + d)
    cuts = [30, 10, 64, 1, 50]
    second = torch.cat([torch.arange(n) >= cut for (_, n), cut in zip(p.pairs, cuts)])
    p.q[..., 0] = 4.0
    p.k[..., 0] = 0.0
    p.k[second, :, 0] = -shift * d ** 0.5 / 4
    p.v[second] *= 1024
    joined = p.forward()
    for first in (True, False):
        rows = torch.nonzero(second != first).flatten().tolist()
        part = Pack([(m, cut if first else n - cut) for (m, n), cut in zip(p.pairs, cuts)], 4, 2, d)
        part.q, part.dout, part.k, part.v = p.q, p.dout, p.k[rows], p.v[rows]
        r = Run(part).build()
        r.out, r.lse = joined[0].bfloat16().cuda(), joined[1].float().cuda()
        # D = rowsum(dO O) of the O that is passed: its rounding is the caller's
        part.forward = lambda: (joined[0].bfloat16().double(), joined[1])
        _check([to_np(x) for x in r.backward(fp32=True)], [x.numpy() for x in part.gradients()], f"first: {first}, {shift}")


def test_short_sources_beside_long_ones_on_one_cta():
    """dQ of one CTA takes more than two seconds, as long as a wait may take, while dK and dV begin with the short source:
    nothing of theirs may wait for the end of dQ under that limit.  All results are those of every CTA, bit for bit."""
    g = torch.Generator(device="cuda").manual_seed(1)
    hq, hkv, d, rows, keys = 32, 8, 128, [45056, 90112], [45056, 100]
    q, dout = (torch.randn((sum(rows), hq, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn((sum(keys), hkv, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    cu, ck = i32([0, rows[0], sum(rows)]), i32([0, keys[0], sum(keys)])
    mask = api.make_mask(api.MASK_CROSS, sum(rows), sum(keys), cu_keys=ck)
    got = []
    for ctas in (0, 1):
        params = api.make_params(hq, hkv, c_tile=api.default_c_tile(d), num_ctas=ctas)
        wl, plan = api.alloc_worklist(2, mask, params), api.alloc_bwd_plan(2, mask, params)
        api.build_worklist(cu, mask, params, wl)
        api.build_bwd_plan(wl, 2, mask, params, plan)
        if ctas == 0:
            out, lse = torch.empty_like(q), torch.empty((hq, sum(rows)), device="cuda")
            api.attn_fwd(q, k, v, cu, mask, params, wl, out, lse)
        grads = [torch.full_like(x, math.nan) for x in (q, k, v)]
        api.attn_bwd(q, k, v, out, lse, dout, cu, 2, mask, params, wl, plan, *grads)
        torch.cuda.synchronize()
        assert api.worklist_error(wl) == 0
        got.append(grads)
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq", [1, 5])
@pytest.mark.parametrize("dispatch", [api.DISPATCH_DYNAMIC, api.DISPATCH_STATIC])
@pytest.mark.parametrize("accumulate", [False, True])
def test_targets_of_one_tile_over_sources_of_many(d, hq, dispatch, accumulate):
    """Targets of up to 128 rows with a kv head of their own, over sources of 2 to 12 tiles, between pairs of one key tile,
    without keys, and of two row tiles; several units a CTA.  Some sources have their largest scores in their last tile."""
    sizes = [(77, 1500), (1, 129), (128, 256), (33, 257), (9, 100), (200, 300), (5, 0), (64, 640), (127, 385), (300, 130), (2, 1024)]
    p = Pack([sizes[(3 * i) % len(sizes)] for i in range(60 if hq == 5 else 22)], hq, hq, d, seed=d + hq, spread=1.5)
    for i, (c, f) in enumerate(zip(p.ck[:-1].tolist(), p.ck[1:].tolist())):
        if i % 3 == 0 and f - c > 128:
            p.k[f - 20:f] *= 4
    r = Run(p, 0, dispatch, fp32=accumulate).build()
    if accumulate:
        r.lse.fill_(-math.inf)
        api.attn_fwd_accumulate(r.q, r.k, r.v, r.cu, r.mask, r.params, r.wl, r.out, r.lse)
    else:
        r.forward()
    torch.cuda.synchronize()
    assert api.worklist_error(r.wl) == 0
    o, l = p.forward()
    seen = torch.isfinite(l[0])  # (accumulated, rows without keys keep what was there)
    assert accumulate or (not r.out.cpu()[~seen].any() and torch.isneginf(r.lse.cpu()[:, ~seen]).all())
    # Scores are sums of d exact products in fp32: off by e <= d 2^-23 sum |q k| scale, and so is the LSE, beside its own
    # logarithm's rounding.  Weights are off by a factor e^+-2e and, as bf16 operands, by 2^-8 of each, the output by 2^-8 of itself.
    e = d * 2.0 ** -23 * p.scale * p.q.abs().double().sum(-1).max() * p.k.abs().max().double()
    assert e < 0.05
    top = p.v.abs().max().double()
    err = (r.out.double().cpu() - o)[seen].abs()
    assert (err <= 2.0 ** -8 * (o[seen].abs() + top) + 3 * e * top).all()
    assert (err.norm() / o[seen].norm()) <= 3e-3  # two roundings to 8 bits, each 2^-8 / sqrt(3) at most in the mean
    assert ((r.lse.double().cpu() - l)[:, seen].abs() <= e + 2.0 ** -21 * (1 + l[:, seen].abs())).all()


def test_captured_with_other_lengths():
    """Worklist, forward, plan and backward in one graph, replayed for other lengths of the same totals."""
    pairs = [[(40, 300), (200, 20), (16, 64)], [(100, 50), (100, 50), (56, 284)], [(0, 384), (255, 0), (1, 0)]]
    p = Pack(pairs[0], 4, 2, 64, seed=12)
    r = Run(p).build().forward()
    plan = api.alloc_bwd_plan(3, r.mask, r.params)
    grads = [torch.empty_like(x) for x in (r.q, r.k, r.v)]

    def step():
        r.build().forward()
        api.build_bwd_plan(r.wl, 3, r.mask, r.params, plan)
        api.attn_bwd(r.q, r.k, r.v, r.out, r.lse, r.dout, r.cu, 3, r.mask, r.params, r.wl, plan, *grads, softmax_scale=p.scale)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for other in pairs:
        p.pairs = other
        p.cu, p.ck = (torch.tensor([0] + [x[i] for x in other]).cumsum(0).to(torch.int32) for i in (0, 1))
        r.cu.copy_(p.cu)
        r.ck.copy_(p.ck)
        graph.replay()
        r.check(str(other))
        _check([to_np(x) for x in grads], [x.numpy() for x in p.gradients()], str(other))


def test_host_buffers_and_the_call_without_allocation():
    p = Pack([(40, 300), (200, 20), (16, 64)], 4, 2, 64, seed=13)
    r = Run(p)
    import ctypes

    from packed_varlen_attention_cu_gb300 import _lib
    rc = _lib.lib().pva_attn_fwd_noalloc(r.q.data_ptr(), r.k.data_ptr(), r.v.data_ptr(), r.cu.data_ptr(), 3, ctypes.byref(r.mask),
                                         ctypes.byref(r.params), 64, r.out.data_ptr(), 0, r.lse.data_ptr(), 0.0,
                                         torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    o, l = p.forward()
    compare(to_np(r.out), to_np(r.lse), o.numpy(), l.numpy(), "noalloc")
    bufs = api.alloc_host_path_buffers(p.q, p.k, 3, r.mask, r.params)
    out, lse = torch.empty_like(p.q).pin_memory(), torch.empty((4, p.tq)).pin_memory()
    api.attn_fwd_host(p.q, p.k, p.v, p.cu, 3, r.mask, r.params, out, lse, bufs)
    torch.cuda.synchronize()
    compare(to_np(out), to_np(lse), o.numpy(), l.numpy(), "host")


# ------------------------------------------------------------------ over the cache

class Source(Problem):
    """A cache of sources; every row of a sequence sees all of its keys."""

    def attend(self, scale=None, drop=None):
        hq, hkv, d = self.hq, self.hkv, self.d
        scale = d ** -0.5 if scale is None else scale
        out = torch.full((self.tokens, hq, d), math.nan, dtype=torch.float64)
        lse = torch.full((hq, self.tokens), math.nan, dtype=torch.float64)
        err, lerr = torch.zeros_like(out), torch.zeros_like(lse)
        for b, (n, m) in enumerate(zip(self.lens, self.news)):
            a = int(self.cu[b])
            j = torch.arange(n)
            j = j[self.table[b, j // self.page] >= 0] if n else j
            if m == 0:
                continue
            if len(j) == 0:
                out[a:a + m], lse[:, a:a + m] = 0, -math.inf
                continue
            k, v = self.cached("k", b)[j], self.cached("v", b)[j]
            q = self.q[a:a + m].double().unflatten(1, (hkv, -1))
            s = torch.einsum("mhgd,lhd->hgml", q, k) * scale
            mag = torch.einsum("mhgd,lhd->hgml", q.abs(), k.abs()) * scale
            ll = torch.logsumexp(s, -1)
            w = (s - ll[..., None]).exp()
            o = torch.einsum("hgml,lhd->mhgd", w, v)
            pv = torch.einsum("hgml,lhd->mhgd", w, v.abs())
            big = torch.einsum("hgml,lhd->mhgd", w, v.abs().amax(-1, keepdim=True).expand_as(v))
            # the bounds of Problem.attend: scores in fp32 (16 times the magnitude for codes around their
            # middle), weights and the result rounded to bf16
            ds = mag.amax(-1) * (d + 4) * 2 * U32 * (16 if self.int4 else 1) + 2e-6
            e16 = U16 * (o.abs() + (2 * big if self.int4 else pv)) + 2 * ds.permute(2, 0, 1)[..., None] * big
            out[a:a + m], err[a:a + m] = o.flatten(1, 2), (e16 + 1e-6 * big).flatten(1, 2) + 1e-30
            lse[:, a:a + m] = ll.flatten(0, 1)
            lerr[:, a:a + m] = (2 * ds + 4 * U32 * ll.abs()).flatten(0, 1)
        return out, lse, err, lerr


def over_cache(p, cu=True, status=None, scale=0.0, fp32=False, strided=False, table=None, cache=None, stream=None):
    q = p.wide.cuda()[:, :p.hq] if strided else p.q.contiguous().cuda()
    out = torch.full((p.tokens, p.hq, p.d), math.nan, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
    lse = torch.full((p.hq, p.tokens), math.nan, device="cuda")
    most = max(p.news + [1])
    ws = api.alloc_cache_workspace(len(p.lens), p.hq, p.hkv, p.d, most)
    ws.fill_(255)
    api.cache_cross_attn(cache or on_gpu(p), q, (p.table if table is None else table).cuda(), i32(p.lens), out, lse, ws,
                         cu_new=p.cu.cuda() if cu else None, max_new=most, softmax_scale=scale, status=status, stream=stream)
    return out, lse


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (3, 3, 64), (14, 2, 64), (5, 1, 128)])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("fp32", [False, True])
def test_rows_see_the_whole_source(int4, hq, hkv, d, page, fp32):
    """1 .. 21 rows, more rows than keys, sources of every length around tiles, no key at all, no row at all."""
    lens = [1, 700, 0, 63, 64, 65, 130, 5, 1000]
    news = [4, 3, 2, 1, 8, 0, 21, 9, 5]
    p = Source(lens, news, hq, hkv, d, page, int4, seed=d + page, spare_rows=2, strided=fp32)
    status = word()
    out, lse = over_cache(p, status=status, fp32=fp32, strided=fp32)
    assert api.cache_status(status) == 0
    check_attention(p, out, lse, p.attend(), f"{int4} {page}")
    t = int(p.cu[-1])
    assert bool(torch.isnan(out[t:]).all()) and bool(torch.isnan(lse[:, t:]).all())


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("hq,hkv,d,most", [(4, 2, 128, 8), (8, 2, 128, 4), (8, 2, 64, 7), (8, 2, 128, 12), (14, 2, 64, 11), (4, 4, 64, 60),
                                           (16, 1, 128, 9)])
@pytest.mark.parametrize("page", [16, 32, 256])
def test_many_rows(int4, hq, hkv, d, most, page):
    """9 to 144 rows a kv head: every variant that divides rows over warps, sources around tiles of 64 keys, cut over
    CTAs and whole, without keys, without rows."""
    lens = [64, 1, 0, 65, 3000, 129, 15, 16, 17, 192, 10000, 63]
    news = [most, 1, most, 2, most, 0, most, 3, 1, most, most, most]
    p = Source(lens, news, hq, hkv, d, page, int4, seed=d + page + most, spare_rows=1, strided=page == 32)
    status = word()
    out, lse = over_cache(p, status=status, fp32=page == 256, strided=page == 32)
    assert api.cache_status(status) == 0
    check_attention(p, out, lse, p.attend(), f"{int4} {hq}/{hkv} {most}")
    assert bool(torch.isnan(out[-1]).all()) and bool(torch.isnan(lse[:, -1]).all())
    again = over_cache(p, fp32=page == 256, strided=page == 32)
    assert torch.equal(out[:-1], again[0][:-1]) and torch.equal(lse[:, :-1], again[1][:, :-1])


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("most", [1, 4, 5, 8, 9, 16, 17])
def test_weights_have_16_bits_for_any_number_of_rows(int4, d, most):
    """4 to 68 rows a kv head, fp32 results.  Queries are whole numbers and so are cached keys (4 bits: codes - 8), so scores
    and their products with the scale 2^-4 are exact.  Weights: 2^-16 of each as the sum of two bf16 numbers, 2^-19 for the
    exponent's argument and the exponential.  4 bits: they meet scale * (code - 8), no larger than 8 scale, and
    middle = low + 8 scale, rounded to fp32.  Sums in fp32: 50 tiles of 64 keys and their joins, each 2^-23 of a sum of
    magnitudes: 2^-17.  In all less than 2^-15 of the weighted magnitudes; one bf16 number a weight is off by up to 2^-8."""
    p = Source([3000, 40, 7, 1, 130], [most, most, 1, most, most], 8, 2, d, 64, int4, seed=most + d)
    g = torch.Generator().manual_seed(most)
    p.q = torch.randint(-2, 3, p.q.shape, generator=g).bfloat16()
    garbage = torch.isnan(p.k_scales if int4 else p.k)
    if int4:
        code = unpack(p.k)
        pair = torch.tensor([1.0, -8.0]).expand(p.k_scales.shape)
        p.rows["k"] = values(code, pair[..., 0], pair[..., 1])
        p.k_scales = torch.where(garbage, torch.nan, pair).bfloat16()
        scale, low = p.v_scales.double().nan_to_num().unbind(-1)
        size = (8 * scale + (low + 8 * scale).abs())[..., None].expand(code.shape[:-1] + (d // 64, 64)).flatten(-2)
    else:
        k = torch.randint(-3, 4, p.k.shape, generator=g).double()
        p.rows["k"] = k
        p.k = torch.where(garbage, torch.nan, k).bfloat16()
        size = p.rows["v"].abs().nan_to_num()
    out, lse = over_cache(p, scale=2.0 ** -4, fp32=True)
    o, l, _, _ = p.attend(scale=2.0 ** -4)
    p.rows["v"] = size
    bound = 2.0 ** -15 * p.attend(scale=2.0 ** -4)[0]
    off = (out.double().cpu() - o).abs()
    assert bool((off <= bound).all()), f"{(off / bound).max():.3g} of the bound"
    # a sum of weights, its logarithm, the maximum in base 2 (below 2^6) and back
    assert bool(((lse.double().cpu() - l).abs() <= 2.0 ** -17).all())


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("most", [5, 12])
def test_many_rows_with_missing_pages(int4, most):
    p = Source([200, 100, 640], [most, 3, most], 8, 2, 128, 16, int4, seed=8)
    p.table[0, 2] = p.table[2, 4] = p.table[2, 5] = -1
    p.table[1, :] = 10 ** 6
    status = word()
    out, lse = over_cache(p, status=status)
    assert api.cache_status(status) == 300
    p.table[1, :] = -1
    check_attention(p, out, lse, p.attend())


@pytest.mark.parametrize("int4", [False, True])
def test_long_sources_of_many_rows_have_no_bias(int4):
    """Equal weights over values of mean 1: sums of 40000 products that all go one way."""
    p = Source([40000], [6], 8, 2, 64, 64, int4, seed=9)
    for x in "v":
        rows = p.rows[x] * 0.05 + 1
        if int4:
            code, scale, low = quantise(rows.float().bfloat16())
            p.v, p.v_scales = pack(code), torch.stack((scale, low), -1).bfloat16()
            p.rows[x] = values(code, scale, low)
        else:
            p.v = rows.bfloat16()
            p.rows[x] = p.v.double()
    p.v_scales = p.v_scales.nan_to_num() if int4 else None
    p.wide = None
    p.q = torch.zeros_like(p.q)
    out, lse = over_cache(p, fp32=True)
    o, l, _, _ = p.attend()
    # weights are 1 (exact in bf16; with 4 bits times the scale: 2^-9 of 8 scales, averaged over 40000 random codes), a
    # tile's sum of up to eight products rounded towards 0 (2^-21) and about 300 additions of fp32 a piece, joined
    tol = 2.0 ** -20 + (8 * 2.0 ** -9 * 0.05 * 8 / 15 / 40000 ** 0.5 * 4 if int4 else 0) + 64 * U32
    off = (out.double().cpu() - o).abs().mean()
    assert off <= tol, (off, tol)


@pytest.mark.parametrize("int4", [False, True])
def test_scores_and_values_that_are_not_finite(int4):
    """A NaN among the keys that rows see makes their results NaN, in other sequences nothing changes; weights of 0 meet
    values that are not finite."""
    p = Source([100, 90, 80], [5, 5, 5], 8, 2, 128, 16, int4, seed=10)
    o, l, e, le = p.attend()
    cache = on_gpu(p)
    at = int(p.table[1, 2])
    if int4:
        cache.k_scales[at, 0, 3, 0, 1] = math.nan
    else:
        cache.k[at, 0, 3, 7] = math.nan
    out, lse = over_cache(p, cache=cache)
    bad = torch.zeros_like(l, dtype=torch.bool)
    bad[:4, 5:10] = True  # the heads of kv head 0, sequence 1
    assert bool(torch.isnan(lse.cpu()[bad]).all()) and bool(torch.isnan(out.cpu()[bad.t()]).all())
    l2, o2 = l.clone(), o.clone()
    fin = ~bad
    assert bool(((lse.cpu().double() - l).abs()[fin] <= le[fin]).all())
    assert bool(((out.cpu().double() - o).abs()[fin.t()] <= e[fin.t()]).all())


@pytest.mark.parametrize("int4", [False, True])
def test_one_row_each_and_padded_batch(int4):
    lens = [40, 0, 300, 1]
    p = Source(lens, [1] * 4, 8, 2, 128, 16, int4, seed=3)
    status = word()
    out, lse = over_cache(p, cu=False, status=status)
    assert api.cache_status(status) == 0
    check_attention(p, out, lse, p.attend())


def test_long_source_cut_over_many_ctas():
    p = Source([9001, 20000], [7, 2], 4, 2, 64, 64, seed=4)
    out, lse = over_cache(p, scale=0.3)
    check_attention(p, out, lse, p.attend(scale=0.3))


def test_one_row_equals_the_causal_call():
    """The last new token sees every cached key: both calls give the same bits."""
    p = Source([500, 77, 3], [1, 1, 1], 8, 2, 128, 32, seed=5)
    out, lse = over_cache(p)
    o, l = torch.empty_like(out), torch.empty_like(lse)
    ws = api.alloc_cache_workspace(3, 8, 2, 128)
    api.cache_attn(on_gpu(p), p.q.contiguous().cuda(), p.table.cuda(), i32(p.lens), o, l, ws)
    assert torch.equal(o, out) and torch.equal(l, lse)


def test_pages_that_are_missing_and_lengths_past_the_table():
    p = Source([200, 100], [3, 3], 4, 2, 64, 16, seed=6)
    p.table[0, 2] = -1
    status = word()
    out, lse = over_cache(p, status=status)
    assert api.cache_status(status) == 300
    check_attention(p, out, lse, p.attend())
    p = Source([200, 100], [3, 3], 4, 2, 64, 16, seed=6)
    lens, p.lens = p.lens, [2 ** 31 - 1, 100]
    status = word()
    out, lse = over_cache(p, status=status)
    p.lens = [16 * p.table.shape[1], 100]
    assert api.cache_status(status) == 300
    check_attention(p, out, lse, p.attend())
    p.lens = [-5, 100]
    status = word()
    out, lse = over_cache(p, status=status)
    p.lens = [0, 100]
    assert api.cache_status(status) == 301
    check_attention(p, out, lse, p.attend())


def test_on_another_stream():
    p = Source([500, 77, 300], [4, 4, 4], 8, 2, 128, 32, seed=7)
    side = torch.cuda.Stream()
    cache = on_gpu(p)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        out, lse = over_cache(p, cache=cache)
    side.synchronize()
    check_attention(p, out, lse, p.attend())


def test_a_source_from_its_pack():
    """A source's keys and values go into the cache by the append (no rotation), and beams over it give what the packs give."""
    p = Pack([(5, 400), (3, 90)], 8, 2, 128, seed=14)
    r = Run(p).build().forward().check()
    cache = api.KVCache.alloc(16, 2, 128, page_size=64)
    table = torch.arange(16, dtype=torch.int32, device="cuda").view(2, 8)
    lens = i32([400, 90])
    api.cache_append(cache, r.k, r.v, table, lens, cu_new=r.ck)
    out, lse = torch.empty_like(r.q), torch.empty_like(r.lse)
    ws = api.alloc_cache_workspace(2, 8, 2, 128, max_new=5)
    api.cache_cross_attn(cache, r.q, table, lens, out, lse, ws, cu_new=r.cu, max_new=5)
    o, l = p.forward()
    compare(to_np(out), to_np(lse), o.numpy(), l.numpy(), "cached")
    assert np.abs(to_np(lse) - to_np(r.lse)).max() < 1e-4
