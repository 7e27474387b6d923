"""Beam search on the GPU: selection against the ranking in 64 bits, reordering
against copies, and both with the cache calls as a model decodes with them."""
import math

import numpy as np
import pytest
import torch

from cache_util import U16, U32, angles, pack, quantise, rotate, values
from packed_varlen_attention_cu_gb300 import api
from test_gpu_cache import i32, word

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ selection

def ranking(logits, scores, k, finished=None, norms=None, end=0):
    """(scores float64, beams, tokens, finished) [groups, k] by the rules of the header, and which rows offer something wrong."""
    groups, beams = scores.shape
    x = logits.double().view(groups, beams, -1).numpy()
    out_s = np.full((groups, k), -np.inf)
    out_b, out_t, out_f = (np.full((groups, k), v) for v in (-1, -1, 0))
    told = False
    for g in range(groups):
        cand = []  # (rank, beam, logit, token, score)
        for b in range(beams):
            s = float(scores[g, b])
            w = 1.0 if norms is None else float(norms[g, b])
            if math.isnan(s) or s == math.inf or not (0 < w < math.inf):
                told = True
                continue
            if s == -math.inf:
                continue
            if finished is not None and finished[g, b]:
                cand.append((s * w, b, 0.0, end, s))
                continue
            row = x[g, b]
            if np.isnan(row).any() or (row == np.inf).any():
                told = True
                continue
            ok = np.nonzero(row > -np.inf)[0]
            if len(ok) == 0:
                continue
            top = row[ok].max()
            lse = top + math.log(np.exp(row[ok] - top).sum())
            best = ok[np.argsort(-row[ok], kind="stable")[:k]]
            cand += [((s - lse + row[t]) * w, b, row[t], int(t), s - lse + row[t]) for t in best]
        cand.sort(key=lambda c: (-c[0], c[1], -c[2], c[3]))
        for i, (_, b, _, t, s) in enumerate(cand[:k]):
            out_s[g, i], out_b[g, i], out_t[g, i] = s, b, t
            out_f[g, i] = t == end or (finished is not None and bool(finished[g, b]))
    return out_s, out_b, out_t, out_f, told


class Select:
    def __init__(self, logits, scores, k, finished=None, norms=None, end=0, status=None, ws=None, stream=None):
        groups, beams = scores.shape
        self.os = torch.full((groups, k), 7.0, device="cuda")
        self.ob, self.ot = (torch.full((groups, k), 7, dtype=torch.int32, device="cuda") for _ in range(2))
        self.of = torch.full((groups, k), 7, dtype=torch.uint8, device="cuda")
        if ws is None:
            ws = api.alloc_beam_workspace(groups, beams, logits.shape[1], k)
            ws.fill_(255)
        self.args = (logits, scores.cuda(), self.os, self.ob, self.ot, ws)
        self.kw = dict(end_token=end, finished=None if finished is None else finished.cuda(), norms=None if norms is None else norms.cuda(),
                       out_finished=self.of, status=status, stream=stream)
        self.again()

    def again(self):
        api.beam_select(*self.args, **self.kw)

    def check(self, ref):
        s, b, t, f, _ = ref
        np.testing.assert_array_equal(self.ob.cpu().numpy(), b)
        np.testing.assert_array_equal(self.ot.cpu().numpy(), t)
        np.testing.assert_array_equal(self.of.cpu().numpy(), f)
        got = self.os.double().cpu().numpy()
        np.testing.assert_array_equal(np.isneginf(got), np.isneginf(s))
        fin = np.isfinite(s)
        # the result's rounding; an exponential's 2^-22, once more where a sum's reference moves (by 1 at least, so
        # that all moves together stay below the last one's 2^-22) and twice where threads and parts are joined; at
        # most 32 additions of a thread in fp32; log2(e) and the differences rounded: 2^-23 of the entropy, below 22
        tol = U32 * np.abs(s[fin]) + 2.0 ** -20 + 32 * U32 + 22 * 2.0 ** -23
        assert (np.abs(got[fin] - s[fin]) <= tol).all(), np.abs(got[fin] - s[fin]).max()


def rows_of(kind, groups, beams, vocab, seed, spread=2.5, pad=0, offset=0):
    """Logits on the GPU as a view into a wider tensor that holds NaN around them, and on the CPU."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((groups * beams, vocab), generator=g) * spread).to(kind)
    wide = torch.full((groups * beams, vocab + pad + offset), math.nan, dtype=kind, device="cuda")
    view = wide[:, offset:offset + vocab]
    view.copy_(x)
    return view, x


def scores_of(groups, beams, seed):
    return -3 * torch.randn((groups, beams), generator=torch.Generator().manual_seed(seed + 1)).abs()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("groups,beams,vocab,k,pad,offset", [
    (1, 1, 1, 1, 0, 0), (1, 1, 1, 5, 0, 0), (2, 3, 2, 8, 1, 1), (3, 4, 7, 4, 0, 0), (5, 2, 64, 64, 3, 5), (2, 4, 255, 8, 0, 1),
    (3, 5, 1000, 10, 7, 2), (1, 4, 8191, 8, 0, 3), (2, 8, 8192, 16, 0, 0), (2, 8, 8193, 16, 0, 7), (1, 4, 32003, 8, 0, 0),
    (7, 3, 50021, 6, 0, 0), (1, 64, 5000, 64, 1, 0), (2, 16, 33333, 32, 0, 0), (1, 1, 262144, 64, 0, 0), (40, 16, 20011, 32, 5, 0),
    (200, 4, 3001, 4, 0, 0), (1, 2, 1000003, 4, 0, 1)])
def test_select(kind, groups, beams, vocab, k, pad, offset):
    seed = vocab + k
    view, x = rows_of(kind, groups, beams, vocab, seed, pad=pad, offset=offset)
    scores, status = scores_of(groups, beams, seed), word()
    Select(view, scores, k, status=status).check(ranking(x, scores, k))
    assert api.cache_status(status) == 0


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_finished_dead_and_weighed_rows(kind):
    groups, beams, vocab, k = 12, 5, 4001, 10
    view, x = rows_of(kind, groups, beams, vocab, 3)
    scores = scores_of(groups, beams, 3)
    g = torch.Generator().manual_seed(4)
    finished = (torch.rand((groups, beams), generator=g) < 0.4).to(torch.uint8)
    norms = (1 + torch.randint(0, 100, (groups, beams), generator=g).float()) ** -0.7
    scores[1, 2] = scores[2] = -math.inf            # one beam, a whole group dead
    finished[3] = 1                                 # a whole group finished: fewer candidates than places
    finished[4], scores[4, 1:] = 0, -math.inf       # the first step: one beam alive
    view[5 * beams] = math.nan                      # a finished row's logits are not read
    finished[5, 0] = 1
    status = word()
    ref = ranking(x, scores, k, finished, norms, end=2)
    Select(view, scores, k, finished, norms, end=2, status=status).check(ref)
    assert api.cache_status(status) == 0 and not ref[4]
    Select(view, scores, k, finished, end=2).check(ranking(x, scores, k, finished, end=2))


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("order", ["up", "down", "flat", "few", "saw", "one"])
def test_logits_in_bad_orders_and_equal_ones(kind, order):
    """Every tile above the one before it, nothing but equal logits, few values: the lower beam and token win."""
    groups, beams, vocab, k = 2, 3, 40000, 12
    i = torch.arange(vocab, dtype=torch.float64)
    row = {"up": i / vocab * 20 - 10, "down": 10 - i / vocab * 20, "flat": 0 * i, "few": (i * 7919 % 5).floor(),
           "saw": (i % 100) / 10, "one": torch.where(i == 39999, 30.0, -5.0)}[order].to(kind)
    x = row.expand(groups * beams, vocab).contiguous()
    scores = torch.tensor([[-1.0, -1.0, -1.0], [-2.0, -1.0, -math.inf]])
    Select(x.cuda(), scores, k).check(ranking(x, scores, k))
    Select(x.cuda(), scores, 64).check(ranking(x, scores, 64))


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("low", ["inf", "lowest"])
def test_masked_logits(kind, low):
    """Masks of -inf or the type's lowest value (a logit like any other: a row of nothing else is a uniform one): all
    tokens but few, all of one row, a whole tile, all rows."""
    groups, beams, vocab, k = 3, 4, 30001, 8
    _, x = rows_of(kind, groups, beams, vocab, 5)
    none = -math.inf if low == "inf" else torch.finfo(kind).min
    x[0, 3:] = none
    x[1] = none
    x[2, :8192] = none
    x[3, 1::2] = none
    x[4:8] = none
    x[5, 29999] = -1.5
    x[8:] = none
    x[8, 30000], x[9, 0] = 3.0, 3.0
    scores = scores_of(groups, beams, 5)
    status = word()
    ref = ranking(x, scores, k)
    assert low == "lowest" or ((ref[1][1] == 1).sum() == 1 and (ref[1][2] == -1).sum() == k - 2)
    Select(x.cuda(), scores, k, status=status).check(ref)
    assert api.cache_status(status) == 0


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("what", ["nan", "inf", "score", "score_inf", "norm0", "norm_nan", "norm_inf"])
def test_rows_that_cannot_be_ranked_are_left_out(kind, what):
    groups, beams, vocab, k = 2, 3, 9000, 5
    _, x = rows_of(kind, groups, beams, vocab, 6)
    scores, norms = scores_of(groups, beams, 6), torch.ones((groups, beams))
    if what in ("nan", "inf"):
        x[1, 8999] = {"nan": math.nan, "inf": math.inf}[what]
    elif what.startswith("score"):
        scores[0, 1] = math.inf if what == "score_inf" else math.nan
    else:
        norms[0, 1] = {"norm0": 0.0, "norm_nan": math.nan, "norm_inf": math.inf}[what]
    ref = ranking(x, scores, k, norms=norms)
    status = word()
    Select(x.cuda(), scores, k, norms=norms, status=status).check(ref)
    assert ref[4] and api.cache_status(status) == 304 and not (ref[1][0] == 1).any()


def test_large_logits_keep_their_logarithm():
    """Values far from 0, up to fp32's largest: the differences from about the largest logit are taken first."""
    g = torch.Generator().manual_seed(7)
    x = torch.randn((4, 20000), generator=g)
    for shift in (1e4, -1e4, 3e8, -1e30, 3e38):
        y = x + shift
        y[0, 77], y[1, 78] = torch.finfo(torch.float32).max, torch.finfo(torch.float32).min
        scores = torch.zeros((1, 4))
        Select(y.cuda(), scores, 8).check(ranking(y, scores, 8))


def test_rows_past_32_bits():
    """Rows whose offsets leave 32 bits."""
    vocab, stride = 5000, 1_300_000_007
    wide = torch.empty(2 * stride + vocab, dtype=torch.bfloat16, device="cuda")
    _, x = rows_of(torch.bfloat16, 1, 3, vocab, 8)
    for b in range(3):
        wide[b * stride:b * stride + vocab] = x[b].cuda()
    scores = scores_of(1, 3, 8)
    Select(torch.as_strided(wide, (3, vocab), (stride, 1)), scores, 6).check(ranking(x, scores, 6))


def test_same_bits_again_captured_and_on_another_stream():
    view, x = rows_of(torch.bfloat16, 6, 5, 70001, 9)
    _, y = rows_of(torch.bfloat16, 6, 5, 70001, 10)
    scores = scores_of(6, 5, 9)
    a = Select(view, scores, 10)
    first = [t.clone() for t in (a.os, a.ob, a.ot)]
    for _ in range(3):
        a.again()
        assert all(torch.equal(p, q) for p, q in zip(first, (a.os, a.ob, a.ot)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.again()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, (a.os, a.ob, a.ot)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.again()
    for z in (y, x):
        view.copy_(z)
        graph.replay()
        a.check(ranking(z, scores, 10))


def test_two_streams_with_their_own_workspaces():
    runs = []
    for i in range(2):
        s = torch.cuda.Stream()
        view, x = rows_of(torch.float32, 8, 4, 30011, 20 + i)
        torch.cuda.synchronize()
        runs.append((s, Select(view, scores_of(8, 4, 20 + i), 8, stream=s), x, scores_of(8, 4, 20 + i)))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, r, _, _ in runs:
            r.again()
    torch.cuda.synchronize()
    for s, r, x, scores in runs:
        r.check(ranking(x, scores, 8))


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_one_workspace_for_a_batch_that_shrinks(kind):
    beams, vocab, k = 8, 40001, 16
    ws = api.alloc_beam_workspace(40, beams, vocab, k)
    for groups in (40, 39, 17, 16, 9, 8, 3, 1):
        view, x = rows_of(kind, groups, beams, vocab, groups)
        s = scores_of(groups, beams, groups)
        ws.fill_(255)
        Select(view, s, k, ws=ws).check(ranking(x, s, k))


def test_select_refusals_of_the_binding():
    view, _ = rows_of(torch.float32, 2, 3, 50, 1)
    s, i = torch.zeros((2, 3), device="cuda"), torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    ws = api.alloc_beam_workspace(2, 3, 50, 3)
    api.beam_select(view, s, torch.empty_like(s), i, i.clone(), ws)
    for args, kw in (((view.double(), s, s, i, i, ws), {}), ((view[:5], s, s, i, i, ws), {}), ((view.t(), s, s, i, i, ws), {}),
                     ((view, s.cpu(), s, i, i, ws), {}), ((view, s, s, i.float(), i, ws), {}), ((view, s, s, i, i[:, :2], ws), {}),
                     ((view, s, s, i, i, ws.cpu()), {}), ((view, s, s, i, i, ws), dict(norms=i)),
                     ((view, s, s, i, i, ws), dict(finished=i)), ((view, s, s, i, i, ws), dict(out_finished=i))):
        with pytest.raises(ValueError):
            api.beam_select(*args, **kw)
    with pytest.raises(Exception, match="BUFFER_TOO_SMALL"):
        api.beam_select(view, s, torch.empty_like(s), i, i.clone(), ws[:256])


# ------------------------------------------------------------------ reordering

class Beams:
    """Caches of several layers and states on the GPU, and copies of them on the CPU to compare with."""

    def __init__(self, lens, beams, layers=2, heads=3, d=64, page=16, int4=False, seed=0, states=(), extra=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.beams, self.page, self.groups = lens, beams, page, len(lens)
        rows = self.groups * beams
        width = max(n // page + 1 for n in lens) + extra
        self.width = width
        # every row owns all pages of its table (prompts' pages may as well be shared)
        count = rows * width + 2
        self.table = torch.randperm(count, generator=g)[:rows * width].view(rows, width).to(torch.int32)
        shape = (count, heads, page)

        def raw(*s, kind=torch.bfloat16):
            if kind == torch.uint8:
                return torch.randint(0, 256, s, generator=g, dtype=torch.uint8)
            return torch.randn(s, generator=g).to(kind)

        if int4:
            self.data = [[raw(*shape, d // 2, kind=torch.uint8), raw(*shape, d // 2, kind=torch.uint8), raw(*shape, d // 64, 2),
                          raw(*shape, d // 64, 2)] for _ in range(layers)]
        else:
            self.data = [[raw(*shape, d), raw(*shape, d)] for _ in range(layers)]
        self.states = [raw(rows, *s[1:], kind=s[0]) if s[0].is_floating_point else
                       torch.randint(-99, 99, (rows, *s[1:]), generator=g, dtype=s[0]) for s in states]
        self.g_data = [[x.cuda() for x in layer] for layer in self.data]
        self.caches = [api.KVCache(*layer) for layer in self.g_data]
        self.g_table, self.g_states = self.table.cuda(), [x.cuda() for x in self.states]
        self.g_lens = i32([n for n in lens for _ in range(beams)])

    def run(self, parents, status=None, **kw):
        self.before = ([[x.clone() for x in layer] for layer in self.data], self.table.clone(), [x.clone() for x in self.states])
        api.beam_reorder(parents.cuda(), self.caches, self.g_table, self.g_lens, states=self.g_states, status=status, **kw)

    def expect(self, parents, skip=()):
        """What the call leaves, row by row."""
        data, table, states = self.before
        for g, n in enumerate(self.lens):
            if g in skip:
                continue
            last, part = n // self.page, n % self.page
            for j in range(self.beams):
                p = int(parents[g, j])
                if p < 0 or p >= self.beams:
                    continue
                row, up = g * self.beams + j, g * self.beams + p
                self.table[row, :last] = table[up, :last]
                for now, old in zip(self.states, states):
                    now[row] = old[up]
                if part == 0:
                    continue
                here, there = int(table[row, last]), int(table[up, last])
                if min(here, there) < 0 or max(here, there) >= self.data[0][0].shape[0]:
                    continue
                for layer, olds in zip(self.data, data):
                    for now, old in zip(layer, olds):
                        now[here, :, :part] = old[there, :, :part]

    def check(self):
        torch.cuda.synchronize()
        assert torch.equal(self.g_table.cpu(), self.table)
        for a, b in zip(self.g_states, self.states):
            assert torch.equal(a.cpu(), b)
        for layer, ref in zip(self.g_data, self.data):
            # (4 bits: up to two slots of no token behind the last token's scales may be copied too)
            for x, y in zip(layer, ref):
                x, y = x.cpu(), y.clone()
                if x.dim() == 5:
                    slot = torch.arange(self.page)
                    for g, n in enumerate(self.lens):
                        last, part = n // self.page, n % self.page
                        behind = (slot >= part) & (slot < part + 4)
                        for r in range(g * self.beams, (g + 1) * self.beams):
                            q = int(self.table[r, last])
                            if part and 0 <= q < y.shape[0]:
                                y[q][:, behind] = x[q][:, behind]
                assert torch.equal(x.view(torch.int16) if x.dtype == torch.bfloat16 else x, y.view(torch.int16) if y.dtype == torch.bfloat16 else y)


def random_parents(groups, beams, seed):
    return torch.randint(0, beams, (groups, beams), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)


STATES = [(torch.int32, 37), (torch.float32, 5, 7), (torch.bfloat16, 48), (torch.float32, 1), (torch.int64, 3)]


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("beams,d,page", [(1, 64, 16), (2, 128, 16), (4, 64, 64), (5, 128, 32), (13, 64, 16), (64, 128, 16), (3, 128, 256)])
def test_reorder(int4, beams, d, page):
    lens = [0, 1, page - 1, page, 3 * page + 5, 2 * page]
    b = Beams(lens, beams, d=d, page=page, int4=int4, seed=beams + page, states=STATES, extra=1)
    status = word()
    for step in range(3):  # one after the other, each from what the one before left
        parents = random_parents(len(lens), beams, step)
        b.run(parents, status)
        b.expect(parents)
        b.check()
    assert api.cache_status(status) == 0


def test_cycles_exchanges_and_rows_that_stay():
    perms = [[1, 0, 3, 2, 4, 5], [1, 2, 3, 4, 5, 0], [0, 1, 2, 3, 4, 5], [5, 5, 5, 5, 5, 5], [-1, 0, -1, 2, 2, -1], [2, 0, 1, 4, 3, 3]]
    parents = torch.tensor(perms, dtype=torch.int32)
    b = Beams([40, 17, 9, 64, 33, 100], 6, seed=3, states=STATES)
    b.run(parents)
    b.expect(parents)
    b.check()


def test_many_layers_many_states_and_long_rows():
    """More caches and states than one launch takes, pages longer than a piece, states of many pieces."""
    b = Beams([1000, 2047], 3, layers=67, heads=1, page=1024, seed=4,
              states=[(torch.int32, 1 + i) for i in range(18)] + [(torch.float32, 10001), (torch.bfloat16, 40000)])
    parents = random_parents(2, 3, 5)
    b.run(parents)
    b.expect(parents)
    b.check()


def test_states_without_caches_and_of_strided_rows():
    wide = torch.randn((12, 3, 50), device="cuda")
    x, whole = wide[:, 1], wide.clone()
    y = torch.randint(0, 9, (12, 8), dtype=torch.int32, device="cuda")
    parents = random_parents(3, 4, 6)
    up = (torch.arange(3)[:, None] * 4 + parents).flatten().cuda()
    want = y[up]
    api.beam_reorder(parents.cuda(), states=(x, y))
    whole[:, 1] = whole[up, 1]
    assert torch.equal(wide, whole) and torch.equal(y, want)


@pytest.mark.parametrize("int4", [False, True])
def test_groups_and_pages_that_do_not_fit(int4):
    lens = [40, 33, 21, 50, 40]
    b = Beams(lens, 4, int4=int4, seed=7, states=STATES)
    parents = random_parents(5, 4, 8)
    parents[0], parents[4] = torch.tensor([1, 0, 0, 2]), torch.tensor([1, 0, 7, -9])
    b.g_lens[4] = 32                      # group 1: one row has another length
    b.g_lens[8:12] = -1                   # group 2: negative
    b.g_lens[12:16] = 16 * b.width + 16   # group 3: past the table
    b.table[1, 2] = -1                    # group 0: row 1 has no last page: neither it nor its children are copied
    b.g_table.copy_(b.table)
    status = word()
    b.run(parents, status)
    b.expect(parents, skip=(1, 2, 3))
    b.check()
    assert api.cache_status(status) in (300, 301, 305)
    for other, code in ((dict(rows=(4, 5), to=32), 301), (dict(rows=(12, 16), to=16 * b.width + 16), 300), (None, 305)):
        c = Beams(lens, 4, int4=int4, seed=7)
        if other:
            c.g_lens[other["rows"][0]:other["rows"][1]] = other["to"]
        p = parents.clamp(0, 3)
        if not other:
            p[2, 1] = 4
        status = word()
        c.run(p, status)
        assert api.cache_status(status) == code


@pytest.mark.parametrize("int4", [False, True])
def test_a_length_whose_last_page_is_past_the_table(int4):
    """One token past the table's last column is past the table: nothing of the group moves, its table and states neither."""
    b = Beams([47, 31, 47], 4, int4=int4, seed=12, states=STATES)  # tables of three pages
    assert b.width == 3
    for at, n in ((0, 49), (8, 63)):
        b.g_lens[at:at + 4] = n
    parents = random_parents(3, 4, 13)
    parents[0], parents[2] = torch.tensor([1, 0, 0, 2]), torch.tensor([3, 3, 0, 0])
    status = word()
    b.run(parents, status)
    b.expect(parents, skip=(0, 2))
    b.check()
    assert api.cache_status(status) == 300


@pytest.mark.parametrize("first", [True, False])
def test_lengths_that_differ_and_pass_the_table(first):
    """Numbers of a group that differ are told of as that, whatever else is wrong with them."""
    b = Beams([47, 47], 4, seed=14, states=STATES)
    b.g_lens[0 if first else 1] = 1000
    b.g_lens[2] = 999
    parents = torch.tensor([[1, 0, 0, 2], [1, 0, 0, 2]])
    status = word()
    b.run(parents.int(), status)
    b.expect(parents, skip=(0,))
    b.check()
    assert api.cache_status(status) == 301


def test_a_table_with_a_stride_and_a_full_one():
    b = Beams([48, 31], 4, seed=9)  # 48 tokens: three full pages, and the table's last column is the next one
    wide = torch.full((8, b.width + 5), -7, dtype=torch.int32, device="cuda")
    wide[:, :b.width] = b.g_table
    b.g_table = wide[:, :b.width]
    parents = random_parents(2, 4, 10)
    b.run(parents)
    b.expect(parents)
    b.check()
    assert bool((wide[:, b.width:] == -7).all())
    b = Beams([47, 47], 4, seed=9)
    b.lens = [48, 48]  # exactly the table
    b.table, b.g_table = b.table[:, :3].contiguous(), b.g_table[:, :3].contiguous()
    b.g_lens.fill_(48)
    status = word()
    b.run(parents, status)
    b.expect(parents)
    b.check_table = None
    torch.cuda.synchronize()
    assert torch.equal(b.g_table.cpu(), b.table) and api.cache_status(status) == 0


def test_reorder_captured():
    b = Beams([40, 17], 4, seed=11, states=STATES)
    parents = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    b.run(torch.tensor([[0, 1, 2, 3]] * 2, dtype=torch.int32))
    with torch.cuda.graph(graph):
        api.beam_reorder(parents, b.caches, b.g_table, b.g_lens, states=b.g_states)
    for step in range(3):
        p = random_parents(2, 4, 20 + step)
        parents.copy_(p)
        b.before = ([[x.clone() for x in layer] for layer in b.data], b.table.clone(), [x.clone() for x in b.states])
        graph.replay()
        b.expect(p)
        b.check()


def test_reorder_refusals_of_the_binding():
    b = Beams([20], 4)
    p = random_parents(1, 4, 0).cuda()
    ok = (p, b.caches, b.g_table, b.g_lens)
    api.beam_reorder(*ok)
    for args, kw in (((p.long(), *ok[1:]), {}), ((p[0], *ok[1:]), {}), ((p, b.caches), {}), ((p, b.caches, b.g_table[:3], b.g_lens), {}),
                     ((p, b.caches, b.g_table.long(), b.g_lens), {}), ((p, b.caches, b.g_table, b.g_lens[:3]), {}),
                     (ok, dict(states=(torch.zeros((3, 4), device="cuda"),))), (ok, dict(states=(torch.zeros((4, 4)),))),
                     (ok, dict(states=(torch.zeros((4, 4, 4), device="cuda").transpose(1, 2),))),
                     (ok, dict(states=(torch.zeros((1, 4), device="cuda").expand(4, 4),)))):
        with pytest.raises(ValueError):
            api.beam_reorder(*args, **kw)
    with pytest.raises(Exception, match="INVALID"):
        api.beam_reorder(*ok, states=(torch.zeros((4, 3), dtype=torch.uint8, device="cuda"),))


# ------------------------------------------------------------------ together

class Decoder:
    """Two layers of a decoder over sources, `beams` beams a request: the cache calls on the GPU, and every beam's own
    list of keys and values on the CPU."""

    def __init__(self, prompts, sources, beams, int4, page, steps, seed=0, hq=4, hkv=2, d=64):
        self.g = torch.Generator().manual_seed(seed)
        self.beams, self.int4, self.page, self.hq, self.hkv, self.d = beams, int4, page, hq, hkv, d
        self.groups = len(prompts)
        self.rows = self.groups * beams
        kind = api.CACHE_INT4 if int4 else api.CACHE_BF16
        width = (max(prompts) + steps) // page + 1
        self.caches = [api.KVCache.alloc(self.rows * width + 1, hkv, d, page, kind) for _ in range(2)]
        self.table = torch.randperm(self.rows * width, generator=self.g).view(self.rows, width).to(torch.int32)
        for i, n in enumerate(prompts):  # a prompt's full pages belong to all its beams
            self.table[i * beams:(i + 1) * beams, :n // page] = self.table[i * beams, :n // page]
        self.table = self.table.cuda()
        self.lens = i32([n for n in prompts for _ in range(beams)])
        self.angles = angles(max(prompts) + steps + 1, d)
        self.g_angles = self.angles.cuda()
        self.history = torch.zeros((self.rows, steps), dtype=torch.int32, device="cuda")
        self.held = [[None] * self.rows for _ in range(2)]  # layer, row: (keys, values) float64 [n, hkv, d]
        cu = i32([0] + list(np.cumsum(prompts)))
        for layer, cache in enumerate(self.caches):
            k, v = (self.randn(sum(prompts), hkv, d) for _ in "kv")
            api.cache_append(cache, k.cuda(), v.cuda(), self.table[::beams], i32(prompts), cu_new=cu, table=self.g_angles)
            a = 0
            for i, n in enumerate(prompts):
                rows = (self.as_held(rotate(k[a:a + n], self.angles, torch.arange(n), False)[0]), self.as_held(v[a:a + n].double()))
                for j in range(beams):
                    self.held[layer][i * beams + j] = rows
                a += n
        # the prompt's last, partly filled page lies in the first beam's own page: every beam becomes its copy
        api.beam_reorder(torch.zeros((self.groups, beams), dtype=torch.int32, device="cuda"), self.caches, self.table, self.lens)
        self.src = api.KVCache.alloc(sum(-(-n // page) for n in sources) + 1, hkv, d, page, kind)
        wide = max(-(-n // page) for n in sources)
        self.src_table = torch.full((self.groups, wide), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(sources):
            self.src_table[i, :-(-n // page)] = torch.arange(at, at - (-n // page))
            at -= -n // page
        self.src_table, self.src_lens = self.src_table.cuda(), i32(sources)
        self.src_cu = torch.arange(self.groups + 1, dtype=torch.int32, device="cuda") * beams
        k, v = (self.randn(sum(sources), hkv, d) for _ in "kv")
        api.cache_append(self.src, k.cuda(), v.cuda(), self.src_table, self.src_lens, cu_new=i32([0] + list(np.cumsum(sources))))
        ends = [0] + list(np.cumsum(sources))
        self.src_held = [(self.as_held(k[a:e].double()), self.as_held(v[a:e].double())) for a, e in zip(ends, ends[1:])]
        self.self_ws = api.alloc_cache_workspace(self.rows, hq, hkv, d)
        self.src_ws = api.alloc_cache_workspace(self.groups, hq, hkv, d, max_new=beams)
        self.out, self.src_out = (torch.empty((self.rows, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.lse, self.src_lse = (torch.empty((hq, self.rows), device="cuda") for _ in range(2))
        self.scores = torch.zeros((self.groups, beams), device="cuda")
        self.finished = torch.zeros((self.groups, beams), dtype=torch.uint8, device="cuda")
        self.picked = [torch.empty((self.groups, beams), device="cuda")] + \
            [torch.empty((self.groups, beams), dtype=torch.int32, device="cuda") for _ in range(2)]
        self.vocab = 5003
        self.beam_ws = api.alloc_beam_workspace(self.groups, beams, self.vocab, beams)
        self.logits = torch.empty((self.rows, self.vocab), dtype=torch.bfloat16, device="cuda")
        self.q, self.k, self.v = (torch.empty((2, self.rows, h, d), dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
        self.src_q, self.q_rot = torch.empty_like(self.out), torch.empty_like(self.q)
        self.status, self.step_no = word(), 0

    def randn(self, *s):
        return torch.randn(s, generator=self.g).bfloat16()

    def as_held(self, rows):
        rows = rows.bfloat16()
        if not self.int4 or len(rows) == 0:
            return rows.double()
        return values(*quantise(rows))

    def new_inputs(self):
        self.inputs = [self.randn(self.rows, self.vocab) * 2.5, *(self.randn(*x.shape) for x in (self.q, self.k, self.v, self.src_q))]
        for x, y in zip((self.logits, self.q, self.k, self.v, self.src_q), self.inputs):
            x.copy_(y)

    def gpu_step(self):
        """What a decoding program launches for one token of every beam."""
        s, b, t = self.picked
        api.beam_select(self.logits, self.scores, s, b, t, self.beam_ws, end_token=3, finished=self.finished,
                        out_finished=self.finished_new, status=self.status)
        api.beam_reorder(b, self.caches, self.table, self.lens, states=(self.history,), status=self.status)
        self.lens += 1
        for layer, cache in enumerate(self.caches):
            api.cache_append(cache, self.k[layer], self.v[layer], self.table, self.lens, table=self.g_angles, q=self.q[layer],
                             q_out=self.q_rot[layer], status=self.status)
        api.cache_attn(self.caches[1], self.q_rot[1], self.table, self.lens, self.out, self.lse, self.self_ws, status=self.status)
        api.cache_cross_attn(self.src, self.src_q, self.src_table, self.src_lens, self.src_out, self.src_lse, self.src_ws,
                             cu_new=self.src_cu, max_new=self.beams, status=self.status)
        self.scores.copy_(s)
        self.finished.copy_(self.finished_new)

    def check_step(self, before):
        scores, finished, history = before
        s, b, t, f, _ = ranking(self.inputs[0], scores, self.beams, finished, end=3)
        np.testing.assert_array_equal(self.picked[1].cpu().numpy(), b)
        np.testing.assert_array_equal(self.picked[2].cpu().numpy(), t)
        np.testing.assert_array_equal(self.finished.cpu().numpy(), f)
        assert np.abs(self.scores.cpu().numpy() - s).max() <= 1e-4
        up = [g * self.beams + int(b[g, j]) for g in range(self.groups) for j in range(self.beams)]
        assert torch.equal(self.history.cpu(), history[up])
        self.held = [[layer[u] for u in up] for layer in self.held]
        _, q, k, v, src_q = self.inputs
        for layer in range(2):
            for r in range(self.rows):
                old = self.held[layer][r]
                at = torch.tensor([len(old[0])])
                self.held[layer][r] = (torch.cat((old[0], self.as_held(rotate(k[layer, r:r + 1], self.angles, at, False)[0]))),
                                       torch.cat((old[1], self.as_held(v[layer, r:r + 1].double()))))
        for r in range(self.rows):
            keys, vals = self.held[1][r]
            turned = rotate(q[1, r:r + 1], self.angles, torch.tensor([len(keys) - 1]), False)[0].bfloat16().double()
            self.check_row(turned[0], keys, vals, self.out[r], self.lse[:, r])
            self.check_row(src_q[r].double(), *self.src_held[r // self.beams], self.src_out[r], self.src_lse[:, r])
        assert api.cache_status(self.status) == 0

    def check_row(self, q, k, v, out, lse):
        s = torch.einsum("hgd,lhd->hgl", q.unflatten(0, (self.hkv, -1)), k) * self.d ** -0.5
        mag = torch.einsum("hgd,lhd->hgl", q.abs().unflatten(0, (self.hkv, -1)), k.abs()) * self.d ** -0.5
        ll = torch.logsumexp(s, -1)
        w = (s - ll[..., None]).exp()
        o = torch.einsum("hgl,lhd->hgd", w, v).flatten(0, 1)
        big = torch.einsum("hgl,lhd->hgd", w, v.abs().amax(-1, keepdim=True).expand_as(v)).flatten(0, 1)
        # as in cache_util: scores in fp32, the weights and the result rounded to bf16; and a rotated query may round the
        # other way than the 64-bit one, a step of bf16 of one of its dims (2^-7 of a score's largest term)
        ds = mag.amax(-1) * (self.d + 4) * 2 * U32 * (16 if self.int4 else 1) + 2e-6 + 2.0 ** -7 * 4 * self.d ** -0.5
        e = U16 * (o.abs() + 2 * big) + 2 * ds.flatten()[:, None] * big + 1e-6 * big
        assert bool(((out.double().cpu() - o).abs() <= e).all())
        assert bool(((lse.double().cpu() - ll.flatten()).abs() <= 2 * ds.flatten() + 4 * U32 * ll.flatten().abs()).all())

    def step(self, launch):
        self.new_inputs()
        before = self.scores.cpu(), self.finished.cpu(), self.history.cpu()
        launch()
        torch.cuda.synchronize()
        self.check_step(before)
        self.history[:, self.step_no] = self.picked[2].flatten()
        self.step_no += 1


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("captured", [False, True])
def test_decoding_steps(int4, captured):
    """Two requests with four beams through 37 steps, over two page borders: tokens, histories, both attentions."""
    d = Decoder([21, 16], [70, 33], 4, int4, 16, 40, seed=1 + int4)
    d.finished_new = torch.empty_like(d.finished)
    d.step(d.gpu_step)
    if not captured:
        for _ in range(36):
            d.step(d.gpu_step)
        return
    # the step writes its own inputs (lengths, scores, tables): they are put back after the capture, which runs nothing
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.gpu_step()
    for _ in range(36):
        d.step(graph.replay)
