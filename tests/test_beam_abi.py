"""Refusals and sizes of the beam search calls: all on the host, before any device work."""
import pytest
import torch

from packed_varlen_attention_cu_gb300 import _lib, api
from test_cache_abi import A, BAD_CACHE, INVALID, L, SMALL, UNSUPPORTED, cache  # noqa: F401


def select(L, logits=A, stride=0, f32=0, groups=2, beams=3, vocab=100, k=4, scores=A, finished=None, norms=None, end=5,
           os=A, ob=A, ot=A, of=None, status=None, ws=A, n=1 << 40):
    return L.pva_beam_select(logits, stride, f32, groups, beams, vocab, k, scores, finished, norms, end, os, ob, ot, of, status,
                             ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(f32=2), INVALID), (dict(groups=-1), INVALID), (dict(beams=0), INVALID), (dict(vocab=0), INVALID), (dict(k=0), INVALID),
    (dict(beams=65), UNSUPPORTED), (dict(k=65), UNSUPPORTED), (dict(vocab=2 ** 31 - 1), UNSUPPORTED),
    (dict(groups=2 ** 31 - 1, beams=64), UNSUPPORTED), (dict(stride=99), INVALID), (dict(stride=-1), INVALID),
    (dict(finished=A, end=-1), INVALID), (dict(finished=A, end=100), INVALID), (dict(of=A, end=100), INVALID),
    (dict(logits=None), INVALID), (dict(scores=None), INVALID), (dict(os=None), INVALID), (dict(ob=None), INVALID),
    (dict(ot=None), INVALID), (dict(ws=None), INVALID), (dict(logits=A + 1), INVALID), (dict(logits=A + 2, f32=1), INVALID),
    (dict(scores=A + 2), INVALID), (dict(norms=A + 2), INVALID), (dict(os=A + 2), INVALID), (dict(ob=A + 1), INVALID),
    (dict(ot=A + 2), INVALID), (dict(status=A + 2), INVALID), (dict(ws=A + 128), INVALID), (dict(n=100), SMALL)])
def test_select_refuses(L, kw, code):
    assert select(L, **kw) == code


def test_no_group_is_nothing_to_do(L):
    assert select(L, groups=0, logits=None, scores=None, os=None, ob=None, ot=None, ws=None, n=256) == 0


def test_workspace_sizes(L):
    size = L.pva_beam_select_bytes
    for bad in ((-1, 4, 100, 4), (1, 0, 100, 4), (1, 65, 100, 4), (1, 4, 0, 4), (1, 4, 100, 0), (1, 4, 100, 65), (1, 4, 2 ** 31 - 1, 4)):
        assert size(*bad) == 0
    assert size(0, 4, 100, 4) > 0
    # one part of a short row: a sum and num_out keys
    assert size(3, 4, 100, 7) == 256 + 12 * (16 + 8 * 7)
    # never more than a join's threads hold of a group
    for groups, beams, k in ((1, 64, 64), (1, 1, 1), (1, 4, 8), (64, 8, 16), (500, 3, 6)):
        per_row = (size(groups, beams, 2 ** 20, k) - 256) // (groups * beams)
        assert per_row % (16 + 8 * k) == 0 and per_row // (16 + 8 * k) * beams * k <= 8192


@pytest.mark.parametrize("beams,k", [(1, 1), (4, 4), (4, 8), (8, 16), (5, 5), (64, 64), (3, 6), (7, 1)])
@pytest.mark.parametrize("vocab", [100, 32000, 50021, 131071, 2 ** 20, 2 ** 31 - 100])
def test_a_workspace_serves_fewer_groups_and_smaller_vocabularies(L, beams, k, vocab):
    """A batch shrinks as requests finish, and fewer rows are cut into more parts each."""
    size = L.pva_beam_select_bytes
    most = 0
    for groups in list(range(0, 700)) + [1000, 5000]:
        n = size(groups, beams, vocab, k)
        assert n >= most > -1
        most = n
    for groups in (1, 16, 600):
        assert size(groups, beams, vocab, k) >= max(size(groups, beams, v, k) for v in (1, vocab // 3 + 1, vocab // 2 + 1, vocab - 1))


def reorder(L, parents=A, groups=2, beams=3, caches=None, n=None, table=A, stride=4, width=4, lens=A, states=(), status=None):
    caches = [cache()] if caches is None else caches
    c = (_lib.CacheDesc * len(caches))(*caches) if caches else None
    s = (_lib.StateDesc * len(states))(*[_lib.StateDesc(*x) for x in states]) if states else None
    return L.pva_beam_reorder(parents, groups, beams, c, len(caches) if n is None else n, table, stride, width, lens, s, len(states),
                              status, None)


@pytest.mark.parametrize("kw,code", [
    (dict(groups=-1), INVALID), (dict(beams=0), INVALID), (dict(beams=65), UNSUPPORTED), (dict(groups=2 ** 31 - 1), UNSUPPORTED),
    (dict(n=-1), INVALID), (dict(caches=[], n=1), INVALID), (dict(parents=None), INVALID), (dict(parents=A + 2), INVALID),
    (dict(table=None), INVALID), (dict(table=A + 2), INVALID), (dict(lens=None), INVALID), (dict(lens=A + 1), INVALID),
    (dict(stride=3), INVALID), (dict(width=-1), INVALID), (dict(status=A + 2), INVALID),
    (dict(states=[(A, 8, 4)]), INVALID), (dict(states=[(A, 6, 8)]), INVALID), (dict(states=[(A, 8, 10)]), INVALID),
    (dict(states=[(A + 2, 8, 8)]), INVALID), (dict(states=[(None, 8, 8)]), INVALID), (dict(states=[(A, -4, 8)]), INVALID),
    (dict(caches=[cache(), cache(num_pages=5)]), INVALID), (dict(caches=[cache(), cache(num_kv_heads=3)]), INVALID),
    (dict(caches=[cache(), cache(page_size=32)]), INVALID), (dict(caches=[cache(), cache(head_dim=128)]), INVALID),
    (dict(caches=[cache(), cache(kind=1, k_scales=A, v_scales=A)]), INVALID)])
def test_reorder_refuses(L, kw, code):
    assert reorder(L, **kw) == code


@pytest.mark.parametrize("kw,code", BAD_CACHE)
def test_reorder_refuses_bad_caches(L, kw, code):
    assert reorder(L, caches=[cache(**kw)]) == code
    assert reorder(L, caches=[cache(), cache(**kw)]) == code


B = A + (1 << 20)


@pytest.mark.parametrize("caches,states", [
    ([cache(v_pages=A)], ()),                                               # one array for K and V
    ([cache(v_pages=B), cache(v_pages=B + 4096)], ()),                      # two layers with the same K
    ([cache(v_pages=B), cache(k_pages=B + 4096, v_pages=B)], ()),           # ... the same V
    ([cache(v_pages=B), cache(k_pages=B + 4096, v_pages=A)], ()),           # ... K of one as V of the other
    ([], [(A, 8, 8), (B, 8, 8), (A, 4, 8)]), ([], [(A, 16, 16), (A, 16, 16)])])
def test_reorder_refuses_what_would_move_twice(L, caches, states):
    assert reorder(L, caches=caches, states=states) == INVALID


C, D, E, F = (A + (n << 21) for n in range(1, 5))


def four(k=C, v=D, ks=E, vs=F):
    return cache(kind=1, k_pages=k, v_pages=v, k_scales=ks, v_scales=vs)


@pytest.mark.parametrize("kw", [
    dict(caches=[four(ks=C)]), dict(caches=[four(vs=E)]), dict(caches=[four(ks=D)]),                # inside one cache
    dict(caches=[four(), four(B, B + 4096, E, B + 8192)]), dict(caches=[four(), four(B, B + 4096, B + 8192, E)]),  # scales of another
    dict(caches=[four(), four(F, B + 4096, B + 8192, B + 12288)]),                                  # pages that are scales of another
    dict(caches=[four()], states=[(C, 8, 8)]), dict(caches=[four()], states=[(F, 8, 8)]),           # a state that is a cache's
    dict(caches=[four()], states=[(A, 8, 8)]), dict(caches=[four()], states=[(B, 8, 8)]),           # ... the parents, the lengths
    dict(caches=[four()], states=[(B + 4096, 8, 8)]), dict(caches=[], states=[(A, 8, 8)]),          # ... the table
    dict(caches=[four()], table=A), dict(caches=[four()], table=B), dict(caches=[four(k=A)]), dict(caches=[four(vs=B + 4096)])])
def test_reorder_refuses_addresses_that_are_listed_twice(L, kw):
    """Whatever they are listed as: pages, scales, states, and what the call reads (parents at A, lengths at B, table at B + 4096)."""
    assert reorder(L, **{**dict(lens=B, table=B + 4096), **kw}) == INVALID


def test_nothing_to_reorder(L):
    assert reorder(L, groups=0, parents=None, table=None, lens=None) == 0
    assert reorder(L, caches=[], parents=None, table=None, lens=None) == 0


def test_the_binding_wants_gpu_tensors():
    x = torch.zeros((2, 3))
    i = x.int()
    with pytest.raises(ValueError):
        api.beam_select(torch.zeros((6, 10)), x, x, i, i, x)
    with pytest.raises(ValueError):
        api.beam_reorder(i)
