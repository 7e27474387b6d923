"""Refusals and sizes of cross attention (the CROSS mask and the call over the cache),
which happen on the host before any device work."""
import ctypes

import pytest
import torch

from packed_varlen_attention_cu_gb300 import _lib, api
from test_cache_abi import A, BAD_BATCH, BAD_CACHE, INVALID, L, SMALL, batch, cache  # noqa: F401


def mask(kind=api.MASK_CROSS, q=100, k=200, keys=A):
    m = _lib.MaskDesc()
    m.kind, m.q_tokens, m.k_tokens, m.cu_keys = kind, q, k, keys
    return m


def test_cross_mask_needs_aligned_offsets_of_the_keys(L):
    p = api.make_params(4, 2, num_ctas=152, pack_docs=1)

    def size(m):
        return L.pva_worklist_bytes(7, ctypes.byref(m), ctypes.byref(p))

    assert size(mask()) > 0
    for bad in (mask(keys=None), mask(keys=A + 2), mask(q=-1), mask(k=-1)):
        assert size(bad) == 0
        assert L.pva_bwd_plan_bytes(7, ctypes.byref(bad), ctypes.byref(p)) == 0
        assert L.pva_build_worklist(A, 7, ctypes.byref(bad), ctypes.byref(p), A, 1 << 40, None) == INVALID
    # other kinds do not look at the field
    assert size(mask(kind=api.MASK_CAUSAL, k=100, keys=A + 2)) > 0
    # without offsets of the targets there is nothing to build
    assert L.pva_build_worklist(None, 7, ctypes.byref(mask()), ctypes.byref(p), A, 1 << 40, None) == INVALID
    # the shared tiles of short pairs need room for their intervals
    q = api.make_params(4, 2, num_ctas=152)
    m = mask()
    assert size(m) - L.pva_worklist_bytes(7, ctypes.byref(m), ctypes.byref(q)) >= 7 * (512 - 16) - 256


def test_cross_backward_refusals(L):
    p = api.make_params(4, 2, num_ctas=152)

    def bwd(m, q=A, k=A, v=A, out=A, dq=A, dk=A, dv=A, d=64):
        return L.pva_attn_bwd(q, k, v, out, A, A, A, 7, ctypes.byref(m), ctypes.byref(p), d, A, A, dq, dk, dv, 0, 0.0, None)

    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(dq=None), dict(dk=None), dict(dv=None),
               dict(dk=A + 8)):
        assert bwd(mask(), **kw) == INVALID
    assert bwd(mask(), d=96) == 4
    # other kinds keep their rule: every tensor is there
    causal = mask(kind=api.MASK_CAUSAL, q=0, k=0)
    assert bwd(causal, q=None) == INVALID and bwd(causal, dk=None) == INVALID


def test_more_documents_than_a_backward_plan_holds(L):
    p = api.make_params(4, 2, num_ctas=152)
    m = mask(q=20000, k=20000)
    assert L.pva_bwd_plan_bytes(8192, ctypes.byref(m), ctypes.byref(p)) > 0
    assert L.pva_bwd_plan_bytes(8193, ctypes.byref(m), ctypes.byref(p)) == 0


def test_make_mask_wants_the_offsets_on_the_device():
    with pytest.raises(ValueError):
        api.make_mask(api.MASK_CROSS, 10, 10)
    with pytest.raises(ValueError):
        api.make_mask(api.MASK_CROSS, 10, 10, cu_keys=torch.tensor([0, 10], dtype=torch.int32))


def cross(L, c=None, b=None, q=A, qs=0, hq=4, new=1, scale=0.0, out=A, f32=0, lse=A, ws=A, n=1 << 40):
    return L.pva_cache_cross_attn(c or cache(), b or batch(), q, qs, hq, new, scale, out, f32, lse, ws, n, None)


@pytest.mark.parametrize("kw,code", BAD_CACHE)
def test_bad_cache(L, kw, code):
    assert cross(L, c=cache(**kw)) == code


@pytest.mark.parametrize("kw,code", BAD_BATCH)
def test_bad_batch(L, kw, code):
    assert cross(L, b=batch(**kw)) == code


@pytest.mark.parametrize("kw,code", [(dict(hq=3), INVALID), (dict(hq=0), INVALID), (dict(new=0), INVALID), (dict(f32=2), INVALID),
                                     (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(lse=None), INVALID),
                                     (dict(ws=None), INVALID), (dict(ws=A + 128), INVALID), (dict(q=A + 8), INVALID),
                                     (dict(qs=4 * 64 - 8), INVALID), (dict(qs=4 * 64 + 4), INVALID), (dict(n=100), SMALL),
                                     (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID)])
def test_bad_call(L, kw, code):
    assert cross(L, **kw) == code


def test_nothing_to_do(L):
    assert cross(L, b=batch(num_seqs=0), q=None, out=None, lse=None, ws=None) == 0
    assert cross(L, b=batch(num_tokens=0), q=None, out=None, lse=None, ws=None) == 0
