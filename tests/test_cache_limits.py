"""Ends of the rotation and cache calls' ranges that need no GPU: refusals, calls with nothing to do, and that
the attention's error bounds notice what they are there for."""
import pytest
import torch

import cache_bounds
from cache_util import Problem
from packed_varlen_attention_cu_gb300 import api
from test_cache_abi import A, INVALID, UNSUPPORTED, L, append, attn, batch, cache, rope  # noqa: F401


@pytest.mark.parametrize("kind,most,over", [(0, 2e38, 3e38), (1, 3.9e17, 4.1e17)])
def test_scales_past_the_kernels_numbers_are_refused(L, kind, most, over):  # noqa: F811
    """The scale goes in times log2(e), with 4 bits times 2^69 as well; every smaller one is taken."""
    c = cache(kind=kind, k_scales=A, v_scales=A)
    empty = batch(num_tokens=0, cu_new=A)  # nothing to do: returns behind the checks
    assert attn(L, c=c, b=empty, scale=over) == INVALID
    for scale in (most, 1.0, 1e-30, 1e-38, 1e-45):
        assert attn(L, c=c, b=empty, scale=scale) == 0


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_bounds_notice_lost_keys_and_coarse_weights(int4, d):
    p = Problem([5000, 300], [1, 2], 4, 2, d, 16, int4)
    ref = cache_bounds.attend(p)
    cache_bounds.check(ref[0].float(), ref[1].float(), ref)
    with pytest.raises(AssertionError):
        cache_bounds.check(torch.zeros_like(ref[0]), ref[1], ref)
    for at in ((0, 0), (0, 2496), (0, 4984), (1, 160)):
        lost = cache_bounds.attend(p, drop=at)
        with pytest.raises(AssertionError, match="row"):
            cache_bounds.check(lost[0], ref[1], ref)
        with pytest.raises(AssertionError, match="lse"):
            cache_bounds.check(ref[0], lost[1], ref)
    with pytest.raises(AssertionError, match="row"):
        cache_bounds.check(ref[0].bfloat16(), ref[1], ref)
    if int4:
        with pytest.raises(AssertionError, match="row"):
            cache_bounds.check(cache_bounds.attend(p, eight=True)[0], ref[1], ref)


def test_an_empty_batch_needs_no_pointers(L):  # noqa: F811
    """Empty tensors have no address: no new tokens, with or without queries, is nothing to do."""
    for b in (batch(num_tokens=0, cu_new=A), batch(num_tokens=0), batch(num_seqs=0)):
        assert append(L, b=b, k=None, v=None, q=None, hq=4, qo=None) == 0
        assert append(L, b=b, k=None, v=None, q=None, hq=0, qo=None) == 0
        assert append(L, b=b, hq=-1) == INVALID
        assert attn(L, b=b, q=None, out=None, lse=None, ws=None) == 0


def test_head_counts_past_the_grid_are_refused(L):  # noqa: F811
    """Counts whose sum leaves 32 bits, or that fill more blocks than a grid has."""
    top = 2 ** 31 - 1

    def turn(hq, hkv):
        return L.pva_rope(A, 0, A, 0, 5, hq, hkv, 64, 0, rope(), None, 0, None, 0, A, 0, A, 0, None, None)
    assert turn(top, top) == turn(top, 1) == turn(2 ** 30, 2 ** 30) == turn(top, 0) == turn(0, top) == UNSUPPORTED
    for hq, hkv in ((top, 2), (4, 2 ** 30), (top, 2 ** 30), (4, top), (2, 2 ** 30 - 1)):
        assert append(L, c=cache(num_kv_heads=hkv), hq=hq) == UNSUPPORTED
    assert append(L, c=cache(num_kv_heads=top), q=None, hq=0, qo=None) == UNSUPPORTED


def test_the_binding_needs_no_private_function_of_torch(monkeypatch):
    """The stream's handle comes from a private function of torch where there is one, else from the Stream."""
    class Stream:
        cuda_stream = 0x1234
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream)
    monkeypatch.setattr(api, "_raw_stream", None)
    assert api._queue(None, 0) == 0x1234 and api._queue(Stream, 0) == 0x1234 and api._queue(7, 0) == 7
    monkeypatch.setattr(api, "_raw_stream", lambda dev: 0x5678 + dev)
    assert api._queue(None, 1) == 0x5679 and api._queue(Stream, 1) == 0x1234 and api._queue(0, 1) == 0
