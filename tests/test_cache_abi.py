"""Refusals of the rotation and cache calls: all of them happen on the host, before
any device work, so they are tested without a GPU."""
import ctypes

import pytest
import torch

from packed_varlen_attention_cu_gb300 import _lib, api
from packed_varlen_attention_cu_gb300 import build as pva_build

INVALID, SMALL, UNSUPPORTED = 1, 2, 4
A = 4096  # an address with every alignment; never dereferenced by a refused call


@pytest.fixture(scope="module")
def L():
    pva_build.build()
    return _lib.lib()


def cache(**kw):
    f = dict(kind=0, num_kv_heads=2, head_dim=64, page_size=16, num_pages=4, k_pages=A, v_pages=A,
             k_scales=None, v_scales=None)
    f.update(kw)
    return _lib.CacheDesc(**f)


def batch(**kw):
    f = dict(num_seqs=2, num_tokens=2, max_pages=3, table_stride=3, page_table=A, kv_lens=A,
             cu_new=None, status=None)
    f.update(kw)
    return _lib.CacheBatch(**f)


def rope(**kw):
    f = dict(table=A, max_pos=10, rot_dim=64, interleaved=0)
    f.update(kw)
    return _lib.RopeDesc(**f)


BAD_CACHE = [(dict(kind=2), INVALID), (dict(kind=-1), INVALID), (dict(num_kv_heads=0), INVALID),
             (dict(head_dim=96), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
             (dict(page_size=8), UNSUPPORTED), (dict(page_size=2048), UNSUPPORTED),
             (dict(page_size=0), UNSUPPORTED), (dict(num_pages=-1), INVALID),
             (dict(num_pages=1 << 31), INVALID), (dict(k_pages=None), INVALID),
             (dict(v_pages=A + 8), INVALID), (dict(kind=1), INVALID),
             (dict(kind=1, k_scales=A, v_scales=A + 4), INVALID)]
BAD_BATCH = [(dict(num_seqs=-1), INVALID), (dict(num_tokens=-1), INVALID), (dict(max_pages=-1), INVALID),
             (dict(table_stride=2), INVALID), (dict(page_table=None), INVALID), (dict(page_table=A + 2), INVALID),
             (dict(cu_new=A + 1), INVALID), (dict(status=A + 2), INVALID),
             (dict(num_tokens=1), INVALID)]  # one row for each sequence is needed without offsets
BAD_ROPE = [(dict(rot_dim=80), INVALID), (dict(rot_dim=-16), INVALID), (dict(rot_dim=24), UNSUPPORTED),
            (dict(interleaved=2), INVALID), (dict(max_pos=-1), INVALID), (dict(table=None), INVALID),
            (dict(table=A + 8), INVALID)]


def append(L, c=None, b=None, r=None, k=A, ks=0, v=A, vs=0, q=A, qs=0, hq=4, qo=A, qos=0, ko=None, kos=0):
    return L.pva_cache_append(c or cache(), b or batch(), r or rope(), k, ks, v, vs, q, qs, hq, qo, qos, ko,
                              kos, None)


def attn(L, c=None, b=None, q=A, qs=0, hq=4, new=1, window=0, scale=0.0, out=A, f32=0, lse=A, ws=A,
         n=1 << 40):
    return L.pva_cache_attn(c or cache(), b or batch(), q, qs, hq, new, window, scale, out, f32, lse, ws, n,
                            None)


@pytest.mark.parametrize("kw,code", BAD_CACHE)
def test_bad_cache(L, kw, code):
    c = cache(**kw)
    assert append(L, c=c) == code and attn(L, c=c) == code
    assert L.pva_cache_read(c, batch(), None, A, A, None) == code


@pytest.mark.parametrize("kw,code", BAD_BATCH)
def test_bad_batch(L, kw, code):
    b = batch(**kw)
    assert append(L, b=b) == code and attn(L, b=b) == code
    assert L.pva_cache_read(cache(), b, None, A, A, None) == code


def test_lengths_are_needed_where_they_are_used(L):
    assert append(L, b=batch(kv_lens=None)) == INVALID and attn(L, b=batch(kv_lens=None)) == INVALID
    assert attn(L, b=batch(kv_lens=A + 2)) == INVALID


@pytest.mark.parametrize("kw,code", BAD_ROPE)
def test_bad_rope(L, kw, code):
    assert append(L, r=rope(**kw)) == code
    assert L.pva_rope(A, 0, A, 0, 5, 4, 2, 64, 0, rope(**kw), None, 0, None, 0, A, 0, A, 0, None, None) == code


def test_bad_append(L):
    assert append(L, q=None) == INVALID and append(L, qo=None) == INVALID and append(L, hq=0) == INVALID
    assert append(L, hq=-1) == INVALID
    assert append(L, k=None) == INVALID and append(L, v=A + 2) == INVALID and append(L, ko=A + 8) == INVALID
    for bad in (8, 127, 132):  # shorter than a row, odd, not a multiple of 16 bytes
        assert append(L, ks=bad) == INVALID and append(L, vs=bad) == INVALID
    assert append(L, qs=128) == INVALID and append(L, qos=260) == INVALID and append(L, ko=A, kos=4) == INVALID


def test_bad_rope_call(L):
    def call(q=A, k=A, t=5, hq=4, hkv=2, d=64, f32=0, r=None, cu=None, nd=0, pos=None, inv=0, qo=A, ko=A, st=None,
             qs=0):
        return L.pva_rope(q, qs, k, 0, t, hq, hkv, d, f32, r or rope(), cu, nd, pos, inv, qo, 0, ko, 0, st, None)
    assert call(t=-1) == call(hq=-1) == call(hkv=-1) == call(f32=2) == call(inv=2) == INVALID
    assert call(d=80) == UNSUPPORTED
    assert call(q=None) == call(k=None) == call(qo=None) == call(ko=None) == call(q=A + 8) == INVALID
    assert call(cu=A, nd=1, pos=A) == INVALID and call(nd=-1) == INVALID and call(pos=A + 2) == INVALID
    assert call(qs=100) == INVALID and call(qs=260) == INVALID
    assert L.pva_rope(A, 0, A, 0, 5, 4, 2, 64, 0, None, None, 0, None, 0, A, 0, A, 0, None, None) == INVALID
    # nothing to do is done without a device
    assert call(t=0) == 0 and call(hq=0, hkv=0, q=None, k=None, qo=None, ko=None) == 0


def test_bad_read(L):
    assert L.pva_cache_read(cache(), batch(), None, None, A, None) == INVALID
    assert L.pva_cache_read(cache(), batch(), None, A, A + 8, None) == INVALID
    assert L.pva_cache_read(cache(), batch(), A + 1, A, A, None) == INVALID
    assert L.pva_cache_read(cache(num_kv_heads=353), batch(), None, A, A, None) == UNSUPPORTED
    assert L.pva_cache_read(cache(num_kv_heads=177, head_dim=128), batch(), None, A, A, None) == UNSUPPORTED


def test_bad_attention(L):
    assert attn(L, hq=3) == attn(L, hq=0) == attn(L, new=0) == attn(L, window=-1) == attn(L, f32=2) == INVALID
    assert attn(L, scale=float("nan")) == attn(L, scale=float("inf")) == INVALID
    assert attn(L, c=cache(page_size=1024, head_dim=128, num_kv_heads=8192), hq=8192) == UNSUPPORTED  # 2 GB a page
    assert attn(L, q=None) == attn(L, out=None) == attn(L, lse=None) == attn(L, ws=None) == INVALID
    assert attn(L, q=A + 2) == attn(L, out=A + 8) == attn(L, lse=A + 2) == attn(L, ws=A + 16) == INVALID
    assert attn(L, qs=100) == attn(L, qs=260) == INVALID
    assert attn(L, n=16) == SMALL


def test_nothing_to_do(L):
    for b in (batch(num_seqs=0), batch(num_tokens=0, cu_new=A)):
        assert append(L, b=b) == 0 and attn(L, b=b) == 0
        assert L.pva_cache_read(cache(), b, None, A, A, None) == 0


def test_workspace_bytes(L):
    assert api.cache_attn_bytes(1, 4, 2, 64) > 0
    assert api.cache_attn_bytes(0, 4, 2, 64) > 0
    for bad in ((-1, 4, 2, 64, 1), (1, 0, 2, 64, 1), (1, 4, 3, 64, 1), (1, 4, 2, 80, 1), (1, 4, 2, 64, 0)):
        assert L.pva_cache_attn_bytes(*bad) == 0
        with pytest.raises(_lib.PvaError):
            api.cache_attn_bytes(*bad)


def test_status_word_is_needed(L):
    code = ctypes.c_int32(0)
    assert L.pva_cache_status(None, ctypes.byref(code), None) == INVALID
    assert L.pva_cache_status(A, None, None) == INVALID
    assert L.pva_cache_status(A + 2, ctypes.byref(code), None) == INVALID


def test_binding_refuses_host_tensors_and_wrong_shapes():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        api.KVCache(k, k)
    with pytest.raises(ValueError, match="bf16 or uint8"):
        api.KVCache(k.float(), k.float())
    with pytest.raises(ValueError, match="scales"):
        api.KVCache(k.view(torch.uint8), k.view(torch.uint8))
    with pytest.raises(ValueError, match="kind"):
        api.KVCache.alloc(4, 2, 64, kind=2, device="cpu")
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    table = api.rope_table(8, 64, device="cpu")
    with pytest.raises(ValueError):
        api.rope(x, None, table, x, None)
    with pytest.raises(ValueError):
        api.rope(x.half(), None, table, x.half(), None)
    with pytest.raises(ValueError):
        api.rope(x, None, table, None, None)


def test_rope_table_is_computed_in_64_bits():
    t = api.rope_table(200001, 32, base=5e5, device="cpu")
    assert t.shape == (200001, 16, 2) and t.dtype == torch.float32
    import math
    for p in (0, 1, 7, 15):
        a = 200000 * 5e5 ** (-2 * p / 32)
        assert abs(float(t[200000, p, 0]) - math.cos(a)) <= 2 ** -24 + 1e-9
        assert abs(float(t[200000, p, 1]) - math.sin(a)) <= 2 ** -24 + 1e-9
    mine = api.rope_table(5, 4, inv_freq=torch.tensor([0.5, 0.25], dtype=torch.float64), device="cpu")
    assert abs(float(mine[3, 1, 1]) - math.sin(0.75)) <= 2 ** -24
