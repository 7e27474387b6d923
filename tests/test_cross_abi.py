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


ROWS, KEYS, LSE = (30, 4, 64), (70, 2, 64), (4, 30)


def tensors(**other):
    """Everything that the attention calls take for 30 rows of 4 heads over 70 keys of 2, on the CPU."""
    t = {n: torch.zeros(ROWS, dtype=torch.bfloat16) for n in ("q", "out", "dout", "dq")}
    t |= {n: torch.zeros(KEYS, dtype=torch.bfloat16) for n in ("k", "v", "dk", "dv")}
    t |= dict(lse=torch.zeros(LSE), o_run=torch.zeros(ROWS), cu=torch.zeros(4, dtype=torch.int32), ws=torch.zeros(256, dtype=torch.uint8))
    t |= {n: torch.zeros(shape, dtype=t[n].dtype) for n, shape in other.items()}
    return t


def calls(t, kind=api.MASK_CROSS):
    m = mask(kind, 30, 70)
    m._cu_keys_keep = torch.zeros(4, dtype=torch.int32)
    p = api.make_params(4, 2, num_ctas=152)
    bufs = dict(q=t["q"], k=t["k"], v=t["v"], out=t["out"], lse=t["lse"], cu=t["cu"], worklist=t["ws"])
    return dict(
        fwd=lambda: api.attn_fwd(t["q"], t["k"], t["v"], t["cu"], m, p, t["ws"], t["out"], t["lse"], stream=0),
        acc=lambda: api.attn_fwd_accumulate(t["q"], t["k"], t["v"], t["cu"], m, p, t["ws"], t["o_run"], t["lse"], stream=0),
        bwd=lambda: api.attn_bwd(t["q"], t["k"], t["v"], t["out"], t["lse"], t["dout"], t["cu"], 3, m, p, t["ws"], t["ws"], t["dq"],
                                 t["dk"], t["dv"], stream=0),
        host=lambda: api.attn_fwd_host(t["q"], t["k"], t["v"], t["cu"], 3, m, p, t["out"], t["lse"], bufs, stream=0))


@pytest.mark.parametrize("call,name,shape", [
    (call, name, shape) for call, names in (("fwd", "q k v out lse cu"), ("acc", "q k v o_run lse cu"), ("host", "q k v out lse cu"),
                                            ("bwd", "q k v out lse dout dq dk dv cu"))
    for name in names.split()
    for shape in ([(5,), (1,)] if name == "cu" else [(4, 70), (30, 4), (2, 30)] if name == "lse" else
                  [ROWS[::-1], (70, 4, 64), (29, 4, 64)] if name in ("q", "out", "o_run", "dout", "dq") else
                  [(30, 2, 64), (70, 4, 64), (69, 2, 64), (70, 2, 128)])])
def test_tensors_that_are_not_the_masks(call, name, shape):
    """A pack of the other side, or of another batch, would be read or written past its end."""
    with pytest.raises(ValueError, match="cu_seqlens" if name == "cu" else "mask"):
        calls(tensors(**{name: shape}))[call]()
    with pytest.raises(ValueError):  # swapped
        calls(tensors(q=KEYS, k=ROWS))[call]()


@pytest.mark.parametrize("name", ["q", "k", "v", "out", "lse", "cu"])
def test_device_buffers_without_room(name):
    t = tensors()
    m, p = mask(q=30, k=70), api.make_params(4, 2, num_ctas=152)
    bufs = dict({n: t[n] for n in ("q", "k", "v", "out", "lse", "cu")}, worklist=t["ws"])
    bufs[name] = bufs[name].flatten()[1:]
    with pytest.raises(ValueError, match="room"):
        api.attn_fwd_host(t["q"], t["k"], t["v"], t["cu"], 3, m, p, t["out"], t["lse"], bufs, stream=0)


@pytest.mark.parametrize("call", ["fwd", "acc", "bwd"])
def test_tensors_that_are_the_masks(call):
    with pytest.raises(AssertionError):  # the next check: they are not on a GPU
        calls(tensors())[call]()
    with pytest.raises(AssertionError):  # other masks keep their rules
        calls(tensors(k=(30, 2, 64)), kind=api.MASK_CAUSAL)[call]()


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
