"""Thin Python binding of the C ABI (include/pva.h).

Argument marshalling only: tensors are passed by ``data_ptr()`` and the
current CUDA stream; every step of the computation runs in the library's
kernels.  PyTorch supplies device memory and streams.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional, Sequence

import numpy as np
import torch

from . import _lib
from ._lib import CacheBatch, MaskDesc, RopeDesc, Slice, WorklistParams, check, lib
from .workloads import (MASK_CAUSAL, MASK_CROSS, MASK_SHARED_QUESTION, MASK_SLICES, MASK_SLIDING_WINDOW,
                        MASK_ZIGZAG_PAIR, MASK_ZIGZAG_STEP)

SLICE_FULL, SLICE_CAUSAL, SLICE_INV_CAUSAL, SLICE_BI_CAUSAL = 0, 1, 2, 3
TILE = 128


# The current stream's handle without making a Stream object (2.5 us less a call), in the
# versions of torch that have this function.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if _raw_stream is None else \
            _raw_stream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def make_mask(kind: int = MASK_CAUSAL, q_tokens: int = 0, k_tokens: int = 0, window: int = 0,
              num_prefix_docs: int = 0, cp: int = 0, q_rank: int = 0, k_rank: int = 0,
              slices: Optional[np.ndarray] = None, ring_step: int = 0,
              cu_keys: Optional[torch.Tensor] = None) -> MaskDesc:
    """pva_mask_desc.  ``slices``: int32 [n, 8] rows (q_row0, q_len, q_pos0, k_row0, k_len,
    k_pos0, type, window); the array is kept alive on the returned object.  ``cu_keys``:
    offsets of the sources (MASK_CROSS; int32 [docs + 1] on the device, kept alive too)."""
    m = MaskDesc()
    m.kind, m.window, m.num_prefix_docs = kind, window, num_prefix_docs
    m.cp, m.q_rank, m.k_rank = cp, q_rank, k_rank
    m.ring_step = ring_step
    m.q_tokens, m.k_tokens = q_tokens, k_tokens
    if slices is not None:
        arr = np.ascontiguousarray(slices, dtype=np.int32).reshape(-1, 8)
        m._slices_keep = arr
        m.slices = arr.ctypes.data_as(ctypes.POINTER(Slice))
        m.num_slices = arr.shape[0]
    if cu_keys is not None:
        if kind != MASK_CROSS or cu_keys.dtype != torch.int32 or not cu_keys.is_cuda or \
                cu_keys.dim() != 1 or not cu_keys.is_contiguous():
            raise ValueError("cu_keys: a contiguous int32 CUDA tensor [docs + 1], for MASK_CROSS")
        m._cu_keys_keep = cu_keys
        m.cu_keys = cu_keys.data_ptr()
    elif kind == MASK_CROSS:
        raise ValueError("MASK_CROSS needs cu_keys")
    return m


DISPATCH_DYNAMIC, DISPATCH_STATIC = 0, 1  # pva_dispatch

# Kernels one pva_build_worklist launches: plan, units, then for static
# dispatch chunk sort + merge rank (LPT order), LPT, chunk sort + merge rank
# (per-CTA order); for dynamic dispatch chunk sort + merge rank (dispatch order).
def worklist_build_kernels(params) -> int:
    return 4 if params.dispatch == DISPATCH_DYNAMIC else 7


def default_c_tile(head_dim: int) -> int:
    """Per-tile fixed cost (pair units) that balanced CTA busy time best on GB300:
    a computed 128 x 128 tile costs about its 16384 pairs of MMA work plus a
    softmax/hand-off term that does not shrink with the head dimension, so the
    fixed term doubles when d halves (32768 at d = 128, 65536 at d = 64)."""
    return 32768 * 128 // int(head_dim)


def make_params(num_q_heads: int, num_kv_heads: int, num_ctas: int = 0, c_tile: int = 0,
                tile_m: int = TILE, tile_n: int = TILE, refine_iters: int = 0,
                dispatch: int = DISPATCH_DYNAMIC, pack_docs: int = 0) -> WorklistParams:
    """pva_worklist_params.  pack_docs = 1: short documents share tiles."""
    p = WorklistParams()
    p.refine_iters = refine_iters
    p.dispatch = dispatch
    p.pack_docs = pack_docs
    p.tile_m, p.tile_n = tile_m, tile_n
    p.num_q_heads, p.num_kv_heads = num_q_heads, num_kv_heads
    p.num_ctas, p.c_tile = num_ctas, c_tile
    return p


def worklist_bytes(num_docs: int, mask: MaskDesc, params: WorklistParams) -> int:
    n = lib().pva_worklist_bytes(num_docs, ctypes.byref(mask), ctypes.byref(params))
    if n == 0:
        raise _lib.PvaError("pva_worklist_bytes", 1)
    return int(n)


def alloc_worklist(num_docs: int, mask: MaskDesc, params: WorklistParams,
                   device="cuda") -> torch.Tensor:
    """Caller-owned device buffer for the worklist (256-byte aligned by the allocator)."""
    return torch.empty(worklist_bytes(num_docs, mask, params), dtype=torch.uint8, device=device)


def build_worklist(cu_seqlens: Optional[torch.Tensor], mask: MaskDesc, params: WorklistParams,
                   worklist: torch.Tensor, stream=None) -> None:
    nd = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    if cu_seqlens is not None:
        assert cu_seqlens.dtype == torch.int32 and cu_seqlens.is_cuda
    if mask.kind == MASK_CROSS:
        keys = mask._cu_keys_keep
        if cu_seqlens is None or keys.numel() != nd + 1 or keys.device != cu_seqlens.device:
            raise ValueError("build_worklist: cu_seqlens and cu_keys on one device, of docs + 1 entries each")
    check("pva_build_worklist", lib().pva_build_worklist(
        _ptr(cu_seqlens), nd, ctypes.byref(mask), ctypes.byref(params), _ptr(worklist),
        worklist.numel(), _stream(stream)))


def _cross_sizes(mask: MaskDesc, params: WorklistParams, cu_seqlens, rows: dict, keys: dict, lse) -> None:
    """Under a CROSS mask targets and sources have lengths of their own: the tensors of either side are
    compared with the mask's (the library sees addresses only)."""
    if mask.kind != MASK_CROSS:
        return
    d = rows["q"].shape[-1]
    for names, shape in ((rows, (mask.q_tokens, params.num_q_heads, d)), (keys, (mask.k_tokens, params.num_kv_heads, d)),
                         (lse, (params.num_q_heads, mask.q_tokens))):
        for name, t in names.items():
            if t.shape != shape:
                raise ValueError(f"{name}: {tuple(t.shape)}, the mask and the head counts ask for {shape}")
    offsets = getattr(mask, "_cu_keys_keep", None)
    if cu_seqlens is None or (offsets is not None and offsets.numel() != cu_seqlens.numel()):
        raise ValueError("cu_seqlens: one entry for each of the mask's cu_keys")


def attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
             cu_seqlens: Optional[torch.Tensor], mask: MaskDesc, params: WorklistParams,
             worklist: torch.Tensor, out: torch.Tensor, lse: torch.Tensor,
             softmax_scale: float = 0.0, cta_busy: Optional[torch.Tensor] = None,
             stream=None) -> None:
    """out [Tq, Hq, d] bf16 or fp32, lse [Hq, Tq] fp32 (written by the kernel)."""
    _cross_sizes(mask, params, cu_seqlens, {"q": q, "out": out}, {"k": k, "v": v}, {"lse": lse})
    for t in (q, k, v, out, lse):
        assert t.is_cuda and t.is_contiguous()
    assert q.dtype == k.dtype == v.dtype == torch.bfloat16
    assert lse.dtype == torch.float32 and out.dtype in (torch.bfloat16, torch.float32)
    check("pva_attn_fwd", lib().pva_attn_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), ctypes.byref(mask), ctypes.byref(params),
        q.shape[-1], _ptr(worklist), _ptr(out), 1 if out.dtype == torch.float32 else 0,
        _ptr(lse), float(softmax_scale), _ptr(cta_busy), _stream(stream)))


def attn_fwd_host(q_host: torch.Tensor, k_host: torch.Tensor, v_host: torch.Tensor,
                  cu_host: Optional[torch.Tensor], num_docs: int, mask: MaskDesc,
                  params: WorklistParams, out_host: torch.Tensor, lse_host: torch.Tensor,
                  dev_bufs: dict, softmax_scale: float = 0.0, stream=None) -> None:
    """pva_attn_fwd_host: copies in, worklist, attention and copies out on one
    stream.  Host tensors (pinned for asynchronous copies) hold the inputs and
    receive O and LSE; dev_bufs holds the device buffers "q", "k", "v", "cu",
    "worklist", "out", "lse" (see alloc_host_path_buffers)."""
    _cross_sizes(mask, params, cu_host, {"q": q_host, "out": out_host}, {"k": k_host, "v": v_host}, {"lse": lse_host})
    if mask.kind == MASK_CROSS:
        for name, t in (("q", q_host), ("k", k_host), ("v", v_host), ("out", out_host), ("lse", lse_host), ("cu", cu_host)):
            if dev_bufs[name].numel() < t.numel():
                raise ValueError(f"dev_bufs: {name} has less room than the mask's tensor")
    for t in (q_host, k_host, v_host, out_host, lse_host):
        assert not t.is_cuda and t.is_contiguous()
    wl = dev_bufs["worklist"]
    check("pva_attn_fwd_host", lib().pva_attn_fwd_host(
        _ptr(q_host), _ptr(k_host), _ptr(v_host), _ptr(cu_host), num_docs, ctypes.byref(mask),
        ctypes.byref(params), q_host.shape[-1], _ptr(out_host), _ptr(lse_host),
        float(softmax_scale), _ptr(dev_bufs["q"]), _ptr(dev_bufs["k"]), _ptr(dev_bufs["v"]),
        _ptr(dev_bufs["cu"]), _ptr(wl), wl.numel(), _ptr(dev_bufs["out"]), _ptr(dev_bufs["lse"]),
        _stream(stream)))


def alloc_host_path_buffers(q_host: torch.Tensor, k_host: torch.Tensor, num_docs: int,
                            mask: MaskDesc, params: WorklistParams, device=None) -> dict:
    """Device buffers for attn_fwd_host with the shapes of q_host / k_host."""
    dev = device or torch.device("cuda")
    tq, hq, d = q_host.shape
    return {"q": torch.empty(q_host.shape, dtype=torch.bfloat16, device=dev),
            "k": torch.empty(k_host.shape, dtype=torch.bfloat16, device=dev),
            "v": torch.empty(k_host.shape, dtype=torch.bfloat16, device=dev),
            "cu": torch.empty((num_docs + 1,), dtype=torch.int32, device=dev),
            "worklist": alloc_worklist(num_docs, mask, params, dev),
            "out": torch.empty((tq, hq, d), dtype=torch.bfloat16, device=dev),
            "lse": torch.empty((hq, tq), dtype=torch.float32, device=dev)}


def attn_fwd_accumulate(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                        cu_seqlens: Optional[torch.Tensor], mask: MaskDesc,
                        params: WorklistParams, worklist: torch.Tensor, o_run: torch.Tensor,
                        lse_run: torch.Tensor, softmax_scale: float = 0.0,
                        cta_busy: Optional[torch.Tensor] = None, stream=None) -> None:
    """Fused ring step: merge this call's attention into the running fp32
    o_run [Tq, Hq, d] and lse_run [Hq, Tq] in place (start with lse_run = -inf)."""
    _cross_sizes(mask, params, cu_seqlens, {"q": q, "o_run": o_run}, {"k": k, "v": v}, {"lse_run": lse_run})
    for t in (q, k, v, o_run, lse_run):
        assert t.is_cuda and t.is_contiguous()
    assert q.dtype == k.dtype == v.dtype == torch.bfloat16
    assert o_run.dtype == lse_run.dtype == torch.float32
    check("pva_attn_fwd_accumulate", lib().pva_attn_fwd_accumulate(
        _ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), ctypes.byref(mask), ctypes.byref(params),
        q.shape[-1], _ptr(worklist), _ptr(o_run), _ptr(lse_run), float(softmax_scale),
        _ptr(cta_busy), _stream(stream)))


def zigzag_shard_len(cu_seqlens_host: np.ndarray, cp: int, rank: int) -> int:
    cu = np.ascontiguousarray(cu_seqlens_host, dtype=np.int32)
    n = lib().pva_zigzag_shard_len(cu.ctypes.data_as(ctypes.c_void_p), cu.shape[0] - 1, cp, rank)
    if n < 0:
        raise _lib.PvaError("pva_zigzag_shard_len", 1)
    return int(n)


def zigzag_shard(cu_seqlens: torch.Tensor, cp: int, rank: int, gather_map: torch.Tensor,
                 chunk_table: Optional[torch.Tensor] = None, stream=None) -> None:
    check("pva_zigzag_shard", lib().pva_zigzag_shard(
        _ptr(cu_seqlens), cu_seqlens.numel() - 1, cp, rank, _ptr(gather_map), _ptr(chunk_table),
        _stream(stream)))


def zigzag_ring_map(cu_seqlens: torch.Tensor, cp: int, ring_map: torch.Tensor,
                    stream=None) -> None:
    """Ring order of all cp zigzag shards (pva_zigzag_ring_map) into ring_map [T] int32."""
    check("pva_zigzag_ring_map", lib().pva_zigzag_ring_map(
        _ptr(cu_seqlens), cu_seqlens.numel() - 1, cp, _ptr(ring_map), _stream(stream)))


def gather_rows(src: torch.Tensor, index_map: torch.Tensor, dst: torch.Tensor,
                scatter: bool = False, stream=None) -> None:
    """dst[i] = src[map[i]] (or dst[map[i]] = src[i]) over the first dimension."""
    rows = index_map.numel()
    # the library sees raw pointers: the map's own side must hold `rows` rows
    if (src if scatter else dst).shape[0] < rows:
        raise ValueError("gather_rows: the map has more entries than the tensor it fills has rows")
    row_bytes = src[0].numel() * src.element_size()
    indexed = dst.shape[0] if scatter else src.shape[0]
    check("pva_gather_rows", lib().pva_gather_rows(
        _ptr(src), _ptr(index_map), _ptr(dst), rows, row_bytes, indexed, 1 if scatter else 0,
        _stream(stream)))


def merge_partials(o_a: torch.Tensor, lse_a: torch.Tensor, o_b: torch.Tensor,
                   lse_b: torch.Tensor, out: torch.Tensor, lse_out: torch.Tensor,
                   stream=None) -> None:
    tokens, heads, d = o_a.shape
    check("pva_merge_partials", lib().pva_merge_partials(
        _ptr(o_a), _ptr(lse_a), _ptr(o_b), _ptr(lse_b), _ptr(out), _ptr(lse_out), tokens, heads,
        d, 1 if o_a.dtype == torch.float32 else 0, _stream(stream)))


def worklist_error(worklist: torch.Tensor, stream=None) -> int:
    code = ctypes.c_int32(0)
    check("pva_worklist_error", lib().pva_worklist_error(_ptr(worklist), ctypes.byref(code),
                                                         _stream(stream)))
    return int(code.value)


def fit_tile_cost(worklists: Sequence[torch.Tensor], cta_busy: Sequence[torch.Tensor],
                  stream=None):
    """Per-tile cost fitted to the per-CTA times of several runs (one worklist and
    one busy-stamp tensor per run): (c_tile, (a ns per pair, c ns per tile))."""
    n = len(worklists)
    assert n == len(cta_busy) and n > 0
    wl = (ctypes.c_void_p * n)(*[w.data_ptr() for w in worklists])
    bz = (ctypes.c_void_p * n)(*[b.data_ptr() for b in cta_busy])
    ct = ctypes.c_int64(0)
    coef = (ctypes.c_double * 2)()
    check("pva_fit_tile_cost", lib().pva_fit_tile_cost(wl, bz, n, ctypes.byref(ct), coef,
                                                       _stream(stream)))
    return int(ct.value), (coef[0], coef[1])


def worklist_refine_rounds(worklist: torch.Tensor) -> int:
    """Move/swap rounds the worklist build applied after LPT (header field)."""
    off = _HDR.itemsize + 8  # after lpt_steps and refine_iters
    return int(np.frombuffer(worklist[off:off + 4].cpu().numpy().tobytes(), dtype="<i4")[0])


# ------------------------------------------------------ backward
def bwd_plan_bytes(num_docs: int, mask: MaskDesc, params: WorklistParams) -> int:
    n = lib().pva_bwd_plan_bytes(num_docs, ctypes.byref(mask), ctypes.byref(params))
    if n == 0:
        raise _lib.PvaError("pva_bwd_plan_bytes", 4)
    return int(n)


def alloc_bwd_plan(num_docs: int, mask: MaskDesc, params: WorklistParams,
                   device="cuda") -> torch.Tensor:
    return torch.empty(bwd_plan_bytes(num_docs, mask, params), dtype=torch.uint8, device=device)


def build_bwd_plan(worklist: torch.Tensor, num_docs: int, mask: MaskDesc,
                   params: WorklistParams, plan: torch.Tensor, stream=None) -> None:
    check("pva_build_bwd_plan", lib().pva_build_bwd_plan(
        _ptr(worklist), num_docs, ctypes.byref(mask), ctypes.byref(params), _ptr(plan),
        plan.numel(), _stream(stream)))


def attn_bwd(q, k, v, out, lse, dout, cu_seqlens: Optional[torch.Tensor], num_docs: int,
             mask: MaskDesc, params: WorklistParams, worklist: torch.Tensor, plan: torch.Tensor,
             dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor, softmax_scale: float = 0.0,
             stream=None) -> None:
    """Gradients into dq [Tq, Hq, d], dk/dv [Tk, Hkv, d] (all bf16 or all fp32)."""
    _cross_sizes(mask, params, cu_seqlens, {"q": q, "out": out, "dout": dout, "dq": dq},
                 {"k": k, "v": v, "dk": dk, "dv": dv}, {"lse": lse})
    for t in (q, k, v, out, lse, dout, dq, dk, dv):
        assert t.is_cuda and t.is_contiguous()
    assert dq.dtype == dk.dtype == dv.dtype and dq.dtype in (torch.bfloat16, torch.float32)
    check("pva_attn_bwd", lib().pva_attn_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(cu_seqlens), num_docs,
        ctypes.byref(mask), ctypes.byref(params), q.shape[-1], _ptr(worklist), _ptr(plan),
        _ptr(dq), _ptr(dk), _ptr(dv), 1 if dq.dtype == torch.float32 else 0,
        float(softmax_scale), _stream(stream)))


# ------------------------------------------------------ positions and the key/value cache
CACHE_BF16, CACHE_INT4 = 0, 1  # pva_cache_kind
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


# A decoding step is a few microseconds of GPU work for each call, so the checks below
# ask a tensor as few questions as they can and format a message only to raise it.
def _device(t: torch.Tensor, name: str) -> int:
    """The current device, which the call's first tensor must live on."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: a CUDA tensor is needed")
    current = torch.cuda.current_device()
    if dev != current:
        raise ValueError(f"{name}: tensor on cuda:{dev}, current device is cuda:{current}")
    return dev


def _queue(stream, dev: int) -> int:
    return _stream(stream) if stream is not None or _raw_stream is None else _raw_stream(dev)


def _rows3(t: torch.Tensor, name: str, dev: int, dtype=_BF16) -> int:
    """Token stride of a [tokens, heads, head_dim] tensor whose heads and dims are contiguous."""
    if t.dtype is not dtype or t.get_device() != dev or t.dim() != 3:
        raise ValueError(f"{name}: a {dtype} tensor [tokens, heads, head_dim] on cuda:{dev} is needed")
    if t.is_contiguous():
        return 0
    (n, h, d), (st, sh, sd) = t.shape, t.stride()
    if (sd != 1 and d != 1) or (sh != d and h != 1) or (st < h * d and n > 1):
        raise ValueError(f"{name}: heads and dims must be contiguous and rows must not overlap")
    return st if n > 1 else 0


def _whole(t: torch.Tensor, name: str, dev: int, shape, *dtypes) -> int:
    if t.dtype not in dtypes or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor {list(shape)} of {dtypes} on cuda:{dev} is needed")
    return t.data_ptr()


def _ints(t: Optional[torch.Tensor], n: int, name: str, dev: int) -> Optional[int]:
    """Pointer of a contiguous int32 vector of at least n entries (None stays None)."""
    if t is None:
        return None
    if t.dtype is not _I32 or t.get_device() != dev or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous int32 tensor of at least {n} entries on cuda:{dev} is needed")
    return t.data_ptr()


def _need(ok, what: str) -> None:
    if not ok:
        raise ValueError(what)


def rope_table(max_pos: int, rot_dim: int, base: float = 10000.0, device="cuda",
               inv_freq: Optional[torch.Tensor] = None) -> torch.Tensor:
    """(cos, sin) of position t and pair p, fp32 [max_pos, rot_dim / 2, 2]: angle
    t * base^(-2 p / rot_dim), or t * inv_freq[p] (float64 [rot_dim / 2]); computed in 64 bits."""
    if inv_freq is None:
        inv_freq = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    a = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * \
        inv_freq.to(device=device, dtype=torch.float64)
    return torch.stack((a.cos(), a.sin()), -1).float()


def _rope_desc(table: Optional[torch.Tensor], interleaved: bool, dev: int) -> Optional[RopeDesc]:
    if table is None:
        return None
    if table.dtype is not _F32 or table.get_device() != dev or table.dim() != 3 or not table.is_contiguous():
        raise ValueError(f"table: a contiguous fp32 tensor [max_pos, rot_dim / 2, 2] on cuda:{dev} is needed")
    n, pairs, two = table.shape
    if two != 2:
        raise ValueError("table: fp32 [max_pos, rot_dim / 2, 2]")
    return RopeDesc(table.data_ptr(), n, 2 * pairs, 1 if interleaved else 0)


def rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], table: torch.Tensor,
         q_out: Optional[torch.Tensor], k_out: Optional[torch.Tensor],
         cu_seqlens: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
         interleaved: bool = False, inverse: bool = False,
         status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Rotate a pack's queries and keys ([tokens, heads, head_dim], bf16 or fp32) by
    their positions: inside the documents of cu_seqlens, or `positions` (int32
    [tokens], e.g. of a zigzag shard).  inverse: turn back (the gradient).
    q or k may be None; q_out is q (in place) is allowed."""
    x = q if q is not None else k
    _need(x is not None and (q is None) == (q_out is None) and (k is None) == (k_out is None),
          "rope: queries or keys, each with its output")
    kind = x.dtype
    _need(kind is _BF16 or kind is _F32, "rope: bf16 or fp32")
    _need(cu_seqlens is None or positions is None, "rope: cu_seqlens or positions, not both")
    dev = _device(x, "rope")
    _need(x.dim() == 3, "rope: [tokens, heads, head_dim]")
    t, _, d = x.shape
    hq = hkv = qs = ks = qo = ko = 0
    if q is not None:
        qs, qo, hq = _rows3(q, "q", dev, kind), _rows3(q_out, "q_out", dev, kind), q.shape[1]
        _need(q.shape == q_out.shape, "rope: q and q_out differ in shape")
    if k is not None:
        ks, ko, hkv = _rows3(k, "k", dev, kind), _rows3(k_out, "k_out", dev, kind), k.shape[1]
        _need(k.shape == k_out.shape and k.shape[0] == t and k.shape[2] == d,
              "rope: k and k_out [tokens, kv heads, head_dim]")
    check("pva_rope", lib().pva_rope(
        _ptr(q), qs, _ptr(k), ks, t, hq, hkv, d, 1 if kind is _F32 else 0,
        _rope_desc(table, interleaved, dev), _ints(cu_seqlens, 1, "cu_seqlens", dev),
        0 if cu_seqlens is None else cu_seqlens.numel() - 1, _ints(positions, t, "positions", dev),
        1 if inverse else 0, _ptr(q_out), qo, _ptr(k_out), ko, _ints(status, 1, "status", dev),
        _queue(stream, dev)))


class KVCache:
    """A paged key/value cache over tensors that the caller owns: bf16 rows
    [num_pages, kv heads, page_size, head_dim], or 4-bit rows (uint8
    [.., head_dim / 2]) with their scales (bf16 [.., head_dim / 64, 2])."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scales: Optional[torch.Tensor] = None,
                 v_scales: Optional[torch.Tensor] = None):
        int4 = k.dtype == torch.uint8
        _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype and
              k.dtype in (_BF16, torch.uint8), "KVCache: k and v bf16 or uint8 [pages, heads, page_size, row]")
        pages, heads, page, row = k.shape
        self.kind, self.head_dim = (CACHE_INT4, 2 * row) if int4 else (CACHE_BF16, row)
        self.num_pages, self.num_kv_heads, self.page_size = pages, heads, page
        _need((k_scales is not None and v_scales is not None) if int4 else
              (k_scales is None and v_scales is None), "KVCache: scales go with 4-bit rows")
        for s in (k_scales, v_scales) if int4 else ():
            _need(s.dtype == _BF16 and tuple(s.shape) == (pages, heads, page, self.head_dim // 64, 2),
                  "KVCache: scales bf16 [pages, heads, page_size, head_dim / 64, 2]")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        for t in (k, v, k_scales, v_scales):
            _need(t is None or (t.is_cuda and t.is_contiguous() and t.device == k.device),
                  "KVCache: contiguous CUDA tensors of one device")
        self.device, self.index = k.device, k.get_device()
        self.desc = _lib.CacheDesc(self.kind, heads, self.head_dim, page, pages, _ptr(k), _ptr(v),
                                   _ptr(k_scales), _ptr(v_scales))
        self.raw = bytes(self.desc)  # for calls that take the caches of several layers

    @classmethod
    def alloc(cls, num_pages: int, num_kv_heads: int, head_dim: int, page_size: int = 64,
              kind: int = CACHE_BF16, device="cuda") -> "KVCache":
        _need(kind in (CACHE_BF16, CACHE_INT4), "KVCache: kind is CACHE_BF16 or CACHE_INT4")
        shape = (num_pages, num_kv_heads, page_size)
        if kind == CACHE_BF16:
            return cls(*(torch.zeros(shape + (head_dim,), dtype=_BF16, device=device) for _ in "kv"))
        return cls(*(torch.zeros(shape + (head_dim // 2,), dtype=torch.uint8, device=device) for _ in "kv"),
                   *(torch.zeros(shape + (head_dim // 64, 2), dtype=_BF16, device=device) for _ in "kv"))


def _cache_batch(cache: KVCache, page_table, num_tokens: int, kv_lens, cu_new, status, dev: int) -> CacheBatch:
    if page_table.dtype is not _I32 or page_table.get_device() != dev or page_table.dim() != 2:
        raise ValueError(f"page_table: an int32 tensor [sequences, pages] on cuda:{dev} is needed")
    if cache.index != dev:
        raise ValueError(f"the cache is on cuda:{cache.index}, the call's tensors on cuda:{dev}")
    n, width = page_table.shape
    stride = width
    if not page_table.is_contiguous():
        stride, one = page_table.stride()
        _need(one == 1 or width <= 1, "page_table: rows must be contiguous")
        if n <= 1:
            stride = width
        _need(stride >= width, "page_table: rows overlap")
    return CacheBatch(n, num_tokens, width, stride, page_table.data_ptr(),
                      None if kv_lens is None else _ints(kv_lens, n, "kv_lens", dev),
                      None if cu_new is None else _ints(cu_new, n + 1, "cu_new", dev),
                      None if status is None else _ints(status, 1, "status", dev))


def cache_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor,
                 kv_lens: torch.Tensor, cu_new: Optional[torch.Tensor] = None,
                 table: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                 interleaved: bool = False, status: Optional[torch.Tensor] = None,
                 stream=None) -> None:
    """Append the new tokens' keys and values ([tokens, kv heads, head_dim] bf16) to
    the cache.  Sequence b owns rows cu_new[b] .. cu_new[b + 1] (None: row b) and
    kv_lens[b] counts its tokens with the new ones; page_table [sequences, pages].
    With an angle table the keys are rotated on the way (k_out: a copy of them for
    attn_fwd), and the queries q into q_out."""
    dev = _device(k, "k")
    ks, vs = _rows3(k, "k", dev), _rows3(v, "v", dev)
    shape = k.shape
    t, h, d = shape
    if v.shape != shape or h != cache.num_kv_heads or d != cache.head_dim:
        raise ValueError("cache_append: k and v [tokens, kv heads, head_dim] of the cache")
    hq = qs = qo = ko = 0
    if (q is None) != (q_out is None):
        raise ValueError("cache_append: q goes with q_out")
    if q is not None:
        qs, qo = _rows3(q, "q", dev), _rows3(q_out, "q_out", dev)
        q_shape = q.shape
        hq = q_shape[1]
        if q_shape != q_out.shape or q_shape[0] != t or q_shape[2] != d:
            raise ValueError("cache_append: q and q_out [tokens, heads, head_dim]")
    if k_out is not None:
        ko = _rows3(k_out, "k_out", dev)
        _need(k_out.shape == shape, "cache_append: k_out has k's shape")
    rc = (_lib._lib or lib()).pva_cache_append(
        cache.desc, _cache_batch(cache, page_table, t, kv_lens, cu_new, status, dev),
        None if table is None else _rope_desc(table, interleaved, dev), k.data_ptr(), ks,
        v.data_ptr(), vs, None if q is None else q.data_ptr(), qs, hq,
        None if q is None else q_out.data_ptr(), qo, None if k_out is None else k_out.data_ptr(), ko,
        _queue(stream, dev))
    if rc:
        check("pva_cache_append", rc)


def cache_read(cache: KVCache, page_table: torch.Tensor, cu_out: torch.Tensor,
               k_out: torch.Tensor, v_out: torch.Tensor, starts: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Cached rows as a contiguous pack: rows cu_out[b] .. cu_out[b + 1] of k_out and
    v_out (bf16 [tokens, kv heads, head_dim]) are the tokens of sequence b from
    position starts[b] (None: 0) on.  Other rows are left as they were."""
    dev = _device(k_out, "k_out")
    t = k_out.shape[0]
    shape = (t, cache.num_kv_heads, cache.head_dim)
    ko, vo = _whole(k_out, "k_out", dev, shape, _BF16), _whole(v_out, "v_out", dev, shape, _BF16)
    _need(cu_out is not None, "cache_read: cu_out is needed")
    b = _cache_batch(cache, page_table, t, None, cu_out, status, dev)
    check("pva_cache_read", lib().pva_cache_read(
        cache.desc, b, _ints(starts, page_table.shape[0], "starts", dev), ko, vo,
        _queue(stream, dev)))


def cache_attn_bytes(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                     max_new: int = 1) -> int:
    n = lib().pva_cache_attn_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, max_new)
    if n == 0:
        raise _lib.PvaError("pva_cache_attn_bytes", 1)
    return int(n)


def alloc_cache_workspace(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                          max_new: int = 1, device="cuda") -> torch.Tensor:
    """Workspace of cache_attn for up to num_seqs sequences; one call at a time uses it."""
    return torch.empty(cache_attn_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, max_new),
                       dtype=torch.uint8, device=device)


def cache_attn(cache: KVCache, q: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
               out: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor,
               cu_new: Optional[torch.Tensor] = None, max_new: int = 1, window: int = 0,
               softmax_scale: float = 0.0, status: Optional[torch.Tensor] = None,
               stream=None) -> None:
    """Attention of the new tokens' queries ([tokens, heads, head_dim] bf16, rotated)
    over their sequences' cached keys: token i of sequence b's n new ones stands at
    position kv_lens[b] - n + i and sees the keys up to it (window > 0: the last
    `window` of them).  out bf16 or fp32 like q, lse fp32 [heads, tokens]; max_new:
    an upper bound of n."""
    dev, t, args = _attn_args("cache_attn", cache, q, out, lse, workspace)
    rc = (_lib._lib or lib()).pva_cache_attn(
        cache.desc, _cache_batch(cache, page_table, t, kv_lens, cu_new, status, dev), *args[:3],
        max_new, window, softmax_scale, *args[3:], _queue(stream, dev))
    if rc:
        check("pva_cache_attn", rc)


def _attn_args(name: str, cache: KVCache, q, out, lse, workspace):
    """(device, tokens, the C call's q, q_stride, heads, out, out_is_fp32, lse, workspace, its bytes)."""
    dev = _device(q, "q")
    qs = _rows3(q, "q", dev)
    shape = q.shape
    t, h, d = shape
    if d != cache.head_dim:
        raise ValueError(f"{name}: head_dim differs from the cache's")
    o, l = _whole(out, "out", dev, shape, _BF16, _F32), _whole(lse, "lse", dev, (h, t), _F32)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on cuda:{dev} is needed")
    return dev, t, (q.data_ptr(), qs, h, o, 1 if out.dtype is _F32 else 0, l, workspace.data_ptr(),
                    workspace.nbytes)


def cache_cross_attn(cache: KVCache, q: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
                     out: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor,
                     cu_new: Optional[torch.Tensor] = None, max_new: int = 1,
                     softmax_scale: float = 0.0, status: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """Attention of every row of a sequence (beams, or tokens that answer about a source)
    over all kv_lens cached keys of that sequence.  Sequence b owns rows cu_new[b] ..
    cu_new[b + 1] of q (None: row b), at most max_new; the rest as cache_attn."""
    dev, t, args = _attn_args("cache_cross_attn", cache, q, out, lse, workspace)
    rc = (_lib._lib or lib()).pva_cache_cross_attn(
        cache.desc, _cache_batch(cache, page_table, t, kv_lens, cu_new, status, dev), *args[:3],
        max_new, softmax_scale, *args[3:], _queue(stream, dev))
    if rc:
        check("pva_cache_cross_attn", rc)


# ------------------------------------------------------ beam search
_U8 = torch.uint8


def beam_workspace_bytes(groups: int, beams: int, vocab: int, num_out: int) -> int:
    n = lib().pva_beam_select_bytes(groups, beams, vocab, num_out)
    if n == 0:
        raise _lib.PvaError("pva_beam_select_bytes", 1)
    return int(n)


def alloc_beam_workspace(groups: int, beams: int, vocab: int, num_out: int, device="cuda") -> torch.Tensor:
    """Workspace of beam_select for these sizes, and for fewer groups; one call at a time uses it."""
    return torch.empty(beam_workspace_bytes(groups, beams, vocab, num_out), dtype=_U8, device=device)


def beam_select(logits: torch.Tensor, scores: torch.Tensor, out_scores: torch.Tensor,
                out_beams: torch.Tensor, out_tokens: torch.Tensor, workspace: torch.Tensor,
                end_token: int = -1, finished: Optional[torch.Tensor] = None,
                norms: Optional[torch.Tensor] = None, out_finished: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None, stream=None) -> None:
    """The best continuations of every group of beams: logits [groups * beams, vocab]
    (bf16 or fp32, rows of any stride), scores fp32 [groups, beams], into out_scores
    (fp32), out_beams (the parents) and out_tokens (int32), [groups, num_out], best
    first.  finished (uint8 [groups, beams]): rows that offer only themselves, at
    their own score with the end token; norms (fp32 [groups, beams]): scores are
    ranked times these; out_finished (uint8 [groups, num_out])."""
    dev = _device(logits, "logits")
    kind = logits.dtype
    if (kind is not _BF16 and kind is not _F32) or logits.dim() != 2 or scores.dim() != 2 or out_scores.dim() != 2:
        raise ValueError("beam_select: logits bf16 or fp32 [groups * beams, vocab], scores [groups, beams], "
                         "out_scores [groups, num_out]")
    rows, vocab = logits.shape
    shape, out = scores.shape, out_scores.shape
    groups, beams = shape
    if rows != groups * beams or out[0] != groups:
        raise ValueError("beam_select: a row of logits for every beam, a row of results for every group")
    stride, one = logits.stride()
    if (one != 1 and vocab > 1) or (stride < vocab and rows > 1):
        raise ValueError("logits: rows must be contiguous and must not overlap")
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on cuda:{dev} is needed")
    s = _whole(scores, "scores", dev, shape, _F32)
    o = _whole(out_scores, "out_scores", dev, out, _F32)
    ob, ot = _whole(out_beams, "out_beams", dev, out, _I32), _whole(out_tokens, "out_tokens", dev, out, _I32)
    f = None if finished is None else _whole(finished, "finished", dev, shape, _U8)
    n = None if norms is None else _whole(norms, "norms", dev, shape, _F32)
    of = None if out_finished is None else _whole(out_finished, "out_finished", dev, out, _U8)
    rc = (_lib._lib or lib()).pva_beam_select(
        logits.data_ptr(), stride if rows > 1 else 0, 1 if kind is _F32 else 0, groups, beams, vocab, out[1],
        s, f, n, end_token, o, ob, ot, of, None if status is None else _ints(status, 1, "status", dev),
        workspace.data_ptr(), workspace.nbytes, _queue(stream, dev))
    if rc:
        check("pva_beam_select", rc)


def beam_reorder(parents: torch.Tensor, caches: Sequence[KVCache] = (),
                 page_table: Optional[torch.Tensor] = None, kv_lens: Optional[torch.Tensor] = None,
                 states: Sequence[torch.Tensor] = (), status: Optional[torch.Tensor] = None,
                 stream=None) -> None:
    """Every beam's row becomes a copy of its parent's, in place: parents int32
    [groups, beams] (beam_select's out_beams where num_out = beams).  caches: those
    of all layers, which share page_table (int32 [groups * beams, pages], updated:
    full pages are shared, the last one is copied) and kv_lens (int32, the tokens
    cached so far).  states: tensors [groups * beams, ...] of contiguous rows."""
    dev = _device(parents, "parents")
    if parents.dtype is not _I32 or parents.dim() != 2 or not parents.is_contiguous():
        raise ValueError("parents: a contiguous int32 tensor [groups, beams]")
    groups, beams = parents.shape
    rows = groups * beams
    n, table, stride, width, lens, descs = len(caches), None, 0, 0, None, None
    if n:
        if page_table is None or kv_lens is None:
            raise ValueError("beam_reorder: caches go with page_table and kv_lens")
        if page_table.dtype is not _I32 or page_table.get_device() != dev or page_table.dim() != 2 or \
                page_table.shape[0] != rows:
            raise ValueError(f"page_table: an int32 tensor [groups * beams, pages] on cuda:{dev} is needed")
        width = stride = page_table.shape[1]
        if not page_table.is_contiguous():
            stride, one = page_table.stride()
            _need(one == 1 or width <= 1, "page_table: rows must be contiguous")
            stride = width if rows <= 1 else stride
            _need(stride >= width, "page_table: rows overlap")
        table, lens = page_table.data_ptr(), _ints(kv_lens, rows, "kv_lens", dev)
        for c in caches:
            if c.index != dev:
                raise ValueError(f"a cache is on cuda:{c.index}, the call's tensors on cuda:{dev}")
        descs = b"".join([c.raw for c in caches])
    rc = (_lib._lib or lib()).pva_beam_reorder(
        parents.data_ptr(), groups, beams, descs, n, table, stride, width, lens,
        b"".join([_state(t, rows, dev) for t in states]) if states else None, len(states),
        None if status is None else _ints(status, 1, "status", dev), _queue(stream, dev))
    if rc:
        check("pva_beam_reorder", rc)


_STATE = struct.Struct("Pqq")  # pva_state_desc


def _state(t: torch.Tensor, rows: int, dev: int) -> bytes:
    """The bytes of the pva_state_desc of a tensor [rows, ...] of contiguous rows."""
    if t.get_device() != dev or t.dim() < 1 or t.shape[0] != rows:
        raise ValueError(f"states: tensors [groups * beams, ...] of contiguous rows on cuda:{dev} are needed")
    if rows == 0:
        return _STATE.pack(t.data_ptr(), 0, 0)
    if t.is_contiguous():
        size = t.numel() // rows * t.element_size()
        return _STATE.pack(t.data_ptr(), size, size)
    if not t[0].is_contiguous():
        raise ValueError("states: rows must be contiguous")
    size = t[0].numel() * t.element_size()
    stride = t.stride(0) * t.element_size() if rows > 1 else size
    if stride < size:
        raise ValueError("states: rows overlap")
    return _STATE.pack(t.data_ptr(), size, stride)


def cache_status(status: torch.Tensor, stream=None) -> int:
    """The first failure met on the device by the calls that were given this status word
    (int32, 0 before them): 0, or a code of pva.h.  Synchronizes the stream."""
    dev = _device(status, "status")
    code = ctypes.c_int32(0)
    check("pva_cache_status", lib().pva_cache_status(
        _ints(status, 1, "status", dev), ctypes.byref(code), _queue(stream, dev)))
    return int(code.value)


# ------------------------------------------------------ sharding solvers
def chunk_areas(cu_seqlens: torch.Tensor, mask: MaskDesc, chunk_size: int,
                areas: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Allowed pairs of every chunk of chunk_size query rows (device int64)."""
    n = (mask.q_tokens + chunk_size - 1) // chunk_size
    if areas is None:
        areas = torch.empty((n,), dtype=torch.int64, device=cu_seqlens.device)
    check("pva_chunk_areas", lib().pva_chunk_areas(
        _ptr(cu_seqlens), cu_seqlens.numel() - 1, ctypes.byref(mask), chunk_size, _ptr(areas),
        _stream(stream)))
    return areas


def dispatch_chunks(areas: torch.Tensor, cp: int, bucket: Optional[torch.Tensor] = None,
                    bucket_area: Optional[torch.Tensor] = None, stream=None):
    """Greedy min-heap dispatch: (bucket [n] int32, bucket_area [cp] int64), device."""
    n = areas.numel()
    if bucket is None:
        bucket = torch.empty((max(n, 1),), dtype=torch.int32, device=areas.device)
    if bucket_area is None:
        bucket_area = torch.empty((cp,), dtype=torch.int64, device=areas.device)
    check("pva_dispatch_chunks", lib().pva_dispatch_chunks(
        _ptr(areas), n, cp, _ptr(bucket), _ptr(bucket_area), _stream(stream)))
    return bucket[:n], bucket_area


def striped_shard_len(total_tokens: int, cp: int, rank: int, stripe: int) -> int:
    n = lib().pva_striped_shard_len(total_tokens, cp, rank, stripe)
    if n < 0:
        raise _lib.PvaError("pva_striped_shard_len", 1)
    return int(n)


def striped_shard(total_tokens: int, cp: int, rank: int, stripe: int, map_out: torch.Tensor,
                  stream=None) -> None:
    check("pva_striped_shard", lib().pva_striped_shard(
        total_tokens, cp, rank, stripe, _ptr(map_out), _stream(stream)))


def wlb_choose(cu_seqlens_host: np.ndarray, cp: int, tile: int, head_dim: int):
    """(choice 0 per-sequence / 1 per-document, costs [2, cp] int64)."""
    cu = np.ascontiguousarray(cu_seqlens_host, dtype=np.int32)
    costs = np.zeros(2 * cp, dtype=np.int64)
    rc = lib().pva_wlb_choose(cu.ctypes.data_as(ctypes.c_void_p), cu.shape[0] - 1, cp, tile,
                              head_dim, costs.ctypes.data_as(ctypes.c_void_p))
    if rc < 0:
        raise _lib.PvaError("pva_wlb_choose", 1)
    return int(rc), costs.reshape(2, cp)


def debug_withhold_kv_load(enable: bool) -> None:
    """Test hook (see pva_debug_withhold_kv_load): while enabled, one CTA of each
    attention launch (CTA 0 under static dispatch, the one that claimed the
    first unit under dynamic dispatch) waits for a K/V copy that is never
    issued, so its bounded wait expires and worklist_error() reports the site."""
    lib().pva_debug_withhold_kv_load(1 if enable else 0)


def worklist_counts(worklist: torch.Tensor, stream=None) -> dict:
    out = (ctypes.c_int64 * 7)()
    st = lib().pva_worklist_counts(_ptr(worklist), out, _stream(stream))
    names = ("segs", "slices", "units", "runs", "pairs_per_head", "tiles_per_head", "lpt_steps")
    res = dict(zip(names, (int(x) for x in out)))
    res["status"] = int(st)
    return res


# ----------------------------------------------------------------- decoding
_HDR = np.dtype([("i32", "<i4", 20), ("c_tile", "<i8"), ("pair_sum", "<u8"), ("tile_sum", "<u8"),
                 ("off", "<i8", 14)])
_OFF = ("slices", "segs", "units_enum", "keys", "order", "assign", "units", "runs",
        "cta_off", "doc_scan", "dorder", "cls_work", "smask", "total")


def decode_worklist(worklist: torch.Tensor) -> dict:
    """Copy a built worklist to the host and split it into numpy arrays:
    segments, slices, runs and the units.  A static-dispatch worklist gives
    its units in CTA order with the CSR offsets of the CTAs; a dynamic one
    gives them in enumeration (uid) order (cta -1, no offsets) with the
    dispatch order of the uids."""
    raw = worklist.detach().cpu().numpy()
    h = np.frombuffer(raw[:_HDR.itemsize].tobytes(), dtype=_HDR)[0]
    i32 = h["i32"]
    names = ("magic", "version", "error", "num_ctas", "tile_m", "tile_n", "hq", "hkv", "kind",
             "q_tokens", "k_tokens", "num_docs", "cap_slices", "cap_segs", "cap_units",
             "cap_runs", "nslices", "nsegs", "nunits", "nruns")
    hd = {n: int(x) for n, x in zip(names, i32)}
    off = {n: int(x) for n, x in zip(_OFF, h["off"])}
    # after the offsets: lpt_steps, refine_iters, refine_rounds, dispatch_next,
    # dispatch_done, dispatch, dispatch_split, pack_docs
    tail = np.frombuffer(raw[_HDR.itemsize:_HDR.itemsize + 32].tobytes(), dtype="<i4")
    dispatch = tail[5]

    def arr(name, dtype, n, width):
        b = raw[off[name]: off[name] + n * width * np.dtype(dtype).itemsize]
        return np.frombuffer(b.tobytes(), dtype=dtype).reshape(n, width) if width > 1 else \
            np.frombuffer(b.tobytes(), dtype=dtype)

    dynamic = dispatch == DISPATCH_DYNAMIC
    # dynamic dispatch: no per-CTA lists; the units in enumeration (uid) order
    units = arr("units_enum" if dynamic else "units", "<i4", hd["nunits"], 16)
    costs = units[:, 12:14].copy().view("<i8").reshape(-1)
    pairs = units[:, 14:16].copy().view("<i8").reshape(-1)
    return {"header": hd, "pair_sum": int(h["pair_sum"]), "tile_sum": int(h["tile_sum"]),
            "slices": arr("slices", "<i4", hd["nslices"], 8),
            "slice_masks": arr("smask", "<u4", hd["nslices"], 4),
            "pack_docs": int(tail[7]),
            "segs": arr("segs", "<i4", hd["nsegs"], 8),
            "units": units[:, :10].copy(), "unit_ntiles": units[:, 10].copy(),
            "unit_cost": costs, "unit_pairs": pairs,
            "runs": arr("runs", "<i4", hd["nruns"], 4)[:, :3].copy(),
            "cta_off": None if dynamic else arr("cta_off", "<i4", hd["num_ctas"] + 1, 1).copy(),
            "dispatch": int(dispatch), "dispatch_split": int(tail[6]),
            "dispatch_order": arr("dorder", "<i4", hd["nunits"], 1).copy() if dynamic else None}


class PackedAttention:
    """Convenience holder: builds the worklist once for a pack/mask and runs
    the forward on it.  Buffers come from PyTorch; all work is in libpva."""

    def __init__(self, cu_seqlens: Optional[torch.Tensor], mask: MaskDesc,
                 num_q_heads: int, num_kv_heads: int, num_ctas: int = 0,
                 c_tile: Optional[int] = None, head_dim: int = 128):
        self.cu = cu_seqlens
        self.mask = mask
        if c_tile is None:
            c_tile = default_c_tile(head_dim)
        self.params = make_params(num_q_heads, num_kv_heads, num_ctas, c_tile)
        nd = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
        dev = cu_seqlens.device if cu_seqlens is not None else torch.device("cuda")
        self.worklist = alloc_worklist(nd, mask, self.params, dev)

    def plan(self, stream=None) -> None:
        build_worklist(self.cu, self.mask, self.params, self.worklist, stream)

    def forward(self, q, k, v, out=None, lse=None, out_fp32: bool = False, softmax_scale=0.0,
                cta_busy=None, stream=None):
        tq, hq, d = q.shape
        if out is None:
            out = torch.empty((tq, hq, d), dtype=torch.float32 if out_fp32 else torch.bfloat16,
                              device=q.device)
        if lse is None:
            lse = torch.empty((hq, tq), dtype=torch.float32, device=q.device)
        attn_fwd(q, k, v, self.cu, self.mask, self.params, self.worklist, out, lse,
                 softmax_scale, cta_busy, stream)
        return out, lse


def mask_for_workload(w, q_tokens: Optional[int] = None, k_tokens: Optional[int] = None,
                      **kw) -> MaskDesc:
    t = w.total_tokens
    return make_mask(w.mask_kind, q_tokens if q_tokens is not None else t,
                     k_tokens if k_tokens is not None else t, window=w.window,
                     num_prefix_docs=w.num_prefix_docs, **kw)
