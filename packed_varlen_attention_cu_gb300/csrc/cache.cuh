// cache.cuh -- what the rotation and key/value cache kernels share: the batch
// of sequences as the device sees it, lookups of a token's sequence and of a
// position's page, the 4-bit row format, and the host's argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/pva.h"

namespace pva {

// Device status words of the cache calls (pva_cache_status).
constexpr int kErrPage = 300;      // no page, or a page outside the cache
constexpr int kErrLength = 301;    // lengths that do not fit the batch
constexpr int kErrPosition = 303;  // a position outside the angle table

__device__ __forceinline__ void raise_status(int32_t* status, int code) {
    if (status) atomicCAS(status, 0, code);
}

// Lengths, offsets and pages may have been written by the kernel before, which may
// still run when this one is launched (see wait_previous): they are read after the wait,
// and by ordinary loads, not through the read-only path.

// Sequence b with cu[b] <= t < cu[b + 1], or -1; called by whole warps.  Each
// round every lane probes one offset, so a batch of up to 1024 sequences takes
// two rounds.  Whatever cu holds, the reads stay inside cu[0 .. n].
__device__ __forceinline__ int32_t find_seq(const int32_t* cu, int32_t n, int32_t t) {
    const int lane = threadIdx.x & 31;
    int32_t lo = 0, hi = n;
    while (hi - lo > 1) {
        const int32_t step = (hi - lo + 31) / 32;
        const int64_t at = lo + (int64_t)lane * step;
        const bool le = at < hi && cu[at] <= t;
        const int c = __popc(__ballot_sync(0xffffffffu, le));
        lo += (c > 0 ? c - 1 : 0) * step;
        hi = min(hi, lo + step);
    }
    return (n > 0 && cu[lo] <= t && t < cu[lo + 1]) ? lo : -1;
}

// Dependent launches.  A kernel of these calls may be launched while the kernel before
// it in the stream runs out, and waits for its end: a chain of short kernels (append,
// attention, join) pays less for its launches (0.3 to 1 us each; letting the next kernel
// start any earlier than the last blocks' exit was no better and cost the long ones 1%).
// All reads and writes come after the wait, and no thread block leaves without having
// waited, so that the end of a kernel is the end of all before it.
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                                const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

constexpr int kMaxDevices = 64;

// SMs of the current device (asked once for each), or 0.
inline int sm_count() {
    static std::atomic<int> known[kMaxDevices];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
    if (dev < kMaxDevices && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < kMaxDevices) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

// The sequences of one call, as pva_cache_batch describes them.
struct SeqView {
    const int32_t* page_table;
    const int32_t* kv_lens;
    const int32_t* cu;  // null: one token for each sequence
    int32_t* status;
    int64_t table_stride;
    int64_t num_pages;
    int32_t num_seqs, num_tokens, max_pages, page_shift;
};

// Do the rows of sequence b, which find_seq has found, lie inside the tensor?  Those of a
// sequence that says otherwise are left out: its count is not to be trusted, and positions
// and slots follow from it.
__device__ __forceinline__ bool rows_fit(const SeqView& s, int32_t b) {
    return s.cu[b] >= 0 && s.cu[b + 1] <= s.num_tokens;
}

// Offsets that decrease or leave the tensor are told of, a sequence a thread (thread i of n).
// Rows that such offsets place in no sequence meet no other check.
__device__ __forceinline__ void tell_offsets(const SeqView& s, int64_t i, int64_t n) {
    if (!s.cu || !s.status) return;
#pragma unroll 1
    for (; i < s.num_seqs; i += n) {
        const int32_t first = s.cu[i], end = s.cu[i + 1];
        if (first < 0 || end < first || end > s.num_tokens) raise_status(s.status, kErrLength);
    }
}

// Page of key position `pos` of sequence b, or -1 where there is none.
__device__ __forceinline__ int64_t page_of(const SeqView& s, int32_t b, int32_t pos) {
    const int32_t i = pos >> s.page_shift;
    if (pos < 0 || i >= s.max_pages) return -1;
    const int32_t p = s.page_table[b * s.table_stride + i];
    return (p < 0 || p >= s.num_pages) ? -1 : p;
}

// ---- 4-bit rows.  A row of d dims is d / 64 groups of 64; a group has a
// (scale, low) pair of bf16 and value = low + code * scale, code in 0..15.
// Eight dims share a 32-bit word, dim i of the eight at bit
// 4 * (i / 2) + 16 * (i % 2): one AND with 0x000f000f, after a shift by 4 * p,
// leaves dims 2p and 2p + 1 in the halves that a pair of bf16 occupies.
// Octet o of a row is word (o % 8) * (d / 64) + o / 8: the words of both groups
// of a 128-dim row lie side by side, so that one thread's load feeds both.
template <int D>
__device__ __forceinline__ constexpr int word_of_octet(int o) {
    return (o % 8) * (D / 64) + o / 8;
}

// ---- host checks
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// log2 of a page size the kernels take (16 .. 1024, a power of two), or -1.
inline int page_shift_of(int32_t page_size) {
    for (int s = 4; s <= 10; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

inline pva_status check_cache(const pva_cache_desc* c) {
    if (!c || c->num_kv_heads <= 0 || c->num_pages < 0 || c->num_pages > INT32_MAX)
        return PVA_ERR_INVALID_ARG;
    if (c->kind != PVA_CACHE_BF16 && c->kind != PVA_CACHE_INT4) return PVA_ERR_INVALID_ARG;
    if ((c->head_dim != 64 && c->head_dim != 128) || page_shift_of(c->page_size) < 0)
        return PVA_ERR_UNSUPPORTED;
    if (c->num_pages > 0 &&
        (!c->k_pages || !c->v_pages || !aligned16(c->k_pages) || !aligned16(c->v_pages)))
        return PVA_ERR_INVALID_ARG;
    if (c->kind == PVA_CACHE_INT4 && c->num_pages > 0 &&
        (!c->k_scales || !c->v_scales || !aligned16(c->k_scales) || !aligned16(c->v_scales)))
        return PVA_ERR_INVALID_ARG;
    return PVA_OK;
}

inline pva_status check_batch(const pva_cache_batch* b, bool need_lens) {
    if (!b || b->num_seqs < 0 || b->num_tokens < 0 || b->max_pages < 0 ||
        b->table_stride < b->max_pages)
        return PVA_ERR_INVALID_ARG;
    if (!aligned4(b->page_table) || !aligned4(b->kv_lens) || !aligned4(b->cu_new) ||
        !aligned4(b->status))
        return PVA_ERR_INVALID_ARG;
    if (b->num_seqs > 0 && b->num_tokens > 0) {
        if (need_lens && !b->kv_lens) return PVA_ERR_INVALID_ARG;
        if (b->max_pages > 0 && !b->page_table) return PVA_ERR_INVALID_ARG;
        if (!b->cu_new && b->num_tokens < b->num_seqs) return PVA_ERR_INVALID_ARG;
    }
    return PVA_OK;
}

inline SeqView seq_view(const pva_cache_desc* c, const pva_cache_batch* b) {
    SeqView s;
    s.page_table = b->page_table;
    s.kv_lens = b->kv_lens;
    s.cu = b->cu_new;
    s.status = b->status;
    s.table_stride = b->table_stride;
    s.num_pages = c->num_pages;
    s.num_seqs = b->num_seqs;
    s.num_tokens = b->num_tokens;
    s.max_pages = b->max_pages;
    s.page_shift = page_shift_of(c->page_size);
    return s;
}

// A token stride in elements (0: contiguous heads * dim) that keeps every row
// 16-byte aligned; -1 if it is none.
inline int64_t row_stride(int64_t stride, int64_t heads, int64_t dim, int elem_bytes) {
    if (stride == 0) stride = heads * dim;
    return (stride < heads * dim || stride * elem_bytes % 16 != 0) ? -1 : stride;
}

}  // namespace pva
