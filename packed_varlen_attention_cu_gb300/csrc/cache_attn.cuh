// cache_attn.cuh -- what the kernels of the attention over the paged cache share: arguments, the
// line of units and how it is cut over CTAs, tensor-core and copy instructions, and the kernel that
// joins what was cut.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "../../include/pva.h"
#include "cache.cuh"

namespace pva {

struct AttnArgs {
    const __nv_bfloat16* q;
    const uint8_t *k_pages, *v_pages;
    const uint8_t *k_scales, *v_scales;
    void* out;
    float* lse;
    int64_t* ws_cum;    // [num_seqs]: first unit of each sequence
    int64_t* ws_per;    // units of a piece
    float* ws_o;        // [2 * kMaxCtas][R][D]: sums of cut items, not normalised
    float2* ws_ml;      // [2 * kMaxCtas][R]: their (maximum in base 2, sum)
    int64_t q_stride;
    SeqView s;
    int32_t hq, hkv, group, window, out_fp32;
    int32_t cross;  // every row sees all that its sequence has cached
    uint32_t num_pages, page_bytes;  // page_bytes: codes or values of a page, one of K and V
    float c;      // softmax scale * log2(e), times 2^69 with 4 bits (whose scores carry 2^-69)
    float slack;  // kSlack / c
};

namespace {

constexpr int kMaxCtas = 512;   // pieces the workspace has room for
constexpr int64_t kSpreadRows = 1024;  // rows (tokens * heads) up to which the join spreads a row
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum moves only when a tile exceeds it by 2^8: weights stay below
// 2^8, sums far inside fp32's range, and the accumulators are rescaled rarely.
constexpr float kSlack = 8.f;


__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm(uint32_t* r, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t* r, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The first product of a sum.
__device__ __forceinline__ void mma0(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float lo_f(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_f(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
// 4-bit codes as bf16 without arithmetic: a bf16 whose sign and upper seven exponent
// bits are 0 is its low eight bits as a whole number, times 2^-133 (subnormals and the
// first binade lie on one line).  So a mask alone makes code * 2^-133 of bits 0 .. 3 of
// each half and 16 * code * 2^-133 of bits 4 .. 7; the products, which are exact in
// fp32, stay in range because the other operand carries 2^64.
__device__ __forceinline__ uint32_t low_codes(uint32_t w) { return w & 0x000f000fu; }
__device__ __forceinline__ uint32_t high_codes(uint32_t w) { return w & 0x00f000f0u; }
__device__ __forceinline__ uint32_t both_codes(uint32_t w) { return w & 0x00ff00ffu; }
__device__ __forceinline__ uint32_t upper_bytes(uint32_t w) { return __byte_perm(w, 0, 0x4341); }
constexpr float kUp64 = 18446744073709551616.f;           // 2^64
constexpr float kUp69 = 590295810358705651712.f;          // 2^69 = 2^133 / 2^64

// ---------------------------------------------------------------- the line of units
struct SeqInfo {
    int32_t row0, n;      // rows of the new tokens
    int32_t pos0;         // position of the first of them
    int32_t klo, khi;     // keys any of them may see
    int32_t nrb;          // row blocks
    int32_t blo, nb;      // first block of keys, number of blocks
};

template <class Sh>
__device__ __forceinline__ SeqInfo seq_info(const AttnArgs& a, int32_t b, bool tell) {
    constexpr int R = Sh::R, BLOCK = Sh::kBlock;
    SeqInfo s;
    s.row0 = b;
    s.n = 1;
    bool bad = false;
    if (a.s.cu) {
        s.row0 = a.s.cu[b];
        const int32_t end = a.s.cu[b + 1];
        bad = s.row0 < 0 || end < s.row0 || end > a.s.num_tokens;
        s.n = bad ? 0 : end - s.row0;
    }
    const int32_t kv = a.s.kv_lens[b];
    const int64_t room = (int64_t)a.s.max_pages << a.s.page_shift;
    if (tell) {
        // (without offsets a length of 0 is a row of no sequence: a padded batch)
        if (bad || (a.cross ? kv < 0 : kv < s.n && (a.s.cu || kv != 0))) raise_status(a.s.status, kErrLength);
        if (s.n > 0 && kv > room) raise_status(a.s.status, kErrPage);
    }
    const int32_t kvp = max(kv, 0);
    // Cross: each row stands at the last key or past it (by its number: no sum overflows), where
    // the causal rule lets it see every key.
    s.pos0 = a.cross ? min(kvp - 1, INT32_MAX - 1 - s.n) : kvp - s.n;
    s.khi = (int32_t)min((int64_t)kvp, min(room, (int64_t)INT32_MAX - 2 * BLOCK));
    s.klo = a.window > 0 ? (int32_t)max((int64_t)s.pos0 - a.window + 1, (int64_t)0) : 0;
    s.nrb = (int32_t)(((int64_t)s.n * a.group + R - 1) / R);
    s.blo = s.klo / BLOCK;
    s.nb = max((s.khi + BLOCK - 1) / BLOCK - s.blo, 0);
    return s;
}
// x / y of whole numbers >= 0, by 32 bits where they fit.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
    return ((x | y) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}
template <class Sh>
__device__ __forceinline__ int64_t units_of(const AttnArgs& a, const SeqInfo& s) {
    return (int64_t)a.hkv * s.nrb * (Sh::kFixed + s.nb);
}

// The calling CTA's piece [u0, u1) of the line, and the sequence b that it starts in, whose first
// unit is ub; false where there is none.  Every thread sums a run of sequences; a scan over the
// threads gives each run's first unit.
template <class Sh>
__device__ __forceinline__ bool find_piece(const AttnArgs& a, int64_t& u0, int64_t& u1, int32_t& b, int64_t& ub) {
    constexpr int W = Sh::kWarps;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t ns = a.s.num_seqs, per_thread = (ns + Sh::kThreads - 1) / Sh::kThreads;
    const int32_t s0 = min((int64_t)tid * per_thread, (int64_t)ns), s1 = min(s0 + per_thread, ns);
    int64_t sum = 0;
    for (int32_t x = s0; x < s1; ++x)
        sum += units_of<Sh>(a, seq_info<Sh>(a, x, blockIdx.x == 0));
    int64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    __shared__ int64_t wsum[W];
    __shared__ int32_t found_b;
    __shared__ int64_t found_u;
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        before += w < warp ? wsum[w] : 0;
        total += wsum[w];
    }
    inc += before;
    int64_t per = quotient(total + gridDim.x - 1, gridDim.x);
    per = max(per, (int64_t)2);
    u0 = per * blockIdx.x;
    u1 = min(u0 + per, total);
    if (blockIdx.x == 0) {  // for the join
        if (tid == 0) *a.ws_per = per;
        int64_t u = inc - sum;
        for (int32_t x = s0; x < s1; ++x) {
            a.ws_cum[x] = u;
            u += units_of<Sh>(a, seq_info<Sh>(a, x, false));
        }
    }
    if (u0 >= total) return false;
    if (u0 >= inc - sum && u0 < inc) {
        int64_t u = inc - sum;
        for (int32_t x = s0; x < s1; ++x) {
            const int64_t len = units_of<Sh>(a, seq_info<Sh>(a, x, false));
            if (u0 < u + len) {
                found_b = x;
                found_u = u;
                break;
            }
            u += len;
        }
    }
    __syncthreads();
    b = found_b;
    ub = found_u;
    return true;
}

// Joins the partial sums of every item that was cut, in the order of the pieces.
// What it costs is latency: one load for the piece, one for the sums.  So a row's
// partials are spread over WARPS warps, four at a time in flight in each, and every warp
// keeps its own maximum until the end.  (32 partials of a row of 128: 13 us with one warp,
// 3 us with eight.)  Where rows are many, pieces are few and each warp takes a row.
template <int D, class Sh, int WARPS>
__global__ void __launch_bounds__(256) join_kernel(const AttnArgs a) {
    constexpr int R = Sh::R, E = D / 32;
    __shared__ float sm_o[WARPS][D], sm_m[WARPS], sm_l[WARPS];
    wait_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = WARPS > 1 ? blockIdx.x : (int64_t)blockIdx.x * 8 + warp;
    const int32_t t = (int32_t)quotient(row, a.hq), h = (int32_t)(row - (int64_t)t * a.hq);
    if (t >= a.s.num_tokens) return;
    int32_t b = t;
    if (a.s.cu) b = find_seq(a.s.cu, a.s.num_seqs, t);
    if (b < 0 || b >= a.s.num_seqs) return;
    const SeqInfo s = seq_info<Sh>(a, b, false);
    if (s.nb == 0 || t - s.row0 >= s.n) return;
    const int32_t kvh = h / a.group;
    const int64_t rr = (int64_t)(t - s.row0) * a.group + h - kvh * a.group;
    const int32_t rb = (int32_t)(rr / R), r = (int32_t)(rr - (int64_t)rb * R);
    const int64_t per = *a.ws_per, first = a.ws_cum[b] + ((int64_t)rb * a.hkv + kvh) * (Sh::kFixed + s.nb);
    const int32_t cf = (int32_t)quotient(first + Sh::kFixed, per);
    const int32_t cl = (int32_t)quotient(first + Sh::kFixed + s.nb - 1, per);
    if (cf == cl) return;  // one piece holds it all
    const int32_t n = cl - cf + 1;
    float mm = -INFINITY, l = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int k0 = WARPS > 1 ? warp : 0; k0 < n; k0 += 4 * WARPS) {
        float2 ml[4];
        float v[4][E];
#pragma unroll
        for (int u = 0; u < 4; ++u) {  // (past the end the last one again, with weight 0)
            const int k = min(k0 + u * WARPS, n - 1);
            const int64_t at = (int64_t)(k == 0 ? 2 * cf + 1 : 2 * (cf + k)) * R + r;
            ml[u] = a.ws_ml[at];
            const float* src = a.ws_o + at * D + lane * E;
            if (E == 4) {
                const float4 f = *reinterpret_cast<const float4*>(src);
                v[u][0] = f.x;
                v[u][1] = f.y;
                v[u][E - 2] = f.z;
                v[u][E - 1] = f.w;
            } else {
                const float2 f = *reinterpret_cast<const float2*>(src);
                v[u][0] = f.x;
                v[u][1] = f.y;
            }
        }
        float mn = mm;
#pragma unroll
        for (int u = 0; u < 4; ++u) mn = fmaxf(mn, ml[u].x);
        const float old = mm == -INFINITY ? 0.f : ex2(mm - mn);
        l *= old;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= old;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            // A piece of which the row sees no key has the sum 0 and no part in the result (its sums may
            // hold a NaN of values that only other rows see).  Any other has, whatever its weight: scores
            // that are NaN raise no maximum, so that -inf beside a sum of NaN is no empty piece, and a
            // weight of 0 must meet a value that is not finite.
            const bool none = k0 + u * WARPS >= n || ml[u].y == 0.f;
            const float f = ex2(ml[u].x - mn);
            l += none ? 0.f : f * ml[u].y;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += none ? 0.f : f * v[u][e];
        }
        mm = mn;
    }
    if (WARPS > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = acc[e];
        if (lane == 0) {
            sm_m[warp] = mm;
            sm_l[warp] = l;
        }
        __syncthreads();
        if (warp > 0) return;
        mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) mm = fmaxf(mm, sm_m[w]);
        l = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float f = sm_m[w] == -INFINITY ? 0.f : ex2(sm_m[w] - mm);
            l = fmaf(f, sm_l[w], l);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(f, sm_o[w][lane * E + e], acc[e]);
        }
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const int64_t to = ((int64_t)t * a.hq + h) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = l != 0.f ? acc[e] * inv : 0.f;
    if (a.out_fp32) {
#pragma unroll
        for (int e = 0; e < E; ++e) ((float*)a.out)[to + e] = acc[e];
    } else {
#pragma unroll
        for (int e = 0; e < E; e += 2)
            *reinterpret_cast<uint32_t*>((__nv_bfloat16*)a.out + to + e) = pack2(acc[e], acc[e + 1]);
    }
    if (lane == 0) a.lse[(int64_t)h * a.s.num_tokens + t] = l != 0.f ? fmaf(mm, kLn2, logf(l)) : -INFINITY;
}

inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Where the workspace holds what.
template <class Sh>
inline void place_workspace(AttnArgs& a, uint8_t* ws) {
    a.ws_per = reinterpret_cast<int64_t*>(ws);
    a.ws_cum = reinterpret_cast<int64_t*>(ws + 256);
    ws += 256 + up256((size_t)a.s.num_seqs * 8);
    a.ws_ml = reinterpret_cast<float2*>(ws);
    a.ws_o = reinterpret_cast<float*>(ws + (size_t)2 * kMaxCtas * Sh::R * 8);
}

// The join after a kernel of shape Sh.
template <int D, class Sh>
inline cudaError_t launch_join(const AttnArgs& a, cudaStream_t st) {
    const int64_t rows = (int64_t)a.s.num_tokens * a.hq;
    const bool spread = rows <= kSpreadRows;
    const dim3 grid((unsigned)(spread ? rows : (rows + 7) / 8));
    return spread ? launch_after(join_kernel<D, Sh, 8>, grid, 256, 0, st, a)
                  : launch_after(join_kernel<D, Sh, 1>, grid, 256, 0, st, a);
}

}  // namespace

// cache_rows.cu: cross attention of more than kRowsMin rows of a kv head.
pva_status launch_many_rows(int32_t kind, int32_t head_dim, int64_t rows, const AttnArgs& a, uint8_t* ws,
                            cudaStream_t st);
constexpr int kRowsMin = 16;
// Rows of an item in the workspace.
inline int workspace_rows(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

}  // namespace pva
