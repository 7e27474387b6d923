// rope.cu -- rotation of queries and keys by their positions, alone (a pack and
// its gradient) and on the way into the paged cache; and the way back, cached
// rows as a contiguous pack.
//
// A pair (a, b) of a head's dims at position t turns by the angle w_p t of its
// pair index p:  (a cos - b sin, b cos + a sin).  The turn is orthogonal, so
// the gradient goes back through the same kernel with the sign of sin changed.
// The angles come as a table of (cos, sin) in fp32: far positions need 64 bits
// for w_p t, which the caller spends once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pva.h"
#include "cache.cuh"

namespace pva {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
enum { kNoCache = -1 };
// Passes whose loads a lane has in flight, where there is work for every SM.
template <bool F32, int KIND>
struct Unroll {
    static constexpr int value = F32 ? 4 : KIND == kNoCache ? 5 : 3;
};

struct RotArgs {
    const void *q, *k, *v;
    void *q_out, *k_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
    const float* table;  // [max_pos][rot / 2][2], or null: no rotation
    const int32_t* positions;
    void *k_pages, *v_pages, *k_scales, *v_scales;
    SeqView s;  // cu: documents (rotation alone) or new tokens (append)
    int32_t max_pos, rot, inter, inverse;
    int32_t hq, hkv, nslots;
};

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// 16 bytes of a row: eight bf16 or four fp32 dims.
template <bool F32>
struct Vec {
    static constexpr int kDims = F32 ? 4 : 8;
    uint4 r;
    __device__ __forceinline__ void load(const void* row, int v) {
        r = __ldcs(reinterpret_cast<const uint4*>(row) + v);
    }
    __device__ __forceinline__ void store(void* row, int v) const {
        reinterpret_cast<uint4*>(row)[v] = r;
    }
    __device__ __forceinline__ void get(float* x) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (F32) {
                x[i] = __uint_as_float(w[i]);
            } else {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
    __device__ __forceinline__ void set(const float* x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (F32) {
                w[i] = __float_as_uint(x[i]);
            } else {
                const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&p);
            }
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Products and sums are rounded one by one (no contraction), as the formula
// writes them: a 4-bit code then depends on the formula's own values alone.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

// Codes of eight values of a group with (low, inv): one 32-bit word.  up is a power of two
// that inv has been divided by.
__device__ __forceinline__ uint32_t encode(const float* x, float low, float up, float inv) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float c = fminf(fmaxf(rintf(__fmul_rn(__fmul_rn(__fsub_rn(x[i], low), up), inv)), 0.f), 15.f);
        w |= (uint32_t)c << (4 * (i / 2) + 16 * (i % 2));
    }
    return w;
}

// Sequence (or document) of row t0 + lane, for a warp's run of `rows` rows; -1: none, or
// one whose offsets leave the tensor.
__device__ __forceinline__ int32_t seq_of_lane(const SeqView& s, int32_t t0, int32_t rows) {
    const int lane = threadIdx.x & 31;
    const int32_t t = t0 + lane;
    if (!s.cu) return lane < rows && t < s.num_seqs ? t : -1;
    const int32_t b0 = find_seq(s.cu, s.num_seqs, t0);
    if (lane >= rows) return -1;
    if (b0 >= 0 && t < s.cu[b0 + 1]) return rows_fit(s, b0) ? b0 : -1;
    // the run goes on into another sequence, or begins before the first
    int32_t lo = max(b0, 0), hi = s.num_seqs;
    while (hi - lo > 1) {
        const int32_t mid = lo + (hi - lo) / 2;
        if (s.cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return s.num_seqs > 0 && s.cu[lo] <= t && t < s.cu[lo + 1] && rows_fit(s, lo) ? lo : -1;
}

// One warp takes kUnroll passes of a token, whose loads go out before the token's place is
// looked up; a pass is 32 / (D / 2 / dims) heads.  A lane holds two 16-byte vectors of its
// head: with half-split pairs (p, p + rot / 2) those that turn against each other; with
// interleaved pairs, which lie inside a vector, one of each half of the head.  So a
// rotation needs no shuffle, a warp's accesses are whole lines, and a lane's angles serve
// all its heads.  The heads of q, k and v form one list of slots, whatever their counts.
// Bounded by HBM; three CTAs an SM (80 registers, of which five passes of bf16 spill 32 bytes)
// measured best: 131072 tokens of 40 heads of 128, bf16: 419 us (95% of the copy rate), 488 us
// with two, 547 us with four.
template <int D, bool F32, int KIND, int kUnroll>
__global__ void __launch_bounds__(kThreads, 3) rotate_kernel(const RotArgs a) {
    constexpr int kV = Vec<F32>::kDims;
    constexpr int kLph = D / (2 * kV);   // lanes a head
    constexpr int kHpw = 32 / kLph;      // heads a pass
    constexpr int kElem = F32 ? 4 : 2;
    wait_previous();
    const int lane = threadIdx.x & 31;
    const int j = lane % kLph, sub = lane / kLph;
    const int pairs = a.rot / (2 * kV);  // vectors of the first half of the rotated dims
    int oa, ob;           // the lane's vectors
    bool rot_a, rot_b;    // are they rotated?
    if (a.inter) {
        oa = j;
        ob = j + kLph;
        rot_a = oa < 2 * pairs;
        rot_b = ob < 2 * pairs;
    } else {
        rot_a = rot_b = j < pairs;
        oa = rot_a ? j : j + pairs;
        ob = rot_a ? j + pairs : j + kLph;
    }
    const int slot0 = blockIdx.y * kUnroll * kHpw + sub;
    const int64_t stride = (int64_t)gridDim.x * kWarps;
    if (blockIdx.y == 0) tell_offsets(a.s, (int64_t)blockIdx.x * kThreads + threadIdx.x, (int64_t)gridDim.x * kThreads);
    for (int64_t tt = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); tt < a.s.num_tokens;
         tt += stride) {
        const int32_t t = (int32_t)tt;
        // A lane without a head loads the token's first one again: a branch around the loads
        // would make each wait for the one before it.
        Vec<F32> xa[kUnroll], xb[kUnroll];
        const char* q_row = (const char*)a.q + t * a.q_stride * kElem;
        const char* k_row = (const char*)a.k + t * a.k_stride * kElem;
        const char* v_row = (const char*)a.v + t * a.v_stride * kElem;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int slot = slot0 + u * kHpw;
            const char* row = a.hq > 0 ? q_row : k_row;
            if (slot < a.hq) row = q_row + slot * (D * kElem);
            else if (slot < a.hq + a.hkv) row = k_row + (slot - a.hq) * (D * kElem);
            else if (KIND != kNoCache && slot < a.nslots) row = v_row + (slot - a.hq - a.hkv) * (D * kElem);
            xa[u].load(row, oa);
            xb[u].load(row, ob);
        }
        // position of the token, and its cached row (of head 0; -1: it has no page)
        int64_t p = t, row_at = -1;
        if (KIND != kNoCache) {
            int32_t b = t, first = t, n = 1;
            if (a.s.cu) {
                b = find_seq(a.s.cu, a.s.num_seqs, t);
                if (b < 0 || !rows_fit(a.s, b)) continue;
                first = a.s.cu[b];
                n = a.s.cu[b + 1] - first;
            } else if (b >= a.s.num_seqs || a.s.kv_lens[b] == 0) {
                continue;  // (a length of 0: a padded batch)
            }
            p = (int64_t)a.s.kv_lens[b] - n + (t - first);
            const int64_t page = p < 0 ? -1 : page_of(a.s, b, (int32_t)p);
            if (page >= 0) row_at = ((page * a.hkv) << a.s.page_shift) + (p & ((1 << a.s.page_shift) - 1));
        } else if (a.positions) {
            p = a.positions[t];
        } else if (a.s.cu) {
            const int32_t b = find_seq(a.s.cu, a.s.num_seqs, t);
            if (b < 0 || !rows_fit(a.s, b)) continue;
            p = t - a.s.cu[b];
        }
        if (p < 0 || (a.rot > 0 && p >= a.max_pos)) {
            if (lane == 0) raise_status(a.s.status, KIND != kNoCache && p < 0 ? kErrLength : kErrPosition);
            continue;
        }
        if (KIND != kNoCache && row_at < 0 && lane == 0) raise_status(a.s.status, kErrPage);
        const int32_t pos = (int32_t)p;
        // angles: of pairs kV * j on, or of kV / 2 pairs of each vector
        float c[kV], s[kV];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h == 0 ? rot_a : rot_b) {
                const int first = a.inter ? kV / 2 * (h == 0 ? oa : ob) : kV * j + kV / 2 * h;
                const float4* cs =
                    reinterpret_cast<const float4*>(a.table + ((int64_t)pos * (a.rot / 2) + first) * 2);
#pragma unroll
                for (int i = 0; i < kV / 4; ++i) {
                    const float4 f = cs[i];
                    const int at = h * (kV / 2) + 2 * i;
                    c[at] = f.x;
                    s[at] = a.inverse ? -f.y : f.y;
                    c[at + 1] = f.z;
                    s[at + 1] = a.inverse ? -f.w : f.w;
                }
            } else {  // no turn
#pragma unroll
                for (int i = 0; i < kV / 2; ++i) {
                    c[h * (kV / 2) + i] = 1.f;
                    s[h * (kV / 2) + i] = 0.f;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int slot = slot0 + u * kHpw;
            const bool live = slot < a.nslots;
            const bool is_q = slot < a.hq, is_k = !is_q && slot < a.hq + a.hkv;
            if (live && (is_q || is_k) && (rot_a || rot_b)) {
                float x[2 * kV];
                xa[u].get(x);
                xb[u].get(x + kV);
                if (a.inter) {
#pragma unroll
                    for (int i = 0; i < kV; ++i) turn(x[2 * i], x[2 * i + 1], c[i], s[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < kV; ++i) turn(x[i], x[kV + i], c[i], s[i]);
                }
                if (rot_a) xa[u].set(x);
                if (rot_b) xb[u].set(x + kV);
            }
            if (live && is_q) {
                void* o = (char*)a.q_out + (t * a.q_out_stride + (int64_t)slot * D) * kElem;
                xa[u].store(o, oa);
                xb[u].store(o, ob);
            }
            if (live && is_k && a.k_out) {
                void* o =
                    (char*)a.k_out + (t * a.k_out_stride + (int64_t)(slot - a.hq) * D) * kElem;
                xa[u].store(o, oa);
                xb[u].store(o, ob);
            }
            if (KIND != kNoCache) {
                const bool put = live && !is_q && row_at >= 0;
                const int h = is_k ? slot - a.hq : slot - a.hq - a.hkv;
                const int64_t at = row_at + ((int64_t)h << a.s.page_shift);  // cached row
                if (KIND == PVA_CACHE_BF16) {
                    if (put) {
                        char* o = (char*)(is_k ? a.k_pages : a.v_pages) + at * D * 2;
                        xa[u].store(o, oa);
                        xb[u].store(o, ob);
                    }
                } else if (__any_sync(0xffffffffu, live && !is_q)) {
                    // lowest and highest value of each group, over the head's lanes
                    constexpr int kG = D / 64;
                    float x[16], lo[kG], hi[kG];
                    if (live) {
                        xa[u].get(x);
                        xb[u].get(x + 8);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = 0.f;
                    }
                    float la = x[0], ha = x[0], lb = x[8], hb = x[8];
#pragma unroll
                    for (int i = 1; i < 8; ++i) {
                        la = min_nan(la, x[i]);
                        ha = max_nan(ha, x[i]);
                        lb = min_nan(lb, x[8 + i]);
                        hb = max_nan(hb, x[8 + i]);
                    }
                    const int ga = oa / 8, gb = ob / 8;
#pragma unroll
                    for (int g = 0; g < kG; ++g) {
                        lo[g] = INFINITY;
                        hi[g] = -INFINITY;
                        if (ga == g) {
                            lo[g] = min_nan(lo[g], la);
                            hi[g] = max_nan(hi[g], ha);
                        }
                        if (gb == g) {
                            lo[g] = min_nan(lo[g], lb);
                            hi[g] = max_nan(hi[g], hb);
                        }
#pragma unroll
                        for (int o = 1; o < kLph; o <<= 1) {
                            lo[g] = min_nan(lo[g], __shfl_xor_sync(0xffffffffu, lo[g], o));
                            hi[g] = max_nan(hi[g], __shfl_xor_sync(0xffffffffu, hi[g], o));
                        }
                    }
                    // The scale is kept in bf16 and the codes are taken against the kept one;
                    // low is one of the bf16 values, so it is kept exactly.  Scales down to 2^-133
                    // have a reciprocal in fp32 times 2^100 (a power of two changes no rounding).
                    float inv[kG], up[kG];
                    uint32_t pair[kG];
#pragma unroll
                    for (int g = 0; g < kG; ++g) {
                        const __nv_bfloat16 sc =
                            __float2bfloat16_rn(__fmul_rn(__fsub_rn(hi[g], lo[g]), 1.f / 15.f));
                        constexpr float kUp100 = 1267650600228229401496703205376.f;  // 2^100
                        const float f = __bfloat162float(sc);
                        up[g] = f < 1.f / kUp100 ? kUp100 : 1.f;
                        inv[g] = f == 0.f ? 0.f : __frcp_rn(f * up[g]);
                        pair[g] = (uint32_t)__bfloat16_as_ushort(sc) |
                                  (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(lo[g])) << 16;
                    }
                    if (put) {
                        uint32_t* o = (uint32_t*)(is_k ? a.k_pages : a.v_pages) + at * (D / 8);
                        uint32_t* so = (uint32_t*)(is_k ? a.k_scales : a.v_scales) + at * kG;
                        const bool ia = kG == 2 && ga > 0, ib = kG == 2 && gb > 0;  // of the second group
                        o[word_of_octet<D>(oa)] = encode(x, ia ? lo[kG - 1] : lo[0], ia ? up[kG - 1] : up[0],
                                                         ia ? inv[kG - 1] : inv[0]);
                        o[word_of_octet<D>(ob)] = encode(x + 8, ib ? lo[kG - 1] : lo[0], ib ? up[kG - 1] : up[0],
                                                         ib ? inv[kG - 1] : inv[0]);
                        if (j == 0) {
#pragma unroll
                            for (int g = 0; g < kG; ++g) so[g] = pair[g];
                        }
                    }
                }
            }
        }
    }
}

// ------------------------------------------------------------------ read
struct ReadArgs {
    const void *k_pages, *v_pages, *k_scales, *v_scales;
    void *k_out, *v_out;  // [rows, hkv, D] bf16
    const int32_t* starts;
    SeqView s;
    int32_t hkv;
};

// One warp takes `run` (at most 32) consecutive rows: lane i finds the page of row i, so
// that the lookups of a run go on at once, then the warp passes over rows and heads,
// kUnroll passes' loads in flight.  A lane holds 16 bytes of a bf16 row; of a 4-bit row
// the word or two (one of each group) that become one or two octets.
// Bounded by HBM: 37423 rows of 4 heads of 128 dims from 4 bits 18 us (98 MB, 79% of the copy
// rate, cold), 123214 rows of 2 heads of 64 dims in bf16 26 us (127 MB, 72%).  A branch around
// the loads made each wait for the one before it: 52 us.
template <int D, int KIND>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadArgs a, int32_t run) {
    constexpr bool kInt4 = KIND == PVA_CACHE_INT4;
    constexpr int kLph = kInt4 ? 8 : D / 8, kHpw = 32 / kLph, kUnroll = 4, kG = D / 64;
    wait_previous();
    const int lane = threadIdx.x & 31;
    const int o = lane % kLph, sub = lane / kLph;
    const int ppr = (2 * a.hkv + kHpw - 1) / kHpw;  // passes a row
    // p / ppr for p below 32 * ppr + kUnroll as a product: exact while 33 ppr^2 < 2^20
    const uint32_t inv = ((1u << 20) + ppr - 1) / ppr;
    const int64_t runs = ((int64_t)a.s.num_tokens + run - 1) / run;
    for (int64_t ri = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); ri < runs;
         ri += (int64_t)gridDim.x * kWarps) {
        const int32_t t0 = (int32_t)(ri * run);
        const int32_t rows = min(run, a.s.num_tokens - t0);
        // the cached row (of head 0) that lane i's row is
        int64_t at = -1;
        {
            const int32_t t = t0 + lane, b = seq_of_lane(a.s, t0, rows);
            const int32_t i = b >= 0 && a.s.cu ? t - a.s.cu[b] : 0;
            if (b >= 0) {
                const int64_t pos = (a.starts ? a.starts[b] : 0) + (int64_t)i;
                const int64_t page = pos > INT32_MAX ? -1 : page_of(a.s, b, (int32_t)pos);
                if (page < 0) raise_status(a.s.status, kErrPage);
                else at = ((page * a.hkv) << a.s.page_shift) + (pos & ((1 << a.s.page_shift) - 1));
            }
        }
        if (!__any_sync(0xffffffffu, at >= 0)) continue;  // (a cache may have no page at all)
        for (int p0 = 0; p0 < rows * ppr; p0 += kUnroll) {
            uint4 x[kUnroll];
            uint2 sc[kUnroll];
            bool live[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int r = (int)(((uint32_t)(p0 + u) * inv) >> 20), slot = (p0 + u - r * ppr) * kHpw + sub;
                const int64_t row0 = __shfl_sync(0xffffffffu, at, r & 31);
                const bool is_k = slot < a.hkv;
                const int h = is_k ? slot : slot - a.hkv;
                // (lanes without a row load the first one, so that no branch parts the loads)
                live[u] = r < rows && h < a.hkv && row0 >= 0;
                const int64_t row = live[u] ? row0 + ((int64_t)h << a.s.page_shift) : 0;
                const void* pages = is_k ? a.k_pages : a.v_pages;
                if (!kInt4) {
                    x[u] = __ldcs((const uint4*)pages + row * kLph + o);
                } else {
                    const void* scales = is_k ? a.k_scales : a.v_scales;
                    if (kG == 2) {
                        const uint2 w = __ldcs((const uint2*)pages + row * 8 + o);
                        x[u].x = w.x;
                        x[u].y = w.y;
                        sc[u] = ((const uint2*)scales)[row];
                    } else {
                        x[u].x = __ldcs((const uint32_t*)pages + row * 8 + o);
                        sc[u].x = ((const uint32_t*)scales)[row];
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (!live[u]) continue;
                const int r = (int)(((uint32_t)(p0 + u) * inv) >> 20), slot = (p0 + u - r * ppr) * kHpw + sub;
                const bool is_k = slot < a.hkv;
                const int h = is_k ? slot : slot - a.hkv;
                uint4* out = (uint4*)(is_k ? a.k_out : a.v_out) + ((int64_t)(t0 + r) * a.hkv + h) * (D / 8);
                if (!kInt4) {
                    out[o] = x[u];
                } else {
#pragma unroll
                    for (int g = 0; g < kG; ++g) {
                        const uint32_t w = g == 0 ? x[u].x : x[u].y, s = g == 0 ? sc[u].x : sc[u].y;
                        // low + code * scale by one fused operation on bf16 pairs: the product is
                        // exact and the sum is rounded once.  128 + code is a mask and an OR.
                        const uint32_t sw = __byte_perm(s, 0, 0x1010), lw = __byte_perm(s, 0, 0x3232);
                        uint32_t y[4];
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const uint32_t m = ((w >> (4 * p)) & 0x000f000fu) | 0x43004300u;
                            const uint32_t k128 = 0x43004300u;
                            const __nv_bfloat162 code = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                                                *reinterpret_cast<const __nv_bfloat162*>(&k128));
                            const __nv_bfloat162 v = __hfma2(code, *reinterpret_cast<const __nv_bfloat162*>(&sw),
                                                             *reinterpret_cast<const __nv_bfloat162*>(&lw));
                            y[p] = *reinterpret_cast<const uint32_t*>(&v);
                        }
                        out[8 * g + o] = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
            }
        }
    }
    tell_offsets(a.s, (int64_t)blockIdx.x * kThreads + threadIdx.x, (int64_t)gridDim.x * kThreads);
}

// CTAs along the runs: up to 64 on an SM, then a stride.
int grid_x(int64_t tokens, int32_t run, int grid_y, int sms) {
    const int64_t blocks = ((tokens + run - 1) / run + kWarps - 1) / kWarps;
    const int64_t cap = ((int64_t)sms * 64 + grid_y - 1) / grid_y;
    return (int)(blocks < cap ? (blocks > 0 ? blocks : 1) : cap);
}

template <int D, bool F32, int KIND, int kUnroll>
pva_status launch_unrolled(const RotArgs& a, int sms, cudaStream_t st) {
    constexpr int per = kUnroll * (32 / (D / (2 * Vec<F32>::kDims)));
    const int gy = (a.nslots + per - 1) / per;
    if (gy > 65535) return PVA_ERR_UNSUPPORTED;
    const dim3 grid(grid_x(a.s.num_tokens, 1, gy, sms), gy);
    return launch_after(rotate_kernel<D, F32, KIND, kUnroll>, grid, kThreads, 0, st, a) == cudaSuccess
               ? PVA_OK
               : PVA_ERR_CUDA;
}

// A few tokens take one pass a warp: what they cost is latency (96 tokens of 24 heads into
// 4 bits: 5.7 us with three passes a warp, 3.6 us with one).  Of many, heads that fill one or two
// passes take no more (bf16, interleaved: 32768 tokens of 16 heads of 64, two passes: 34.9 us
// with five, 31.4 us with two; 20383 of 8 heads, one pass: 18.0 and 13.8 us).  All others run
// Unroll's number a warp, and what the last warp has no heads for it loads in vain: of 131072
// tokens with heads of 128 in bf16, 40 heads (ten passes) reach 95% of the copy rate, 32 (eight)
// 89%, 16 (four) 86%, 24 (six) 80%.
template <int D, bool F32, int KIND>
pva_status launch_rotate(const RotArgs& a, cudaStream_t st) {
    const int sms = sm_count();
    if (sms <= 0) return PVA_ERR_CUDA;
    constexpr int per = 32 / (D / (2 * Vec<F32>::kDims));
    const int passes = (a.nslots + per - 1) / per;
    if (passes <= 1 || (int64_t)a.s.num_tokens * passes <= (int64_t)sms * 3 * kWarps)
        return launch_unrolled<D, F32, KIND, 1>(a, sms, st);
    if (passes == 2) return launch_unrolled<D, F32, KIND, 2>(a, sms, st);
    return launch_unrolled<D, F32, KIND, Unroll<F32, KIND>::value>(a, sms, st);
}

template <int D, int KIND>
pva_status launch_read(const ReadArgs& a, cudaStream_t st) {
    if ((2 * (int64_t)a.hkv * (KIND == PVA_CACHE_INT4 ? 8 : D / 8) + 31) / 32 > 176)
        return PVA_ERR_UNSUPPORTED;  // the kernel's division (352 kv heads, 176 of 128 bf16 dims)
    const int sms = sm_count();
    if (sms <= 0) return PVA_ERR_CUDA;
    int32_t run = 32;  // as many rows a warp as leave every SM two CTAs of work
    while (run > 1 && a.s.num_tokens / run < sms * 2 * kWarps) run /= 2;
    const dim3 grid(grid_x(a.s.num_tokens, run, 1, sms));
    return launch_after(read_kernel<D, KIND>, grid, kThreads, 0, st, a, run) == cudaSuccess ? PVA_OK
                                                                                            : PVA_ERR_CUDA;
}

// Heads of one token past which no grid has blocks for them (65535 of at most 40), and far
// below which sums of counts stay in 32 bits.
constexpr int64_t kMaxSlots = 1 << 24;

// The angle table: rot_dim 0 (or no descriptor) means no rotation.
pva_status check_rope(const pva_rope_desc* r, int32_t head_dim) {
    if (!r) return PVA_OK;
    if (r->rot_dim < 0 || r->rot_dim > head_dim || r->max_pos < 0 ||
        (r->interleaved != 0 && r->interleaved != 1))
        return PVA_ERR_INVALID_ARG;
    if (r->rot_dim % 16 != 0) return PVA_ERR_UNSUPPORTED;
    if (r->rot_dim > 0 && r->max_pos > 0 && (!r->table || !aligned16(r->table)))
        return PVA_ERR_INVALID_ARG;
    return PVA_OK;
}

void set_rope(RotArgs* a, const pva_rope_desc* r) {
    a->rot = r ? r->rot_dim : 0;
    a->table = r ? r->table : nullptr;
    a->max_pos = r ? r->max_pos : 0;
    a->inter = r ? r->interleaved : 0;
}

}  // namespace
}  // namespace pva

using namespace pva;

extern "C" pva_status pva_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                               int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                               int32_t head_dim, int32_t is_fp32, const pva_rope_desc* rope,
                               const int32_t* cu_seqlens_dev, int32_t num_docs,
                               const int32_t* positions_dev, int32_t inverse, void* q_out,
                               int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                               int32_t* status_dev, void* stream) {
    if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads < 0 || num_docs < 0 || !rope ||
        (is_fp32 != 0 && is_fp32 != 1) || (inverse != 0 && inverse != 1))
        return PVA_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return PVA_ERR_UNSUPPORTED;
    const pva_status rs = check_rope(rope, head_dim);
    if (rs != PVA_OK) return rs;
    if ((int64_t)num_q_heads + num_kv_heads > kMaxSlots) return PVA_ERR_UNSUPPORTED;
    if (cu_seqlens_dev && positions_dev) return PVA_ERR_INVALID_ARG;
    if (!aligned4(cu_seqlens_dev) || !aligned4(positions_dev) || !aligned4(status_dev))
        return PVA_ERR_INVALID_ARG;
    const int eb = is_fp32 ? 4 : 2;
    RotArgs a = {};
    a.q_stride = row_stride(q_stride, num_q_heads, head_dim, eb);
    a.k_stride = row_stride(k_stride, num_kv_heads, head_dim, eb);
    a.q_out_stride = row_stride(q_out_stride, num_q_heads, head_dim, eb);
    a.k_out_stride = row_stride(k_out_stride, num_kv_heads, head_dim, eb);
    if (a.q_stride < 0 || a.k_stride < 0 || a.q_out_stride < 0 || a.k_out_stride < 0)
        return PVA_ERR_INVALID_ARG;
    if (num_tokens == 0 || num_q_heads + num_kv_heads == 0) return PVA_OK;
    if ((num_q_heads > 0 && (!q || !q_out)) || (num_kv_heads > 0 && (!k || !k_out)) ||
        !aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out))
        return PVA_ERR_INVALID_ARG;
    a.q = q;
    a.k = k;
    a.q_out = q_out;
    a.k_out = k_out;
    a.positions = positions_dev;
    a.inverse = inverse;
    a.hq = num_q_heads;
    a.hkv = num_kv_heads;
    a.nslots = num_q_heads + num_kv_heads;
    set_rope(&a, rope);
    a.s.cu = cu_seqlens_dev;
    a.s.num_seqs = num_docs;
    a.s.num_tokens = num_tokens;
    a.s.status = status_dev;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (head_dim == 128)
        return is_fp32 ? launch_rotate<128, true, kNoCache>(a, st)
                       : launch_rotate<128, false, kNoCache>(a, st);
    return is_fp32 ? launch_rotate<64, true, kNoCache>(a, st)
                   : launch_rotate<64, false, kNoCache>(a, st);
}

extern "C" pva_status pva_cache_append(const pva_cache_desc* cache, const pva_cache_batch* batch,
                                       const pva_rope_desc* rope, const void* k, int64_t k_stride,
                                       const void* v, int64_t v_stride, const void* q,
                                       int64_t q_stride, int32_t num_q_heads, void* q_out,
                                       int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                                       void* stream) {
    pva_status st = check_cache(cache);
    if (st == PVA_OK) st = check_batch(batch, true);
    if (st == PVA_OK) st = check_rope(rope, cache->head_dim);
    if (st != PVA_OK) return st;
    const int32_t d = cache->head_dim, hkv = cache->num_kv_heads;
    if (num_q_heads < 0) return PVA_ERR_INVALID_ARG;
    if (num_q_heads + 2 * (int64_t)hkv > kMaxSlots) return PVA_ERR_UNSUPPORTED;
    RotArgs a = {};
    a.q_stride = row_stride(q_stride, num_q_heads, d, 2);
    a.k_stride = row_stride(k_stride, hkv, d, 2);
    a.v_stride = row_stride(v_stride, hkv, d, 2);
    a.q_out_stride = row_stride(q_out_stride, num_q_heads, d, 2);
    a.k_out_stride = row_stride(k_out_stride, hkv, d, 2);
    if (a.q_stride < 0 || a.k_stride < 0 || a.v_stride < 0 || a.q_out_stride < 0 ||
        a.k_out_stride < 0)
        return PVA_ERR_INVALID_ARG;
    if (batch->num_tokens == 0 || batch->num_seqs == 0) return PVA_OK;  // (empty tensors have no address)
    if ((num_q_heads > 0) != (q != nullptr) || (q == nullptr) != (q_out == nullptr)) return PVA_ERR_INVALID_ARG;
    if (!k || !v || !aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out) ||
        !aligned16(k_out))
        return PVA_ERR_INVALID_ARG;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.k_out = k_out;
    a.k_pages = cache->k_pages;
    a.v_pages = cache->v_pages;
    a.k_scales = cache->k_scales;
    a.v_scales = cache->v_scales;
    a.hq = num_q_heads;
    a.hkv = hkv;
    a.nslots = num_q_heads + 2 * hkv;
    set_rope(&a, rope);
    a.s = seq_view(cache, batch);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cache->kind == PVA_CACHE_BF16)
        return d == 128 ? launch_rotate<128, false, PVA_CACHE_BF16>(a, s)
                        : launch_rotate<64, false, PVA_CACHE_BF16>(a, s);
    return d == 128 ? launch_rotate<128, false, PVA_CACHE_INT4>(a, s)
                    : launch_rotate<64, false, PVA_CACHE_INT4>(a, s);
}

extern "C" pva_status pva_cache_read(const pva_cache_desc* cache, const pva_cache_batch* batch,
                                     const int32_t* starts_dev, void* k_out, void* v_out,
                                     void* stream) {
    pva_status st = check_cache(cache);
    if (st == PVA_OK) st = check_batch(batch, false);
    if (st != PVA_OK) return st;
    if (!aligned4(starts_dev)) return PVA_ERR_INVALID_ARG;
    if (batch->num_tokens == 0 || batch->num_seqs == 0) return PVA_OK;
    if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)) return PVA_ERR_INVALID_ARG;
    ReadArgs a = {};
    a.k_pages = cache->k_pages;
    a.v_pages = cache->v_pages;
    a.k_scales = cache->k_scales;
    a.v_scales = cache->v_scales;
    a.k_out = k_out;
    a.v_out = v_out;
    a.starts = starts_dev;
    a.s = seq_view(cache, batch);
    a.hkv = cache->num_kv_heads;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cache->kind == PVA_CACHE_BF16)
        return cache->head_dim == 128 ? launch_read<128, PVA_CACHE_BF16>(a, s)
                                      : launch_read<64, PVA_CACHE_BF16>(a, s);
    return cache->head_dim == 128 ? launch_read<128, PVA_CACHE_INT4>(a, s)
                                  : launch_read<64, PVA_CACHE_INT4>(a, s);
}

extern "C" pva_status pva_cache_status(const int32_t* status_dev, int32_t* code_out,
                                       void* stream) {
    if (!status_dev || !code_out || !aligned4(status_dev)) return PVA_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (cudaMemcpyAsync(code_out, status_dev, sizeof(int32_t), cudaMemcpyDeviceToHost, st) !=
            cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return PVA_ERR_CUDA;
    return PVA_OK;
}
