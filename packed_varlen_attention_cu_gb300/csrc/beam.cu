// beam.cu -- one step of beam search: the best continuations of every group of
// beams, and caches and states that follow the chosen parents.
//
// Selection.  Row b of a group offers every token t with the score
//   s_b + x_bt - ln sum_t e^(x_bt),
// and the num_out best of the group are wanted, ranked by score * norm_b.  The
// logits are read once: while a CTA streams its part of a row it keeps the sum
// of exponentials and the num_out largest logits that it has met (inside a row
// the order of scores is the order of logits).  A second, dependent kernel joins
// the parts: a row's logarithm, then the group's best among the parts' lists.
//
// Reordering.  Row j of a group becomes a copy of its parent: full pages of the
// paged cache by the page table, the tokens of the last, partly filled page by
// copies in all layers, plain states by copies, all of it in place.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pva.h"
#include "cache.cuh"

namespace pva {
namespace {

constexpr int kErrLogits = 304;  // a row with a NaN or +inf, a score or norm that is no number to rank by
constexpr int kErrParent = 305;  // a parent outside the group

constexpr int kMaxBeams = 64, kMaxOut = 64;
constexpr int kScan = 256;           // threads of a scan CTA
constexpr int kVecs = 4;             // 16-byte loads of a thread and tile
constexpr int kTile = kScan * kVecs; // 16-byte vectors of a tile
constexpr int kJoin = 1024;          // threads of a join CTA
constexpr int kJoinEach = 8;         // candidates of a thread
constexpr int kTargetCtas = 608;     // four CTAs on each of 152 SMs

constexpr float kC = 1.4426950408889634f;  // log2(e)

typedef unsigned long long u64;

struct PartHead {
    double sum;   // sum of e^(x - ref)
    float ref;    // about the largest logit; -inf where the part has none above -inf
    int32_t count;
};

struct SelectArgs {
    const void* logits;
    int64_t row_stride;
    const float* scores;
    const uint8_t* finished;
    const float* norms;
    float* out_scores;
    int32_t *out_beams, *out_tokens;
    uint8_t* out_finished;
    int32_t* status;
    PartHead* heads;  // [rows][parts]
    u64* lists;       // [rows][parts][k]: keys, largest first
    int32_t groups, beams, vocab, k, parts, per, end_token;  // per: vectors of a part
};

__device__ __forceinline__ float ex2_of(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// A key orders logits, the lower token first among equal ones: no two are the same.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);  // (-0 is 0)
    return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float((o >> 31) ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ u64 key_of(float x, int32_t token) {
    return (u64)ordered(x) << 32 | (uint32_t)~token;
}
constexpr u64 kNoKey = (u64)0x007fffffu << 32 | 0xffffffffu;  // -inf: every candidate's key is larger

__device__ __forceinline__ uint4 load16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

enum { kRowNone = 0, kRowLive = 1, kRowDone = 2 };

// What a row offers: nothing (dead, or a score or norm to tell of), its tokens, or itself.
__device__ __forceinline__ int row_state(const SelectArgs& a, int64_t row, bool& bad) {
    const float s = a.scores[row];
    const float w = a.norms ? a.norms[row] : 1.f;
    bad = !(s <= 3.4028234e38f) || !(w > 0.f && w <= 3.4028234e38f);
    if (bad || s == -INFINITY) return kRowNone;
    return a.finished && a.finished[row] ? kRowDone : kRowLive;
}

// One part of one row a CTA.  F32: fp32 logits, else bf16.
template <bool F32>
__global__ void __launch_bounds__(kScan, 4) scan_kernel(const SelectArgs a) {
    constexpr int VE = F32 ? 4 : 8;  // logits of a vector
    constexpr int E = VE * kVecs;    // of a thread and tile
    __shared__ u64 cand[kMaxOut + kMaxOut * E];  // the list, then what a tile adds to it
    __shared__ u64 best[kMaxOut];
    __shared__ u64 tops[kScan];
    __shared__ u64 s_bound;
    __shared__ int s_tops, s_new;
    __shared__ double sm_sum[kScan / 32];
    __shared__ float sm_ref[kScan / 32];
    wait_previous();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / (unsigned)a.parts;
    const int part = blockIdx.x - (int)row * a.parts;
    bool bad;
    if (row_state(a, row, bad) != kRowLive) return;
    const int k = a.k;

    // Vectors start at 16-byte boundaries: vector v holds logits v * VE - shift on, the first
    // and last ones fewer than VE of the row's.
    const char* base = reinterpret_cast<const char*>(a.logits) + row * a.row_stride * (F32 ? 4 : 2);
    const int shift = (int)(reinterpret_cast<uintptr_t>(base) & 15u) / (F32 ? 4 : 2);
    const int32_t nv = (int32_t)(((int64_t)shift + a.vocab + VE - 1) / VE);
    const int32_t v0 = min((int64_t)part * a.per, (int64_t)nv), v1 = min((int64_t)v0 + a.per, (int64_t)nv);
    auto load = [&](uint4 (&v)[kVecs], int32_t tile) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int32_t x = tile + j * kScan + tid;
            const int64_t e0 = (int64_t)x * VE - shift;
            const uint32_t none = F32 ? 0xff800000u : 0xff80ff80u;
            v[j] = make_uint4(none, none, none, none);
            if (x >= v1) continue;
            if (e0 >= 0 && e0 + VE <= a.vocab) {
                v[j] = load16(base + e0 * (F32 ? 4 : 2));
            } else {
                uint32_t w[4] = {none, none, none, none};
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    if (e0 + i < 0 || e0 + i >= a.vocab) continue;
                    if (F32) {
                        w[i & 3] = reinterpret_cast<const uint32_t*>(base)[e0 + i];
                    } else {
                        const uint32_t y = reinterpret_cast<const uint16_t*>(base)[e0 + i];
                        w[i >> 1] = i & 1 ? (w[i >> 1] & 0xffffu) | y << 16 : (w[i >> 1] & 0xffff0000u) | y;
                    }
                }
                v[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    };
    auto word = [&](const uint4 (&v)[kVecs], int i) {
        const uint4 q = v[i >> 2];
        return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
    };
    auto logit = [&](const uint4 (&v)[kVecs], int e) {
        if (F32) return __uint_as_float(word(v, e));
        const uint32_t w = word(v, e >> 1);
        return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
    };

    float ref = -INFINITY, sum = 0.f;
    u64 bound = kNoKey;           // a candidate's key is larger
    float bound_x = -INFINITY;    // its logit
    int count = 0;                // entries of the list
    uint4 v[kVecs], next[kVecs];
    load(v, v0);
    for (int32_t tile = v0; tile < v1; tile += kTile) {
        load(next, tile + kTile);  // (past the part's end: nothing)
        float top;
        if (F32) {
            top = logit(v, 0);
#pragma unroll
            for (int e = 1; e < E; ++e) top = fmaxf(top, logit(v, e));
        } else {
            uint32_t w0 = word(v, 0);
            __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&w0);
#pragma unroll
            for (int i = 1; i < E / 2; ++i) {
                const uint32_t w = word(v, i);
                m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&w));
            }
            top = fmaxf(__low2float(m), __high2float(m));
        }
        // Sum of e^(x - ref), the difference first: c x alone, rounded, is off by more than an
        // exponent holds for logits past 2^30.  ref is a whole number, so it moves by 1 at least
        // and the rounding of the sum's factors dies away.
        const float want = rintf(top);
        if (want > ref) {
            sum *= ex2_of((ref - want) * kC);
            ref = want;
        }
        const float neg = ref == -INFINITY ? 0.f : -ref;
        {
            float2 part2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const float2 c2 = make_float2(kC, kC), n2 = make_float2(neg, neg);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 y = __fmul2_rn(__fadd2_rn(make_float2(logit(v, e), logit(v, e + 1)), n2), c2);
                part2[(e >> 1) & 1] = __fadd2_rn(part2[(e >> 1) & 1], make_float2(ex2_of(y.x), ex2_of(y.y)));
            }
            sum += (part2[0].x + part2[1].x) + (part2[0].y + part2[1].y);
        }
        // ---- candidates: logits above the list's last.  (Tokens ascend, so an equal one is no better.)
        const int above = __syncthreads_count(top > bound_x);
        if (above > 0) {
            u64 least = bound + 1;  // the smallest key that is taken
            if (above > k) {
                // More threads than places hold one.  The k-th largest of the threads' largest keys is
                // a bound: k keys reach it, and at most k threads hold any that do.
                u64 mine = 0;
                if (top > bound_x) {
                    int32_t at = 0;
#pragma unroll
                    for (int e = E - 1; e >= 0; --e) at = logit(v, e) == top ? e : at;
                    mine = key_of(top, (tile + (at / VE) * kScan + tid) * VE - shift + at % VE);
                }
                int ahead = 0;
#pragma unroll
                for (int o = 1; o < 32; ++o) ahead += __shfl_xor_sync(0xffffffffu, mine, o) > mine;
                if (tid == 0) s_tops = 0;
                __syncthreads();
                if (mine != 0 && ahead < k) tops[atomicAdd(&s_tops, 1)] = mine;
                __syncthreads();
                const int n = s_tops;
                if (tid < n) {
                    const u64 x = tops[tid];
                    int r = 0;
                    for (int i = 0; i < n; ++i) r += tops[i] > x;
                    if (r == k - 1) s_bound = x;
                }
                __syncthreads();
                least = s_bound;
            }
            if (tid == 0) s_new = 0;
            __syncthreads();
            if (top > bound_x && ordered(top) >= (uint32_t)(least >> 32)) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float x = logit(v, e);
                    if (x > bound_x) {
                        const u64 key = key_of(x, (tile + (e / VE) * kScan + tid) * VE - shift + e % VE);
                        if (key >= least) cand[count + atomicAdd(&s_new, 1)] = key;
                    }
                }
            }
            __syncthreads();
            const int n = count + s_new;
            for (int i = tid; i < n; i += kScan) {
                const u64 x = cand[i];
                int r = 0;
                for (int j = 0; j < n; ++j) r += cand[j] > x;
                if (r < k) best[r] = x;
            }
            __syncthreads();
            count = min(n, k);
            if (tid < count) cand[tid] = best[tid];
            if (count == k) {
                bound = best[k - 1];
                bound_x = unordered((uint32_t)(bound >> 32));
            }
            // (the next tile's barrier comes before anything is added to the list or put into `best`)
        }
#pragma unroll
        for (int j = 0; j < kVecs; ++j) v[j] = next[j];
    }
    // ---- the part's sum, in 64 bits over the threads, and its list
    float r = ref;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, o));
    double d = ref == -INFINITY ? (double)sum : (double)(sum * ex2_of((ref - r) * kC));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) {
        sm_ref[warp] = r;
        sm_sum[warp] = d;
    }
    __syncthreads();
    const int64_t at = row * a.parts + part;
    if (tid == 0) {
        float rr = sm_ref[0];
        for (int w = 1; w < kScan / 32; ++w) rr = fmaxf(rr, sm_ref[w]);
        double dd = 0;
        for (int w = 0; w < kScan / 32; ++w)
            dd += sm_ref[w] == -INFINITY ? sm_sum[w] : sm_sum[w] * (double)ex2_of((sm_ref[w] - rr) * kC);
        a.heads[at] = PartHead{dd, rr, count};
    }
    if (tid < count) a.lists[at * k + tid] = cand[tid];
}

// One group a CTA: every row's logarithm from its parts, then the best candidates of all lists.
// The k-th largest score is bracketed by halving over the scores' order as whole numbers (rounded
// to fp32, which keeps the order) until few candidates are left, and those are ranked in 64 bits.
__global__ void __launch_bounds__(kJoin) join_kernel(const SelectArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ double add[kMaxBeams];  // what a row adds to its logits
    __shared__ double norm[kMaxBeams];
    __shared__ int state[kMaxBeams];
    __shared__ int s_count[3], s_kept;
    wait_previous();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row0 = (int64_t)blockIdx.x * a.beams;
    const int k = a.k, parts = a.parts, total = a.beams * parts * k;
    double* rank = reinterpret_cast<double*>(smem);        // [total]
    u64* keys = reinterpret_cast<u64*>(rank + total);      // [total]
    int* from = reinterpret_cast<int*>(keys + total);      // [total]
    for (int b = warp; b < a.beams; b += kJoin / 32) {
        bool bad;
        int st = row_state(a, row0 + b, bad);
        double lse = 0;
        if (st == kRowLive) {
            const PartHead* h = a.heads + (row0 + b) * parts;
            float r = -INFINITY;
            for (int p = lane; p < parts; p += 32) r = fmaxf(r, h[p].ref);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, o));
            double s = 0;
            for (int p = lane; p < parts; p += 32)
                s += h[p].ref == -INFINITY ? h[p].sum : h[p].sum * (double)ex2_of((h[p].ref - r) * kC);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (!(s - s == 0)) {  // a NaN or +inf among the logits
                bad = true;
                st = kRowNone;
            } else if (s == 0) {  // nothing above -inf
                st = kRowNone;
            } else {
                lse = (double)r + log(s);
            }
        }
        if (lane == 0) {
            if (bad) raise_status(a.status, kErrLogits);
            state[b] = st;
            add[b] = (double)a.scores[row0 + b] - lse;
            norm[b] = a.norms ? (double)a.norms[row0 + b] : 1.0;
        }
    }
    if (tid < 3) s_count[tid] = 0;
    if (tid == 0) s_kept = 0;
    __syncthreads();
    // candidate i of the group: entry i % k of list i / k
    auto score_of = [&](int b, u64 key) {
        return state[b] == kRowDone ? add[b] : add[b] + (double)unordered((uint32_t)(key >> 32));
    };
    uint32_t coarse[kJoinEach];
    u64 mine[kJoinEach];
#pragma unroll
    for (int e = 0; e < kJoinEach; ++e) {
        const int i = e * kJoin + tid;
        coarse[e] = 0;
        mine[e] = 0;
        if (i >= total) continue;
        const int list = i / k, b = list / parts, at = i - list * k;
        const int64_t l = row0 * parts + list;
        if (state[b] == kRowDone ? at == 0 && list == b * parts : state[b] == kRowLive && at < a.heads[l].count) {
            mine[e] = state[b] == kRowDone ? 0 : a.lists[l * k + at];
            // (a score that fp32 rounds to -inf, or that its norm takes there, is no candidate's)
            const double x = score_of(b, mine[e]);
            const float f = (float)(x * norm[b]);
            coarse[e] = f == -INFINITY || (float)x == -INFINITY ? 0 : ordered(f);
        }
    }
    int round = 0;
    auto reaching = [&](uint32_t x) {  // candidates whose order is at least x
        int n = 0;
#pragma unroll
        for (int e = 0; e < kJoinEach; ++e) n += coarse[e] >= x;
        n = __reduce_add_sync(0xffffffffu, n);
        const int now = round % 3;
        if (lane == 0 && n) atomicAdd(&s_count[now], n);
        if (tid == 0) s_count[(now + 1) % 3] = 0;
        __syncthreads();
        ++round;
        return s_count[now];
    };
    const int few = k + 32;
    uint32_t lo = 1, hi = 0xffffffffu;  // at least min(k, all) candidates reach lo, fewer than k reach hi
    int n = reaching(1);
    if (n > few) {
        while (hi - lo > 1) {
            const uint32_t mid = lo + (hi - lo) / 2;
            const int m = reaching(mid);
            if (m >= k) {
                lo = mid;
                n = m;
                if (n <= few) break;
            } else {
                hi = mid;
            }
        }
    }
#pragma unroll
    for (int e = 0; e < kJoinEach; ++e) {
        if (coarse[e] < lo) continue;
        const int b = (e * kJoin + tid) / k / parts, at = atomicAdd(&s_kept, 1);
        rank[at] = score_of(b, mine[e]) * norm[b];
        keys[at] = mine[e];
        from[at] = b;
    }
    __syncthreads();
    // larger score first, then the lower beam, then the larger logit, then the lower token
    const int64_t out = (int64_t)blockIdx.x * k;
    for (int i = tid; i < n; i += kJoin) {
        const double x = rank[i];
        const u64 key = keys[i];
        const int b = from[i];
        int r = 0;
        for (int j = 0; j < n; ++j) {
            const double y = rank[j];
            r += y > x || (y == x && (from[j] < b || (from[j] == b && keys[j] > key)));
        }
        if (r >= k) continue;
        const bool done = state[b] == kRowDone;
        const int32_t token = done ? a.end_token : (int32_t)~(uint32_t)key;
        a.out_scores[out + r] = (float)score_of(b, key);
        a.out_beams[out + r] = b;
        a.out_tokens[out + r] = token;
        if (a.out_finished) a.out_finished[out + r] = done || token == a.end_token;
    }
    for (int i = n + tid; i < k; i += kJoin) {  // fewer candidates than places
        a.out_scores[out + i] = -INFINITY;
        a.out_beams[out + i] = a.out_tokens[out + i] = -1;
        if (a.out_finished) a.out_finished[out + i] = 0;
    }
}

// Parts that a row is cut into: whole tiles, enough CTAs for the machine where rows are few, and
// no more candidates than the join's threads hold.
int parts_of(int64_t rows, int32_t beams, int32_t k, int64_t vectors) {
    const int64_t tiles = (vectors + kTile - 1) / kTile;
    int64_t parts = (kTargetCtas + rows - 1) / rows;
    const int64_t most = (int64_t)kJoin * kJoinEach / (beams * k);
    parts = parts < most ? parts : most;
    parts = parts < tiles ? parts : tiles;
    const int64_t each = (tiles + parts - 1) / parts;
    return (int)((tiles + each - 1) / each);
}

int64_t vectors_of(int32_t vocab, bool f32) {  // of a row that starts anywhere
    const int ve = f32 ? 4 : 8;
    return ((int64_t)vocab + ve - 1 + ve - 1) / ve;
}

// ---------------------------------------------------------------- reordering

constexpr int kMove = 256;            // threads of a CTA
constexpr int kStage = 6144;          // bytes of a warp's staging buffer
constexpr int kLaunchCaches = 64, kLaunchStates = 16;
constexpr int kPiece = 16384;         // bytes of a row that a warp takes at a time, at most

struct MoveState {
    uint8_t* data;
    int64_t row_bytes, row_stride;
    int32_t pieces, wide;  // wide: 16-byte units, else 4
};

struct MoveArgs {
    const int32_t *parents, *lens;
    int32_t* table;
    int32_t* status;
    int64_t table_stride, num_pages;
    int32_t beams, max_pages, page_shift, heads, row_bytes, scale_bytes;  // of one cached row of a head
    int32_t caches, states, write_table, tell;
    int32_t head_pieces;  // pieces of a page's rows of one head
    uint8_t* k[kLaunchCaches];
    uint8_t* v[kLaunchCaches];
    uint8_t* ks[kLaunchCaches];
    uint8_t* vs[kLaunchCaches];
    MoveState state[kLaunchStates];
};

__device__ __forceinline__ void cp_unit(uint32_t to, const uint8_t* from, bool wide) {
    if (wide) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}

// A CTA belongs to one group; its warps take regions (one head's rows of one page array, a piece
// of a state, the page table) independently.  A warp reads a run of bytes of every row that some
// other row copies into its staging buffer, then writes the run of every row that moves: any
// parents, cycles among them, are right in place, since nothing else touches these bytes.
__global__ void __launch_bounds__(kMove) move_kernel(const __grid_constant__ MoveArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int32_t s_parent[kMaxBeams], s_page[kMaxBeams];
    __shared__ int32_t s_len;
    __shared__ int s_bad;
    __shared__ u64 s_moved, s_source;
    wait_previous();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row0 = (int64_t)blockIdx.x * a.beams;
    if (tid == 0) {
        s_bad = 0;
        s_moved = s_source = 0;
        s_len = a.lens ? a.lens[row0] : 0;
    }
    __syncthreads();
    const int32_t len = s_len;
    const int32_t full = len < 0 ? 0 : len >> a.page_shift, part = len < 0 ? 0 : len & ((1 << a.page_shift) - 1);
    if (tid < a.beams) {
        int32_t p = a.parents[row0 + tid];
        if (p < 0 || p >= a.beams) {
            if (p != -1 && a.tell && blockIdx.y == 0) raise_status(a.status, kErrParent);
            p = tid;
        }
        s_parent[tid] = p;
        int32_t page = -1;
        if (a.lens) {
            if (a.lens[row0 + tid] != len || len < 0) s_bad = kErrLength;
            else if (full > a.max_pages) s_bad = kErrPage;
            if (part > 0 && full < a.max_pages) {
                page = a.table[(row0 + tid) * a.table_stride + full];
                if (page < 0 || page >= a.num_pages) page = -1;
            }
        }
        s_page[tid] = page;
        if (p != tid) {
            atomicOr(&s_moved, 1ull << tid);
            atomicOr(&s_source, 1ull << p);
        }
    }
    __syncthreads();
    // A group whose lengths differ, or lie past its table, is left as it was.
    if (s_bad) {
        if (tid == 0 && a.tell && blockIdx.y == 0) raise_status(a.status, s_bad);
        return;
    }
    const u64 moved = s_moved, source = s_source;
    if (moved == 0) return;
    if (a.lens && part > 0 && tid < a.beams && blockIdx.y == 0 && a.tell && (moved >> tid & 1) &&
        (s_page[tid] < 0 || s_page[s_parent[tid]] < 0))
        raise_status(a.status, kErrPage);
    const int ns = __popcll(source);
    uint8_t* stage = smem + warp * kStage;
    const uint32_t stage_at = (uint32_t)__cvta_generic_to_shared(stage);

    // Bytes [0, bytes) of each row, row j at at(j) (null: the row is left out), in units of 16 or 4 bytes.
    auto move = [&](auto at, int64_t bytes, bool wide) {
        const int shift = wide ? 4 : 2;
        const int64_t units = bytes >> shift;
        const int chunk = ns * 512 <= kStage ? (kStage >> 9) / ns * 32 : 0;  // 16-byte units of a source in the stage
        // more sources than the stage has room for 32 units each: fewer lanes read
        const int run = chunk > 0 ? chunk : (kStage >> 4) / ns;
        for (int64_t u0 = 0; u0 < units; u0 += run) {
            const int m = (int)min((int64_t)run, units - u0);
            int slot = 0;
            for (u64 s = source; s; s &= s - 1, ++slot) {
                const uint8_t* from = at(__ffsll((long long)s) - 1);
                if (!from) continue;
                from += (u0 << shift);
                for (int i = lane; i < m; i += 32)
                    cp_unit(stage_at + ((slot * run + i) << shift), from + ((int64_t)i << shift), wide);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
            for (u64 d = moved; d; d &= d - 1) {
                const int j = __ffsll((long long)d) - 1, p = s_parent[j];
                uint8_t* to = at(j);
                if (!to || !at(p)) continue;
                to += (u0 << shift);
                const uint8_t* got = stage + ((__popcll(source & ((1ull << p) - 1)) * run) << shift);
                if (wide)
                    for (int i = lane; i < m; i += 32)
                        reinterpret_cast<uint4*>(to)[i] = reinterpret_cast<const uint4*>(got)[i];
                else
                    for (int i = lane; i < m; i += 32)
                        reinterpret_cast<uint32_t*>(to)[i] = reinterpret_cast<const uint32_t*>(got)[i];
            }
            __syncwarp();
        }
    };

    const int64_t w0 = (int64_t)blockIdx.y * (kMove / 32) + warp, ws = (int64_t)gridDim.y * (kMove / 32);
    // ---- the last pages: items (cache, K or V, head, piece)
    const int64_t per_cache = (int64_t)2 * a.heads * a.head_pieces;
    const int64_t items = part > 0 ? a.caches * per_cache : 0;
    for (int64_t i = w0; i < items; i += ws) {
        const int c = (int)(i / per_cache);
        int64_t rest = i - c * per_cache;
        const bool v = rest >= (int64_t)a.heads * a.head_pieces;
        if (v) rest -= (int64_t)a.heads * a.head_pieces;
        const int32_t h = (int32_t)(rest / a.head_pieces), piece = (int32_t)(rest - (int64_t)h * a.head_pieces);
        const int64_t head_rows = ((int64_t)h << a.page_shift), page_rows = ((int64_t)a.heads << a.page_shift);
        auto region = [&](uint8_t* pages, int32_t row_bytes) {
            const int64_t off = (int64_t)piece * kPiece;
            // (rows of 4-bit scales are 4 or 8 bytes: the last unit may reach into slots of no token)
            const int64_t bytes = min((int64_t)kPiece, (((int64_t)part * row_bytes + 15) & ~(int64_t)15) - off);
            if (bytes <= 0) return;
            move([&](int j) -> uint8_t* {
                const int32_t page = s_page[j];
                return page < 0 ? nullptr : pages + ((int64_t)page * page_rows + head_rows) * row_bytes + off;
            }, bytes, true);
        };
        region(v ? a.v[c] : a.k[c], a.row_bytes);
        if (a.scale_bytes) region(v ? a.vs[c] : a.ks[c], a.scale_bytes);
    }
    // ---- states and the table, on the warps that the pages leave over first
    int64_t first = items;
    for (int s = 0; s < a.states; ++s) {
        const MoveState& st = a.state[s];
        for (int64_t i = (w0 + ws - first % ws) % ws; i < st.pieces; i += ws) {
            const int64_t off = i * kPiece;
            move([&](int j) { return st.data + (row0 + j) * st.row_stride + off; },
                 min((int64_t)kPiece, st.row_bytes - off), st.wide);
        }
        first += st.pieces;
    }
    if (a.write_table && w0 == first % ws)
        move([&](int j) { return reinterpret_cast<uint8_t*>(a.table + (row0 + j) * a.table_stride); },
             (int64_t)full * 4, false);
}

}  // namespace
}  // namespace pva

using namespace pva;

extern "C" size_t pva_beam_select_bytes(int32_t num_groups, int32_t beams, int32_t vocab, int32_t num_out) {
    if (num_groups < 0 || beams < 1 || beams > kMaxBeams || vocab < 1 || vocab > INT32_MAX - 64 ||
        num_out < 1 || num_out > kMaxOut)
        return 0;
    const int64_t rows = (int64_t)num_groups * beams;
    if (rows > INT32_MAX / kTargetCtas) return 0;
    if (rows == 0) return 256;
    // (fp32 rows have more vectors, so at least as many parts)
    const int a = parts_of(rows, beams, num_out, vectors_of(vocab, true));
    const int b = parts_of(rows, beams, num_out, vectors_of(vocab, false));
    return 256 + (size_t)rows * (a > b ? a : b) * (sizeof(PartHead) + 8 * (size_t)num_out);
}

extern "C" pva_status pva_beam_select(const void* logits, int64_t row_stride, int32_t logits_are_fp32,
                                      int32_t num_groups, int32_t beams, int32_t vocab,
                                      int32_t num_out, const float* scores, const uint8_t* finished,
                                      const float* norms, int32_t end_token, float* out_scores,
                                      int32_t* out_beams, int32_t* out_tokens, uint8_t* out_finished,
                                      int32_t* status_dev, void* workspace, size_t workspace_bytes,
                                      void* stream) {
    if (logits_are_fp32 != 0 && logits_are_fp32 != 1) return PVA_ERR_INVALID_ARG;
    if (num_groups < 0 || beams < 1 || vocab < 1 || num_out < 1) return PVA_ERR_INVALID_ARG;
    if (beams > kMaxBeams || num_out > kMaxOut || vocab > INT32_MAX - 64) return PVA_ERR_UNSUPPORTED;
    const bool f32 = logits_are_fp32 != 0;
    if (row_stride == 0) row_stride = vocab;
    if (row_stride < vocab || row_stride > (int64_t)1 << 40) return PVA_ERR_INVALID_ARG;
    if ((finished || out_finished) && (end_token < 0 || end_token >= vocab)) return PVA_ERR_INVALID_ARG;
    const size_t need = pva_beam_select_bytes(num_groups, beams, vocab, num_out);
    if (need == 0) return PVA_ERR_UNSUPPORTED;
    if (!aligned4(scores) || !aligned4(norms) || !aligned4(out_scores) || !aligned4(out_beams) ||
        !aligned4(out_tokens) || !aligned4(status_dev) ||
        (reinterpret_cast<uintptr_t>(logits) & (f32 ? 3u : 1u)) != 0)
        return PVA_ERR_INVALID_ARG;
    if (num_groups == 0) return PVA_OK;
    if (!logits || !scores || !out_scores || !out_beams || !out_tokens || !workspace ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return PVA_ERR_INVALID_ARG;
    if (workspace_bytes < need) return PVA_ERR_BUFFER_TOO_SMALL;
    const int64_t rows = (int64_t)num_groups * beams, vectors = vectors_of(vocab, f32);
    SelectArgs a = {};
    a.logits = logits;
    a.row_stride = row_stride;
    a.scores = scores;
    a.finished = finished;
    a.norms = norms;
    a.out_scores = out_scores;
    a.out_beams = out_beams;
    a.out_tokens = out_tokens;
    a.out_finished = out_finished;
    a.status = status_dev;
    a.groups = num_groups;
    a.beams = beams;
    a.vocab = vocab;
    a.k = num_out;
    a.end_token = finished || out_finished ? end_token : -1;
    a.parts = parts_of(rows, beams, num_out, vectors);
    a.per = (int32_t)((vectors + a.parts - 1) / a.parts);
    a.heads = reinterpret_cast<PartHead*>(workspace);
    a.lists = reinterpret_cast<u64*>(a.heads + rows * a.parts);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const size_t smem = (size_t)beams * a.parts * num_out * 20;
    if (cudaFuncSetAttribute(join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kJoin * kJoinEach * 20) != cudaSuccess)
        return PVA_ERR_CUDA;
    const dim3 grid((unsigned)(rows * a.parts));
    cudaError_t e = f32 ? launch_after(scan_kernel<true>, grid, kScan, 0, st, a)
                        : launch_after(scan_kernel<false>, grid, kScan, 0, st, a);
    if (e == cudaSuccess) e = launch_after(join_kernel, dim3((unsigned)num_groups), kJoin, smem, st, a);
    return e == cudaSuccess ? PVA_OK : PVA_ERR_CUDA;
}

extern "C" pva_status pva_beam_reorder(const int32_t* parents, int32_t num_groups, int32_t beams,
                                       const pva_cache_desc* caches, int32_t num_caches,
                                       int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                       const int32_t* kv_lens, const pva_state_desc* states,
                                       int32_t num_states, int32_t* status_dev, void* stream) {
    if (num_groups < 0 || beams < 1 || num_caches < 0 || num_states < 0 || (num_caches > 0 && !caches) ||
        (num_states > 0 && !states))
        return PVA_ERR_INVALID_ARG;
    if (beams > kMaxBeams || (int64_t)num_groups * beams > INT32_MAX) return PVA_ERR_UNSUPPORTED;
    if (!aligned4(parents) || !aligned4(page_table) || !aligned4(kv_lens) || !aligned4(status_dev))
        return PVA_ERR_INVALID_ARG;
    const pva_cache_desc* c0 = caches;
    for (int32_t i = 0; i < num_caches; ++i) {
        const pva_cache_desc& c = caches[i];
        const pva_status st = check_cache(&c);
        if (st != PVA_OK) return st;
        // one page table serves them all
        if (c.kind != c0->kind || c.num_kv_heads != c0->num_kv_heads || c.head_dim != c0->head_dim ||
            c.page_size != c0->page_size || c.num_pages != c0->num_pages)
            return PVA_ERR_INVALID_ARG;
    }
    if (num_caches > 0 && (max_pages < 0 || table_stride < max_pages)) return PVA_ERR_INVALID_ARG;
    for (int32_t i = 0; i < num_states; ++i) {
        const pva_state_desc& s = states[i];
        if (s.row_bytes < 0 || s.row_bytes % 4 != 0 || s.row_stride % 4 != 0 || s.row_stride < s.row_bytes ||
            (s.row_bytes > 0 && num_groups > 0 && !s.data) || !aligned4(s.data) || s.row_bytes > (int64_t)1 << 40)
            return PVA_ERR_INVALID_ARG;
    }
    if (num_groups == 0 || (num_caches == 0 && num_states == 0)) return PVA_OK;
    if (!parents || (num_caches > 0 && (!kv_lens || (max_pages > 0 && !page_table)))) return PVA_ERR_INVALID_ARG;
    MoveArgs a = {};
    a.parents = parents;
    a.status = status_dev;
    a.beams = beams;
    if (num_caches > 0) {
        a.lens = kv_lens;
        a.table = page_table;
        a.table_stride = table_stride;
        a.max_pages = max_pages;
        a.num_pages = c0->num_pages;
        a.page_shift = page_shift_of(c0->page_size);
        a.heads = c0->num_kv_heads;
        const bool int4 = c0->kind == PVA_CACHE_INT4;
        a.row_bytes = int4 ? c0->head_dim / 2 : 2 * c0->head_dim;
        a.scale_bytes = int4 ? c0->head_dim / 16 : 0;
        a.head_pieces = (int32_t)(((int64_t)c0->page_size * a.row_bytes + kPiece - 1) / kPiece);
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (cudaFuncSetAttribute(move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMove / 32 * kStage) !=
        cudaSuccess)
        return PVA_ERR_CUDA;
    // As many launches as the caches and states need, all with the lengths; the table goes last
    // (no launch reads the columns that it changes).
    int32_t c = 0, s = 0;
    do {
        const bool first = c == 0 && s == 0;
        a.caches = num_caches - c < kLaunchCaches ? num_caches - c : kLaunchCaches;
        a.states = num_states - s < kLaunchStates ? num_states - s : kLaunchStates;
        for (int32_t i = 0; i < a.caches; ++i) {
            a.k[i] = reinterpret_cast<uint8_t*>(caches[c + i].k_pages);
            a.v[i] = reinterpret_cast<uint8_t*>(caches[c + i].v_pages);
            a.ks[i] = reinterpret_cast<uint8_t*>(caches[c + i].k_scales);
            a.vs[i] = reinterpret_cast<uint8_t*>(caches[c + i].v_scales);
        }
        int64_t work = (int64_t)a.caches * 2 * a.heads * a.head_pieces + 1;
        for (int32_t i = 0; i < a.states; ++i) {
            const pva_state_desc& x = states[s + i];
            MoveState& m = a.state[i];
            m.data = reinterpret_cast<uint8_t*>(x.data);
            m.row_bytes = x.row_bytes;
            m.row_stride = x.row_stride;
            m.pieces = (int32_t)((x.row_bytes + kPiece - 1) / kPiece);
            m.wide = x.row_bytes % 16 == 0 && x.row_stride % 16 == 0 && aligned16(x.data);
            work += m.pieces;
        }
        c += a.caches;
        s += a.states;
        const bool last = c == num_caches && s == num_states;
        a.write_table = last && num_caches > 0;
        a.tell = first;
        int64_t y = (work + kMove / 32 - 1) / (kMove / 32);
        const int64_t room = (kTargetCtas + num_groups - 1) / num_groups;
        y = y < room ? y : room;
        if (launch_after(move_kernel, dim3((unsigned)num_groups, (unsigned)y), kMove, kMove / 32 * kStage, st, a) !=
            cudaSuccess)
            return PVA_ERR_CUDA;
    } while (c < num_caches || s < num_states);
    return PVA_OK;
}
