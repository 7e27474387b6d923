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
constexpr int kScanCtas = 4;         // scan CTAs on an SM
constexpr int kRoom = 2048;          // candidates of a run that a scan CTA has room for
constexpr int kHits = 1024;          // vectors that hold candidates of a run
constexpr int kPlenty = 768;         // more than these are not ranked: a better bound is found first
constexpr int kJoin = 1024;          // threads of a join CTA, at most
constexpr int kJoinEach = 8;         // candidates of a thread
constexpr int kFewCandidates = 128;  // up to which each candidate of a group counts the others
constexpr int kPieceCost = 4;        // in tiles
constexpr int kTargetCtas = 608;     // four CTAs on each of 152 SMs

constexpr float kC = 1.4426950408889634f;  // log2(e)

typedef unsigned long long u64;

// x / y of whole numbers >= 0, by 32 bits where they fit.
__device__ __forceinline__ int64_t quotient(int64_t x, int32_t y) {
    return (x >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}

struct PartHead {
    float hi, lo;   // hi + lo: sum of e^(x - ref)
    float ref;      // about the largest logit; -inf where the part has none above -inf
    int32_t pad;
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
    u64* lists;       // [rows][parts][k]: keys, largest first; 0 where there is none
    int32_t groups, beams, vocab, k, end_token;
    int32_t tiles, per, parts;  // tiles of a row and of a CTA, room for a row's parts
    int32_t whole;              // CTAs of a row, or 0: CTAs take pieces of the line of all rows
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

// (a, b) becomes a sum of two floats that keeps what their addition rounds off.
__device__ __forceinline__ void add_exact(float& hi, float& lo, float x, float y) {
    const float s = hi + x, t = s - hi;
    lo += (hi - (s - t)) + (x - t) + y;
    hi = s;
}

// A CTA takes an equal piece of the line of all rows' tiles (16 KB each), so a row is cut into
// parts where pieces end.  F32: fp32 logits, else bf16.
//
// What bounds it is HBM, so candidates must cost next to nothing.  Threads note the vectors in which
// a logit passes a bound; warps stream without meeting.  After 1, 4, 16, ... tiles the noted vectors'
// candidates go to a list, which is ranked and cut to its k best, and the bound is raised: each run
// adds about 3 k.
// (512 rows of 131071 bf16 logits, both kernels: a barrier and a count for each tile 78 us; warps
// that look through their logits where they find one 55; vectors noted 42, 40 since
// no tile past a row's end is read; without candidates 28.)
// Should a run hold more than the lists, as ascending logits do, it is read again tile by tile
// with a better bound.
// The first bound is the smallest of the largest logits of 8, 16, 32 or 64 groups of threads: as
// many logits as places reach it, and a few times as many in all.
template <bool F32>
__global__ void __launch_bounds__(kScan, kScanCtas) scan_kernel(const SelectArgs a) {
    constexpr int VE = F32 ? 4 : 8;  // logits of a vector
    constexpr int E = VE * kVecs;    // of a thread and tile
    static_assert(kMaxOut * E <= kRoom, "what a tile may add after a bound by threads");
    __shared__ uint4 hits[kHits];     // vectors that hold candidates of the run, and their numbers
    __shared__ int32_t numbers[kHits];
    __shared__ u64 cand[kRoom];       // the candidates in them
    __shared__ u64 best[2][kMaxOut];  // the k best so far, largest first, and those before them
    __shared__ u64 tops[kScan];
    __shared__ u64 s_bound;
    __shared__ int s_tops, s_n, s_hits;
    __shared__ float sm_hi[kScan / 32], sm_lo[kScan / 32], sm_ref[kScan / 32];
    wait_previous();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int k = a.k;
    int64_t u = (int64_t)blockIdx.x * a.per, u1 = min(u + a.per, (int64_t)a.groups * a.beams * a.tiles);
    if (a.whole) {
        const int64_t row = quotient(blockIdx.x, a.whole);
        u = row * a.tiles + (blockIdx.x - row * a.whole) * a.per;
        u1 = min(u + a.per, (row + 1) * a.tiles);
    }
    for (; u < u1;) {
        const int64_t row = quotient(u, a.tiles);
        const int32_t t0 = (int32_t)(u - row * a.tiles);
        int32_t t1 = (int32_t)min((int64_t)a.tiles, t0 + u1 - u);
        const int part = a.whole ? t0 / a.per : (int)blockIdx.x - (int)quotient(row * a.tiles, a.per);
        u += t1 - t0;

        // Vectors start at 16-byte boundaries: vector v holds logits v * VE - shift on, the first
        // and last ones fewer than VE of the row's.
        const char* base = reinterpret_cast<const char*>(a.logits) + row * a.row_stride * (F32 ? 4 : 2);
        const int shift = (int)(reinterpret_cast<uintptr_t>(base) & 15u) / (F32 ? 4 : 2);
        const int32_t nv = (int32_t)(((int64_t)shift + a.vocab + VE - 1) / VE);
        // (rows have tiles for any start; the last one may be empty: 512 rows of 131071, 42.2 -> 40.2 us;
        // tiles on their way to L2 by prefetches, 1, 2, 4, 8 or 16 ahead, 40.8 to 45.4)
        t1 = min(t1, (nv + kTile - 1) / kTile);
        const int32_t whole0 = shift > 0 ? 1 : 0, whole1 = (int32_t)(((int64_t)shift + a.vocab) / VE);
        // Vector x of the row; what is not the row's is -inf.
        auto vector = [&](int32_t x) {
            const int64_t e0 = (int64_t)x * VE - shift;
            if (x >= whole0 && x < whole1) return load16(base + e0 * (F32 ? 4 : 2));
            const uint32_t none = F32 ? 0xff800000u : 0xff80ff80u;
            uint32_t w[4] = {none, none, none, none};
            if (x < nv) {
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
            }
            return make_uint4(w[0], w[1], w[2], w[3]);
        };
        auto load = [&](uint4 (&v)[kVecs], int32_t t) {
            const int32_t x = t * kTile + tid;
            if (t * kTile >= whole0 && t * kTile + kTile <= whole1) {
                const char* at = base + ((int64_t)x * VE - shift) * (F32 ? 4 : 2);
#pragma unroll
                for (int j = 0; j < kVecs; ++j) v[j] = load16(at + j * kScan * 16);
            } else {
#pragma unroll
                for (int j = 0; j < kVecs; ++j) v[j] = vector(x + j * kScan);
            }
        };
        uint4 v[kVecs];
        load(v, t0);  // (beside the row's score, not after it)
        bool bad;
        if (row_state(a, row, bad) != kRowLive) continue;
        if (tid == 0) s_n = s_hits = 0;

        auto word = [&](int i) {
            const uint4 q = v[i >> 2];
            return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
        };
        auto logit = [&](int e) {
            if (F32) return __uint_as_float(word(e));
            const uint32_t w = word(e >> 1);
            return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
        };
        float ref = -INFINITY, sum = 0.f;
        u64 bound = kNoKey;           // a candidate's key is larger
        float bound_x = -INFINITY;    // its logit: a candidate's is larger (tokens ascend, so an equal one is no better)
        float least_x = -INFINITY;    // a candidate's is at least this
        int count = 0;                // entries of the list when it was cut
        float tops4[kVecs], top;      // largest logits of a tile's vectors, and of all
        auto find_top = [&]() {
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                if (F32) {
                    tops4[j] = fmaxf(fmaxf(logit(4 * j), logit(4 * j + 1)), fmaxf(logit(4 * j + 2), logit(4 * j + 3)));
                } else {
                    __nv_bfloat162 m[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t w = word(4 * j + i);
                        m[i] = *reinterpret_cast<const __nv_bfloat162*>(&w);
                    }
                    m[0] = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
                    tops4[j] = fmaxf(__low2float(m[0]), __high2float(m[0]));
                }
            }
            top = fmaxf(fmaxf(tops4[0], tops4[1]), fmaxf(tops4[2], tops4[3]));
        };
        // Notes this thread's vectors that hold a candidate.  (Looking for it here would have a warp run
        // through its logits for the sake of one lane.)
        auto note = [&](int32_t t) {
            if (!(top > bound_x && top >= least_x)) return;
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
                if (tops4[j] > bound_x && tops4[j] >= least_x) {
                    const int at = atomicAdd(&s_hits, 1);
                    if (at < kHits) {
                        hits[at] = v[j];
                        numbers[at] = t * kTile + j * kScan + tid;
                    }
                }
        };
        // Takes the candidates out of the noted vectors, ranks them with the k best so far and keeps the
        // k best of all.  False, and nothing done, where there are more than `most`.
        int now = 0;  // which of best[] holds the list
        auto cut = [&](int most) {
            __syncthreads();
            const int noted = s_hits;
            if (noted > kHits) return false;
            for (int i = tid; i < noted; i += kScan) {
                const uint4 q = hits[i];
                const int32_t first = numbers[i] * VE - shift;
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const uint32_t w = (F32 ? e : e >> 1) == 0 ? q.x : (F32 ? e : e >> 1) == 1 ? q.y
                                       : (F32 ? e : e >> 1) == 2 ? q.z : q.w;
                    const float y = __uint_as_float(F32 ? w : e & 1 ? w & 0xffff0000u : w << 16);
                    if (y > bound_x && y >= least_x) {
                        const int at = atomicAdd(&s_n, 1);
                        if (at < kRoom) cand[at] = key_of(y, first + e);
                    }
                }
            }
            __syncthreads();
            const int fresh = s_n, n = count + fresh;
            if (fresh > most) return false;
            if (tid == 0) s_hits = 0;
            const u64* list = best[now];
            // (a short list's entries are compared by two or four lanes each)
            const int lanes = n <= kScan / 4 ? 4 : n <= kScan / 2 ? 2 : 1;
            for (int i = tid / lanes; i < ((n + 31) & ~31); i += kScan) {
                const u64 x = i < count ? list[i] : cand[min(i - count, kRoom - 1)];
                int r = 0;
                for (int j = tid & (lanes - 1); j < count; j += lanes) r += list[j] > x;
#pragma unroll 4
                for (int j = tid & (lanes - 1); j < fresh; j += lanes) r += cand[j] > x;
                if (lanes > 1) r += __shfl_xor_sync(0xffffffffu, r, 1);
                if (lanes > 2) r += __shfl_xor_sync(0xffffffffu, r, 2);
                if (i < n && r < k) best[now ^ 1][r] = x;
            }
            __syncthreads();
            if (tid == 0) s_n = 0;  // (appended to after the next call's first barrier only)
            now ^= 1;
            count = min(n, k);
            if (count == k) {
                bound = best[now][k - 1];
                bound_x = unordered((uint32_t)(bound >> 32));
            }
            least_x = -INFINITY;
            return true;
        };
        // Tiles ta .. tb once more, from the list of the last cut.  Where more threads than places
        // hold a logit above the bound, the k-th largest of the threads' largest keys is a better one:
        // k keys reach it, and at most k threads hold any that do.
        auto again = [&](int32_t ta, int32_t tb) {
#pragma unroll 1
            for (int32_t t = ta; t < tb; ++t) {
                load(v, t);
                find_top();
                __syncthreads();
                if (tid == 0) s_n = s_tops = s_hits = 0;
                const int above = __syncthreads_count(top > bound_x);
                u64 least = bound + 1;
                if (above > k) {
                    u64 mine = 0;
                    if (top > bound_x) {
                        int32_t at = 0;
#pragma unroll
                        for (int e = E - 1; e >= 0; --e) at = logit(e) == top ? e : at;
                        mine = key_of(top, (t * kTile + (at / VE) * kScan + tid) * VE - shift + at % VE);
                    }
                    int ahead = 0;
#pragma unroll 1
                    for (int o = 1; o < 32; ++o) ahead += __shfl_xor_sync(0xffffffffu, mine, o) > mine;
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
                if (top > bound_x && ordered(top) >= (uint32_t)(least >> 32)) {
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const u64 key = key_of(logit(e), (t * kTile + (e / VE) * kScan + tid) * VE - shift + e % VE);
                        if (logit(e) > bound_x && key >= least) cand[atomicAdd(&s_n, 1)] = key;
                    }
                }
                cut(kRoom);
            }
        };
        int32_t from = t0, goal = t0 + 1;  // first tile of the run, and where it ends
        for (int32_t t = t0; t < t1; ++t) {
            find_top();
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
                    const float2 y = __fmul2_rn(__fadd2_rn(make_float2(logit(e), logit(e + 1)), n2), c2);
                    part2[(e >> 1) & 1] = __fadd2_rn(part2[(e >> 1) & 1], make_float2(ex2_of(y.x), ex2_of(y.y)));
                }
                sum += (part2[0].x + part2[1].x) + (part2[0].y + part2[1].y);
            }
            if (t == t0) {
                const int group = k <= 8 ? 32 : k <= 16 ? 16 : k <= 32 ? 8 : 4;  // threads
                float x = top == top ? top : -INFINITY;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {  // the largest of a group, then the smallest of the groups
                    const float y = __shfl_xor_sync(0xffffffffu, x, o);
                    x = o < group ? fmaxf(x, y) : fminf(x, y);
                }
                if (lane == 0) sm_ref[warp] = x;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < kScan / 32; ++w) x = fminf(x, sm_ref[w]);
                least_x = x;
            }
            note(t);
            // (Warps are at different tiles, so others compute while one waits; a second tile in registers
            // was slower, 71 against 65 us.)
            if (t + 1 < t1) load(v, t + 1);
            if (t + 1 == goal || t + 1 == t1) {
                if (!cut(kPlenty)) {
                    again(from, t + 1);
                    if (t + 1 < t1) load(v, t + 1);
                }
                from = t + 1;
                goal = t0 + 4 * (goal - t0);
            }
        }
        // ---- the part's sum, two floats wide over the threads, and its list
        float r = ref;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, o));
        float hi = ref == -INFINITY ? sum : sum * ex2_of((ref - r) * kC), lo = 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            add_exact(hi, lo, __shfl_xor_sync(0xffffffffu, hi, o), __shfl_xor_sync(0xffffffffu, lo, o));
        if (lane == 0) {
            sm_ref[warp] = r;
            sm_hi[warp] = hi;
            sm_lo[warp] = lo;
        }
        __syncthreads();
        const int64_t at = row * a.parts + part;
        if (tid == 0) {
            float rr = sm_ref[0];
#pragma unroll
            for (int w = 1; w < kScan / 32; ++w) rr = fmaxf(rr, sm_ref[w]);
            float h = 0.f, l = 0.f;
#pragma unroll
            for (int w = 0; w < kScan / 32; ++w) {
                const float f = sm_ref[w] == -INFINITY ? 1.f : ex2_of((sm_ref[w] - rr) * kC);
                add_exact(h, l, f * sm_hi[w], f * sm_lo[w]);
            }
            a.heads[at] = PartHead{h, l, rr, 0};
        }
        if (tid < k) a.lists[at * k + tid] = tid < count ? best[now][tid] : 0;
        __syncthreads();  // the next row's piece may write what this one reads
    }
}

// One group a CTA: every row's logarithm from its parts, then the best candidates of all lists.
// 64-bit arithmetic is slow here (two operations a clock and SM), so candidates are first judged by
// an interval around their rank in fp32: what k others are surely above is dropped (few candidates:
// each counts the others; many: the k-th largest lower end is bracketed by halving), and the rest is
// ranked in 64 bits.
// EACH: candidates of a thread.  (One where they suffice: this code runs once, and waits for its
// instructions more than for anything else.)
template <int EACH>
__global__ void __launch_bounds__(kJoin) join_kernel(const SelectArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ double add[kMaxBeams];  // what a row adds to its logits
    __shared__ double norm[kMaxBeams];
    __shared__ float add_f[kMaxBeams], norm_f[kMaxBeams], refs[kMaxBeams];
    __shared__ float sums[kMaxBeams], rests[kMaxBeams];
    __shared__ int state[kMaxBeams], cuts[kMaxBeams];
    __shared__ int s_count[3], s_kept;
    __shared__ uint32_t s_max;
    wait_previous();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
    const int64_t row0 = (int64_t)blockIdx.x * a.beams;
    const int k = a.k, parts = a.parts, total = a.beams * parts * k;
    u64* rank = reinterpret_cast<u64*>(smem);              // [total]: in the order of the ranks
    u64* keys = rank + total;                              // [total]
    int* from = reinterpret_cast<int*>(keys + total);      // [total]
    float* low = reinterpret_cast<float*>(smem);           // [total], before the ranks
    bool bad = false;
    int st = kRowNone;
    float score = 0.f, weight = 1.f;
    if (tid < a.beams) {
        st = row_state(a, row0 + tid, bad);
        score = a.scores[row0 + tid];
        if (a.norms) weight = a.norms[row0 + tid];
    }
    // this thread's candidates: entry i % k of list i / k
    u64 mine[EACH];
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        const int i = e * threads + tid;
        mine[e] = i < total ? a.lists[row0 * parts * k + i] : 0;
    }
    // parts that row b was cut into
    auto parts_here = [&](int b) {
        if (a.whole) return a.whole;
        const int64_t first = (row0 + b) * a.tiles;
        return (int)(quotient(first + a.tiles - 1, a.per) - quotient(first, a.per)) + 1;
    };
    for (int b = warp; b < a.beams; b += threads / 32) {
        const PartHead* h = a.heads + (row0 + b) * parts;
        const int cut = parts_here(b);
        float r = -INFINITY;
        for (int p = lane; p < cut; p += 32) r = fmaxf(r, h[p].ref);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, o));
        float hi = 0.f, lo = 0.f;
        for (int p = lane; p < cut; p += 32) {
            const float f = h[p].ref == -INFINITY ? 1.f : ex2_of((h[p].ref - r) * kC);
            add_exact(hi, lo, f * h[p].hi, f * h[p].lo);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            add_exact(hi, lo, __shfl_xor_sync(0xffffffffu, hi, o), __shfl_xor_sync(0xffffffffu, lo, o));
        if (lane == 0) {
            cuts[b] = cut;
            refs[b] = r;
            sums[b] = hi;
            rests[b] = lo;
        }
    }
    if (tid < 3) s_count[tid] = 0;
    if (tid == 0) s_kept = s_max = 0;
    __syncthreads();
    if (tid < a.beams) {
        double lse = 0;
        if (st == kRowLive) {
            float s = sums[tid];
            if (!(s - s == 0.f)) {  // a NaN or +inf among the logits
                bad = true;
                st = kRowNone;
            } else if (s == 0.f) {  // nothing above -inf
                st = kRowNone;
            } else {
                // ln(s + rest), s = m 2^e: a float's logarithm of m near 1 is off by 3e-8 at most, which the
                // logarithm of s itself would not be
                int e;
                const float rest = rests[tid] / s;
                s = frexpf(s, &e);
                if (s < 0.70710678f) {
                    s *= 2.f;
                    --e;
                }
                lse = (double)refs[tid] + (double)e * 0.6931471805599453 + (double)(logf(s) + rest);
            }
        }
        if (bad) raise_status(a.status, kErrLogits);
        state[tid] = st;
        add[tid] = (double)score - lse;
        add_f[tid] = (float)add[tid];
        norm_f[tid] = weight;
        norm[tid] = (double)weight;
    }
    __syncthreads();
    auto score_of = [&](int b, u64 key) {
        return state[b] == kRowDone ? add[b] : add[b] + (double)unordered((uint32_t)(key >> 32));
    };
    // the interval of a candidate's rank: four roundings of fp32 on either side
    float up[EACH];
    uint32_t lows[EACH];
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        const int i = e * threads + tid;
        up[e] = -INFINITY;
        lows[e] = 0;
        if (i < total) {
            const int list = i / k, b = list / parts;
            const bool done = state[b] == kRowDone && i == b * parts * k;
            if (done || (state[b] == kRowLive && list - b * parts < cuts[b] && mine[e] != 0)) {
                const float x = done ? 0.f : unordered((uint32_t)(mine[e] >> 32));
                const float y = (add_f[b] + x) * norm_f[b];
                const float err = (fabsf(add_f[b]) + fabsf(x)) * norm_f[b] * 2.4e-7f + 1e-37f;
                // (a score that fp32 rounds to -inf, or that its norm takes there, is no candidate's)
                if (y > -3.4e38f || ((float)score_of(b, mine[e]) != -INFINITY &&
                                     (float)(score_of(b, mine[e]) * norm[b]) != -INFINITY)) {
                    up[e] = fmaxf(y + err, -3.4028234e38f);
                    lows[e] = ordered(fmaxf(y - err, -3.4028234e38f));
                }
            }
            if (total <= kFewCandidates) low[i] = lows[e] ? unordered(lows[e]) : -INFINITY;
        }
    }
    uint32_t keep = 1;  // order of the upper end that a kept candidate has at least
    bool kept[EACH];
    int n = 0;
    if (total <= kFewCandidates) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            kept[e] = lows[e] != 0;
            if (!kept[e]) continue;
            int surely = 0;
#pragma unroll 8
            for (int j = 0; j < total; ++j) surely += low[j] > up[e];
            kept[e] = surely < k;
        }
        __syncthreads();
    } else {
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < EACH; ++e) top = max(top, lows[e]);
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) atomicMax(&s_max, top);
        __syncthreads();
        top = s_max;
        int round = 0;
        auto reaching = [&](uint32_t x) {  // candidates whose lower end is x in order at least
            int m = 0;
#pragma unroll
            for (int e = 0; e < EACH; ++e) m += lows[e] >= x;
            m = __reduce_add_sync(0xffffffffu, m);
            const int now = round % 3;
            if (lane == 0 && m) atomicAdd(&s_count[now], m);
            if (tid == 0) s_count[(now + 1) % 3] = 0;
            __syncthreads();
            ++round;
            return s_count[now];
        };
        // k candidates or all there are reach lo, fewer than k reach hi: from the largest down in
        // growing steps, then by halves, until not many more than k are left
        uint32_t lo = top, hi = top + 1, step = 1u << 20;
        int m = reaching(lo);
        while (m < k && lo > 1) {
            hi = lo;
            lo = lo > step ? lo - step : 1;
            step *= 2;
            m = reaching(lo);
        }
        while (m > k + 32 && hi - lo > 1) {
            const uint32_t mid = lo + (hi - lo) / 2;
            const int c = reaching(mid);
            if (c >= k) {
                lo = mid;
                m = c;
            } else {
                hi = mid;
            }
        }
        keep = lo;
#pragma unroll
        for (int e = 0; e < EACH; ++e) kept[e] = lows[e] != 0 && ordered(up[e]) >= keep;
    }
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        if (!kept[e]) continue;
        const int b = (e * threads + tid) / k / parts, at = atomicAdd(&s_kept, 1);
        const u64 key = state[b] == kRowDone ? 0 : mine[e];
        // (64-bit floats in the order of whole numbers, whose comparison is cheap; -0 is 0)
        const u64 bits = (u64)__double_as_longlong(score_of(b, key) * norm[b] + 0.0);
        rank[at] = bits >> 63 ? ~bits : bits | (u64)1 << 63;
        keys[at] = key;
        from[at] = b;
    }
    __syncthreads();
    n = s_kept;
    // larger score first, then the lower beam, then the larger logit, then the lower token
    const int64_t out = (int64_t)blockIdx.x * k;
    for (int i = tid; i < n; i += threads) {
        const u64 x = rank[i], key = keys[i];
        const int b = from[i];
        int r = 0;
        for (int j = 0; j < n; ++j) {
            const u64 y = rank[j];
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
    for (int i = n + tid; i < k; i += threads) {  // fewer candidates than places
        a.out_scores[out + i] = -INFINITY;
        a.out_beams[out + i] = a.out_tokens[out + i] = -1;
        if (a.out_finished) a.out_finished[out + i] = 0;
    }
}

// No more candidates of a group than the join's threads hold.
int64_t parts_most(int32_t beams, int32_t k) { return (int64_t)kJoin * kJoinEach / ((int64_t)beams * k); }

// How the rows' tiles are cut: tiles of a CTA, room for a row's parts, CTAs of a row or 0.
struct Cut {
    int64_t tiles, per, parts, whole;
};
// A piece of a row costs about four tiles more than it has, so rows are cut into equal parts of
// their own unless that leaves the last round of CTAs too empty (512 rows of 16 tiles: 42 us a CTA
// a row, 48 in 581 pieces of the line, 1.9 rows each; 120 rows of 13: 15.5 and 19.9 us).
Cut cut_of(int64_t rows, int32_t beams, int32_t k, int64_t vectors) {
    Cut c;
    c.tiles = (vectors + kTile - 1) / kTile;
    const int64_t most = parts_most(beams, k);
    int64_t parts = rows < kTargetCtas ? kTargetCtas / rows : 1;
    parts = parts < most ? parts : most;
    parts = parts < c.tiles ? parts : c.tiles;
    c.per = (c.tiles + parts - 1) / parts;
    c.parts = c.whole = (c.tiles + c.per - 1) / c.per;
    const int64_t rounds = (rows * c.whole + kTargetCtas - 1) / kTargetCtas;
    const int64_t line = (rows * c.tiles + kTargetCtas - 1) / kTargetCtas;
    if (rounds * (c.per + kPieceCost) <= line + kPieceCost * (line / c.tiles + 2)) return c;
    // (a row may touch one piece more than it fills)
    c.whole = 0;
    for (c.per = line;; ++c.per) {
        c.parts = (c.tiles + c.per - 2) / c.per + 1;
        if (c.parts <= most) return c;
    }
}

int64_t vectors_of(int32_t vocab, bool f32) {  // of a row that starts anywhere
    const int ve = f32 ? 4 : 8;
    return ((int64_t)vocab + ve - 1 + ve - 1) / ve;
}

// Parts of a row that the workspace has room for: the most that any number of rows is cut into (one for each
// tile at most), so that a workspace serves every smaller number of groups, whose rows have more parts each.
int64_t parts_room(int32_t beams, int32_t k, int32_t vocab) {
    const int64_t most = parts_most(beams, k), tiles = (vectors_of(vocab, true) + kTile - 1) / kTile;
    return most < tiles ? most : tiles;
}

// ---------------------------------------------------------------- reordering

constexpr int kMove = 256;            // threads of a CTA
constexpr int kStage = 8192;          // bytes of a warp's staging buffer
constexpr int kLaunchCaches = 64, kLaunchStates = 16;
constexpr int kPiece = 8192;          // bytes of a row that a warp takes at a time, at most

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
            if (a.lens[row0 + tid] != len || len < 0) s_bad = 1;
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
    // A group whose lengths differ, or need a page past its table, is left as it was.
    const int bad = s_bad ? kErrLength : a.lens && full + (part > 0) > a.max_pages ? kErrPage : 0;
    if (bad) {
        if (tid == 0 && a.tell && blockIdx.y == 0) raise_status(a.status, bad);
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
                if (wide) {
                    uint4* out = reinterpret_cast<uint4*>(to);
                    const uint4* in = reinterpret_cast<const uint4*>(got);
                    int i = lane;
                    for (; i + 96 < m; i += 128) {  // (four at a time: one by one they wait for shared memory)
                        const uint4 a0 = in[i], a1 = in[i + 32], a2 = in[i + 64], a3 = in[i + 96];
                        out[i] = a0;
                        out[i + 32] = a1;
                        out[i + 64] = a2;
                        out[i + 96] = a3;
                    }
                    for (; i < m; i += 32) out[i] = in[i];
                } else
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
    return 256 + (size_t)rows * parts_room(beams, num_out, vocab) * (sizeof(PartHead) + 8 * (size_t)num_out);
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
    const Cut c = cut_of(rows, beams, num_out, vectors);
    a.tiles = (int32_t)c.tiles;
    a.per = (int32_t)c.per;
    a.parts = (int32_t)c.parts;
    a.heads = reinterpret_cast<PartHead*>(workspace);
    a.lists = reinterpret_cast<u64*>(a.heads + rows * a.parts);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const size_t smem = (size_t)beams * a.parts * num_out * 20;
    a.whole = (int32_t)c.whole;
    const dim3 grid((unsigned)(c.whole ? rows * c.whole : (rows * c.tiles + c.per - 1) / c.per));
    cudaError_t e = f32 ? launch_after(scan_kernel<true>, grid, kScan, 0, st, a)
                        : launch_after(scan_kernel<false>, grid, kScan, 0, st, a);
    if (e == cudaSuccess) {
        const int total = (int)(beams * c.parts * num_out);
        const dim3 groups((unsigned)num_groups);
        if (total <= kJoin) {
            const int threads = total <= 64 ? 64 : (total + 31) / 32 * 32;  // (a thread for every beam)
            e = launch_after(join_kernel<1>, groups, threads, smem, st, a);
        } else {
            e = cudaFuncSetAttribute(join_kernel<kJoinEach>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kJoin * kJoinEach * 20);
            if (e == cudaSuccess) e = launch_after(join_kernel<kJoinEach>, groups, kJoin, smem, st, a);
        }
    }
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
    // What is listed twice would be moved twice, by warps that do not meet; what the call reads must not move.
    const bool scales = num_caches > 0 && c0->kind == PVA_CACHE_INT4, pages = num_caches > 0 && c0->num_pages > 0;
    const int arrays = pages ? (scales ? 4 : 2) : 0;
    struct Arrays {
        const void* at[4];
    };
    auto arrays_of = [&](int32_t i) {
        const pva_cache_desc& c = caches[i];
        return Arrays{{c.k_pages, c.v_pages, c.k_scales, c.v_scales}};
    };
    const void* const given[3] = {parents, num_caches > 0 ? kv_lens : nullptr, num_caches > 0 ? page_table : nullptr};
    auto is_given = [&](const void* x) { return x == given[0] || x == given[1] || x == given[2]; };
    if (given[2] && (given[2] == given[0] || given[2] == given[1])) return PVA_ERR_INVALID_ARG;
    for (int32_t i = 0; i < num_caches && arrays > 0; ++i) {
        const Arrays x = arrays_of(i);
        for (int k = 0; k < arrays; ++k) {
            if (is_given(x.at[k])) return PVA_ERR_INVALID_ARG;
            for (int m = 0; m < k; ++m)
                if (x.at[k] == x.at[m]) return PVA_ERR_INVALID_ARG;
        }
        for (int32_t j = 0; j < i; ++j) {
            const Arrays y = arrays_of(j);
            bool same = false;
            for (int k = 0; k < arrays; ++k)
                for (int m = 0; m < arrays; ++m) same |= x.at[k] == y.at[m];
            if (same) return PVA_ERR_INVALID_ARG;
        }
    }
    for (int32_t i = 0; i < num_states; ++i) {
        const void* x = states[i].data;
        if (states[i].row_bytes == 0) continue;
        if (is_given(x)) return PVA_ERR_INVALID_ARG;
        for (int32_t j = 0; j < i; ++j)
            if (x == states[j].data && states[j].row_bytes > 0) return PVA_ERR_INVALID_ARG;
        for (int32_t j = 0; j < num_caches; ++j) {
            const Arrays y = arrays_of(j);
            for (int k = 0; k < arrays; ++k)
                if (x == y.at[k]) return PVA_ERR_INVALID_ARG;
        }
    }
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
