// cache_attn.cu -- attention of new tokens over the paged cache.
//
// For every new token (row) of a sequence, over the keys j it may see,
//   s_j = scale q.k_j,  O = sum_j e^(s_j) v_j / sum_j e^(s_j),  LSE = ln sum_j e^(s_j).
// A row and its head's group share one kv head, so a key and value row is read
// once for group * new tokens rows: a few multiply-adds a byte, bounded by HBM.
//
// The products run transposed on m16n8k16 tiles, S^T = K Q^T and O^T = V^T P^T:
// keys (or dims) fill the 16 rows of a tile, query rows its 8 columns, so a
// decoding step of up to 8 rows a kv head (one token, groups up to 8) wastes no
// half of every product, of the softmax and of the registers on absent rows.  More
// rows of a bf16 cache take two column tiles on the same K and V fragments, 16 rows an
// item; four column tiles spilled and were slower than reading K and V again from L2
// (32 rows of 128 dims, 64 contexts of 4000 .. 9001 keys: 567 us against 305 us).
// (tcgen05 tiles start at 64 rows of D and take their operands from shared memory,
// where 4-bit rows would have to be written back expanded.)
//
// Each warp streams its own tiles of keys through a private ring of cp.async
// stages: no barrier inside a context, running maximum and sum in registers.
// The warps of a CTA take turns over the blocks of one (sequence, kv head, row
// block) item and join at its end in shared memory.  All items together form one
// line of units, a unit being a block of keys or an item's fixed cost, cut into
// equal pieces over the CTAs; an item cut by a piece's end leaves partial sums in
// the workspace, and a second, dependent kernel joins them in a fixed order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "../../include/pva.h"
#include "cache.cuh"

namespace pva {
namespace {

constexpr int kMaxCtas = 512;   // pieces the workspace has room for
constexpr int64_t kSpreadRows = 1024;  // rows (tokens * heads) up to which the join spreads a row
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum moves only when a tile exceeds it by 2^8: weights stay below
// 2^8, sums far inside fp32's range, and the accumulators are rescaled rarely.
constexpr float kSlack = 8.f;

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
    uint32_t num_pages, page_bytes;  // page_bytes: codes or values of a page, one of K and V
    float c;      // softmax scale * log2(e), times 2^69 with 4 bits (whose scores carry 2^-69)
    float slack;  // kSlack / c
};

// Shape of a variant: warps a CTA, keys a step, ring stages, columns of the join buffer.
template <int D, int KIND, int NT, bool H>
struct Shape {
    static constexpr bool kInt4 = KIND == PVA_CACHE_INT4;
    static constexpr int kWarps = 4;
    static_assert(!kInt4 || NT == 1, "4 bits take one column tile");
    static constexpr int kKeys = kInt4 ? 64 : 16 * (128 / D);
    static constexpr int kStages = kInt4 ? 2 : 3;
    static constexpr int kCtas = kInt4 ? 3 : 2;  // resident on an SM
    static constexpr int kCols = 8 * NT;     // columns of S^T
    static constexpr int R = H ? 4 : kCols;  // rows of an item
    static constexpr int kThreads = 32 * kWarps;
    // Ring sizes: bf16 16 KB (128 dims) a step and warp in flight at 8 warps an SM keep HBM
    // busy (98% of the copy rate on a batch of 64 contexts).  4 bits are bounded by issue slots
    // and the integer pipe, not by HBM: 64 keys a step spread a step's fixed instructions (16
    // keys: 143 us, 32: 91 us, 64: 84 us on 3 contexts of 131072, with weights of 8 bits), and
    // twelve warps with two stages beat eight (84 -> 82 us).  At 128 dims their 168 registers
    // spill 28 (up to four rows) and 48 bytes.
    // An item's fixed cost (queries, join, results) in blocks of keys.  bf16: 256 contexts of
    // 10 .. 1000 tokens 61.6 us at 1, 53.7 us at 3; 4 bits, whose block is four times as
    // long: 96 contexts of 200 .. 16000 with their append 71.1 us at 0, 60.3 at 1, 61.4 at 2.
    static constexpr int kFixed = kInt4 ? 1 : 3;
    static constexpr int kBlock = kWarps * kKeys;  // keys of a unit
    static constexpr int kRowBytes = kInt4 ? D / 2 : 2 * D;
    static constexpr int kGroups = D / 64;
    static constexpr int kScaleBytes = kInt4 ? 4 * kGroups : 0;
    static constexpr int kStageBytes = kKeys * 2 * (kRowBytes + kScaleBytes);
    static constexpr int kTiles = D / 16;  // 16-dim tiles of O^T
    // Dims that the warps' sums are joined by at a time, in the stage that each has just read.
    static constexpr int kJoinDims = NT == 1 ? D : 64;
    static constexpr int kJoinPitch = kJoinDims + 4;
    static_assert(kCols * kJoinPitch * 4 <= kStageBytes, "the sums fit a stage");
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kMeta = kWarps * kStages * 48;
    static constexpr int kJoin = kWarps * (2 * kCols + 4) * 4;
    static constexpr int kSmem = kRing + kMeta + kJoin;
};

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
        if (bad || (kv < s.n && (a.s.cu || kv != 0))) raise_status(a.s.status, kErrLength);
        if (s.n > 0 && kv > room) raise_status(a.s.status, kErrPage);
    }
    const int32_t kvp = max(kv, 0);
    s.pos0 = kvp - s.n;
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

template <int N>
struct Const {
    static constexpr int value = N;
};

// Steps: first and last of an item, nothing to read, the item is all this piece's, some
// key of the tile is not for every row.
enum { kFirst = 1, kLast = 2, kEmpty = 4, kWhole = 8, kPartial = 16 };

// What a step's consumer needs beside its flags: written for first, last and partial steps.
struct Meta {
    int32_t key0, vlo, vhi, missing;  // partial: keys vlo .. vhi are there, bit x: no page for keys 16x ..
    int32_t row0, rows, pos0, rb;     // first token, group * new tokens, first position, row block
    int32_t kvh, slot, pad[2];
};

template <int D, int KIND, int NT, bool H>
__global__ void __launch_bounds__(Shape<D, KIND, NT, H>::kThreads, Shape<D, KIND, NT, H>::kCtas)
    attn_kernel(const AttnArgs a) {
    using Sh = Shape<D, KIND, NT, H>;
    constexpr int R = Sh::R, W = Sh::kWarps, KS = Sh::kKeys, S = Sh::kStages, SUB = KS / 16;
    constexpr int HN = H ? 2 : 1, ST = SUB / HN;  // tiles of keys that share the columns, sets of scores
    constexpr int C = Sh::kCols;
    constexpr int G = Sh::kGroups, T = Sh::kTiles, BLOCK = Sh::kBlock, ROWB = Sh::kRowBytes;
    constexpr bool INT4 = Sh::kInt4;
    extern __shared__ __align__(128) uint8_t smem[];
    wait_previous();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    uint8_t* ring = smem + warp * S * Sh::kStageBytes;
    Meta* meta = reinterpret_cast<Meta*>(smem + Sh::kRing) + warp * S;
    float* join_m = reinterpret_cast<float*>(smem + Sh::kRing + Sh::kMeta);  // [W][C]
    float* join_l = join_m + W * C;                                          // [W][C]
    int* join_at = reinterpret_cast<int*>(join_l + W * C);                   // [W]: stage of the sums
    // ---- plan: this CTA's piece [u0, u1) of the line and the sequence it starts in.
    // Every thread sums a run of sequences; a scan over the threads gives each run's
    // first unit.
    int32_t b, it;       // sequence, item inside it
    int64_t u0, u1, ub;  // ub: first unit of sequence b
    {
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
        if (u0 >= total) return;
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
    }

    // ---- cursor over this warp's steps
    const int32_t own = warp * KS;      // this warp's keys inside a block
    const bool one_page = (1 << a.s.page_shift) >= KS;
    SeqInfo sq = seq_info<Sh>(a, b, false);
    const int32_t* pages = a.s.page_table + b * a.s.table_stride;
    int32_t len = Sh::kFixed + sq.nb;
    it = (int32_t)quotient(u0 - ub, len);
    int32_t rb = it / a.hkv, kvh = it - rb * a.hkv;
    int64_t ui = ub + (int64_t)it * len;  // first unit of the item
    int32_t key = 0, kend = 0;            // the pending step's first key; where the item's steps end
    int32_t rlo = 0, rhi = 0;             // keys that some row of the block may see
    int32_t alo = 0, ahi = 0;             // keys that every row of it sees
    int32_t slot = 0, flags_next = 0;
    uint32_t page = 0;     // lane x < SUB: of the pending step's keys 16x ..
    bool more = true;      // the piece may have another step
    bool pending = false;  // a step waits to be copied
    bool fresh = true;  // the cursor stands before its first item

    // The item at the cursor: false where this piece has no block of it.
    auto open_item = [&]() -> bool {
        const int32_t i0 = (int32_t)((int64_t)rb * R / a.group);
        const int32_t i1 = (int32_t)min(((int64_t)rb * R + R - 1) / a.group, (int64_t)sq.n - 1);
        rlo = alo = 0;
        if (a.window > 0) {
            rlo = (int32_t)max((int64_t)sq.pos0 + i0 - a.window + 1, (int64_t)0);
            alo = (int32_t)max((int64_t)sq.pos0 + i1 - a.window + 1, (int64_t)0);
        }
        rhi = min(sq.pos0 + i1 + 1, sq.khi);
        ahi = min(sq.pos0 + i0 + 1, sq.khi);
        if (sq.nb == 0) {
            key = kend = 0;
            flags_next = kFirst | kLast | kEmpty | kWhole;
            return u0 <= ui;
        }
        const int64_t first = ui + Sh::kFixed, last = ui + len;
        const int32_t t0 = (int32_t)max(u0 - first, (int64_t)0);
        const int32_t t1 = (int32_t)(min(u1, last) - first);
        if (t1 <= t0) return false;
        flags_next = kFirst | (t0 == 0 && t1 == sq.nb ? kWhole : 0);
        slot = 2 * blockIdx.x + (t0 == 0 ? 1 : 0);
        // of blocks blo + t0 .. blo + t1, those whose keys of this warp the rows may see
        const int32_t ta = max(sq.blo + t0, rlo - own < KS ? 0 : (rlo - own - KS + BLOCK) / BLOCK);
        const int32_t tb = min(sq.blo + t1, rhi <= own ? 0 : (rhi - own + BLOCK - 1) / BLOCK);
        key = ta * BLOCK + own;
        kend = tb * BLOCK + own;
        if (ta >= tb) flags_next |= kLast | kEmpty;
        return true;
    };
    auto next = [&]() {
        pending = false;
        key += BLOCK;
        flags_next &= kWhole;
        if (key >= kend) {
            for (;;) {
                if (!fresh) {
                    ui += len;
                    if (++kvh == a.hkv) {
                        kvh = 0;
                        if (++rb == sq.nrb) {
                            rb = 0;
                            do {
                                if (++b >= a.s.num_seqs) {
                                    more = pending = false;
                                    return;
                                }
                                sq = seq_info<Sh>(a, b, false);
                            } while (sq.nrb == 0);
                            len = Sh::kFixed + sq.nb;
                            pages = a.s.page_table + b * a.s.table_stride;
                        }
                    }
                }
                fresh = false;
                if (ui >= u1) {
                    more = false;
                    return;
                }
                if (open_item()) break;
            }
        }
        pending = true;
        if (key >= kend) return;  // an empty step
        if (key + BLOCK >= kend) flags_next |= kLast;
        if (key < alo || key + KS > ahi) flags_next |= kPartial;
        const int32_t i = (key + 16 * min(lane, SUB - 1)) >> a.s.page_shift;
        page = lane < SUB && i < a.s.max_pages ? (uint32_t)pages[i] : ~0u;
    };
    // N * 16 keys from byte `off` of a page's K and V on, into tile x of a stage;
    // [vlo, vhi): rows of the first 16 that are there.
    auto copy = [&](auto tiles, uint32_t kd, int x, uint64_t off, int vlo, int vhi) {
        constexpr int N = decltype(tiles)::value;
        constexpr int CPR = ROWB / 16, PER = CPR / 2;  // 16-byte chunks: a row's, a lane's of 16 keys
        const uint8_t* ks = a.k_pages + off + lane * 16;
        const uint8_t* vs = a.v_pages + off + lane * 16;
        if (!INT4) {
            const int r0 = lane / CPR, ch = lane % CPR;
#pragma unroll
            for (int i = 0; i < N * PER; ++i) {
                const int r = i * (32 / CPR) + r0;
                const uint32_t to = (16 * x + r) * ROWB + ((ch ^ (r & 7)) << 4);
                // rows that are not there are filled with zeros: a weight of 0 must not meet a NaN
                const bool ok = N > 1 || (r >= vlo && r < vhi);
                cp16(kd + to, ok ? ks + i * 512 : a.k_pages, ok ? 16 : 0);
                cp16(kd + KS * ROWB + to, ok ? vs + i * 512 : a.v_pages, ok ? 16 : 0);
            }
        } else {
            // V: 16-byte chunks of a 128-byte line change places with the line's number, so that
            // the rows a warp reads at once lie in other banks
            const int sw = (lane & 7) ^ (2 * ((lane >> 3) & (D == 128 ? 3 : 1)));
            const uint32_t kt = kd + 16 * x * ROWB + lane * 16;
            const uint32_t vt = kd + (KS + 16 * x) * ROWB + ((lane & 24) + sw) * 16;
#pragma unroll
            for (int i = 0; i < N * PER; ++i) {
                cp16(kt + i * 512, ks + i * 512, 16);
                cp16(vt + i * 512, vs + i * 512, 16);
            }
            // scales, an eighth of the codes: of 16 keys (16 * N) kScaleBytes chunks, K's then V's
            constexpr int SC = Sh::kScaleBytes * N, HALF = SC < 16 ? SC : 16;
            const bool v = lane >= HALF;
            const int i0 = v ? lane - HALF : lane;
            const uint8_t* ss = (v ? a.v_scales : a.k_scales) + (off >> 3) + i0 * 16;
            const uint32_t st = kd + 2 * KS * ROWB + ((v ? KS : 0) + 16 * x) * Sh::kScaleBytes + i0 * 16;
            if (lane < 2 * HALF) {
#pragma unroll
                for (int i = 0; i < SC; i += HALF) cp16(st + i * 16, ss + i * 16, 16);
            }
        }
    };
    // Copies of the pending step into a stage.  Returns the step's flags.
    auto issue = [&](int stage) -> int32_t {
        const uint32_t kd = smem_addr(ring + stage * Sh::kStageBytes);
        int32_t flags = flags_next, missing = 0;
        if (!(flags & kEmpty)) {
            const uint32_t mask = (1u << a.s.page_shift) - 1;
            const uint32_t head = (uint32_t)kvh << a.s.page_shift;
            if (!__all_sync(0xffffffffu, lane >= SUB || page < a.num_pages)) flags |= kPartial;
            if (one_page && !(flags & kPartial)) {
                copy(Const<SUB>(), kd, 0,
                     (uint64_t)__shfl_sync(0xffffffffu, page, 0) * a.page_bytes + (head + (key & mask)) * ROWB, 0, 16);
            } else if (!(flags & kPartial)) {
#pragma unroll
                for (int x = 0; x < SUB; ++x)
                    copy(Const<1>(), kd, x,
                         (uint64_t)__shfl_sync(0xffffffffu, page, x) * a.page_bytes +
                             (head + ((key + 16 * x) & mask)) * ROWB, 0, 16);
            } else {
#pragma unroll 1
                for (int x = 0; x < SUB; ++x) {
                    const int32_t k = key + 16 * x;
                    const uint32_t p = __shfl_sync(0xffffffffu, page, x);
                    const int lo = max(rlo - k, 0), hi = min(rhi - k, 16);
                    const bool there = p < a.num_pages;
                    const uint64_t off = (uint64_t)p * a.page_bytes + (head + (k & mask)) * ROWB;
                    if (!there) {
                        missing |= 1 << x;
                        if (lane == 0 && lo < hi) raise_status(a.s.status, kErrPage);
                    }
                    if (!INT4 || there) copy(Const<1>(), kd, x, there ? off : 0, lo, there ? hi : 0);
                }
            }
        }
        if (lane == 0 && (flags & (kFirst | kLast | kPartial))) {
            Meta& m = meta[stage];
            *reinterpret_cast<int4*>(&m.key0) = make_int4(key, rlo, rhi, missing);
            *reinterpret_cast<int4*>(&m.row0) = make_int4(sq.row0, sq.n * a.group, sq.pos0, rb);
            *reinterpret_cast<int2*>(&m.kvh) = make_int2(kvh, slot);
        }
        return flags;
    };

    // ---- state of the item in hand
    // Scores stay as the products leave them; weights are 2^(c (s - m)) (4 bits: times 2^64),
    // base being m, or 0 as long as m is -inf.  The difference is taken first: c m is rounded to
    // its own last bit, which for scores past 2^30 is more than fp32's exponents hold.
    float o[NT][T][4], m_run[NT][2], base[NT][2], l_run[NT][2];
    float zs[INT4 ? G : 1][NT][2];     // 4 bits: sums of weight * middle of the group
    float vs[INT4 ? G : 1][NT][4];     // 4 bits: sums of the rounded weight * scale
    uint32_t qs[HN][NT];                 // 4 bits: sums of the query's dims of a group
    uint32_t qf[HN][NT][D / 16][2];
    int32_t pos[NT][2];

    // (scale, low) of a tile's keys g and g + 8
    auto scales = [&](uint32_t (&sc)[2][G], const uint8_t* at) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            if (D == 128) {
                const uint2 z = *reinterpret_cast<const uint2*>(at + 8 * y * Sh::kScaleBytes);
                sc[y][0] = z.x;
                sc[y][G - 1] = z.y;
            } else {
                sc[y][0] = *reinterpret_cast<const uint32_t*>(at + 8 * y * Sh::kScaleBytes);
            }
        }
    };

    // a slot of no token may hold anything: nothing of it goes into a product
    auto no_token = [&](uint32_t (&sc)[2][G], int32_t j, int32_t vlo, int32_t vhi, bool missing) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int gr = 0; gr < G; ++gr)
                sc[y][gr] = missing || j + 8 * y < vlo || j + 8 * y >= vhi ? 0u : sc[y][gr];
    };

    // Each turn copies step `step + S - 1` (the first turn finds the first step only), then
    // takes step `step`: one place for everything, since short contexts run through the code
    // once and wait for its instructions.
    int32_t queue[S];  // flags of the steps in flight
#pragma unroll
    for (int i = 0; i < S; ++i) queue[i] = 0;
    int issued = 0;
#pragma unroll 1
    for (int step = -S, stage = 0;; ++step, stage = stage + 1 == S ? 0 : stage + 1) {
        __syncwarp();  // the stage before this one is read
#pragma unroll
        for (int i = 0; i + 1 < S; ++i) queue[i] = queue[i + 1];
        if (pending) {
            queue[S - 1] = issue(stage == 0 ? S - 1 : stage - 1);
            ++issued;
        }
        cp_commit();
        if (more) next();
        if (step < 0) continue;
        if (step >= issued) break;
        const int32_t flags = queue[0];
        const uint8_t* buf = ring + stage * Sh::kStageBytes;
        const Meta& mt = meta[stage];
        if (flags & kFirst) {
            const int32_t row0 = mt.row0, rows = mt.rows, pos0 = mt.pos0, r0 = mt.rb * R;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < T; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
                m_run[nt][0] = m_run[nt][1] = -INFINITY;
                base[nt][0] = base[nt][1] = 0.f;
                l_run[nt][0] = l_run[nt][1] = 0.f;
                const int32_t r = r0 + (H ? g & 3 : 8 * nt + g);
                const int32_t tok = r / a.group;
                const __nv_bfloat16* q = a.q + (int64_t)(row0 + tok) * a.q_stride +
                                         (int64_t)(mt.kvh * a.group + r - tok * a.group) * D;
                const bool live = r < rows;
                if (!INT4) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            qf[0][nt][ks][e] =
                                live ? *reinterpret_cast<const uint32_t*>(q + 16 * ks + 8 * e + 2 * c) : 0u;
                } else {
#pragma unroll
                    for (int hh = 0; hh < HN; ++hh) qs[hh][nt] = 0;
                    // the dims in the order in which the codes of a row come out of their words
#pragma unroll
                    for (int gr = 0; gr < G; ++gr) {
                        float sum = 0.f;
#pragma unroll
                        for (int oc = 0; oc < 2; ++oc) {
                            constexpr float kUp60 = kUp64 / 16.f;  // meets 16 * code
                            const uint4 x = live ? *reinterpret_cast<const uint4*>(q + 64 * gr + 16 * c + 8 * oc)
                                                 : make_uint4(0, 0, 0, 0);
                            const uint32_t y[4] = {pack2(lo_f(x.x) * kUp64, hi_f(x.x) * kUp64),
                                                   pack2(lo_f(x.y) * kUp60, hi_f(x.y) * kUp60),
                                                   pack2(lo_f(x.z) * kUp64, hi_f(x.z) * kUp64),
                                                   pack2(lo_f(x.w) * kUp60, hi_f(x.w) * kUp60)};
#pragma unroll
                            for (int hh = 0; hh < HN; ++hh)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    qf[hh][nt][4 * gr + 2 * oc + i / 2][i % 2] = !H || (g >> 2) == hh ? y[i] : 0u;
                            sum += ((lo_f(x.x) + hi_f(x.x)) + (lo_f(x.y) + hi_f(x.y))) +
                                   ((lo_f(x.z) + hi_f(x.z)) + (lo_f(x.w) + hi_f(x.w)));
                        }
                        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                        sum *= 1.f / kUp69;
                        // in three bf16 parts that add up to fp32's bits, one for each of c = 0, 1, 2
#pragma unroll
                        for (int i = 0; i < 3; ++i) {
                            const float part = __bfloat162float(__float2bfloat16_rn(sum));
#pragma unroll
                            for (int hh = 0; hh < HN; ++hh)
                                if (c == i && (!H || (g >> 2) == hh))
                                    qs[hh][nt] |= (__float_as_uint(part) >> 16) << (16 * gr);
                            sum -= part;
                        }
                        zs[gr][nt][0] = zs[gr][nt][1] = 0.f;
#pragma unroll
                        for (int e = 0; e < 4; ++e) vs[gr][nt][e] = 0.f;
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    pos[nt][e] = pos0 + min(r0 + (H ? (2 * c + e) & 3 : 8 * nt + 2 * c + e), rows - 1) / a.group;
            }
        }
        cp_wait<S - 1>();
        __syncwarp();  // every lane's copies of this step are in
        if (!(flags & kEmpty)) {
            const bool partial = flags & kPartial;
            int32_t key0 = 0, vlo = 0, vhi = 0, missing = 0;
            if (partial) {
                const int4 m = *reinterpret_cast<const int4*>(&mt.key0);
                key0 = m.x;
                vlo = m.y;
                vhi = m.z;
                missing = m.w;
            }
            const uint32_t kb = smem_addr(buf), vb = kb + KS * ROWB;
            // Set z of scores: tile z of 16 keys; with H tile 2z in columns 0 .. 3 and tile 2z + 1 in
            // columns 4 .. 7, so that up to four rows leave no column of the softmax empty.  This
            // lane's columns belong to tile HN * z + mine.
            float s[ST][NT][4];
            uint32_t own_sc[INT4 ? ST : 1][2][G];
            const int mine = H ? c >> 1 : 0;
            // ---- S^T
#pragma unroll
            for (int z = 0; z < ST; ++z) {
                if (!INT4) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        uint32_t f[4];
                        const int r = lane & 15, ch = 2 * ks + (lane >> 4);
                        ldsm(f, kb + (16 * z + r) * ROWB + ((ch ^ (r & 7)) << 4));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (ks == 0) mma0(s[z][nt], f, qf[0][nt][ks][0], qf[0][nt][ks][1]);
                            else mma(s[z][nt], f, qf[0][nt][ks][0], qf[0][nt][ks][1]);
                        }
                    }
                } else {
                    float acc[G][NT][4];
#pragma unroll
                    for (int hh = 0; hh < HN; ++hh) {
                        const int x = HN * z + hh;
                        uint32_t w[2][2 * G], sc[2][G];
                        const uint8_t* kr = buf + (16 * x + g) * ROWB + c * (ROWB / 4);
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            if (D == 128) {
                                const uint4 v = *reinterpret_cast<const uint4*>(kr + 8 * y * ROWB);
                                w[y][0] = v.x;
                                w[y][1] = v.y;
                                w[y][2 * G - 2] = v.z;
                                w[y][2 * G - 1] = v.w;
                            } else {
                                const uint2 v = *reinterpret_cast<const uint2*>(kr + 8 * y * ROWB);
                                w[y][0] = v.x;
                                w[y][1] = v.y;
                            }
                        }
#pragma unroll
                        for (int gr = 0; gr < G; ++gr)
#pragma unroll
                            for (int oc = 0; oc < 2; ++oc)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const uint32_t w0 = w[0][G * oc + gr] >> (8 * h), w1 = w[1][G * oc + gr] >> (8 * h);
                                    const uint32_t f[4] = {low_codes(w0), low_codes(w1), high_codes(w0),
                                                           high_codes(w1)};
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt) {
                                        const uint32_t* q2 = qf[hh][nt][4 * gr + 2 * oc + h];
                                        if (hh == 0 && oc == 0 && h == 0) mma0(acc[gr][nt], f, q2[0], q2[1]);
                                        else mma(acc[gr][nt], f, q2[0], q2[1]);
                                    }
                                }
                        // s = sum over groups of scale * (q . codes) + low * (sum of q); the second by
                        // one more product, of the lows of a key with the parts of the sums
                        scales(sc, buf + 2 * KS * ROWB + (16 * x + g) * Sh::kScaleBytes);
                        if (partial) no_token(sc, key0 + 16 * x + g, vlo, vhi, missing >> x & 1);
                        const uint32_t lows[4] = {G == 2 ? __byte_perm(sc[0][0], sc[0][G - 1], 0x7632) : sc[0][0] >> 16,
                                                  G == 2 ? __byte_perm(sc[1][0], sc[1][G - 1], 0x7632) : sc[1][0] >> 16,
                                                  0u, 0u};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (hh == 0) mma0(s[z][nt], lows, qs[hh][nt], 0u);
                            else mma(s[z][nt], lows, qs[hh][nt], 0u);
                        }
                        if (H && hh == 0) {
                            own_sc[z][0][0] = sc[0][0];
                            own_sc[z][0][G - 1] = sc[0][G - 1];
                            own_sc[z][1][0] = sc[1][0];
                            own_sc[z][1][G - 1] = sc[1][G - 1];
                        } else {
#pragma unroll
                            for (int y = 0; y < 2; ++y)
#pragma unroll
                                for (int gr = 0; gr < G; ++gr)
                                    own_sc[z][y][gr] = !H || mine ? sc[y][gr] : own_sc[z][y][gr];
                        }
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int gr = 0; gr < G; ++gr) {
                            const float scl = lo_f(own_sc[z][y][gr]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    s[z][nt][2 * y + e] = fmaf(scl, acc[gr][nt][2 * y + e], s[z][nt][2 * y + e]);
                        }
                }
            }
            // ---- masks; has a score left the range of the running maximum?
            if (partial) {
#pragma unroll
                for (int z = 0; z < ST; ++z)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int x = HN * z + mine;
                            const int32_t j = key0 + 16 * x + g + 8 * (e >> 1), p = pos[nt][e & 1];
                            const bool ok = j >= vlo && j < vhi && j <= p && !(missing >> x & 1) &&
                                            (a.window <= 0 || p - j < a.window);
                            s[z][nt][e] = ok ? s[z][nt][e] : -INFINITY;
                        }
            }
            bool up = false;
            float mx[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[nt][e] = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
                    for (int z = 1; z < ST; ++z)
                        mx[nt][e] = fmaxf(mx[nt][e], fmaxf(s[z][nt][e], s[z][nt][2 + e]));
                    up |= mx[nt][e] > m_run[nt][e] + a.slack;
                }
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int d = H ? 2 : 4; d < 32; d <<= 1)  // (with H both halves of a row)
                            mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], d));
                        const float mn = fmaxf(m_run[nt][e], mx[nt][e]);
                        const float f = m_run[nt][e] == -INFINITY ? 0.f : ex2((m_run[nt][e] - mn) * a.c);
                        m_run[nt][e] = mn;
                        base[nt][e] = mn == -INFINITY ? 0.f : mn;
                        l_run[nt][e] *= f;
#pragma unroll
                        for (int i = 0; i < T; ++i) {
                            o[nt][i][e] *= f;
                            o[nt][i][2 + e] *= f;
                        }
                        if (INT4) {
#pragma unroll
                            for (int gr = 0; gr < G; ++gr) {
                                zs[gr][nt][e] *= f;
                                vs[gr][nt][e] *= f;
                            }
                        }
                    }
            }
            // ---- weights and O^T
#pragma unroll
            for (int z = 0; z < ST; ++z) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[z][nt][e] = ex2(fmaf(s[z][nt][e] - base[nt][e & 1], a.c, INT4 ? 64.f : 0.f));
                        l_run[nt][e & 1] += s[z][nt][e];
                    }
                if (!INT4) {
                    // the values are bf16, so the weights go in as the sum of two bf16 numbers: 16 of
                    // their bits (2^-17), and what a bf16 result loses is its own rounding (2^-8).  One
                    // bf16 number alone adds as much again; the second product hides behind HBM.
                    uint32_t p[NT][2], q[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float p0 = s[z][nt][2 * y], p1 = s[z][nt][2 * y + 1];
                            const uint32_t hi = pack2(p0, p1);
                            p[nt][y] = transpose8(hi);
                            q[nt][y] = transpose8(pack2(p0 - lo_f(hi), p1 - hi_f(hi)));
                        }
#pragma unroll
                    for (int i = 0; i < T; ++i) {
                        uint32_t f[4];
                        const int r = (lane & 7) + ((lane >> 4) << 3), ch = 2 * i + ((lane >> 3) & 1);
                        ldsm_t(f, vb + (16 * z + r) * ROWB + ((ch ^ (r & 7)) << 4));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            // The products round their sums towards 0: over a long context that would be a
                            // bias (64 contexts of 131072, values of mean 1: 2e-4 of the result).  So the products
                            // of 16 keys start from 0 and go onto the sums by additions, which round to nearest.
                            float y[4];
                            mma0(y, f, p[nt][0], p[nt][1]);
                            mma(y, f, q[nt][0], q[nt][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[nt][i][e] += y[e];
                        }
                    }
                } else {
                    // v = middle + scale * (code - 7.5), middle = low + 7.5 scale.  weight * middle stays
                    // in fp32; weight * scale meets the codes as the sum of two bf16 numbers, 16 bits as
                    // with a bf16 cache, and its own sum takes the 7.5 off again at the item's end: so the
                    // rounding meets scale * (code - 7.5), which is no larger than v, and not v - low.
                    // (One number is off by 2^-8: an fp32 result over 32768 random values by 1.7e-3, with
                    // two by 9e-5, most of it the sums' rounding; 82.7 against 86.7 us on 3 contexts of 131072.)
                    // With H a tile's columns are half of the eight, so its low parts take the other half: both
                    // halves of a row stand at one maximum and are added at the item's end.
                    uint32_t sc[2][G], p[2][G][NT][2];
                    const int own_x = HN * z + mine;
                    scales(sc, buf + 2 * KS * ROWB + (KS + 16 * own_x + g) * Sh::kScaleBytes);
                    if (partial) no_token(sc, key0 + 16 * own_x + g, vlo, vhi, missing >> own_x & 1);
#pragma unroll
                    for (int gr = 0; gr < G; ++gr)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const float scl = lo_f(sc[y][gr]), mid = fmaf(7.5f, scl, hi_f(sc[y][gr]));
                                const float p0 = s[z][nt][2 * y] * scl, p1 = s[z][nt][2 * y + 1] * scl;
                                const uint32_t hi = pack2(p0, p1);
                                p[0][gr][nt][y] = transpose8(hi);
                                p[1][gr][nt][y] = transpose8(pack2(p0 - lo_f(hi), p1 - hi_f(hi)));
                                if (H) p[1][gr][nt][y] = __shfl_xor_sync(0xffffffffu, p[1][gr][nt][y], 16);
                                zs[gr][nt][0] = fmaf(s[z][nt][2 * y], mid, zs[gr][nt][0]);
                                zs[gr][nt][1] = fmaf(s[z][nt][2 * y + 1], mid, zs[gr][nt][1]);
                            }
#pragma unroll
                    for (int gr = 0; gr < G; ++gr)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint32_t ones[4] = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
                            mma(vs[gr][nt], ones, p[0][gr][nt][0], p[0][gr][nt][1]);
                            mma(vs[gr][nt], ones, p[1][gr][nt][0], p[1][gr][nt][1]);
                        }
#pragma unroll
                    for (int hh = 0; hh < HN; ++hh) {
                        const int x = HN * z + hh;
                        uint32_t w[4][G];  // keys 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const int r = 16 * x + 2 * c + (y & 1) + 8 * (y >> 1);
                            if (D == 128) {
                                const int line = r >> 1, at = ((r & 1) * 4 + (g >> 1)) ^ (2 * (line & 3));
                                const uint2 v = *reinterpret_cast<const uint2*>(
                                    buf + KS * ROWB + line * 128 + at * 16 + (g & 1) * 8);
                                w[y][0] = v.x;
                                w[y][G - 1] = v.y;
                            } else {
                                const int line = r >> 2, at = ((r & 3) * 2 + (g >> 2)) ^ (2 * (line & 1));
                                w[y][0] = *reinterpret_cast<const uint32_t*>(
                                    buf + KS * ROWB + line * 128 + at * 16 + (g & 3) * 4);
                            }
                        }
#pragma unroll
                        for (int gr = 0; gr < G; ++gr) {
                            // the even dims of two keys in one word, and the odd ones
                            const uint32_t v[4] = {__byte_perm(w[0][gr], w[1][gr], 0x5410),
                                                   __byte_perm(w[0][gr], w[1][gr], 0x7632),
                                                   __byte_perm(w[2][gr], w[3][gr], 0x5410),
                                                   __byte_perm(w[2][gr], w[3][gr], 0x7632)};
                            uint32_t b[NT][2];
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int y = 0; y < 2; ++y)
                                    b[nt][y] = !H || (g >> 2) == hh ? p[0][gr][nt][y] : p[1][gr][nt][y];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                // tile 2h: the lower code of a byte; tile 2h + 1: the whole byte, from
                                // which the lower code is taken off again at the item's end
                                uint32_t f[4], lo[4];
#pragma unroll
                                for (int y = 0; y < 4; ++y) {
                                    f[y] = h == 0 ? both_codes(v[y]) : upper_bytes(v[y]);
                                    lo[y] = low_codes(f[y]);
                                }
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    mma(o[nt][4 * gr + 2 * h], lo, b[nt][0], b[nt][1]);
                                    mma(o[nt][4 * gr + 2 * h + 1], f, b[nt][0], b[nt][1]);
                                    if (!H) {
                                        mma(o[nt][4 * gr + 2 * h], lo, p[1][gr][nt][0], p[1][gr][nt][1]);
                                        mma(o[nt][4 * gr + 2 * h + 1], f, p[1][gr][nt][0], p[1][gr][nt][1]);
                                    }
                                }
                            }
                        }
                    }
                }
            }
            // The products' sums lose up to a last bit a step, always towards 0, and codes are never
            // negative: over thousands of steps that would be a bias against a result that the values
            // average down to.  So every 16 steps the middle goes off the sums, which leaves them small
            // (64 contexts of 131072, equal weights: error 0.025 of the result without, 5e-5 with).
            if (INT4 && step % 16 == 15) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int i = 0; i < T; ++i) {
                            const float mid = vs[INT4 ? i / 4 : 0][nt][e] * (7.5f / kUp64);
                            const float f = (i % 2 ? -17.f : -1.f) / kUp69;  // a byte holds code + 16 code'
                            o[nt][i][e] = fmaf(mid, f, o[nt][i][e]);
                            o[nt][i][2 + e] = fmaf(mid, f, o[nt][i][2 + e]);
                        }
#pragma unroll
                for (int gr = 0; gr < (INT4 ? G : 1); ++gr)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) vs[gr][nt][e] = 0.f;
            }
        }

        // ---- the item's end: the warps' sums are joined
        if (flags & kLast) {
            const int32_t r0 = mt.rb * R;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        l_run[nt][e] += __shfl_xor_sync(0xffffffffu, l_run[nt][e], d);
                        if (INT4) {
#pragma unroll
                            for (int gr = 0; gr < G; ++gr)
                                zs[gr][nt][e] += __shfl_xor_sync(0xffffffffu, zs[gr][nt][e], d);
                        }
                    }
                    // sums in plain units, the maximum in base 2
                    m_run[nt][e] *= a.c;
                    if (INT4) {
                        l_run[nt][e] *= 1.f / kUp64;
#pragma unroll
                        for (int i = 0; i < T; i += 2) {
                            const float z = fmaf(-7.5f, vs[INT4 ? i / 4 : 0][nt][e], zs[INT4 ? i / 4 : 0][nt][e]) * (1.f / kUp64);
#pragma unroll
                            for (int y = e; y < 4; y += 2) {
                                o[nt][i + 1][y] = fmaf(o[nt][i + 1][y] - o[nt][i][y], kUp69 / 16.f, z);
                                o[nt][i][y] = fmaf(o[nt][i][y], kUp69, z);
                            }
                        }
                    }
                }
            constexpr int JT = Sh::kJoinDims / 16, JD = Sh::kJoinDims, JP = Sh::kJoinPitch;
#pragma unroll
            for (int t0 = 0; t0 < T; t0 += JT) {
                if (t0 > 0) __syncthreads();  // the last dims are read
                if (t0 == 0 && lane == 0) join_at[warp] = (warp * S + stage) * Sh::kStageBytes;
                float* join_o = reinterpret_cast<float*>(ring + stage * Sh::kStageBytes);  // [C][JP]
                __syncwarp();  // the stage is read
                if (t0 == 0 && g == 0) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            join_m[warp * C + 8 * nt + 2 * c + e] = m_run[nt][e];
                            join_l[warp * C + 8 * nt + 2 * c + e] = l_run[nt][e];
                        }
                }
#pragma unroll
                for (int i = 0; i < JT; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            // tile i holds dims 16i + g, 16i + g + 8, or with 4 bits dims
                            // 8g + 2i, 8g + 2i + 1 of its group
                            const int at = INT4 ? 64 * (i / 4) + 8 * g + 2 * (i % 4) + (e >> 1)
                                                : 16 * i + g + 8 * (e >> 1);
                            join_o[(8 * nt + 2 * c + (e & 1)) * JP + at] = o[nt][t0 + i][e];
                        }
                __syncthreads();
                for (int idx = tid; idx < R * (JD / 4); idx += Sh::kThreads) {
                    const int r = idx / (JD / 4), d4 = idx % (JD / 4) * 4;
                    if (r0 + r >= mt.rows) continue;
                    float mm = -INFINITY;
#pragma unroll
                    for (int w = 0; w < W * HN; ++w) mm = fmaxf(mm, join_m[w * (C / HN) + r]);
                    float l = 0.f;
                    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < W * HN; ++w) {  // with H two sets of columns a warp
                        const float mw = join_m[w * (C / HN) + r];
                        const float f = mw == -INFINITY ? 0.f : ex2(mw - mm);
                        const float4 v = *reinterpret_cast<const float4*>(
                            smem + join_at[w / HN] + (((w % HN) * (C / HN) + r) * JP + d4) * 4);
                        l = fmaf(f, join_l[w * (C / HN) + r], l);
                        sum.x = fmaf(f, v.x, sum.x);
                        sum.y = fmaf(f, v.y, sum.y);
                        sum.z = fmaf(f, v.z, sum.z);
                        sum.w = fmaf(f, v.w, sum.w);
                    }
                    const int dim = 16 * t0 + d4;  // first of four
                    if (flags & kWhole) {
                        const int32_t tok = (r0 + r) / a.group;
                        const int32_t h = mt.kvh * a.group + (r0 + r) - tok * a.group;
                        const int64_t at = ((int64_t)(mt.row0 + tok) * a.hq + h) * D + dim;
                        const float inv = l != 0.f ? 1.f / l : 0.f;
                        if (l == 0.f) sum = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (a.out_fp32) {
                            *reinterpret_cast<float4*>((float*)a.out + at) =
                                make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
                        } else {
                            *reinterpret_cast<uint2*>((__nv_bfloat16*)a.out + at) =
                                make_uint2(pack2(sum.x * inv, sum.y * inv), pack2(sum.z * inv, sum.w * inv));
                        }
                        if (t0 == 0 && d4 == 0)
                            a.lse[(int64_t)h * a.s.num_tokens + mt.row0 + tok] =
                                l != 0.f ? fmaf(mm, kLn2, logf(l)) : -INFINITY;
                    } else {
                        const int64_t at = (int64_t)mt.slot * R + r;
                        *reinterpret_cast<float4*>(a.ws_o + at * D + dim) = sum;
                        if (t0 == 0 && d4 == 0) a.ws_ml[at] = make_float2(mm, l);
                    }
                }
            }
            __syncthreads();  // the sums are read: the stages may be filled again
        }
    }
}

// Joins the partial sums of every item that was cut, in the order of the pieces.
// What it costs is latency: one load for the piece, one for the sums.  So a row's
// partials are spread over WARPS warps, four at a time in flight in each, and every warp
// keeps its own maximum until the end.  (32 partials of a row of 128: 13 us with one warp,
// 3 us with eight.)  Where rows are many, pieces are few and each warp takes a row.
template <int D, int KIND, int NT, bool H, int WARPS>
__global__ void __launch_bounds__(256) join_kernel(const AttnArgs a) {
    using Sh = Shape<D, KIND, NT, H>;
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

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

template <int D, int KIND, int NT, bool H>
pva_status launch(AttnArgs a, uint8_t* ws, cudaStream_t st) {
    using Sh = Shape<D, KIND, NT, H>;
    static_assert((Sh::kSmem + 1280) * Sh::kCtas <= 228 * 1024, "the CTAs share an SM");
    a.ws_per = reinterpret_cast<int64_t*>(ws);
    a.ws_cum = reinterpret_cast<int64_t*>(ws + 256);
    ws += 256 + up256((size_t)a.s.num_seqs * 8);
    a.ws_ml = reinterpret_cast<float2*>(ws);
    a.ws_o = reinterpret_cast<float*>(ws + (size_t)2 * kMaxCtas * Sh::R * 8);
    const int sms = sm_count();
    if (sms <= 0) return PVA_ERR_CUDA;
    const int ctas = sms * Sh::kCtas < kMaxCtas ? sms * Sh::kCtas : kMaxCtas;
    if (cudaFuncSetAttribute(attn_kernel<D, KIND, NT, H>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Sh::kSmem) != cudaSuccess)
        return PVA_ERR_CUDA;
    if (launch_after(attn_kernel<D, KIND, NT, H>, dim3(ctas), Sh::kThreads, Sh::kSmem, st, a) != cudaSuccess)
        return PVA_ERR_CUDA;
    const int64_t rows = (int64_t)a.s.num_tokens * a.hq;
    const bool spread = rows <= kSpreadRows;
    const dim3 grid((unsigned)(spread ? rows : (rows + 7) / 8));
    const cudaError_t e = spread ? launch_after(join_kernel<D, KIND, NT, H, 8>, grid, 256, 0, st, a)
                                 : launch_after(join_kernel<D, KIND, NT, H, 1>, grid, 256, 0, st, a);
    return e == cudaSuccess ? PVA_OK : PVA_ERR_CUDA;
}

// Variants by rows a kv head: 4 bits up to 4 rows two key tiles in the columns, else items of 8
// rows (two column tiles of 16 rows were slower, with weights of 8 bits: 12 contexts to 49635
// tokens, 12 rows: 52 us against 37 us; 32 contexts to 16000, 32 rows: 85 against 83; now 41 and
// 99 us, append included); bf16 up to 8 rows one column tile, else items of 16 rows (4 contexts of
// 8192: up to 16 rows 33.2 us, 32.6 with items of 8; up to 64 rows 35.5 and 42.5 us; 64 contexts
// of 4000 .. 9001, up to 32 rows: 305 and 443 us).
template <int D, int KIND>
pva_status launch_rows(int64_t rows, const AttnArgs& a, uint8_t* ws, cudaStream_t st) {
    if constexpr (KIND == PVA_CACHE_INT4)
        return rows <= 4 ? launch<D, KIND, 1, true>(a, ws, st) : launch<D, KIND, 1, false>(a, ws, st);
    else
        return rows <= 8 ? launch<D, KIND, 1, false>(a, ws, st) : launch<D, KIND, 2, false>(a, ws, st);
}

}  // namespace
}  // namespace pva

using namespace pva;

extern "C" size_t pva_cache_attn_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                       int32_t head_dim, int32_t max_new) {
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
        (head_dim != 64 && head_dim != 128) || max_new < 1)
        return 0;
    const int64_t rows = (int64_t)(num_q_heads / num_kv_heads) * max_new;
    const size_t r = rows <= 8 ? 8 : 16;
    return 256 + up256((size_t)num_seqs * 8) + (size_t)2 * kMaxCtas * r * (8 + 4 * (size_t)head_dim);
}

extern "C" pva_status pva_cache_attn(const pva_cache_desc* cache, const pva_cache_batch* batch,
                                     const void* q, int64_t q_stride, int32_t num_q_heads,
                                     int32_t max_new, int32_t window, float softmax_scale,
                                     void* out, int32_t out_is_fp32, float* lse, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    pva_status st = check_cache(cache);
    if (st == PVA_OK) st = check_batch(batch, true);
    if (st != PVA_OK) return st;
    const int32_t d = cache->head_dim;
    if (num_q_heads <= 0 || num_q_heads % cache->num_kv_heads != 0 || max_new < 1 || window < 0 ||
        (out_is_fp32 != 0 && out_is_fp32 != 1) || !(softmax_scale - softmax_scale == 0.f))
        return PVA_ERR_INVALID_ARG;
    AttnArgs a = {};
    a.c = (softmax_scale > 0.f ? softmax_scale : 1.f / sqrtf((float)d)) * kLog2e;
    if (cache->kind == PVA_CACHE_INT4) a.c *= kUp69;
    if (!(a.c <= FLT_MAX)) return PVA_ERR_INVALID_ARG;
    // (a slack past fp32's numbers would make -inf + slack a NaN: a first maximum has to rise from -inf)
    a.slack = fminf(kSlack / a.c, FLT_MAX);
    a.q_stride = row_stride(q_stride, num_q_heads, d, 2);
    if (a.q_stride < 0) return PVA_ERR_INVALID_ARG;
    if (batch->num_tokens == 0 || batch->num_seqs == 0) return PVA_OK;
    if (!q || !out || !lse || !workspace || !aligned16(q) || !aligned16(out) || !aligned4(lse) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return PVA_ERR_INVALID_ARG;
    if (workspace_bytes < pva_cache_attn_bytes(batch->num_seqs, num_q_heads, cache->num_kv_heads, d,
                                               max_new))
        return PVA_ERR_BUFFER_TOO_SMALL;
    if (batch->num_tokens > INT32_MAX / num_q_heads) return PVA_ERR_UNSUPPORTED;
    a.q = reinterpret_cast<const __nv_bfloat16*>(q);
    // (a copy of no bytes still names an address)
    a.k_pages = reinterpret_cast<const uint8_t*>(cache->num_pages > 0 ? cache->k_pages : q);
    a.v_pages = reinterpret_cast<const uint8_t*>(cache->num_pages > 0 ? cache->v_pages : q);
    a.k_scales = reinterpret_cast<const uint8_t*>(cache->k_scales);
    a.v_scales = reinterpret_cast<const uint8_t*>(cache->v_scales);
    a.out = out;
    a.lse = lse;
    a.s = seq_view(cache, batch);
    a.hq = num_q_heads;
    a.hkv = cache->num_kv_heads;
    a.group = num_q_heads / cache->num_kv_heads;
    a.window = window;
    a.out_fp32 = out_is_fp32;
    const int64_t page_bytes =
        (int64_t)cache->num_kv_heads * cache->page_size * (cache->kind == PVA_CACHE_INT4 ? d / 2 : 2 * d);
    if (page_bytes > INT32_MAX) return PVA_ERR_UNSUPPORTED;
    a.page_bytes = (uint32_t)page_bytes;
    a.num_pages = (uint32_t)cache->num_pages;
    // Without offsets every sequence has one row, whatever bound was given.
    const int64_t rows = (int64_t)a.group * (batch->cu_new ? max_new : 1);
    uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cache->kind == PVA_CACHE_BF16)
        return d == 128 ? launch_rows<128, PVA_CACHE_BF16>(rows, a, ws, s)
                        : launch_rows<64, PVA_CACHE_BF16>(rows, a, ws, s);
    return d == 128 ? launch_rows<128, PVA_CACHE_INT4>(rows, a, ws, s)
                    : launch_rows<64, PVA_CACHE_INT4>(rows, a, ws, s);
}
