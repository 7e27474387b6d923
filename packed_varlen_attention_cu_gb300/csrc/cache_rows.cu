// cache_rows.cu -- cross attention over the paged cache for many rows of a kv head (beams times the
// heads of a group).
//
// The formulas and the transposed products are those of cache_attn.cu.  There every warp streams keys
// of its own for all rows of an item, 16 of them at most (8 with 4 bits), and an item more reads K and V
// again: 32 rows of a bf16 cache took twice its bytes' time, 48 rows three times (and so still goes up to 16
// rows: with 4 bits 16 rows took 137 us here against 133).  Here the four warps
// of a CTA share each tile of 64 keys and divide the rows, up to 64, between them, so K and V are read
// once.  4-bit tiles are expanded in shared memory once for all rows: masks alone make the codes of K
// numbers (subnormal bf16, see there), those of V are taken around their middle, code - 8, so that
// sums over a long context have no bias; scales stay apart, on the scores and on the weights.
//
// (tcgen05 was slower with 4 bits: with a thread a row the scales of every key are broadcast loads, four
// wavefronts of shared memory each, 24 sources to 30000 keys and 32 rows 109 against 105 us, 64 sources to
// 8192 235 against 191.  Here a lane's keys are its own.)
//
// With 4 bits and up to 32 rows two warps have all rows, 16 each (a warp's K and V fragments then serve
// twice the products: 191 against 202 us with four warps of 8 rows), and the pairs divide the keys of a
// tile; their sums meet at the item's end.
#include "cache_attn.cuh"

namespace pva {
namespace {

// NT column tiles (of 8 rows) a warp, WR warps along the rows, 4 / WR along the keys.
template <int D_, int KIND, int NT_, int WR_>
struct Rows {
    static constexpr bool kInt4 = KIND == PVA_CACHE_INT4;
    static constexpr int D = D_, NT = NT_, WR = WR_, WK = 4 / WR;
    static constexpr int kWarps = 4, kThreads = 128;
    static constexpr int kKeys = 64, kBlock = 64;  // of a tile, of a unit
    static constexpr int Z = 4 / WK;               // tiles of 16 keys of a warp
    static constexpr int R = 8 * NT * WR;          // rows of an item
    static constexpr int kFixed = 3;               // an item's fixed cost in blocks
    // Resident on an SM.  (4 bits, up to 32 rows, three instead of two: 28 rows of 64 dims 35.4 -> 33.7 us;
    // of 128 dims, with spills, 32 rows 105.8 -> 109.1.)
    static constexpr int kCtas = NT == 1 || (kInt4 && WR == 2 && D == 64) ? 3 : 2;
    static constexpr int G = D / 64;
    static constexpr int kRowBytes = kInt4 ? D / 2 : 2 * D;
    static constexpr int kScaleBytes = kInt4 ? 4 * G : 0;
    static constexpr int kStageBytes = 2 * kKeys * (kRowBytes + kScaleBytes);
    static constexpr int kStages = !kInt4 && D == 128 && kCtas == 3 ? 2 : 3;
    static constexpr int kOperand = kInt4 ? kKeys * 2 * D : 0;  // bytes of K's or V's expanded tile
    static constexpr int kPitch = D + 4;                        // floats of a row where warps' sums meet
    static constexpr int kSmem = kStages * kStageBytes + 2 * kOperand;
    static_assert(WK * R * kPitch * 4 <= kSmem, "the sums fit");
};

// Eight codes of a word as bf16, code * 2^-133 (K).
__device__ __forceinline__ uint4 spread_low(uint32_t w) {
    return make_uint4(low_codes(w), low_codes(w >> 4), low_codes(w >> 8), low_codes(w >> 12));
}
// Eight codes of a word as bf16, code - 8 (V): 0x4300 is 128, whose last place is 1.
__device__ __forceinline__ uint32_t centred(uint32_t two) {
    const uint32_t x = two | 0x43004300u, m = 0x43084308u;  // 136
    const __nv_bfloat162 y = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x),
                                     *reinterpret_cast<const __nv_bfloat162*>(&m));
    return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ uint4 spread_centred(uint32_t w) {
    return make_uint4(centred(low_codes(w)), centred(low_codes(w >> 4)), centred(low_codes(w >> 8)),
                      centred(low_codes(w >> 12)));
}

// TWO: weights are operands as the sum of two bf16 numbers, 16 of their bits, else as one.
template <class Sh, bool TWO>
__global__ void __launch_bounds__(128, Sh::kCtas) rows_kernel(const AttnArgs a) {
    constexpr int D = Sh::D, NT = Sh::NT, WR = Sh::WR, WK = Sh::WK, Z = Sh::Z, R = Sh::R, S = Sh::kStages;
    constexpr int G = Sh::G, T = D / 16, KEYS = Sh::kKeys, ROWB = Sh::kRowBytes, JP = Sh::kPitch;
    constexpr bool INT4 = Sh::kInt4;
    constexpr int GA = INT4 ? G : 1;   // groups with products of their own
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float join_m[WK][R], join_l[WK][R];
    wait_previous();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int wr = warp % WR, wk = warp / WR;
    int32_t b;
    int64_t u0, u1, ub;
    if (!find_piece<Sh>(a, u0, u1, b, ub)) return;
    SeqInfo sq = seq_info<Sh>(a, b, false);
    int32_t len = Sh::kFixed + sq.nb;
    int32_t it = (int32_t)quotient(u0 - ub, len);
    int32_t rb = it / a.hkv, kvh = it - rb * a.hkv;
    int64_t ui = ub + (int64_t)it * len;  // first unit of the item
    const uint32_t mask = (1u << a.s.page_shift) - 1;
    uint8_t* operands = smem + S * Sh::kStageBytes;

    while (ui < u1) {
        const int32_t r0 = rb * R, rows = sq.n * a.group;
        const int64_t first = ui + Sh::kFixed;
        const int32_t t0 = (int32_t)max(u0 - first, (int64_t)0);
        const int32_t t1 = (int32_t)(min(u1, ui + len) - first);
        const bool empty = sq.nb == 0;
        if (empty ? u0 <= ui : t1 > t0) {
            const bool whole = empty || (t0 == 0 && t1 == sq.nb);
            const int32_t slot = 2 * blockIdx.x + (t0 == 0 ? 1 : 0);
            const int32_t* pages = a.s.page_table + b * a.s.table_stride;
            const uint32_t head = (uint32_t)kvh << a.s.page_shift;
            // ---- the queries, and with 4 bits their sums over a group's dims
            uint32_t qf[NT][T][2];
            float qs[GA][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int32_t r = r0 + (wr * NT + nt) * 8 + g, tok = r / a.group;
                const __nv_bfloat16* q = a.q + (int64_t)(sq.row0 + tok) * a.q_stride +
                                         (int64_t)(kvh * a.group + r - tok * a.group) * D;
#pragma unroll
                for (int gr = 0; gr < G; ++gr) {
                    float sum = 0.f;
#pragma unroll
                    for (int ks = 4 * gr; ks < 4 * gr + 4; ++ks)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t x = r < rows ? *reinterpret_cast<const uint32_t*>(q + 16 * ks + 8 * e + 2 * c) : 0u;
                            if (INT4) {
                                sum += lo_f(x) + hi_f(x);
                                x = pack2(lo_f(x) * kUp64, hi_f(x) * kUp64);
                            }
                            qf[nt][ks][e] = x;
                        }
                    if (INT4) {
                        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                        sum *= 1.f / kUp69;
#pragma unroll
                        for (int e = 0; e < 2; ++e)  // of rows 2c, 2c + 1: this lane's columns of the scores
                            qs[INT4 ? gr : 0][nt][e] = __shfl_sync(0xffffffffu, sum, 4 * (2 * c + e));
                    }
                }
            }
            float o[NT][T][4], m_run[NT][2], l_run[NT][2], zs[GA][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m_run[nt][e] = -INFINITY;
                    l_run[nt][e] = 0.f;
#pragma unroll
                    for (int gr = 0; gr < GA; ++gr) zs[gr][nt][e] = 0.f;
#pragma unroll
                    for (int i = 0; i < T; ++i) o[nt][i][e] = o[nt][i][2 + e] = 0.f;
                }

            // ---- copies.  Lane x < 4 knows the page of keys 16x .. of the tile to be copied next.
            auto page_at = [&](int32_t t) -> uint32_t {
                const int32_t i = (t * KEYS + 16 * (lane & 3)) >> a.s.page_shift;
                return i < a.s.max_pages ? (uint32_t)pages[i] : ~0u;
            };
            uint32_t page = empty ? ~0u : page_at(t0);
            uint32_t missing = 0;  // four bits a stage: no page for 16 keys
            auto issue = [&](int32_t t, int stage) {
                const uint32_t kd = smem_addr(smem + stage * Sh::kStageBytes);
                const int32_t key0 = t * KEYS;
                const bool none = lane < 4 && key0 + 16 * lane < sq.khi && page >= a.num_pages;
                const uint32_t miss = __ballot_sync(0xffffffffu, none);
                if (none && warp == 0) raise_status(a.s.status, kErrPage);
                missing = (missing & ~(15u << 4 * stage)) | miss << 4 * stage;
                uint64_t off[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t p = __shfl_sync(0xffffffffu, page, x);
                    off[x] = p < a.num_pages ? (uint64_t)p * a.page_bytes + (head + ((key0 + 16 * x) & mask)) * ROWB : ~0ull;
                }
                constexpr int CPR = ROWB / 16;  // 16-byte chunks of a row
                if constexpr (!INT4) {
                    const int r = tid / CPR, ch = tid % CPR;
#pragma unroll
                    for (int i = 0; i < KEYS * CPR / 128; ++i) {
                        const int row = i * (128 / CPR) + r, x = (i * (128 / CPR)) / 16;  // (a pass stays inside 16 keys)
                        const uint32_t to = row * ROWB + ((ch ^ (row & 7)) << 4);
                        // rows that are not there are filled with zeros: a weight of 0 must not meet a NaN
                        const bool ok = off[x] != ~0ull && key0 + row < sq.khi;
                        const uint64_t at = off[x] + (uint64_t)(row - 16 * x) * ROWB + ch * 16;
                        cp16(kd + to, ok ? a.k_pages + at : a.k_pages, ok ? 16 : 0);
                        cp16(kd + KEYS * ROWB + to, ok ? a.v_pages + at : a.v_pages, ok ? 16 : 0);
                    }
                } else {
                    // (what stands for keys without a token are their scales, set to 0 where they are read)
#pragma unroll
                    for (int i = 0; i < KEYS * CPR / 128; ++i) {
                        const int n = i * 128 + tid, x = n / (16 * CPR);
                        const uint64_t o4 = x == 0 ? off[0] : x == 1 ? off[1] : x == 2 ? off[2] : off[3];
                        if (o4 == ~0ull) continue;
                        const uint64_t at = o4 + (uint64_t)(n - x * 16 * CPR) * 16;
                        cp16(kd + n * 16, a.k_pages + at, 16);
                        cp16(kd + KEYS * ROWB + n * 16, a.v_pages + at, 16);
                    }
                    constexpr int SC = KEYS * Sh::kScaleBytes / 16;  // chunks of K's scales
                    if (tid < 2 * SC) {
                        const bool v = tid >= SC;
                        const int n = v ? tid - SC : tid, x = n / (SC / 4);
                        const uint64_t o4 = x == 0 ? off[0] : x == 1 ? off[1] : x == 2 ? off[2] : off[3];
                        if (o4 != ~0ull)
                            cp16(kd + 2 * KEYS * ROWB + tid * 16,
                                 (v ? a.v_scales : a.k_scales) + (o4 >> 3) + (n - x * (SC / 4)) * 16, 16);
                    }
                }
                page = page_at(t + 1);
            };
            if (!empty) {
#pragma unroll
                for (int i = 0; i < S - 1; ++i) {
                    if (t0 + i < t1) issue(t0 + i, i);
                    cp_commit();
                }
                int stage = 0;
#pragma unroll 1
                for (int32_t t = t0; t < t1; ++t) {
                    cp_wait<S - 2>();
                    __syncthreads();  // the tile is in, and every warp has left the one before
                    if (t + S - 1 < t1) issue(t + S - 1, stage == 0 ? S - 1 : stage - 1);
                    cp_commit();
                    const uint8_t* buf = smem + stage * Sh::kStageBytes;
                    const uint32_t miss = missing >> 4 * stage & 15u;
                    const int32_t key0 = t * KEYS;
                    const bool partial = miss != 0 || key0 + KEYS > sq.khi;
                    if (INT4) {
                        constexpr int CPR = ROWB / 16;
#pragma unroll
                        for (int i = 0; i < KEYS * CPR / 128; ++i) {
                            const int n = i * 128 + tid, row = n / CPR, ch = n % CPR;
                            const uint4 kw = *reinterpret_cast<const uint4*>(buf + n * 16);
                            const uint4 vw = *reinterpret_cast<const uint4*>(buf + KEYS * ROWB + n * 16);
                            const uint32_t k4[4] = {kw.x, kw.y, kw.z, kw.w}, v4[4] = {vw.x, vw.y, vw.z, vw.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int wd = 4 * ch + j, octet = wd % G * 8 + wd / G;
                                uint8_t* to = operands + row * 2 * D + ((octet ^ (row & 7)) << 4);
                                *reinterpret_cast<uint4*>(to) = spread_low(k4[j]);
                                *reinterpret_cast<uint4*>(to + Sh::kOperand) = spread_centred(v4[j]);
                            }
                        }
                        __syncthreads();
                    }
                    const uint32_t kb = INT4 ? smem_addr(operands) : smem_addr(buf);
                    const uint32_t vb = INT4 ? kb + Sh::kOperand : kb + KEYS * ROWB;
                    // (scale, low) of keys j and j + 8 of K or V; 0 where there is no token
                    auto scales = [&](uint32_t (&sc)[2][G], bool v, int32_t j) {
#pragma unroll
                        for (int y = 0; y < 2; ++y)
#pragma unroll
                            for (int gr = 0; gr < G; ++gr) {
                                const int32_t x = j + 8 * y;
                                sc[y][gr] = *reinterpret_cast<const uint32_t*>(
                                    buf + 2 * KEYS * ROWB + ((v ? KEYS : 0) + x) * Sh::kScaleBytes + 4 * gr);
                                if (partial && (key0 + x >= sq.khi || (miss >> (x >> 4) & 1))) sc[y][gr] = 0;
                            }
                    };
                    // ---- S^T of this warp's keys and rows
                    float s[Z][NT][4];
#pragma unroll
                    for (int z = 0; z < Z; ++z) {
                        const int x = wk * Z + z;
                        float acc[GA][NT][4];
#pragma unroll
                        for (int ks = 0; ks < T; ++ks) {
                            uint32_t f[4];
                            const int r = lane & 15, ch = 2 * ks + (lane >> 4);
                            ldsm(f, kb + (16 * x + r) * 2 * D + ((ch ^ (r & 7)) << 4));
                            const int gr = INT4 ? ks / 4 : 0;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                if (ks == 0 || (INT4 && ks % 4 == 0)) mma0(acc[gr][nt], f, qf[nt][ks][0], qf[nt][ks][1]);
                                else mma(acc[gr][nt], f, qf[nt][ks][0], qf[nt][ks][1]);
                            }
                        }
                        if (INT4) {
                            // s = sum over groups of scale * (q . codes) + low * (sum of q)
                            uint32_t sc[2][G];
                            scales(sc, false, 16 * x + g);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    float y = 0.f;
#pragma unroll
                                    for (int gr = 0; gr < G; ++gr) {
                                        const uint32_t p = sc[e >> 1][gr];
                                        y = fmaf(hi_f(p), qs[INT4 ? gr : 0][nt][e & 1], y);
                                        y = fmaf(lo_f(p), acc[INT4 ? gr : 0][nt][e], y);
                                    }
                                    s[z][nt][e] = y;
                                }
                        } else {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) s[z][nt][e] = acc[0][nt][e];
                        }
                        if (partial) {
                            const int32_t j = key0 + 16 * x + g;
                            const bool gone = miss >> x & 1;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (gone || j + 8 * (e >> 1) >= sq.khi) s[z][nt][e] = -INFINITY;
                        }
                    }
                    // ---- has a score left the range of the running maximum?
                    bool up = false;
                    float mx[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            mx[nt][e] = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
                            for (int z = 1; z < Z; ++z)
                                mx[nt][e] = fmaxf(mx[nt][e], fmaxf(s[z][nt][e], s[z][nt][2 + e]));
                            up |= mx[nt][e] > m_run[nt][e] + a.slack;
                        }
                    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
#pragma unroll
                                for (int d = 4; d < 32; d <<= 1)
                                    mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], d));
                                const float mn = fmaxf(m_run[nt][e], mx[nt][e]);
                                const float f = m_run[nt][e] == -INFINITY ? 0.f : ex2((m_run[nt][e] - mn) * a.c);
                                m_run[nt][e] = mn;
                                l_run[nt][e] *= f;
#pragma unroll
                                for (int gr = 0; gr < GA; ++gr) zs[gr][nt][e] *= f;
#pragma unroll
                                for (int i = 0; i < T; ++i) {
                                    o[nt][i][e] *= f;
                                    o[nt][i][2 + e] *= f;
                                }
                            }
                    }
                    // ---- weights, in place of the scores
#pragma unroll
                    for (int z = 0; z < Z; ++z)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float base = m_run[nt][e & 1] == -INFINITY ? 0.f : m_run[nt][e & 1];
                                s[z][nt][e] = ex2((s[z][nt][e] - base) * a.c);
                                l_run[nt][e & 1] += s[z][nt][e];
                            }
                    // ---- O^T, group by group of dims.  Operands are the weights, with 4 bits weight * scale, as the sum
                    // of two bf16 numbers where that hides behind HBM (a bf16 cache, up to 32 rows) or the result
                    // is fp32, which keeps the difference.  A bf16 result takes one number otherwise, as the packs do:
                    // 2^-9 of each weight, about what it loses again itself (off by 0.0024, not 0.0017), for 105 us
                    // instead of 121 (24 sources to 30000 keys in 4 bits, 32 rows of 128 dims), 241 instead of 301 (64
                    // sources to 8192, 48 rows), 431 instead of 575 (64 sources of 8192, bf16, 48 rows).  4 bits: what
                    // the weights meet, scale * (code - 8), is no larger than the values; weight * (low + 8 scale)
                    // stays in fp32.
#pragma unroll
                    for (int gr = 0; gr < GA; ++gr) {
                        uint32_t pf[Z][TWO ? 2 : 1][NT][2];
#pragma unroll
                        for (int z = 0; z < Z; ++z) {
                            uint32_t sc[2][G];
                            if (INT4) scales(sc, true, 16 * (wk * Z + z) + g);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    float p0 = s[z][nt][2 * y], p1 = s[z][nt][2 * y + 1];
                                    if (INT4) {
                                        const float scl = lo_f(sc[y][gr]), mid = fmaf(8.f, scl, hi_f(sc[y][gr]));
                                        zs[gr][nt][0] = fmaf(p0, mid, zs[gr][nt][0]);
                                        zs[gr][nt][1] = fmaf(p1, mid, zs[gr][nt][1]);
                                        p0 *= scl;
                                        p1 *= scl;
                                    }
                                    const uint32_t hi = pack2(p0, p1);
                                    pf[z][0][nt][y] = transpose8(hi);
                                    if (TWO) pf[z][TWO ? 1 : 0][nt][y] = transpose8(pack2(p0 - lo_f(hi), p1 - hi_f(hi)));
                                }
                        }
                        // The products round their sums towards 0: those of a tile start from 0 and go onto the sums
                        // by additions, which round to nearest.
                        constexpr int IG = T / GA;  // tiles of 16 dims of a group
#pragma unroll
                        for (int i = gr * IG; i < (gr + 1) * IG; ++i) {
                            float y[NT][4];
#pragma unroll
                            for (int z = 0; z < Z; ++z) {
                                uint32_t f[4];
                                const int r = (lane & 7) + ((lane >> 4) << 3), ch = 2 * i + ((lane >> 3) & 1);
                                ldsm_t(f, vb + (16 * (wk * Z + z) + r) * 2 * D + ((ch ^ (r & 7)) << 4));
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    if (z == 0) mma0(y[nt], f, pf[z][0][nt][0], pf[z][0][nt][1]);
                                    else mma(y[nt], f, pf[z][0][nt][0], pf[z][0][nt][1]);
                                    if (TWO) mma(y[nt], f, pf[z][TWO ? 1 : 0][nt][0], pf[z][TWO ? 1 : 0][nt][1]);
                                }
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[nt][i][e] += y[nt][e];
                        }
                    }
                    stage = stage + 1 == S ? 0 : stage + 1;
                }
            }
            // ---- the item's end: rows leave through shared memory
            cp_wait<0>();
            __syncthreads();  // the last tile is read
            float* sums = reinterpret_cast<float*>(smem) + (int64_t)(wk * R + wr * NT * 8) * JP;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        l_run[nt][e] += __shfl_xor_sync(0xffffffffu, l_run[nt][e], d);
                        if (INT4) {
#pragma unroll
                            for (int gr = 0; gr < GA; ++gr)
                                zs[gr][nt][e] += __shfl_xor_sync(0xffffffffu, zs[gr][nt][e], d);
                        }
                    }
                    if (g == 0) {
                        join_m[wk][(wr * NT + nt) * 8 + 2 * c + e] = m_run[nt][e] * a.c;  // in base 2
                        join_l[wk][(wr * NT + nt) * 8 + 2 * c + e] = l_run[nt][e];
                    }
                }
#pragma unroll
                for (int i = 0; i < T; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sums[(8 * nt + 2 * c + (e & 1)) * JP + 16 * i + g + 8 * (e >> 1)] =
                            INT4 ? o[nt][i][e] + zs[INT4 ? i / 4 : 0][nt][e & 1] : o[nt][i][e];
            }
            __syncthreads();
            for (int idx = tid; idx < R * (D / 4); idx += 128) {
                const int r = idx / (D / 4), dim = idx % (D / 4) * 4;
                if (r0 + r >= rows) continue;
                float mm = join_m[0][r];
#pragma unroll
                for (int w = 1; w < WK; ++w) mm = fmaxf(mm, join_m[w][r]);
                float l = 0.f;
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < WK; ++w) {
                    const float f = join_m[w][r] == -INFINITY ? 0.f : ex2(join_m[w][r] - mm);
                    const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(smem) + (w * R + r) * JP + dim);
                    l = fmaf(f, join_l[w][r], l);
                    sum.x = fmaf(f, v.x, sum.x);
                    sum.y = fmaf(f, v.y, sum.y);
                    sum.z = fmaf(f, v.z, sum.z);
                    sum.w = fmaf(f, v.w, sum.w);
                }
                if (whole) {
                    const int32_t tok = (r0 + r) / a.group;
                    const int32_t h = kvh * a.group + (r0 + r) - tok * a.group;
                    const int64_t at = ((int64_t)(sq.row0 + tok) * a.hq + h) * D + dim;
                    const float inv = l != 0.f ? 1.f / l : 0.f;
                    if (l == 0.f) sum = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (a.out_fp32)
                        *reinterpret_cast<float4*>((float*)a.out + at) =
                            make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
                    else
                        *reinterpret_cast<uint2*>((__nv_bfloat16*)a.out + at) =
                            make_uint2(pack2(sum.x * inv, sum.y * inv), pack2(sum.z * inv, sum.w * inv));
                    if (dim == 0)
                        a.lse[(int64_t)h * a.s.num_tokens + sq.row0 + tok] =
                            l != 0.f ? fmaf(mm, kLn2, logf(l)) : -INFINITY;
                } else {
                    const int64_t at = (int64_t)slot * R + r;
                    *reinterpret_cast<float4*>(a.ws_o + at * D + dim) = sum;
                    if (dim == 0) a.ws_ml[at] = make_float2(mm, l);
                }
            }
            __syncthreads();  // the sums are read: the stages may be filled again
        }
        // ---- the next item
        ui += len;
        if (++kvh == a.hkv) {
            kvh = 0;
            if (++rb == sq.nrb) {
                rb = 0;
                do {
                    if (++b >= a.s.num_seqs) return;
                    sq = seq_info<Sh>(a, b, false);
                } while (sq.nrb == 0);
                len = Sh::kFixed + sq.nb;
            }
        }
    }
}

template <class Sh, bool TWO>
pva_status launch(AttnArgs a, uint8_t* ws, cudaStream_t st) {
    static_assert((Sh::kSmem + 4096) * Sh::kCtas <= 228 * 1024, "the CTAs share an SM");
    place_workspace<Sh>(a, ws);
    const int sms = sm_count();
    if (sms <= 0) return PVA_ERR_CUDA;
    const int ctas = sms * Sh::kCtas < kMaxCtas ? sms * Sh::kCtas : kMaxCtas;
    if (cudaFuncSetAttribute(rows_kernel<Sh, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem) !=
            cudaSuccess ||
        launch_after(rows_kernel<Sh, TWO>, dim3(ctas), Sh::kThreads, Sh::kSmem, st, a) != cudaSuccess)
        return PVA_ERR_CUDA;
    return launch_join<Sh::D, Sh>(a, st) == cudaSuccess ? PVA_OK : PVA_ERR_CUDA;
}

template <int D>
pva_status launch_kind(int32_t kind, int64_t rows, const AttnArgs& a, uint8_t* ws, cudaStream_t st) {
    constexpr int B = PVA_CACHE_BF16, I = PVA_CACHE_INT4;
    const bool f32 = a.out_fp32 != 0;
    if (kind == B) {
        if (rows <= 32) return launch<Rows<D, B, 1, 4>, true>(a, ws, st);
        return f32 ? launch<Rows<D, B, 2, 4>, true>(a, ws, st) : launch<Rows<D, B, 2, 4>, false>(a, ws, st);
    }
    if (rows <= 32) return f32 ? launch<Rows<D, I, 2, 2>, true>(a, ws, st) : launch<Rows<D, I, 2, 2>, false>(a, ws, st);
    return f32 ? launch<Rows<D, I, 2, 4>, true>(a, ws, st) : launch<Rows<D, I, 2, 4>, false>(a, ws, st);
}

}  // namespace

pva_status launch_many_rows(int32_t kind, int32_t head_dim, int64_t rows, const AttnArgs& a, uint8_t* ws,
                            cudaStream_t st) {
    return head_dim == 128 ? launch_kind<128>(kind, rows, a, ws, st) : launch_kind<64>(kind, rows, a, ws, st);
}

}  // namespace pva
