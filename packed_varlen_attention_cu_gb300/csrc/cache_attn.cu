// cache_attn.cu -- attention of new tokens over the paged cache.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pva.h"
#include "cache.cuh"

namespace pva {
namespace {

struct AttnArgs {
    const void* q;
    const void *k_pages, *v_pages, *k_scales, *v_scales;
    void* out;
    float* lse;
    int64_t q_stride;
    SeqView s;
    int32_t hq, hkv, window, out_fp32;
    float scale;
};

// One CTA for a query row and head; its warps take every fourth key.
template <int D, int KIND>
__global__ void __launch_bounds__(128) simple_kernel(const AttnArgs a) {
    constexpr int kE = D / 32;
    __shared__ float sm_m[4], sm_l[4], sm_o[4][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t t = blockIdx.x, h = blockIdx.y, kvh = h / (a.hq / a.hkv);
    int32_t b = t, n = 1, i = 0;
    if (a.s.cu && t == 0 && h == 0)
        for (int32_t x = threadIdx.x; x < a.s.num_seqs; x += 128)
            if (a.s.cu[x] < 0 || a.s.cu[x + 1] < a.s.cu[x] || a.s.cu[x + 1] > a.s.num_tokens)
                raise_status(a.s.status, kErrLength);
    if (a.s.cu) {
        b = find_seq(a.s.cu, a.s.num_seqs, t);
        if (b < 0) return;
        n = a.s.cu[b + 1] - a.s.cu[b];
        i = t - a.s.cu[b];
    }
    if (b >= a.s.num_seqs) return;
    const int32_t pos = (int32_t)max((int64_t)a.s.kv_lens[b] - n + i, (int64_t)-1);
    if (threadIdx.x == 0 && a.s.kv_lens[b] < n) raise_status(a.s.status, kErrLength);
    const int32_t first = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
    const __nv_bfloat16* q = (const __nv_bfloat16*)a.q + t * a.q_stride + (int64_t)h * D;
    auto element = [&](const void* pages, const void* scales, int64_t at, int d) {
        if (KIND == PVA_CACHE_BF16) return __bfloat162float(((const __nv_bfloat16*)pages)[at * D + d]);
        const uint32_t w = ((const uint32_t*)pages)[at * (D / 8) + word_of_octet<D>(d / 8)];
        const uint32_t sc = ((const uint32_t*)scales)[at * (D / 64) + d / 64];
        const float code = (float)(w >> (4 * (d % 8 / 2) + 16 * (d % 2)) & 15u);
        return __uint_as_float(sc & 0xffff0000u) + code * __uint_as_float(sc << 16);
    };
    float m = -INFINITY, l = 0.f, o[kE] = {};
    for (int32_t j = first + warp; j <= pos; j += 4) {
        const int64_t page = page_of(a.s, b, j);
        if (page < 0) {
            if (lane == 0) raise_status(a.s.status, kErrPage);
            continue;
        }
        const int64_t at = ((page * a.hkv + kvh) << a.s.page_shift) + (j & ((1 << a.s.page_shift) - 1));
        float s = 0.f;
        for (int e = 0; e < kE; ++e)
            s += __bfloat162float(q[e * 32 + lane]) * element(a.k_pages, a.k_scales, at, e * 32 + lane);
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= a.scale;
        const float mn = fmaxf(m, s);
        const float old = m == -INFINITY ? 0.f : expf(m - mn), p = s == -INFINITY ? 0.f : expf(s - mn);
        l = l * old + p;
        for (int e = 0; e < kE; ++e)
            o[e] = o[e] * old + p * element(a.v_pages, a.v_scales, at, e * 32 + lane);
        m = mn;
    }
    sm_m[warp] = m;
    sm_l[warp] = l;
    for (int e = 0; e < kE; ++e) sm_o[warp][e * 32 + lane] = o[e];
    __syncthreads();
    if (threadIdx.x < D) {
        float mx = -INFINITY, lt = 0.f, ot = 0.f;
        for (int w = 0; w < 4; ++w) mx = fmaxf(mx, sm_m[w]);
        for (int w = 0; w < 4; ++w) {
            const float f = sm_m[w] == -INFINITY ? 0.f : expf(sm_m[w] - mx);
            lt += f * sm_l[w];
            ot += f * sm_o[w][threadIdx.x];
        }
        const float r = lt > 0.f ? ot / lt : 0.f;
        const int64_t at = ((int64_t)t * a.hq + h) * D + threadIdx.x;
        if (a.out_fp32) ((float*)a.out)[at] = r;
        else ((__nv_bfloat16*)a.out)[at] = __float2bfloat16_rn(r);
        if (threadIdx.x == 0)
            a.lse[(int64_t)h * a.s.num_tokens + t] = lt > 0.f ? mx + logf(lt) : -INFINITY;
    }
}

}  // namespace
}  // namespace pva

using namespace pva;

extern "C" size_t pva_cache_attn_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                       int32_t head_dim, int32_t max_new) {
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
        (head_dim != 64 && head_dim != 128) || max_new < 1)
        return 0;
    return 256;
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
        (out_is_fp32 != 0 && out_is_fp32 != 1) || !(softmax_scale == softmax_scale))
        return PVA_ERR_INVALID_ARG;
    AttnArgs a = {};
    a.q_stride = row_stride(q_stride, num_q_heads, d, 2);
    if (a.q_stride < 0) return PVA_ERR_INVALID_ARG;
    if (batch->num_tokens == 0 || batch->num_seqs == 0) return PVA_OK;
    if (!q || !out || !lse || !workspace || !aligned16(q) || !aligned16(out) || !aligned4(lse) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return PVA_ERR_INVALID_ARG;
    if (workspace_bytes < pva_cache_attn_bytes(batch->num_seqs, num_q_heads, cache->num_kv_heads, d,
                                               max_new))
        return PVA_ERR_BUFFER_TOO_SMALL;
    a.q = q;
    a.k_pages = cache->k_pages;
    a.v_pages = cache->v_pages;
    a.k_scales = cache->k_scales;
    a.v_scales = cache->v_scales;
    a.out = out;
    a.lse = lse;
    a.s = seq_view(cache, batch);
    a.hq = num_q_heads;
    a.hkv = cache->num_kv_heads;
    a.window = window;
    a.out_fp32 = out_is_fp32;
    a.scale = softmax_scale > 0.f ? softmax_scale : rsqrtf((float)d);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const dim3 grid(batch->num_tokens, num_q_heads);
    if (cache->kind == PVA_CACHE_BF16) {
        if (d == 128) simple_kernel<128, PVA_CACHE_BF16><<<grid, 128, 0, s>>>(a);
        else simple_kernel<64, PVA_CACHE_BF16><<<grid, 128, 0, s>>>(a);
    } else {
        if (d == 128) simple_kernel<128, PVA_CACHE_INT4><<<grid, 128, 0, s>>>(a);
        else simple_kernel<64, PVA_CACHE_INT4><<<grid, 128, 0, s>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? PVA_OK : PVA_ERR_CUDA;
}
