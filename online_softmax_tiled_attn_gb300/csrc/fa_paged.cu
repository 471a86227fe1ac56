// fa_paged.cu -- attention of a few queries over the paged key/value cache (fa_fwd_paged).
//
// Row i of sequence b sees the keys j <= kv_len - q_len + i (causal) or j < kv_len; rows at or past
// q_len see none (O = 0, LSE = -inf).  One pass over the cache with the running max and sum of the
// online softmax.
#include <cuda_runtime.h>

#include <cmath>

#include "kv_cache.cuh"
#include "osm_internal.h"
#include "ptx_sm103.cuh"

namespace osm {
namespace {

struct PagedParams {
    const __nv_bfloat16* Q;  // [B, H, Nq, d]
    __nv_bfloat16* O;
    float* LSE;  // [B, H, Nq] or nullptr
    const int32_t *kv_lens, *q_lens;
    int64_t B;
    int H, Nq, causal;
    float scale_log2;
    KvPages pg;
};

// Values of a head's token, E = d / 32 a lane.
template <int D>
__device__ __forceinline__ void token_values(const PagedParams& p, const uint8_t* block, int at,
                                             int lane, float (&x)[D / 32]) {
    constexpr int E = D / 32;
    if (p.pg.format == OSM_KV_BF16) {
        const __nv_bfloat16* row = reinterpret_cast<const __nv_bfloat16*>(block) + at * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = __bfloat162float(row[e]);
        return;
    }
    const uint32_t word = reinterpret_cast<const uint16_t*>(
        block + static_cast<int64_t>(p.pg.page) * (D / 2))
        [at * (D / kKvGroup) + lane * E / kKvGroup];
    const float s = kv4_word_step(word);
    const int base = kv4_word_base(word);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int i = lane * E + e;
        const uint32_t byte = block[at * (D / 2) + i / 2];
        x[e] = s * static_cast<float>(base + static_cast<int>((byte >> (4 * (i & 1))) & 15u));
    }
}

// One CTA a query row; its warps take the keys in turn, each with its own running max and sum.
template <int D>
__global__ void __launch_bounds__(256) paged_row_kernel(const PagedParams p) {
    constexpr int E = D / 32;
    __shared__ float sm[8], sl[8], sacc[8][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x;
    const int i = static_cast<int>(row % p.Nq);
    const int h = static_cast<int>(row / p.Nq % p.H);
    const int64_t b = row / p.Nq / p.H;
    const int kvh = h / (p.H / p.pg.H_kv);
    const int64_t room = p.pg.max_pages * p.pg.page;
    const int64_t len = min(static_cast<int64_t>(max(p.kv_lens[b], 0)), room);
    const int ql = p.q_lens ? min(max(p.q_lens[b], 0), p.Nq) : p.Nq;
    int64_t end = p.causal ? len - ql + i + 1 : len;  // keys below it
    if (i >= ql) end = 0;
    float q[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = __bfloat162float(p.Q[row * D + lane * E + e]);
        acc[e] = 0.f;
    }
    for (int64_t j = warp; j < end; j += 8) {
        const int32_t id = p.pg.table[b * p.pg.max_pages + j / p.pg.page];
        if (id < 0 || id >= p.pg.num_pages) {
            if (lane == 0) kv_bad_page(p.pg);
            continue;
        }
        const int at = static_cast<int>(j % p.pg.page);
        const int64_t off = kv_head_offset(p.pg, id, kvh);
        float x[E], s = 0.f;
        token_values<D>(p, p.pg.k + off, at, lane, x);
#pragma unroll
        for (int e = 0; e < E; ++e) s += q[e] * x[e];
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
        s *= p.scale_log2;
        token_values<D>(p, p.pg.v + off, at, lane, x);
        const float mn = fmaxf(m, s);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float a = exp2f(m - ref), w = exp2f(s - ref);
        m = mn;
        l = l * a + w;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * x[e];
    }
    sm[warp] = m;
    sl[warp] = l;
#pragma unroll
    for (int e = 0; e < E; ++e) sacc[warp][lane * E + e] = acc[e];
    __syncthreads();
    if (warp != 0) return;
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < 8; ++w) M = fmaxf(M, sm[w]);
    const float ref = M == -INFINITY ? 0.f : M;
    float o[E] = {};
    for (int w = 0; w < 8; ++w) {
        const float a = exp2f(sm[w] - ref);
        L += sl[w] * a;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += a * sacc[w][lane * E + e];
    }
    const bool none = L == 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
        p.O[row * D + lane * E + e] = __float2bfloat16_rn(none ? 0.f : o[e] / L);
    if (lane == 0 && p.LSE)
        p.LSE[row] = none ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

}  // namespace

int64_t fa_paged_ws_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int, int64_t, int64_t) {
    return 0;
}

int fa_paged_launch(const void* Q, void* O, float* LSE, const KvPages& pg,
                    const int32_t* kv_lens, const int32_t* q_lens, int64_t B, int64_t H,
                    int64_t Nq, int64_t d, float scale, bool causal, void*,
                    cudaStream_t stream) {
    PagedParams p{static_cast<const __nv_bfloat16*>(Q), static_cast<__nv_bfloat16*>(O), LSE,
                  kv_lens, q_lens, B, static_cast<int>(H), static_cast<int>(Nq), causal ? 1 : 0,
                  scale * 1.4426950408889634f, pg};
    const unsigned grid = static_cast<unsigned>(B * H * Nq);
    if (d == 64)
        paged_row_kernel<64><<<grid, 256, 0, stream>>>(p);
    else
        paged_row_kernel<128><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace osm
