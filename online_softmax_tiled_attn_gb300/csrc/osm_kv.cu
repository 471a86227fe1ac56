// osm_kv.cu -- appending to the paged key/value cache (osm_kv_append) and reading it out
// (osm_kv_gather).
//
// Append: token n of sequence b (n < new_lens[b]) takes position p = cache_lens[b] + n; its key is
// rotated by p, and key and value go to place p % P of page table[b][p / P], as bf16 or in 4 bits
// (kv_cache.cuh).  Optionally the token's queries are rotated too, into [B, H, N, d].
#include <cuda_runtime.h>

#include "kv_cache.cuh"
#include "osm_internal.h"
#include "ptx_sm103.cuh"

namespace osm {
namespace {

struct AppendParams {
    const __nv_bfloat16 *k, *v, *q;  // q may be nullptr
    int64_t ks[3], vs[3], qs[3];     // strides over b, h, n in elements
    __nv_bfloat16* q_out;            // [B, H, N, d]
    int64_t B, N;
    int H, H_kv;                     // H = 0 without q
    const int32_t *cache_lens, *new_lens;
    const int64_t* table;            // rates of the rot / 2 pairs
    int rot, layout;
    float amplitude;
    KvPages pg;
};

// A row is one head of one token's query, key or value.  d / 16 threads take it, 16 values each:
// octets 2 u and 2 u + 1 of the row (octet o holds values 8 o .. 8 o + 7).
//
// Rotated keys in 4 bits are computed in 32 bits, and again in 64 where that could change what is
// stored: a value within kTieWindow steps of the border between two codes, and a group whose step
// would be another one within kStepWindow units of the last place.
constexpr float kTieWindow = 4e-5f;     // |x / s| <= 46 times a few 2^-24
constexpr uint32_t kStepWindow = 32u;

template <int D>
__global__ void __launch_bounds__(256) kv_append_any_kernel(const AppendParams p) {
    constexpr int T = D / 16;       // threads a row
    constexpr int G = D / kKvGroup;
    const int heads = p.H + 2 * p.H_kv;
    const int64_t rows = p.B * p.N * heads;
    const int u = threadIdx.x % T;
    const unsigned lanes = ((1u << T) - 1u) << ((threadIdx.x & 31) / T * T);
    for (int64_t r = (blockIdx.x * 256LL + threadIdx.x) / T; r < rows;
         r += gridDim.x * 256LL / T) {
        const int head = static_cast<int>(r % heads);
        const int64_t n = (r / heads) % p.N, b = r / heads / p.N;
        const int fresh = p.new_lens ? p.new_lens[b] : static_cast<int>(p.N);
        if (n >= fresh) continue;  // the same for the row's threads
        const int64_t place = static_cast<int64_t>(max(p.cache_lens[b], 0)) + n;
        const bool is_q = head < p.H, is_k = !is_q && head < p.H + p.H_kv;
        const int h = is_q ? head : (is_k ? head - p.H : head - p.H - p.H_kv);
        const __nv_bfloat16* x =
            is_q ? p.q + b * p.qs[0] + h * p.qs[1] + n * p.qs[2]
                 : (is_k ? p.k + b * p.ks[0] + h * p.ks[1] + n * p.ks[2]
                         : p.v + b * p.vs[0] + h * p.vs[1] + n * p.vs[2]);
        const int rot = is_q || is_k ? p.rot : 0;
        auto load = [&](int j) { return __bfloat162float(x[j]); };
        auto exact = [&](int j) {
            return rope_value<double>(load, j, place, p.table, rot, p.layout,
                                      static_cast<double>(p.amplitude));
        };
        float val[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
            val[e] = rope_value<float>(load, 16 * u + e, place, p.table, rot, p.layout,
                                       p.amplitude);
        __nv_bfloat16* dst = nullptr;
        uint8_t* block = nullptr;
        if (is_q) {
            dst = p.q_out + ((b * p.H + h) * p.N + n) * D;
        } else {
            const int64_t pi = place / p.pg.page;
            const int32_t id = pi < p.pg.max_pages ? p.pg.table[b * p.pg.max_pages + pi] : -1;
            if (id < 0 || id >= p.pg.num_pages) {
                if (u == 0) kv_bad_page(p.pg);
                continue;
            }
            block = (is_k ? p.pg.k : p.pg.v) + kv_head_offset(p.pg, id, h);
            if (p.pg.format == OSM_KV_BF16)
                dst = reinterpret_cast<__nv_bfloat16*>(block) + (place % p.pg.page) * D;
        }
        if (dst != nullptr) {
#pragma unroll
            for (int o = 0; o < 2; ++o)
                reinterpret_cast<uint4*>(dst + 16 * u)[o] =
                    make_uint4(pack_bf16x2(val[8 * o], val[8 * o + 1]),
                               pack_bf16x2(val[8 * o + 2], val[8 * o + 3]),
                               pack_bf16x2(val[8 * o + 4], val[8 * o + 5]),
                               pack_bf16x2(val[8 * o + 6], val[8 * o + 7]));
            continue;
        }
        // 4 bits.  A thread's 16 values lie in one group; four threads make a group.
        float lo = val[0], hi = val[0];
#pragma unroll
        for (int e = 1; e < 16; ++e) {
            lo = min_nan(lo, val[e]);
            hi = max_nan(hi, val[e]);
        }
#pragma unroll
        for (int m = 1; m < T / G; m <<= 1) {
            lo = min_nan(lo, __shfl_xor_sync(lanes, lo, m));
            hi = max_nan(hi, __shfl_xor_sync(lanes, hi, m));
        }
        float need = kv4_need(lo, hi);
        if (rot > 0) {
            const uint32_t near = (__float_as_uint(need) + kStepWindow) & 0x1fffffu;
            if (__any_sync(lanes, near <= 2 * kStepWindow && need < INFINITY)) {
                double dlo = 0, dhi = 0;
                for (int e = 0; e < 16; ++e) {
                    const double t = exact(16 * u + e);
                    dlo = e == 0 ? t : fmin(dlo, t);
                    dhi = e == 0 ? t : fmax(dhi, t);
                }
                for (int m = 1; m < T / G; m <<= 1) {
                    dlo = fmin(dlo, __shfl_xor_sync(lanes, dlo, m));
                    dhi = fmax(dhi, __shfl_xor_sync(lanes, dhi, m));
                }
                // upwards: a bound just above a step of three bits must not round down to it
                if (need < INFINITY)
                    need = __double2float_ru(fmax((dhi - dlo) / 15., fabs(dlo) / 31.));
            }
        }
        const uint32_t bits = kv4_step_bits(need);
        const float s = kv4_step(bits), inv = 1.f / s;
        const bool live = bits != 0u && bits != 0x3feu;
        int q[16], base = 1 << 20;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            q[e] = live ? kv4_round(val[e], s, inv) : 0;
            if (rot > 0 && live) {
                const float t = val[e] * inv;
                if (fabsf(fabsf(t - rintf(t)) - 0.5f) < kTieWindow)
                    q[e] = static_cast<int>(rint(exact(16 * u + e) / static_cast<double>(s)));
            }
            base = min(base, q[e]);
        }
#pragma unroll
        for (int m = 1; m < T / G; m <<= 1) base = min(base, __shfl_xor_sync(lanes, base, m));
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 16; ++e)
            w[e >> 3] |= static_cast<uint32_t>(min(q[e] - base, 15)) << (4 * (e & 7));
        const int at = static_cast<int>(place % p.pg.page);
        *reinterpret_cast<uint2*>(block + at * (D / 2) + 8 * u) = make_uint2(w[0], w[1]);
        if (u % (T / G) == 0)
            reinterpret_cast<uint16_t*>(block + static_cast<int64_t>(p.pg.page) * (D / 2))
                [at * G + u / (T / G)] = static_cast<uint16_t>(kv4_word(bits, base));
    }
}

struct GatherParams {
    KvPages pg;
    const int32_t* kv_lens;
    __nv_bfloat16 *K, *V;  // [B, H_kv, N, d]
    int64_t B, N;
};

// Eight values a thread: d / 8 threads a token's head, keys and values in turn.
template <int D>
__global__ void __launch_bounds__(256) kv_gather_kernel(const GatherParams p) {
    constexpr int T = D / 8;
    const int64_t half = p.B * p.pg.H_kv * p.N * T;
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < 2 * half; i += gridDim.x * 256LL) {
        const bool is_v = i >= half;
        const int64_t j = is_v ? i - half : i;
        const int u = static_cast<int>(j % T);
        const int64_t n = (j / T) % p.N;
        const int h = static_cast<int>(j / T / p.N % p.pg.H_kv);
        const int64_t b = j / T / p.N / p.pg.H_kv;
        uint4 out = make_uint4(0u, 0u, 0u, 0u);
        if (n < p.kv_lens[b]) {
            const int64_t pi = n / p.pg.page;
            const int at = static_cast<int>(n % p.pg.page);
            const int32_t id = pi < p.pg.max_pages ? p.pg.table[b * p.pg.max_pages + pi] : -1;
            if (id < 0 || id >= p.pg.num_pages) {
                if (u == 0) kv_bad_page(p.pg);
            } else {
                const uint8_t* block = (is_v ? p.pg.v : p.pg.k) + kv_head_offset(p.pg, id, h);
                if (p.pg.format == OSM_KV_BF16) {
                    out = *reinterpret_cast<const uint4*>(block + (at * D + 8 * u) * 2);
                } else {
                    const uint32_t c = *reinterpret_cast<const uint32_t*>(block + at * (D / 2) + 4 * u);
                    const uint32_t word = reinterpret_cast<const uint16_t*>(
                        block + static_cast<int64_t>(p.pg.page) * (D / 2))
                        [at * (D / kKvGroup) + u / 8];
                    const float s = kv4_word_step(word);
                    const int base = kv4_word_base(word);
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = pack_bf16x2(
                            s * static_cast<float>(base + static_cast<int>((c >> (8 * e)) & 15u)),
                            s * static_cast<float>(base + static_cast<int>((c >> (8 * e + 4)) & 15u)));
                    out = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
        reinterpret_cast<uint4*>(is_v ? p.V : p.K)[j] = out;
    }
}

unsigned grid_of(int64_t threads) {
    const int64_t g = (threads + 255) / 256;
    return static_cast<unsigned>(g > 152 * 64 ? 152 * 64 : g);
}

}  // namespace

int osm_kv_append_launch(const void* k, const void* v, const int64_t* ks, const int64_t* vs,
                         const KvPages& pg, const int32_t* cache_lens, const int32_t* new_lens,
                         const int64_t* table, int64_t rot, int layout, float amplitude,
                         const void* q, void* q_out, const int64_t* qs, int64_t B, int64_t H,
                         int64_t N, int64_t d, cudaStream_t stream) {
    AppendParams p{};
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.q_out = static_cast<__nv_bfloat16*>(q_out);
    for (int i = 0; i < 3; ++i) {
        p.ks[i] = ks[i];
        p.vs[i] = vs[i];
        p.qs[i] = q ? qs[i] : 0;
    }
    p.B = B;
    p.N = N;
    p.H = q ? static_cast<int>(H) : 0;
    p.H_kv = pg.H_kv;
    p.cache_lens = cache_lens;
    p.new_lens = new_lens;
    p.table = table;
    p.rot = static_cast<int>(rot);
    p.layout = layout;
    p.amplitude = amplitude;
    p.pg = pg;
    const int64_t threads = B * N * (p.H + 2LL * p.H_kv) * (d / 16);
    if (d == 64)
        kv_append_any_kernel<64><<<grid_of(threads), 256, 0, stream>>>(p);
    else
        kv_append_any_kernel<128><<<grid_of(threads), 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int osm_kv_gather_launch(const KvPages& pg, const int32_t* kv_lens, void* K, void* V, int64_t B,
                         int64_t N, int64_t d, cudaStream_t stream) {
    GatherParams p{pg, kv_lens, static_cast<__nv_bfloat16*>(K), static_cast<__nv_bfloat16*>(V), B,
                   N};
    const int64_t threads = 2 * B * pg.H_kv * N * (d / 8);
    if (d == 64)
        kv_gather_kernel<64><<<grid_of(threads), 256, 0, stream>>>(p);
    else
        kv_gather_kernel<128><<<grid_of(threads), 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace osm
