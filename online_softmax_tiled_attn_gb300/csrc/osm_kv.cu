// osm_kv.cu -- appending to the paged key/value cache (osm_kv_append) and reading it out
// (osm_kv_gather).
//
// Append: token n of sequence b (n < new_lens[b]) takes position p = cache_lens[b] + n; its key is
// rotated by p, and key and value go to place p % P of page table[b][p / P], as bf16 or in 4 bits
// (kv_cache.cuh).  Optionally the token's queries are rotated too, into [B, H, N, d].
//
// Bound by memory at long prompts, by the launch at single tokens.  A row (one head of one token's
// query, key or value) is taken by d / 16 threads, 16 values each; a thread goes through several
// rows of its token, whose angles are the same.
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

// Rotated keys in 4 bits are computed in 32 bits, and again in 64 where that could change what is
// stored: a value within kTieWindow steps of the border between two codes, and a group whose step
// would be another one within kStepWindow units of the last place.
constexpr float kTieWindow = 4e-5f;     // |x / s| <= 46 times a few 2^-24
constexpr uint32_t kStepWindow = 32u;

// 16 values of a row, as two runs of 8: octets o0 and o1 (octet o: values 8 o .. 8 o + 7).  FAST:
// the first rot / 16 threads of a row in the half layout take the two halves of 8 pairs, all others
// two octets in a row, loaded 16 bytes at a time; otherwise (a rotated width that is no multiple of
// 16, rows off a 16-byte boundary) two octets in a row, value by value.
template <int D>
struct Row {
    const AppendParams& p;
    const __nv_bfloat16* x;
    int64_t place;
    int rot;

    __device__ __forceinline__ double exact(int i) const {
        auto load = [&](int j) { return __bfloat162float(x[j]); };
        return rope_value<double>(load, i, place, p.table, rot, p.layout,
                                  static_cast<double>(p.amplitude));
    }
};

// The row's values in 4 bits into its place of a page head.  All threads of the row take part;
// turned: this one's values are rotated (others are exact as they are).
template <int D>
__device__ __forceinline__ void store_int4(const Row<D>& row, const float (&val)[2][8], int o0,
                                           int o1, bool turned, uint8_t* block, int at,
                                           unsigned lanes) {
    constexpr int T = D / 16, G = D / kKvGroup;
    const int oct[2] = {o0, o1};
    float lo[G], hi[G];
#pragma unroll
    for (int k = 0; k < G; ++k) {
        lo[k] = INFINITY;
        hi[k] = -INFINITY;
    }
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        float a = val[o][0], b = val[o][0];
#pragma unroll
        for (int e = 1; e < 8; ++e) {
            a = min_nan(a, val[o][e]);
            b = max_nan(b, val[o][e]);
        }
#pragma unroll
        for (int k = 0; k < G; ++k)
            if (G == 1 || oct[o] >> 3 == k) {
                lo[k] = min_nan(lo[k], a);
                hi[k] = max_nan(hi[k], b);
            }
    }
#pragma unroll
    for (int m = 1; m < T; m <<= 1)
#pragma unroll
        for (int k = 0; k < G; ++k) {
            lo[k] = min_nan(lo[k], __shfl_xor_sync(lanes, lo[k], m));
            hi[k] = max_nan(hi[k], __shfl_xor_sync(lanes, hi[k], m));
        }
    float need[G];
    bool close = false;
#pragma unroll
    for (int k = 0; k < G; ++k) {
        need[k] = kv4_need(lo[k], hi[k]);
        const uint32_t near = (__float_as_uint(need[k]) + kStepWindow) & 0x1fffffu;
        close |= near <= 2 * kStepWindow && need[k] < INFINITY;
    }
    if (row.rot > 0 && close) {  // the same in all threads of the row
#pragma unroll
        for (int k = 0; k < G; ++k) {
            double dlo = INFINITY, dhi = -INFINITY;
            for (int o = 0; o < 2; ++o)
                for (int e = 0; e < 8; ++e)
                    if (oct[o] >> 3 == k) {
                        const double t = row.exact(8 * oct[o] + e);
                        dlo = fmin(dlo, t);
                        dhi = fmax(dhi, t);
                    }
            for (int m = 1; m < T; m <<= 1) {
                dlo = fmin(dlo, __shfl_xor_sync(lanes, dlo, m));
                dhi = fmax(dhi, __shfl_xor_sync(lanes, dhi, m));
            }
            // upwards: a bound just above a step of three bits must not round down to it
            if (need[k] < INFINITY)
                need[k] = __double2float_ru(fmax((dhi - dlo) / 15., fabs(dlo) / 31.));
        }
    }
    uint32_t bits[G];
    float step[G], inv[G];
    int base[G];
#pragma unroll
    for (int k = 0; k < G; ++k) {
        bits[k] = kv4_step_bits(need[k]);
        step[k] = kv4_step(bits[k]);
        inv[k] = 1.f / step[k];
        if (bits[k] == 0u || bits[k] == 0x3feu) inv[k] = 0.f;  // all codes 0
        base[k] = inv[k] == 0.f ? 0 : kv4_round(lo[k], step[k], inv[k]);
    }
    int q[2][8];
    bool tie = false;
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        const bool second = G == 2 && oct[o] >> 3;
        const float s = second ? step[G - 1] : step[0], r = second ? inv[G - 1] : inv[0];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float t = val[o][e] * r;
            q[o][e] = kv4_round(val[o][e], s, r);
            tie |= turned && fabsf(fabsf(t - rintf(t)) - 0.5f) < kTieWindow;
        }
        if (r == 0.f)
#pragma unroll
            for (int e = 0; e < 8; ++e) q[o][e] = 0;
    }
    if (row.rot > 0 && __any_sync(lanes, tie)) {
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const bool second = G == 2 && oct[o] >> 3;
            const float s = second ? step[G - 1] : step[0], r = second ? inv[G - 1] : inv[0];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = val[o][e] * r;
                if (turned && r != 0.f && fabsf(fabsf(t - rintf(t)) - 0.5f) < kTieWindow)
                    q[o][e] = static_cast<int>(
                        rint(row.exact(8 * oct[o] + e) / static_cast<double>(s)));
            }
        }
#pragma unroll
        for (int k = 0; k < G; ++k) {
            int least = 1 << 20;
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (G == 1 || oct[o] >> 3 == k) least = min(least, q[o][e]);
#pragma unroll
            for (int m = 1; m < T; m <<= 1) least = min(least, __shfl_xor_sync(lanes, least, m));
            base[k] = least;
        }
    }
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        const int b = G == 2 && oct[o] >> 3 ? base[G - 1] : base[0];
        uint32_t w = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e) w |= static_cast<uint32_t>(min(q[o][e] - b, 15)) << (4 * e);
        *reinterpret_cast<uint32_t*>(block + at * (D / 2) + 4 * oct[o]) = w;
    }
    if (threadIdx.x % T == 0) {
        uint8_t* word = block + static_cast<int64_t>(row.p.pg.page) * (D / 2) + at * (G * 2);
        if constexpr (G == 2)
            *reinterpret_cast<uint32_t*>(word) =
                kv4_word(bits[0], base[0]) | kv4_word(bits[1], base[1]) << 16;
        else
            *reinterpret_cast<uint16_t*>(word) = static_cast<uint16_t>(kv4_word(bits[0], base[0]));
    }
}

__device__ __forceinline__ void unpack8(const uint4& x, float (&v)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}

// Thread: (token, 16 values), the threads of a row fastest; blockIdx.y: group of `per` rows of the
// token, which are its queries, then keys, then values.
template <int D, bool FAST>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendParams p, int per) {
    constexpr int T = D / 16;  // threads a row
    const int heads = p.H + 2 * p.H_kv;
    const int u = threadIdx.x % T;
    const unsigned lanes = ((1u << T) - 1u) << ((threadIdx.x & 31) / T * T);
    const uint32_t tok = (blockIdx.x * 256u + threadIdx.x) / T;
    const uint32_t b = tok / static_cast<uint32_t>(p.N);
    if (b >= p.B) return;  // whole rows' threads leave together, here and below
    const uint32_t n = tok - b * static_cast<uint32_t>(p.N);
    const int group = blockIdx.y;
    if (p.new_lens && static_cast<int64_t>(n) >= p.new_lens[b]) return;
    const int64_t place = static_cast<int64_t>(max(p.cache_lens[b], 0)) + n;
    // the token's page
    // (places of a table lie below 2^31)
    const uint32_t pi = static_cast<uint32_t>(place) / static_cast<uint32_t>(p.pg.page);
    const int at = static_cast<int>(place - static_cast<int64_t>(pi) * p.pg.page);
    const int32_t id =
        pi < p.pg.max_pages ? p.pg.table[static_cast<int64_t>(b) * p.pg.max_pages + pi] : -1;
    const bool paged = id >= 0 && id < p.pg.num_pages;
    const bool half = p.layout == OSM_ROPE_HALF, turned = 16 * u < p.rot;
    float c[8], s[8];
    const int first = group * per, end = min(first + per, heads);
    if (FAST && turned && first < p.H + p.H_kv) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            rope_cos_sin(rope_phase(place, p.table[8 * u + e]), c[e], s[e]);
            c[e] *= p.amplitude;
            s[e] *= p.amplitude;
        }
    }
    if (!paged && end > p.H && u == 0) kv_bad_page(p.pg);
    for (int head = first; head < end; ++head) {
        const bool is_q = head < p.H, is_k = !is_q && head < p.H + p.H_kv;
        const int h = is_q ? head : (is_k ? head - p.H : head - p.H - p.H_kv);
        if (!is_q && !paged) continue;
        const __nv_bfloat16* x =
            is_q ? p.q + b * p.qs[0] + h * p.qs[1] + n * p.qs[2]
                 : (is_k ? p.k + b * p.ks[0] + h * p.ks[1] + n * p.ks[2]
                         : p.v + b * p.vs[0] + h * p.vs[1] + n * p.vs[2]);
        const Row<D> row{p, x, place, is_q || is_k ? p.rot : 0};
        const bool turn = turned && row.rot > 0;
        const int o0 = FAST && turn && half ? u : 2 * u;
        const int o1 = FAST && turn && half ? p.rot / 16 + u : 2 * u + 1;
        float val[2][8];
        if constexpr (FAST) {
            unpack8(reinterpret_cast<const uint4*>(x)[o0], val[0]);
            unpack8(reinterpret_cast<const uint4*>(x)[o1], val[1]);
            if (turn && half) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = val[0][e], o = val[1][e];
                    val[0][e] = a * c[e] - o * s[e];
                    val[1][e] = o * c[e] + a * s[e];
                }
            } else if (turn) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = val[e >> 2][2 * (e & 3)], o = val[e >> 2][2 * (e & 3) + 1];
                    val[e >> 2][2 * (e & 3)] = a * c[e] - o * s[e];
                    val[e >> 2][2 * (e & 3) + 1] = o * c[e] + a * s[e];
                }
            }
        } else {
            auto load = [&](int j) { return __bfloat162float(x[j]); };
#pragma unroll
            for (int e = 0; e < 16; ++e)
                val[e >> 3][e & 7] = rope_value<float>(load, 16 * u + e, place, p.table, row.rot,
                                                       p.layout, p.amplitude);
        }
        if (is_q || p.pg.format == OSM_KV_BF16) {
            __nv_bfloat16* dst =
                is_q ? p.q_out + ((static_cast<int64_t>(b) * p.H + h) * p.N + n) * D
                     : reinterpret_cast<__nv_bfloat16*>((is_k ? p.pg.k : p.pg.v) +
                                                        kv_head_offset(p.pg, id, h)) +
                           at * D;
            reinterpret_cast<uint4*>(dst)[o0] = pack8(val[0]);
            reinterpret_cast<uint4*>(dst)[o1] = pack8(val[1]);
        } else {
            store_int4<D>(row, val, o0, o1, FAST ? turn : row.rot > 0,
                          (is_k ? p.pg.k : p.pg.v) + kv_head_offset(p.pg, id, h), at, lanes);
        }
    }
}

struct GatherParams {
    KvPages pg;
    const int32_t* kv_lens;
    __nv_bfloat16 *K, *V;  // [B, H_kv, N, d]
    int64_t B, N;
};

// CTA: kGatherTokens tokens of one head of one sequence's keys or values; 16 values a thread.
constexpr int kGatherTokens = 64;

template <int D>
__global__ void __launch_bounds__(256) kv_gather_kernel(const GatherParams p, int tiles) {
    constexpr int T = D / 16, kPer = 256 / T;  // threads a token's head, tokens at a time
    const bool is_v = blockIdx.x & 1;
    const int64_t rest = blockIdx.x >> 1;
    const int64_t n0 = rest % tiles * kGatherTokens;
    const int64_t bh = rest / tiles;
    const int h = static_cast<int>(bh % p.pg.H_kv);
    const int64_t b = bh / p.pg.H_kv;
    const int u = threadIdx.x % T;
    const int64_t len = min(static_cast<int64_t>(p.kv_lens[b]), p.N);
    const int64_t end = min(n0 + kGatherTokens, p.N);
    uint4* out = reinterpret_cast<uint4*>((is_v ? p.V : p.K) + bh * p.N * D);
#pragma unroll
    for (int k = 0; k < kGatherTokens / kPer; ++k) {
        const int64_t n = n0 + k * kPer + threadIdx.x / T;
        if (n >= end) break;
        uint4 a = make_uint4(0u, 0u, 0u, 0u), c = a;
        if (n < len) {
            const uint32_t pi = static_cast<uint32_t>(n) / static_cast<uint32_t>(p.pg.page);
            const int at = static_cast<int>(n) - static_cast<int>(pi) * p.pg.page;
            const int32_t id = pi < p.pg.max_pages ? p.pg.table[b * p.pg.max_pages + pi] : -1;
            if (id < 0 || id >= p.pg.num_pages) {
                if (u == 0) kv_bad_page(p.pg);
            } else {
                const uint8_t* block = (is_v ? p.pg.v : p.pg.k) + kv_head_offset(p.pg, id, h);
                if (p.pg.format == OSM_KV_BF16) {
                    a = reinterpret_cast<const uint4*>(block + at * D * 2)[2 * u];
                    c = reinterpret_cast<const uint4*>(block + at * D * 2)[2 * u + 1];
                } else {
                    const uint2 codes = reinterpret_cast<const uint2*>(block + at * (D / 2))[u];
                    const uint32_t word = reinterpret_cast<const uint16_t*>(
                        block + static_cast<int64_t>(p.pg.page) * (D / 2))
                        [at * (D / kKvGroup) + u / 4];
                    const float s = kv4_word_step(word);
                    const float base = static_cast<float>(kv4_word_base(word));
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t x = (e < 4 ? codes.x : codes.y) >> (8 * (e & 3));
                        // (2^23 + code) - 2^23 + base, exactly
                        w[e] = pack_bf16x2(
                            s * (__uint_as_float(0x4b000000u | (x & 15u)) - (8388608.f - base)),
                            s * (__uint_as_float(0x4b000000u | (x >> 4 & 15u)) -
                                 (8388608.f - base)));
                    }
                    a = make_uint4(w[0], w[1], w[2], w[3]);
                    c = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
        }
        out[n * (D / 8) + 2 * u] = a;
        out[n * (D / 8) + 2 * u + 1] = c;
    }
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
    bool fast = rot % 16 == 0;
    const int64_t n[3] = {B, 0, N};
    for (int i = 0; i < 3; ++i) {
        fast = fast && ((i == 1 ? pg.H_kv : n[i]) == 1 || (ks[i] % 8 == 0 && vs[i] % 8 == 0)) &&
               (!q || (i == 1 ? H : n[i]) == 1 || qs[i] % 8 == 0);
    }
    for (const void* x : {k, v, q}) fast = fast && reinterpret_cast<uintptr_t>(x) % 16 == 0;
    const int64_t heads = p.H + 2LL * p.H_kv, one = B * N * (d / 16);
    // as many rows a thread as leave 64 warps an SM's worth of threads
    int per = 8;
    while (per > 1 && one * ((heads + per - 1) / per) < 152 * 2048) per >>= 1;
    if (one >= (int64_t(1) << 32) || (heads + per - 1) / per > 65535) return FA_ERR_UNSUPPORTED;
    const dim3 g(static_cast<unsigned>((one + 255) / 256),
                 static_cast<unsigned>((heads + per - 1) / per));
    if (d == 64 && fast) kv_append_kernel<64, true><<<g, 256, 0, stream>>>(p, per);
    else if (d == 64) kv_append_kernel<64, false><<<g, 256, 0, stream>>>(p, per);
    else if (fast) kv_append_kernel<128, true><<<g, 256, 0, stream>>>(p, per);
    else kv_append_kernel<128, false><<<g, 256, 0, stream>>>(p, per);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int osm_kv_gather_launch(const KvPages& pg, const int32_t* kv_lens, void* K, void* V, int64_t B,
                         int64_t N, int64_t d, cudaStream_t stream) {
    GatherParams p{pg, kv_lens, static_cast<__nv_bfloat16*>(K), static_cast<__nv_bfloat16*>(V), B,
                   N};
    const int64_t tiles = (N + kGatherTokens - 1) / kGatherTokens;
    const int64_t grid = 2 * B * pg.H_kv * tiles;
    if (grid > INT32_MAX) return FA_ERR_UNSUPPORTED;
    if (d == 64)
        kv_gather_kernel<64><<<static_cast<unsigned>(grid), 256, 0, stream>>>(
            p, static_cast<int>(tiles));
    else
        kv_gather_kernel<128><<<static_cast<unsigned>(grid), 256, 0, stream>>>(
            p, static_cast<int>(tiles));
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace osm
