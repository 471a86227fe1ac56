// osm_rope.cu -- rotary positions: osm_rope and its adjoint osm_rope_bwd.
//
// Pair (a, b) of a head at position p, pair i with rate w_i, turns by t = p w_i:
//     (a, b) -> amplitude (a cos t - b sin t, b cos t + a sin t)
// The map is linear; its adjoint, which the backward pass applies to the output's gradient, turns
// by -t with the same amplitude.  Values past the first rot of a head are copied.
//
// Bound by memory: each value is read and written once.  A thread takes 16 values of a head (two
// runs of 8: a pair's first and second halves, or 16 in a row) and goes through several heads of
// its token, whose angles are the same: at one head a thread the sines and cosines (8 a thread)
// would take as long as the memory.
#include <cuda_runtime.h>

#include "kv_cache.cuh"
#include "osm_internal.h"
#include "ptx_sm103.cuh"

namespace osm {
namespace {

struct RopeParams {
    const void* x;
    void* y;
    int64_t xs[3], ys[3];  // strides over b, h, n in elements
    int64_t B, H, N;
    int d, rot, layout;
    const int32_t* positions;  // or nullptr: position n
    int64_t pos_bs;
    const int64_t* table;
    float amplitude;
    int inverse;
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

// 8 consecutive values.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// d and rot multiples of 16, rows on 16-byte boundaries, below 2^32 units a head.  Thread: (token,
// unit of 16 values), units fastest; blockIdx.y: group of HEADS heads.
template <typename T, int HEADS>
__global__ void __launch_bounds__(256) rope_kernel(const RopeParams p, uint32_t units) {
    const uint32_t i = blockIdx.x * 256u + threadIdx.x;
    const uint32_t tok = i / units, u = i - tok * units;
    const uint32_t b = tok / static_cast<uint32_t>(p.N);
    if (b >= p.B) return;
    const uint32_t n = tok - b * static_cast<uint32_t>(p.N);
    const int h0 = blockIdx.y * HEADS;
    const bool turned = 16 * u < p.rot, half = p.layout == OSM_ROPE_HALF;
    const int i0 = turned && half ? 8 * u : 16 * u;
    const int i1 = turned && half ? p.rot / 2 + 8 * u : 16 * u + 8;
    float c[8], s[8];
    if (turned) {
        const int64_t pos =
            p.positions ? p.positions[b * p.pos_bs + n] : static_cast<int64_t>(n);
        const float down = p.inverse ? -p.amplitude : p.amplitude;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            rope_cos_sin(rope_phase(pos, p.table[8 * u + e]), c[e], s[e]);
            c[e] *= p.amplitude;
            s[e] *= down;
        }
    }
    const T* x = static_cast<const T*>(p.x) + b * p.xs[0] + n * p.xs[2] + h0 * p.xs[1];
    T* y = static_cast<T*>(p.y) + b * p.ys[0] + n * p.ys[2] + h0 * p.ys[1];
    const int heads = static_cast<int>(min(static_cast<int64_t>(HEADS), p.H - h0));
    float v[HEADS > 4 ? 4 : HEADS][2][8];
#pragma unroll
    for (int g = 0; g < HEADS; g += 4) {
#pragma unroll
        for (int k = 0; k < (HEADS > 4 ? 4 : HEADS); ++k)
            if (g + k < heads) {
                load8(x + (g + k) * p.xs[1] + i0, v[k][0]);
                load8(x + (g + k) * p.xs[1] + i1, v[k][1]);
            }
#pragma unroll
        for (int k = 0; k < (HEADS > 4 ? 4 : HEADS); ++k)
            if (g + k < heads) {
                if (turned && half) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float a = v[k][0][e], o = v[k][1][e];
                        v[k][0][e] = a * c[e] - o * s[e];
                        v[k][1][e] = o * c[e] + a * s[e];
                    }
                } else if (turned) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float a = v[k][e >> 2][2 * (e & 3)], o = v[k][e >> 2][2 * (e & 3) + 1];
                        v[k][e >> 2][2 * (e & 3)] = a * c[e] - o * s[e];
                        v[k][e >> 2][2 * (e & 3) + 1] = o * c[e] + a * s[e];
                    }
                }
                store8(y + (g + k) * p.ys[1] + i0, v[k][0]);
                store8(y + (g + k) * p.ys[1] + i1, v[k][1]);
            }
    }
}

template <typename T>
int launch_units(const RopeParams& p, cudaStream_t stream) {
    const uint32_t units = static_cast<uint32_t>(p.d / 16);
    const int64_t one = p.B * p.N * units;  // threads at all heads a thread
    // as many heads a thread as leave 64 warps an SM's worth of threads
    auto fits = [&](int heads) { return one * ((p.H + heads - 1) / heads) >= 152 * 2048; };
    const int heads = fits(8) ? 8 : (fits(4) ? 4 : (fits(2) ? 2 : 1));
    const dim3 g(static_cast<unsigned>((one + 255) / 256),
                 static_cast<unsigned>((p.H + heads - 1) / heads));
    if (heads == 8) rope_kernel<T, 8><<<g, 256, 0, stream>>>(p, units);
    else if (heads == 4) rope_kernel<T, 4><<<g, 256, 0, stream>>>(p, units);
    else if (heads == 2) rope_kernel<T, 2><<<g, 256, 0, stream>>>(p, units);
    else rope_kernel<T, 1><<<g, 256, 0, stream>>>(p, units);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Any alignment, strides and rotated width: one thread a pair (or a copied value).
template <typename T>
__global__ void __launch_bounds__(256) rope_any_kernel(const RopeParams p) {
    const int half = p.rot >> 1, units = half + p.d - p.rot;
    const int64_t total = p.B * p.N * p.H * units;
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < total; i += gridDim.x * 256LL) {
        const int u = static_cast<int>(i % units);
        const int64_t row = i / units;
        const int64_t h = row % p.H, n = (row / p.H) % p.N, b = row / p.H / p.N;
        const T* x = static_cast<const T*>(p.x) + b * p.xs[0] + h * p.xs[1] + n * p.xs[2];
        T* y = static_cast<T*>(p.y) + b * p.ys[0] + h * p.ys[1] + n * p.ys[2];
        if (u >= half) {
            y[p.rot + u - half] = x[p.rot + u - half];
            continue;
        }
        const int32_t pos = p.positions ? p.positions[b * p.pos_bs + n] : static_cast<int32_t>(n);
        float c, s;
        rope_cos_sin(rope_phase(pos, p.table[u]), c, s);
        c *= p.amplitude;
        s *= p.inverse ? -p.amplitude : p.amplitude;
        const int i0 = p.layout == OSM_ROPE_HALF ? u : 2 * u;
        const int i1 = p.layout == OSM_ROPE_HALF ? u + half : 2 * u + 1;
        const float a = to_float(x[i0]), o = to_float(x[i1]);
        y[i0] = from_float<T>(a * c - o * s);
        y[i1] = from_float<T>(o * c + a * s);
    }
}

}  // namespace

int osm_rope_launch(const void* x, void* y, int dtype, int64_t B, int64_t H, int64_t N, int64_t d,
                    const int64_t* xs, const int64_t* ys, const int32_t* positions,
                    int64_t pos_bs, const int64_t* table, int64_t rot, int layout,
                    float amplitude, bool inverse, cudaStream_t stream) {
    RopeParams p{x, y, {xs[0], xs[1], xs[2]}, {ys[0], ys[1], ys[2]}, B, H, N,
                 static_cast<int>(d), static_cast<int>(rot), layout, positions, pos_bs, table,
                 amplitude, inverse ? 1 : 0};
    const int64_t vec = dtype == OSM_BF16 ? 8 : 4;  // elements in 16 bytes
    bool units = d % 16 == 0 && rot % 16 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                 reinterpret_cast<uintptr_t>(y) % 16 == 0 && H <= 65535 &&
                 B * N <= (int64_t(1) << 32) / d;
    const int64_t n[3] = {B, H, N};
    for (int i = 0; i < 3; ++i)
        units = units && (n[i] == 1 || (xs[i] % vec == 0 && ys[i] % vec == 0));
    if (units)
        return dtype == OSM_BF16 ? launch_units<__nv_bfloat16>(p, stream)
                                 : launch_units<float>(p, stream);
    const int64_t total = B * H * N * (d - rot / 2);
    int64_t grid = (total + 255) / 256;
    if (grid > 152 * 64) grid = 152 * 64;
    if (dtype == OSM_BF16)
        rope_any_kernel<__nv_bfloat16><<<static_cast<unsigned>(grid), 256, 0, stream>>>(p);
    else
        rope_any_kernel<float><<<static_cast<unsigned>(grid), 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace osm
