// osm_rope.cu -- rotary positions: osm_rope and its adjoint osm_rope_bwd.
//
// Pair (a, b) of a head at position p, pair i with rate w_i, turns by t = p w_i:
//     (a, b) -> amplitude (a cos t - b sin t, b cos t + a sin t)
// The map is linear; its adjoint, which the backward pass applies to the output's gradient, turns
// by -t with the same amplitude.  Values past the first rot of a head are copied.
#include <cuda_runtime.h>

#include "kv_cache.cuh"
#include "osm_internal.h"

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
