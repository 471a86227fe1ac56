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
// would take as long as the memory.  Measured: 2 x 8192 tokens of 32 heads of 128, bf16: 43.6 us,
// 6.2 TB/s (91 % of a copy's); 3 x 2047 of 16 fp32 heads of 64, 32 of them rotated: 10.1 us, 5.0 TB/s
// (74 %: two waves of a short launch); 64 single tokens: 2.7 us, the launch.
#include <cuda_runtime.h>

#include <type_traits>

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

// A run: the 16 bytes of 8 bf16 or 4 fp32 values.
template <typename T>
struct Run;
template <>
struct Run<__nv_bfloat16> {
    static constexpr int kValues = 8;
    static __device__ __forceinline__ void get(const uint4& x, float* v) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(w[e] << 16);
            v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float* v) {
        return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                          pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
};
template <>
struct Run<float> {
    static constexpr int kValues = 4;
    static __device__ __forceinline__ void get(const uint4& x, float* v) {
        v[0] = __uint_as_float(x.x), v[1] = __uint_as_float(x.y);
        v[2] = __uint_as_float(x.z), v[3] = __uint_as_float(x.w);
    }
    static __device__ __forceinline__ uint4 put(const float* v) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                          __float_as_uint(v[3]));
    }
};

// d and rot multiples of 16, rows on 16-byte boundaries, below 2^32 units a head.  Thread: (token,
// unit of 16 values), units fastest; blockIdx.y: group of HEADS heads.  A unit's runs are chosen so
// that neighbouring threads' lie side by side and each access of a warp is whole lines: in the half
// layout the first rot / 16 units take runs of both halves of the same 8 pairs, the others share the
// copied rest; in the interleaved layout all units share the head.
template <typename T, int HEADS, bool HALF>
__global__ void __launch_bounds__(256, 3) rope_kernel(const RopeParams p, uint32_t units) {
    constexpr int V = Run<T>::kValues, R = 16 / V;
    const uint32_t i = blockIdx.x * 256u + threadIdx.x;
    const uint32_t tok = i / units;
    const int u = static_cast<int>(i - tok * units), U = static_cast<int>(units);
    const uint32_t b = tok / static_cast<uint32_t>(p.N);
    if (b >= p.B) return;
    const uint32_t n = tok - b * static_cast<uint32_t>(p.N);
    const int h0 = blockIdx.y * HEADS;
    const int P = HALF ? p.rot / 16 : 0;  // units that take pairs of the half layout
    const bool paired = HALF && u < P;
    // Run r of the thread: r * stride past the first (and, for pairs, the second half's runs after
    // those of the first).
    const int run0 = HALF && !paired ? u + P * (R - 1) : u;
    const int stride = paired ? P : (HALF ? U - P : U);
    auto run = [&](int r) {
        return run0 + (paired ? r % (R / 2) * stride + r / (R / 2) * (R / 2) * P : r * stride);
    };
    const T* x = static_cast<const T*>(p.x) + b * p.xs[0] + n * p.xs[2] + h0 * p.xs[1];
    T* y = static_cast<T*>(p.y) + b * p.ys[0] + n * p.ys[2] + h0 * p.ys[1];
    const int heads = static_cast<int>(min(static_cast<int64_t>(HEADS), p.H - h0));
    // kBatch heads on their way while the angles, and then the heads before them, are computed
    constexpr int kBatch = HEADS < 2 ? 1 : 2;
    uint4 raw[kBatch][R];
    auto load = [&](int g) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (g + k < heads)
#pragma unroll
                for (int r = 0; r < R; ++r)
                    raw[k][r] = reinterpret_cast<const uint4*>(x + (g + k) * p.xs[1])[run(r)];
    };
    load(0);
    float c[8], s[8];
    if (paired || !HALF) {
        const int64_t pos =
            p.positions ? p.positions[b * p.pos_bs + n] : static_cast<int64_t>(n);
        const float down = p.inverse ? -p.amplitude : p.amplitude;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // pair e of the thread: in the half layout value e of its first runs, else a run's
            // V / 2 pairs after another's
            const int pair = HALF ? run(e / V) * V + e % V : run(e / (V / 2)) * (V / 2) + e % (V / 2);
            c[e] = 1.f;
            s[e] = 0.f;
            if (2 * pair >= p.rot) continue;  // a copied run
            rope_cos_sin(rope_phase(pos, p.table[pair]), c[e], s[e]);
            c[e] *= p.amplitude;
            s[e] *= down;
        }
    }
#pragma unroll
    for (int g = 0; g < HEADS; g += kBatch) {
        uint4 now[kBatch][R];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
#pragma unroll
            for (int r = 0; r < R; ++r) now[k][r] = raw[k][r];
        if (g + kBatch < HEADS) load(g + kBatch);
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (g + k < heads) {
                uint4* out = reinterpret_cast<uint4*>(y + (g + k) * p.ys[1]);
                float v[16];
#pragma unroll
                for (int r = 0; r < R; ++r) Run<T>::get(now[k][r], v + r * V);
                if (paired) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float a = v[e], o = v[8 + e];
                        v[e] = a * c[e] - o * s[e];
                        v[8 + e] = o * c[e] + a * s[e];
                    }
                } else if (!HALF) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float a = v[2 * e], o = v[2 * e + 1];
                        v[2 * e] = a * c[e] - o * s[e];
                        v[2 * e + 1] = o * c[e] + a * s[e];
                    }
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    // a copied run goes as it is (a NaN's bits too)
                    const bool copied = HALF ? !paired : run(r) * V >= p.rot;
                    out[run(r)] = copied ? now[k][r] : Run<T>::put(v + r * V);
                }
            }
    }
}

template <typename T>
int launch_units(const RopeParams& p, cudaStream_t stream) {
    const uint32_t units = static_cast<uint32_t>(p.d / 16);
    const int64_t one = p.B * p.N * units;  // threads at all heads a thread
    // as many heads a thread as leave 32 warps an SM's worth of threads (2 x 8192 tokens, 32 heads
    // of 128, us: 8 heads a thread 43.6, 4 45.8, 2 50.7, 1 74; 3 x 2047, 16 fp32 heads of 64: 10.1,
    // with 64 warps 10.3)
    auto fits = [&](int heads) { return one * ((p.H + heads - 1) / heads) >= 152 * 1024; };
    const int heads = fits(8) ? 8 : (fits(4) ? 4 : (fits(2) ? 2 : 1));
    const dim3 g(static_cast<unsigned>((one + 255) / 256),
                 static_cast<unsigned>((p.H + heads - 1) / heads));
    auto run = [&](auto half) {
        constexpr bool HALF = decltype(half)::value;
        if (heads == 8) rope_kernel<T, 8, HALF><<<g, 256, 0, stream>>>(p, units);
        else if (heads == 4) rope_kernel<T, 4, HALF><<<g, 256, 0, stream>>>(p, units);
        else if (heads == 2) rope_kernel<T, 2, HALF><<<g, 256, 0, stream>>>(p, units);
        else rope_kernel<T, 1, HALF><<<g, 256, 0, stream>>>(p, units);
    };
    if (p.layout == OSM_ROPE_HALF) run(std::true_type{});
    else run(std::false_type{});
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
