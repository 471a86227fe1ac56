// osm_kv.cu -- appending to the paged key/value cache (osm_kv_append) and reading it out
// (osm_kv_gather).
//
// Append: token n of sequence b (n < new_lens[b]) takes position p = cache_lens[b] + n; its key is
// rotated by p, and key and value go to place p % P of page table[b][p / P], as bf16 or in 4 bits
// (kv_cache.cuh).  Optionally the token's queries are rotated too, into [B, H, N, d].
//
// Bound by memory at long prompts, by the launch at single tokens.  A row (one head of one token's
// query, key or value) is taken by d / 16 threads, 16 values each; a thread goes through several
// rows of its token, whose angles are the same.  Measured: prompts of up to 4096 tokens, 32 + 2 x 8
// heads of 128, into bf16 pages: 50.2 us, 5.7 TB/s (84 % of a copy's); 8192 tokens into 4-bit pages:
// queries 25 us, keys and values 31 us (bound by the quantiser, 33 instructions a value at 16 warps
// an SM), the read-out of all 12192 tokens 13 us; 64 single tokens 3.5 us, the launch.
#include <cuda_runtime.h>

#include <type_traits>

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
// stored.  What the 32-bit value a c - o s is off by goes with its pair, not with itself: c and s are
// off by 9.4e-8 (the angle) and 6e-8 (sincospif), and by 2^-24 of themselves from the amplitude, each
// product and sum by 2^-24 more, 2.8e-7 (|a| + |o|) amplitude in all.  |a| + |o| is at most sqrt(2)
// times the pair's length, which the rotation keeps, and that at most sqrt(2) times the largest value
// of the rotated row: kOff times that value, whichever group it is in (in the half layout at d = 128
// the partner is in the other one).
constexpr float kOff = 6e-7f;
// x / s is off by that over s, and by |x / s| <= 46 times 1 / s's 2^-23 and the product's 2^-24.
constexpr float kQuotientOff = 1e-5f;
// The step's bound is off by four units of the last place, and by a fifteenth of two values' kOff.
constexpr float kNeedOff = 5e-7f, kNeedOffRow = 1e-7f;

// How far a quotient may lie from its whole number and have no border of codes within what it is off
// by: most = the row's largest value, inv = 1 / s.
__device__ __forceinline__ float clear_of_ties(float most, float inv) {
    return 0.5f - kQuotientOff - kOff * most * inv;
}

// 16 values of a row, as two runs of 8: octets o0 and o1 (octet o: values 8 o .. 8 o + 7).  FAST: in
// the half layout the first rot / 16 threads of a row take the two halves of 8 pairs; all others
// take octets so that neighbouring threads' lie side by side (each access of a warp is then whole
// lines), 16 bytes at a time.  Otherwise (a rotated width that is no multiple of 16, rows off a
// 16-byte boundary) two octets in a row, value by value.
struct Row {
    const AppendParams& p;
    const __nv_bfloat16* x;
    int64_t place;
    int rot;
};

// Value i of a row in 64 bits (rare: kept out of line for the registers of the rest).
__device__ __noinline__ double row_exact(const __nv_bfloat16* x, int i, int64_t place,
                                         const int64_t* table, int rot, int layout,
                                         float amplitude) {
    auto load = [&](int j) { return __bfloat162float(x[j]); };
    return rope_value<double>(load, i, place, table, rot, layout, static_cast<double>(amplitude));
}

// The row's values in 4 bits into its place of a page head.  All threads of the row take part.
// TURNS: rows that may be rotated; turned: this thread's values are (others are exact as they are).
template <int D, bool TURNS>
__device__ __forceinline__ void store_int4(const Row& row, const float (&val)[2][8], int o0,
                                           int o1, bool turned, uint8_t* block, int at,
                                           unsigned lanes) {
    constexpr int T = D / 16, G = D / kKvGroup;
    const int oct[2] = {o0, o1};
    auto exact = [&](int i) {
        return row_exact(row.x, i, row.place, row.p.table, row.rot, row.p.layout, row.p.amplitude);
    };
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
    // the row's largest value (of a rotated row)
    float most = 0.f;
    if (TURNS && row.rot > 0)
#pragma unroll
        for (int k = 0; k < G; ++k) most = fmaxf(most, fmaxf(fabsf(lo[k]), fabsf(hi[k])));
    float need[G];
    bool close = false;
#pragma unroll
    for (int k = 0; k < G; ++k) {
        need[k] = kv4_need_fast(lo[k], hi[k]);
        const float off = need[k] * kNeedOff + most * kNeedOffRow;
        close |= (kv4_step_bits(need[k] - off) != kv4_step_bits(need[k] + off) || !(off < INFINITY)) &&
                 need[k] < INFINITY;
    }
    if (close && row.rot == 0) {  // the same in all threads of the row, as is the next
#pragma unroll
        for (int k = 0; k < G; ++k) need[k] = kv4_need(lo[k], hi[k]);
    }
    if (TURNS && close && row.rot > 0) {
#pragma unroll
        for (int k = 0; k < G; ++k) {
            // only what can be the least or the largest: a 64-bit value takes microseconds
            const float slack = 2.f * kOff * most;
            double dlo = INFINITY, dhi = -INFINITY;
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if ((G == 1 || oct[o] >> 3 == k) &&
                        (val[o][e] <= lo[k] + slack || val[o][e] >= hi[k] - slack)) {
                        const double t = exact(8 * oct[o] + e);
                        dlo = fmin(dlo, t);
                        dhi = fmax(dhi, t);
                    }
            for (int m = 1; m < T; m <<= 1) {
                dlo = fmin(dlo, __shfl_xor_sync(lanes, dlo, m));
                dhi = fmax(dhi, __shfl_xor_sync(lanes, dhi, m));
            }
            if (need[k] < INFINITY) need[k] = kv4_need(dlo, dhi);
        }
    }
    uint32_t bits[G];
    float inv[G], inv_lo[G];
    int base[G];
#pragma unroll
    for (int k = 0; k < G; ++k) {
        bits[k] = kv4_step_bits(need[k]);
        kv4_inverse(kv4_step(bits[k]), inv[k], inv_lo[k]);
        if (bits[k] == 0u || bits[k] == 0x3feu) inv[k] = inv_lo[k] = lo[k] = 0.f;  // all codes 0
        base[k] = kv4_whole(kv4_rounded(kv4_divide(lo[k], inv[k], inv_lo[k])));
    }
    // rint(x / s) of every value, as kv4_rounded gives it
    float q[2][8];
    bool ties = false;  // one may round the other way than the value in 64 bits
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        const bool second = G == 2 && oct[o] >> 3;
        const float r = second ? inv[G - 1] : inv[0], r_lo = second ? inv_lo[G - 1] : inv_lo[0];
        float off = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // (a rotated value's quotient near a half is seen to below, whatever its last bit)
            const float t = TURNS && turned ? val[o][e] * r : kv4_divide(val[o][e], r, r_lo);
            q[o][e] = kv4_rounded(t);
            if (TURNS) off = fmaxf(off, fabsf(t - (q[o][e] - kKv4Magic)));
        }
        if (TURNS) ties |= off > clear_of_ties(most, r);
    }
    if (TURNS && row.rot > 0 && __any_sync(lanes, turned && ties)) {
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const bool second = G == 2 && oct[o] >> 3;
            const float r = second ? inv[G - 1] : inv[0], r_lo = second ? inv_lo[G - 1] : inv_lo[0];
            const float s = kv4_step(second ? bits[G - 1] : bits[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = kv4_divide(val[o][e], r, r_lo);
                if (turned && r != 0.f &&
                    fabsf(t - (q[o][e] - kKv4Magic)) > clear_of_ties(most, r))
                    q[o][e] = kv4_rounded(0.f) +
                              static_cast<float>(rint(exact(8 * oct[o] + e) /
                                                      static_cast<double>(s)));
            }
        }
#pragma unroll
        for (int k = 0; k < G; ++k) {
            float least = INFINITY;
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (G == 1 || oct[o] >> 3 == k) least = fminf(least, q[o][e]);
#pragma unroll
            for (int m = 1; m < T; m <<= 1)
                least = fminf(least, __shfl_xor_sync(lanes, least, m));
            base[k] = kv4_whole(least);
        }
    }
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        const int b = G == 2 && oct[o] >> 3 ? base[G - 1] : base[0];
        uint32_t w = 0u;
#pragma unroll
        for (int e = 7; e >= 0; --e)
            w = w * 16u + static_cast<uint32_t>(min(kv4_whole(q[o][e]) - b, 15));
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

template <int K>
using Kind = std::integral_constant<int, K>;

// Thread: (token, 16 values), the threads of a row fastest; blockIdx.y: group of `per` rows of the
// token, which are its queries, then keys, then values.
template <int D, int FMT, bool FAST>
__global__ void __launch_bounds__(256, FMT == OSM_KV_BF16 ? 4 : 2)
    kv_append_kernel(const AppendParams p, int per) {
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
    const bool half = p.layout == OSM_ROPE_HALF;
    // Whether this thread's octets are rotated: both or neither in the half layout.
    const bool turned0 = half ? 16 * u < p.rot : 8 * u < p.rot;
    const bool turned1 = half ? turned0 : 8 * (u + T) < p.rot;
    const int first = group * per, end = min(first + per, heads);
    // Row `head` of the token's list, and the octets that this thread takes of a row.
    auto row_of = [&](int head) {
        if (head < p.H) return p.q + b * p.qs[0] + head * p.qs[1] + n * p.qs[2];
        head -= p.H;
        if (head < p.H_kv) return p.k + b * p.ks[0] + head * p.ks[1] + n * p.ks[2];
        return p.v + b * p.vs[0] + (head - p.H_kv) * p.vs[1] + n * p.vs[2];
    };
    auto octet = [&](int kind, int o) {
        if (!FAST) return 2 * u + o;
        if (!half || kind == 2 || p.rot == 0) return u + o * T;
        const int pairs = p.rot / 16;  // threads that take pairs
        return u < pairs ? u + o * pairs : u + pairs + o * (T - pairs);
    };
    uint4 begun[2];  // the first row's values, on their way while the angles are computed
    auto begin = [&](int head) {
        if constexpr (FAST) {
            const int kind = head < p.H ? 0 : (head < p.H + p.H_kv ? 1 : 2);
#pragma unroll
            for (int o = 0; o < 2; ++o)
                begun[o] = reinterpret_cast<const uint4*>(row_of(head))[octet(kind, o)];
        }
    };
    begin(first);
    float c[8], s[8];
    if (FAST && turned0 && first < p.H + p.H_kv) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // half: pairs 8 u ..; else four pairs of each octet
            const int pair = half ? 8 * u + e : 4 * (u + (e >> 2) * T) + (e & 3);
            if (2 * pair >= p.rot) break;
            rope_cos_sin(rope_phase(place, p.table[pair]), c[e], s[e]);
            c[e] *= p.amplitude;
            s[e] *= p.amplitude;
        }
    }
    if (!paged && end > p.H && u == 0) kv_bad_page(p.pg);
    // The heads [h0, h1) of the queries (KIND 0), keys (1) or values (2): each head's values are
    // loaded while the one before is worked on.
    const int64_t page_at = paged ? kv_head_offset(p.pg, id, 0) : 0;
    auto rows = [&](auto kind, const __nv_bfloat16* x, int64_t stride, int h0, int h1,
                    const uint4 (&begun)[2]) {
        constexpr int KIND = decltype(kind)::value;
        const int rot = KIND == 2 ? 0 : p.rot;
        const bool turn = KIND != 2 && turned0, turn1 = KIND != 2 && turned1;
        const int o0 = octet(KIND, 0), o1 = octet(KIND, 1);
        uint4 raw[2] = {begun[0], begun[1]};
        for (int h = h0; h < h1; ++h, x += stride) {
            float val[2][8];
            if constexpr (FAST) {
                unpack8(raw[0], val[0]);
                unpack8(raw[1], val[1]);
                if (h + 1 < h1) {
                    raw[0] = reinterpret_cast<const uint4*>(x + stride)[o0];
                    raw[1] = reinterpret_cast<const uint4*>(x + stride)[o1];
                }
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
                        if (e >= 4 && !turn1) break;
                        const float a = val[e >> 2][2 * (e & 3)], o = val[e >> 2][2 * (e & 3) + 1];
                        val[e >> 2][2 * (e & 3)] = a * c[e] - o * s[e];
                        val[e >> 2][2 * (e & 3) + 1] = o * c[e] + a * s[e];
                    }
                }
            } else {
                auto load = [&](int j) { return __bfloat162float(x[j]); };
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    val[e >> 3][e & 7] = rope_value<float>(load, 16 * u + e, place, p.table, rot,
                                                           p.layout, p.amplitude);
                // q_out may be q: the row is read by all its threads before one of them writes it
                if (KIND == 0) __syncwarp(lanes);
            }
            uint8_t* block =
                KIND == 0 ? nullptr : (KIND == 1 ? p.pg.k : p.pg.v) + page_at + h * p.pg.head_bytes;
            if constexpr (KIND == 0 || FMT == OSM_KV_BF16) {
                __nv_bfloat16* dst =
                    KIND == 0 ? p.q_out + ((static_cast<int64_t>(b) * p.H + h) * p.N + n) * D
                              : reinterpret_cast<__nv_bfloat16*>(block) + at * D;
                reinterpret_cast<uint4*>(dst)[o0] = pack8(val[0]);
                reinterpret_cast<uint4*>(dst)[o1] = pack8(val[1]);
            } else {
                store_int4<D, KIND == 1>(Row{p, x, place, rot}, val, o0, o1,
                                         FAST ? turn : rot > 0, block, at, lanes);
            }
        }
    };
    const int kq = min(end, p.H), kk = min(end, p.H + p.H_kv);
    if (first < kq) rows(Kind<0>{}, row_of(first), p.qs[1], first, kq, begun);
    if (!paged) return;
    const int k0 = max(first, p.H), v0 = max(first, p.H + p.H_kv);
    if (k0 < kk) {
        if (k0 > first) begin(k0);
        rows(Kind<1>{}, row_of(k0), p.ks[1], k0 - p.H, kk - p.H, begun);
    }
    if (v0 < end) {
        if (v0 > first) begin(v0);
        rows(Kind<2>{}, row_of(v0), p.vs[1], v0 - p.H - p.H_kv, end - p.H - p.H_kv, begun);
    }
}

struct GatherParams {
    KvPages pg;
    const int32_t* kv_lens;
    __nv_bfloat16 *K, *V;  // [B, H_kv, N, d]
    int64_t B, N;
    // before an attention (kv_gather_for_attention), else nullptr
    int32_t* irregular;
    const int32_t* q_lens;
    int Nq, causal;
};

// CTA: kGatherTokens tokens of one head of one sequence's keys or values; 16 values a thread, as
// octets u and u + d / 16 so that a warp's accesses are whole lines.
constexpr int kGatherTokens = 128;

template <int D, int FMT, bool ATTN>
__global__ void __launch_bounds__(256) kv_gather_kernel(const GatherParams p, int tiles) {
    constexpr int T = D / 16, kPer = 256 / T;  // threads a token's head, tokens at a time
    constexpr int kTurns = kGatherTokens / kPer;
    const bool is_v = blockIdx.x & 1;
    const uint32_t rest = blockIdx.x >> 1;
    const uint32_t bh = rest / static_cast<uint32_t>(tiles);
    const int n0 = static_cast<int>(rest - bh * tiles) * kGatherTokens;
    const uint32_t b = bh / static_cast<uint32_t>(p.pg.H_kv), h = bh - b * p.pg.H_kv;
    const int u = threadIdx.x % T, row = threadIdx.x / T;
    const int len = min(static_cast<int64_t>(max(p.kv_lens[b], 0)), p.N);
    const int N = ATTN ? min(static_cast<int>(p.N), (len + 127) & ~127) : static_cast<int>(p.N);
    if (n0 >= N) return;
    // the first token that some query may not see
    int hidden = len;
    if (ATTN) {
        const int ql = p.q_lens ? min(max(p.q_lens[b], 0), p.Nq) : p.Nq;
        hidden = ql < p.Nq ? 0 : (p.causal ? len - ql : len);  // padding rows see none
    }
    bool wild = false;
    const uint8_t* head = (is_v ? p.pg.v : p.pg.k) + h * p.pg.head_bytes;
    const int64_t page_bytes = p.pg.head_bytes * p.pg.H_kv;
    const int32_t* table = p.pg.table + static_cast<int64_t>(b) * p.pg.max_pages;
    uint4* out = reinterpret_cast<uint4*>((is_v ? p.V : p.K) + static_cast<int64_t>(bh) * p.N * D) + u;
    // all of a thread's reads first
    uint4 x[kTurns][2];
    uint32_t word[kTurns];
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        const int n = n0 + k * kPer + row;
        x[k][0] = x[k][1] = make_uint4(0u, 0u, 0u, 0u);
        word[k] = 0u;
        if (n >= len) continue;
        const uint32_t pi = static_cast<uint32_t>(n) / static_cast<uint32_t>(p.pg.page);
        const int at = n - static_cast<int>(pi) * p.pg.page;
        const int32_t id = pi < p.pg.max_pages ? table[pi] : -1;
        if (id < 0 || id >= p.pg.num_pages) {
            if (u == 0) kv_bad_page(p.pg);
            wild = true;
            continue;
        }
        const uint8_t* block = head + id * page_bytes;
        if constexpr (FMT == OSM_KV_BF16) {
            x[k][0] = reinterpret_cast<const uint4*>(block + at * D * 2)[u];
            x[k][1] = reinterpret_cast<const uint4*>(block + at * D * 2)[u + T];
        } else {
            x[k][0].x = reinterpret_cast<const uint32_t*>(block + at * (D / 2))[u];
            x[k][1].x = reinterpret_cast<const uint32_t*>(block + at * (D / 2))[u + T];
            const uint8_t* w = block + p.pg.page * (D / 2) + at * (D / 32);
            word[k] = D == 128 ? *reinterpret_cast<const uint32_t*>(w)
                               : *reinterpret_cast<const uint16_t*>(w);
        }
    }
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        const int n = n0 + k * kPer + row;
        if (n >= N) break;
        if constexpr (FMT == OSM_KV_INT4) {
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                // A byte's two codes as the bf16 numbers 128 + code, plus base - 128, times the
                // step: the sum is exact, the product rounded once (kv_cache.cuh: five values).
                const uint32_t w16 = D == 128 && o == 1 ? word[k] >> 16 : word[k];
                const float base = static_cast<float>(kv4_word_base(w16) - 128);
                const float s = kv4_word_step(w16);
                const uint32_t add = pack_bf16x2(base, base), mul = pack_bf16x2(s, s);
                const uint32_t codes = x[k][o].x;
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t byte = __byte_perm(codes, 0u, 0x4440u | e);
                    const uint32_t two = (byte * 0x1001u & 0x000f000fu) | 0x43004300u;
                    uint32_t whole;
                    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(whole) : "r"(two), "r"(add));
                    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(w[e]) : "r"(whole), "r"(mul));
                }
                x[k][o] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        if (ATTN && is_v && n >= hidden) {
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                const uint32_t w[4] = {x[k][o].x, x[k][o].y, x[k][o].z, x[k][o].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    wild |= (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
            }
        }
        out[static_cast<int64_t>(n) * (D / 8)] = x[k][0];
        out[static_cast<int64_t>(n) * (D / 8) + T] = x[k][1];
    }
    if (ATTN && wild) p.irregular[b] = 1;
}

template <bool ATTN>
int launch_gather(const GatherParams& p, int64_t d, cudaStream_t stream) {
    const int64_t tiles = (p.N + kGatherTokens - 1) / kGatherTokens;
    const int64_t grid = 2 * p.B * p.pg.H_kv * tiles;
    if (grid > INT32_MAX) return FA_ERR_UNSUPPORTED;
    const unsigned g = static_cast<unsigned>(grid);
    const int nt = static_cast<int>(tiles);
    if (p.pg.format == OSM_KV_BF16) {
        if (d == 64) kv_gather_kernel<64, OSM_KV_BF16, ATTN><<<g, 256, 0, stream>>>(p, nt);
        else kv_gather_kernel<128, OSM_KV_BF16, ATTN><<<g, 256, 0, stream>>>(p, nt);
    } else {
        if (d == 64) kv_gather_kernel<64, OSM_KV_INT4, ATTN><<<g, 256, 0, stream>>>(p, nt);
        else kv_gather_kernel<128, OSM_KV_INT4, ATTN><<<g, 256, 0, stream>>>(p, nt);
    }
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D>
void launch_append(const AppendParams& p, int per, bool fast, int format, dim3 g,
                   cudaStream_t stream) {
    if (format == OSM_KV_BF16) {
        if (fast) kv_append_kernel<D, OSM_KV_BF16, true><<<g, 256, 0, stream>>>(p, per);
        else kv_append_kernel<D, OSM_KV_BF16, false><<<g, 256, 0, stream>>>(p, per);
    } else {
        if (fast) kv_append_kernel<D, OSM_KV_INT4, true><<<g, 256, 0, stream>>>(p, per);
        else kv_append_kernel<D, OSM_KV_INT4, false><<<g, 256, 0, stream>>>(p, per);
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
    // as many rows a thread as leave 24 warps an SM's worth of threads: the angles are half the work
    // of a row
    if (one >= (int64_t(1) << 32) || heads > 65535) return FA_ERR_UNSUPPORTED;
    auto run = [&](const AppendParams& a, int format) {
        const int64_t rows = a.H + 2LL * a.pg.H_kv;
        int per = 8;  // (at most 4: 51.2 us in place of 50.2 at the prompts above)
        while (per > 1 && one * ((rows + per - 1) / per) < 152 * 768) per >>= 1;
        const dim3 g(static_cast<unsigned>((one + 255) / 256),
                     static_cast<unsigned>((rows + per - 1) / per));
        if (d == 64) launch_append<64>(a, per, fast, format, g, stream);
        else launch_append<128>(a, per, fast, format, g, stream);
    };
    // The 4-bit kernel's registers leave 16 warps an SM, too few for the queries' copies: beyond
    // the size of a launch they go by themselves, through the kernel for bf16 pages (8192 tokens of
    // 32 + 2 x 8 heads and the read-out: 70.5 us, 73.6 in one launch).
    if (pg.format == OSM_KV_INT4 && p.H > 0 && one * heads >= 152 * 2048 * 4) {
        AppendParams a = p;
        a.pg.H_kv = a.H_kv = 0;
        run(a, OSM_KV_BF16);
        p.q = nullptr;
        p.H = 0;
    }
    run(p, pg.format);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int osm_kv_gather_launch(const KvPages& pg, const int32_t* kv_lens, void* K, void* V, int64_t B,
                         int64_t N, int64_t d, cudaStream_t stream) {
    GatherParams p{pg, kv_lens, static_cast<__nv_bfloat16*>(K), static_cast<__nv_bfloat16*>(V), B,
                   N, nullptr, nullptr, 0, 0};
    return launch_gather<false>(p, d, stream);
}

int kv_gather_for_attention(const KvPages& pg, const int32_t* kv_lens, const int32_t* q_lens,
                            int64_t Nq, bool causal, int32_t* irregular, void* K, void* V,
                            int64_t B, int64_t N, int64_t d, cudaStream_t stream) {
    GatherParams p{pg, kv_lens, static_cast<__nv_bfloat16*>(K), static_cast<__nv_bfloat16*>(V), B,
                   N, irregular, q_lens, static_cast<int>(Nq), causal ? 1 : 0};
    return launch_gather<true>(p, d, stream);
}

}  // namespace osm
