// kv_cache.cuh -- what the kernels of the rotated, paged key/value cache share: rotation angles,
// the two page formats, and the 4-bit quantiser.
//
// Page formats, per page and key/value head (P tokens, d values a token, d = 64 or 128):
//   OSM_KV_BF16  bf16 [P, d].
//   OSM_KV_INT4  P * d / 2 bytes of codes, token after token, value 2i in the low half of byte i
//                and value 2i + 1 in the high half; then one 16-bit word for each token and group
//                of 64 values: the step s as the upper ten bits of a float without its sign
//                (eight of exponent, two of fraction) above a signed six-bit base b.  A value is
//                s * (b + code), nine significant bits at most.  bf16 holds all but 7/4 times
//                37, 39, 41, 43 and 45 (times a power of two), which the read-out rounds, off by
//                s / 7; a base below 22, as any group has whose values straddle zero, reaches none
//                of them, and then every path over a 4-bit cache computes with the same values.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "osm_attn.h"

namespace osm {

constexpr int kKvGroup = 64;  // values that share a step and a base

// Bytes of one key/value head of a page.
__host__ __device__ constexpr int64_t kv_page_head_bytes(int format, int64_t page, int64_t d) {
    return format == OSM_KV_BF16 ? page * d * 2 : page * (d / 2 + d / 32);
}

// ------------------------------------------------------------------------------------------
// Rotation.  The rate of pair i is a 64-bit fraction of a turn per position, so position * rate
// modulo 2^64 is the angle modulo one turn without any rounding, however far the position; only
// the rate itself is rounded (osm_rope_table: as a double, by some 2^-53 of itself, and cut off at
// 2^-64 of a turn).
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ uint64_t rope_phase(int64_t pos, int64_t rate) {
    return static_cast<uint64_t>(pos) * static_cast<uint64_t>(rate);
}

// cos and sin of a phase (2^64 = one turn).  The upper 32 bits, as a signed number of half turns
// in [-1, 1), lose 2^-25 of a half turn in the conversion to float: 9e-8 rad.
__device__ __forceinline__ void rope_cos_sin(uint64_t phase, float& c, float& s) {
    const float half_turns =
        static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f;  // 2^-31
    sincospif(half_turns, &s, &c);
}

__device__ __forceinline__ void rope_cos_sin(uint64_t phase, double& c, double& s) {
    const double half_turns =
        static_cast<double>(static_cast<int64_t>(phase)) * 1.0842021724855044e-19;  // 2^-63
    sincospi(half_turns, &s, &c);
}

// Value i of a row after the rotation of its first `rot` values, in type F (float or double).
// load(j) gives value j of the row before.
template <typename F, typename Load>
__device__ __forceinline__ F rope_value(const Load& load, int i, int64_t pos,
                                        const int64_t* __restrict__ table, int rot, int layout,
                                        F amplitude) {
    if (i >= rot) return static_cast<F>(load(i));
    const int half = rot >> 1;
    const bool second = layout == OSM_ROPE_HALF ? i >= half : (i & 1) != 0;
    const int pair = layout == OSM_ROPE_HALF ? (second ? i - half : i) : (i >> 1);
    const int other = layout == OSM_ROPE_HALF ? (second ? i - half : i + half) : (i ^ 1);
    F c, s;
    rope_cos_sin(rope_phase(pos, table[pair]), c, s);
    const F x = static_cast<F>(load(i)), o = static_cast<F>(load(other));
    return (second ? x * c + o * s : x * c - o * s) * amplitude;
}

// ------------------------------------------------------------------------------------------
// The 4-bit quantiser.  For a group with least and largest value lo, hi: s is the least step of
// three significant bits with 15 s >= hi - lo and 31 s >= |lo|, b = rint(lo / s), and the code of
// x is rint(x / s) - b, at most 15; the error is at most s / 2.  The first bound spans the group;
// the second keeps |b| within 31, so that b + code has six significant bits.
// ------------------------------------------------------------------------------------------
// max / min that return NaN when either operand is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The bound that the step must reach, (fast) within four units of the last place, and as a float
// that is never below it.  Rounding upwards twice lands on no wrong side of a step s: 15 s is a float
// (s has three significant bits), so a span of at most 15 s rounds to at most 15 s, its fifteenth to
// at most s; and one above 15 s stays above.  (Rounded to nearest, a span of 15 + 1e-9 would take a
// step of 1.)  Halved operands: hi - lo of bf16 values can pass the largest float.
__device__ __forceinline__ float kv4_need_fast(float lo, float hi) {
    return fmaxf((0.5f * hi - 0.5f * lo) * (1.f / 7.5f), fabsf(lo) * (1.f / 31.f));
}
__device__ __forceinline__ float kv4_need(float lo, float hi) {
    return fmaxf(__fdiv_ru(__fsub_ru(0.5f * hi, 0.5f * lo), 7.5f), __fdiv_ru(fabsf(lo), 31.f));
}
// The same from values in 64 bits (rotated ones, whose least and largest are no bf16 numbers).
__device__ __forceinline__ float kv4_need(double lo, double hi) {
    return __double2float_ru(
        fmax(__ddiv_ru(__dsub_ru(hi, lo), 15.), __ddiv_ru(fabs(lo), 31.)));
}

// The step in its ten bits: `need` rounded up to two fraction bits.  0 below the smallest normal
// float (the group reads back as 0); a group with a NaN or an infinity takes the NaN pattern and
// reads back as NaN.
__device__ __forceinline__ uint32_t kv4_step_bits(float need) {
    const uint32_t u = __float_as_uint(need);
    if (u >= 0x7f000000u) return 0x3feu;  // NaN, infinite, or no float above it with room
    if (u < 0x00800000u) return 0u;
    return (u + 0x1fffffu) >> 21;
}
__device__ __forceinline__ float kv4_step(uint32_t bits) { return __uint_as_float(bits << 21); }

// x / s for a quotient below 2^22, rounded once: inv and inv_lo are 1 / s and what its rounding left
// out (kv4_inverse; any inv near 1 / s will do).  In particular a quotient that is a whole number
// and a half comes out as that, where x * inv alone can land beside it.
__device__ __forceinline__ void kv4_inverse(float s, float& inv, float& inv_lo) {
    asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(s));
    inv_lo = fmaf(-s, inv, 1.f) * inv;
}
__device__ __forceinline__ float kv4_divide(float x, float inv, float inv_lo) {
    const float p = x * inv;
    return fmaf(x, inv_lo, fmaf(x, inv, -p)) + p;
}
// Rounds |t| < 2^22 to the nearest whole number, ties to even; kv4_whole gives the number.
constexpr float kKv4Magic = 12582912.f;  // 1.5 * 2^23
__device__ __forceinline__ float kv4_rounded(float t) { return __fadd_rn(t, kKv4Magic); }
__device__ __forceinline__ int kv4_whole(float rounded) {
    return __float_as_int(rounded) - 0x4b400000;
}

__device__ __forceinline__ uint32_t kv4_word(uint32_t step_bits, int base) {
    return (step_bits << 6) | (static_cast<uint32_t>(base) & 63u);
}
__device__ __forceinline__ float kv4_word_step(uint32_t word) {
    return __uint_as_float((word & 0xffc0u) << 15);
}
__device__ __forceinline__ int kv4_word_base(uint32_t word) {
    return static_cast<int>(word << 26) >> 26;
}

// ------------------------------------------------------------------------------------------
// Pages.  The page table is a device array [B, max_pages]; an entry outside [0, num_pages) that a
// call needs is reported in the device status word, and its tokens take no part.
// ------------------------------------------------------------------------------------------
struct KvPages {
    uint8_t* k;  // pages [num_pages, H_kv] of kv_page_head_bytes each
    uint8_t* v;
    const int32_t* table;  // [B, max_pages]
    int64_t num_pages, max_pages;
    int page, format, H_kv;
    int64_t head_bytes;  // kv_page_head_bytes
    int* status;         // device status word
};

__device__ __forceinline__ void kv_bad_page(const KvPages& pg) {
    atomicCAS(pg.status, 0, FA_ERR_PAGE);
}

// Offset in bytes of key/value head h of page id.
__device__ __forceinline__ int64_t kv_head_offset(const KvPages& pg, int32_t id, int h) {
    return (static_cast<int64_t>(id) * pg.H_kv + h) * pg.head_bytes;
}

}  // namespace osm
