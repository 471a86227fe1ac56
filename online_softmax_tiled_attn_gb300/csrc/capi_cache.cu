// capi_cache.cu -- the extern "C" boundary of the rotary positions and the paged key/value cache
// (declared in include/osm_attn.h).  As in capi.cu, every argument is checked here on the host
// before anything is launched.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "kv_cache.cuh"
#include "osm_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Span {
    uintptr_t at;
    uint64_t bytes;
};

Span span(const void* p, uint64_t bytes) { return {reinterpret_cast<uintptr_t>(p), bytes}; }

bool meet(const Span& a, const Span& b) {
    return a.bytes != 0 && b.bytes != 0 && a.at < b.at + b.bytes && b.at < a.at + a.bytes;
}

// No output meets an input or another output.
bool apart(const Span* outs, int n_out, const Span* ins, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (meet(outs[i], ins[j])) return false;
        for (int j = i + 1; j < n_out; ++j)
            if (meet(outs[i], outs[j])) return false;
    }
    return true;
}

constexpr int64_t kMostElems = int64_t(1) << 60;

// Product of non-negative sizes; false above 2^60.
bool product(std::initializer_list<int64_t> v, int64_t* out) {
    int64_t p = 1;
    for (int64_t x : v) {
        if (x < 0) return false;
        if (x == 0) {
            *out = 0;
            return true;
        }
        if (p > kMostElems / x) return false;
        p *= x;
    }
    *out = p;
    return true;
}

// Elements from the first to past the last of a strided [B, H, N, d] tensor (no dimension 0);
// false for a negative stride or an extent above 2^60.
bool extent(int64_t B, int64_t H, int64_t N, int64_t d, const int64_t* st, int64_t* out) {
    const int64_t n[3] = {B, H, N};
    int64_t e = d;
    for (int i = 0; i < 3; ++i) {
        int64_t t;
        if (st[i] < 0 || !product({n[i] - 1, st[i]}, &t) || e > kMostElems - t) return false;
        e += t;
    }
    *out = e;
    return true;
}

// No two elements of a strided [B, H, N, d] tensor share memory: from the smallest stride up, each
// steps over all that the ones below it span.  (Stricter than needed for strides that interleave.)
bool distinct(int64_t B, int64_t H, int64_t N, int64_t d, const int64_t* st) {
    int64_t n[3] = {B, H, N}, s[3] = {st[0], st[1], st[2]};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i]) {
                const int64_t a = s[i], b = n[i];
                s[i] = s[j], n[i] = n[j];
                s[j] = a, n[j] = b;
            }
    int64_t span = d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (s[i] < span) return false;
        span += (n[i] - 1) * s[i];
    }
    return true;
}

bool rope_ok(int64_t rot, int64_t d, int layout, float amplitude, const int64_t* table) {
    return rot >= 2 && rot <= d && rot % 2 == 0 &&
           (layout == OSM_ROPE_HALF || layout == OSM_ROPE_INTERLEAVED) &&
           std::isfinite(amplitude) && table && aligned(table, 8);
}

int rope_call(const void* x, void* y, int dtype, int64_t B, int64_t H, int64_t N, int64_t d,
              const int64_t* xs, const int64_t* ys, const int32_t* positions, int64_t pos_bs,
              const int64_t* table, int64_t rot, int layout, float amplitude, void* stream,
              bool inverse) {
    int64_t elems;
    if (!product({B, H, N, d}, &elems)) return FA_ERR_INVALID_ARG;
    if (dtype != OSM_BF16 && dtype != OSM_FP32) return FA_ERR_INVALID_ARG;
    if (elems == 0) return FA_OK;
    if (d > 65536) return FA_ERR_UNSUPPORTED;
    if (!rope_ok(rot, d, layout, amplitude, table)) return FA_ERR_INVALID_ARG;
    const int64_t size = dtype == OSM_BF16 ? 2 : 4;
    if (!x || !y || !xs || !ys || !aligned(x, size) || !aligned(y, size) ||
        (positions && (!aligned(positions, 4) || pos_bs < 0)))
        return FA_ERR_INVALID_ARG;
    if (!positions && N > INT32_MAX) return FA_ERR_INVALID_ARG;
    int64_t xe, ye, pe = 0;
    if (!extent(B, H, N, d, xs, &xe) || !extent(B, H, N, d, ys, &ye) ||
        !distinct(B, H, N, d, ys))
        return FA_ERR_INVALID_ARG;
    if (positions && (!product({B - 1, pos_bs}, &pe) || pe > kMostElems - N))
        return FA_ERR_INVALID_ARG;
    bool in_place = x == y;
    const int64_t n[3] = {B, H, N};
    for (int i = 0; i < 3; ++i) in_place = in_place && (n[i] == 1 || xs[i] == ys[i]);
    const Span out = span(y, ye * size);
    const Span ins[3] = {span(x, in_place ? 0 : xe * size),
                         span(positions, positions ? (pe + N) * 4 : 0), span(table, rot / 2 * 8)};
    if (!apart(&out, 1, ins, 3)) return FA_ERR_INVALID_ARG;
    return osm::osm_rope_launch(x, y, dtype, B, H, N, d, xs, ys, positions, pos_bs, table, rot,
                                layout, amplitude, inverse, static_cast<cudaStream_t>(stream));
}

constexpr int64_t kMostPlaces = int64_t(1) << 30;  // of a sequence

// The arguments that describe the cache; `bytes` gets the size of each page array.
int pages_ok(const void* k, const void* v, int format, int64_t num_pages, int64_t page,
             const int32_t* table, int64_t max_pages, int64_t B, int64_t H_kv, int64_t d,
             int64_t* bytes) {
    if (format != OSM_KV_BF16 && format != OSM_KV_INT4) return FA_ERR_INVALID_ARG;
    if (num_pages < 0 || page < 1 || max_pages < 0) return FA_ERR_INVALID_ARG;
    if (page > 1024 || page % 16 != 0) return FA_ERR_UNSUPPORTED;
    int64_t places, entries;
    if (num_pages > INT32_MAX || !product({max_pages, page}, &places) || places > kMostPlaces ||
        !product({B, max_pages}, &entries) ||
        !product({num_pages, H_kv, osm::kv_page_head_bytes(format, page, d)}, bytes))
        return FA_ERR_INVALID_ARG;
    if (*bytes > 0 && (!k || !v || !aligned(k, 16) || !aligned(v, 16))) return FA_ERR_INVALID_ARG;
    if (entries > 0 && (!table || !aligned(table, 4))) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

osm::KvPages make_pages(const void* k, const void* v, int format, int64_t num_pages, int64_t page,
                        const int32_t* table, int64_t max_pages, int64_t H_kv, int64_t d) {
    osm::KvPages pg{};
    pg.k = static_cast<uint8_t*>(const_cast<void*>(k));
    pg.v = static_cast<uint8_t*>(const_cast<void*>(v));
    pg.table = table;
    pg.num_pages = num_pages;
    pg.max_pages = max_pages;
    pg.page = static_cast<int>(page);
    pg.format = format;
    pg.H_kv = static_cast<int>(H_kv);
    pg.head_bytes = osm::kv_page_head_bytes(format, page, d);
    pg.status = osm::device_status_word();
    return pg;
}

}  // namespace

extern "C" {

int osm_rope_rates(int64_t rot_dim, double base, int scaling, double factor, double orig_len,
                   double low, double high, double* rates) {
    if (!rates || rot_dim < 2 || rot_dim % 2 != 0 || !std::isfinite(base) || !(base > 0))
        return FA_ERR_INVALID_ARG;
    if (scaling < OSM_ROPE_PLAIN || scaling > OSM_ROPE_BANDS) return FA_ERR_INVALID_ARG;
    if (scaling != OSM_ROPE_PLAIN && (!std::isfinite(factor) || !(factor >= 1)))
        return FA_ERR_INVALID_ARG;
    if (scaling == OSM_ROPE_BASE) {
        if (rot_dim <= 2) return FA_ERR_INVALID_ARG;
        base *= std::pow(factor, static_cast<double>(rot_dim) / static_cast<double>(rot_dim - 2));
    }
    if (scaling == OSM_ROPE_BANDS &&
        (!std::isfinite(orig_len) || !(orig_len > 0) || !std::isfinite(low) ||
         !std::isfinite(high) || !(high > low)))
        return FA_ERR_INVALID_ARG;
    for (int64_t i = 0; i < rot_dim / 2; ++i) {
        double r = std::pow(base, -2.0 * static_cast<double>(i) / static_cast<double>(rot_dim));
        if (scaling == OSM_ROPE_LINEAR) r /= factor;
        if (scaling == OSM_ROPE_BANDS) {
            const double turns = orig_len * r / 6.283185307179586;
            double w = (turns - low) / (high - low);
            w = w < 0 ? 0 : (w > 1 ? 1 : w);
            r *= w + (1 - w) / factor;
        }
        rates[i] = r;
    }
    return FA_OK;
}

int osm_rope_table(const double* rates, int64_t n, int64_t* table) {
    if (n < 0 || (n > 0 && (!rates || !table))) return FA_ERR_INVALID_ARG;
    for (int64_t i = 0; i < n; ++i)
        if (!std::isfinite(rates[i]) || rates[i] < 0) return FA_ERR_INVALID_ARG;
    for (int64_t i = 0; i < n; ++i) {
        const double turns = rates[i] / 6.283185307179586;
        const double part = turns - std::floor(turns);  // exact
        // part * 2^64 < 2^64 (the largest double below 1 is 1 - 2^-53)
        table[i] = static_cast<int64_t>(static_cast<uint64_t>(std::ldexp(part, 64)));
    }
    return FA_OK;
}

int osm_rope(const void* x, void* y, int dtype, int64_t B, int64_t H, int64_t N, int64_t d,
             const int64_t* x_strides, const int64_t* y_strides, const int32_t* positions,
             int64_t pos_b_stride, const int64_t* table, int64_t rot_dim, int layout,
             float amplitude, void* stream) {
    return rope_call(x, y, dtype, B, H, N, d, x_strides, y_strides, positions, pos_b_stride, table,
                     rot_dim, layout, amplitude, stream, false);
}

int osm_rope_bwd(const void* dy, void* dx, int dtype, int64_t B, int64_t H, int64_t N, int64_t d,
                 const int64_t* dy_strides, const int64_t* dx_strides, const int32_t* positions,
                 int64_t pos_b_stride, const int64_t* table, int64_t rot_dim, int layout,
                 float amplitude, void* stream) {
    return rope_call(dy, dx, dtype, B, H, N, d, dy_strides, dx_strides, positions, pos_b_stride,
                     table, rot_dim, layout, amplitude, stream, true);
}

int osm_kv_page_bytes(int format, int64_t page_size, int64_t d, int64_t* bytes) {
    if (!bytes || page_size < 1 || d < 0 || (format != OSM_KV_BF16 && format != OSM_KV_INT4))
        return FA_ERR_INVALID_ARG;
    if (page_size > 1024 || page_size % 16 != 0 || (d != 64 && d != 128))
        return FA_ERR_UNSUPPORTED;
    *bytes = osm::kv_page_head_bytes(format, page_size, d);
    return FA_OK;
}

int osm_kv_append(const void* k, const void* v, const int64_t* k_strides,
                  const int64_t* v_strides, void* k_pages, void* v_pages, int format,
                  int64_t num_pages, int64_t page_size, const int32_t* page_table,
                  int64_t max_pages, const int32_t* cache_lens, const int32_t* new_lens,
                  const int64_t* table, int64_t rot_dim, int layout, float amplitude,
                  const void* q, void* q_out, const int64_t* q_strides, int64_t B, int64_t H,
                  int64_t H_kv, int64_t N, int64_t d, void* stream) {
    int64_t kv_elems, q_elems = 0, page_bytes;
    if (!product({B, H_kv, N, d}, &kv_elems)) return FA_ERR_INVALID_ARG;
    if ((q == nullptr) != (q_out == nullptr) || H < 0) return FA_ERR_INVALID_ARG;
    if (q && (!product({B, H, N, d}, &q_elems) || H > INT32_MAX / 4)) return FA_ERR_INVALID_ARG;
    if (kv_elems == 0) return q_elems == 0 ? FA_OK : FA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if (H_kv > INT32_MAX / 4 || N > INT32_MAX) return FA_ERR_INVALID_ARG;
    if (q && H < 1) return FA_ERR_INVALID_ARG;
    const int st = pages_ok(k_pages, v_pages, format, num_pages, page_size, page_table, max_pages,
                            B, H_kv, d, &page_bytes);
    if (st != FA_OK) return st;
    if (rot_dim != 0 && !rope_ok(rot_dim, d, layout, amplitude, table)) return FA_ERR_INVALID_ARG;
    if (!k || !v || !k_strides || !v_strides || !aligned(k, 2) || !aligned(v, 2) || !cache_lens ||
        !aligned(cache_lens, 4) || (new_lens && !aligned(new_lens, 4)))
        return FA_ERR_INVALID_ARG;
    int64_t ke, ve, qe = 0;
    if (!extent(B, H_kv, N, d, k_strides, &ke) || !extent(B, H_kv, N, d, v_strides, &ve))
        return FA_ERR_INVALID_ARG;
    bool in_place = false;
    if (q) {
        if (!q_strides || !aligned(q, 2) || !aligned(q_out, 16) ||
            !extent(B, H, N, d, q_strides, &qe))
            return FA_ERR_INVALID_ARG;
        in_place = q == q_out && (N == 1 || q_strides[2] == d) &&
                   (H == 1 || q_strides[1] == N * d) && (B == 1 || q_strides[0] == H * N * d);
    }
    const Span outs[3] = {span(k_pages, page_bytes), span(v_pages, page_bytes),
                          span(q_out, q_elems * 2)};
    const Span ins[7] = {span(k, ke * 2), span(v, ve * 2), span(q, in_place ? 0 : qe * 2),
                         span(page_table, B * max_pages * 4), span(cache_lens, B * 4),
                         span(new_lens, new_lens ? B * 4 : 0),
                         span(table, rot_dim ? rot_dim / 2 * 8 : 0)};
    if (!apart(outs, 3, ins, 7)) return FA_ERR_INVALID_ARG;
    const osm::KvPages pg = make_pages(k_pages, v_pages, format, num_pages, page_size, page_table,
                                       max_pages, H_kv, d);
    if (!pg.status) return FA_ERR_CUDA;
    return osm::osm_kv_append_launch(k, v, k_strides, v_strides, pg, cache_lens, new_lens, table,
                                     rot_dim, layout, amplitude, q, q_out, q_strides, B, H, N, d,
                                     static_cast<cudaStream_t>(stream));
}

int osm_kv_gather(const void* k_pages, const void* v_pages, int format, int64_t num_pages,
                  int64_t page_size, const int32_t* page_table, int64_t max_pages,
                  const int32_t* kv_lens, void* K, void* V, int64_t B, int64_t H_kv, int64_t N,
                  int64_t d, void* stream) {
    int64_t elems, page_bytes;
    if (!product({B, H_kv, N, d}, &elems)) return FA_ERR_INVALID_ARG;
    if (elems == 0) return FA_OK;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if (H_kv > INT32_MAX || N > INT32_MAX) return FA_ERR_INVALID_ARG;
    const int st = pages_ok(k_pages, v_pages, format, num_pages, page_size, page_table, max_pages,
                            B, H_kv, d, &page_bytes);
    if (st != FA_OK) return st;
    if (!K || !V || !aligned(K, 16) || !aligned(V, 16) || !kv_lens || !aligned(kv_lens, 4))
        return FA_ERR_INVALID_ARG;
    const Span outs[2] = {span(K, elems * 2), span(V, elems * 2)};
    const Span ins[4] = {span(k_pages, page_bytes), span(v_pages, page_bytes),
                         span(page_table, B * max_pages * 4), span(kv_lens, B * 4)};
    if (!apart(outs, 2, ins, 4)) return FA_ERR_INVALID_ARG;
    const osm::KvPages pg = make_pages(k_pages, v_pages, format, num_pages, page_size, page_table,
                                       max_pages, H_kv, d);
    if (!pg.status) return FA_ERR_CUDA;
    return osm::osm_kv_gather_launch(pg, kv_lens, K, V, B, N, d,
                                     static_cast<cudaStream_t>(stream));
}

int fa_fwd_paged_plan(int64_t B, int64_t H, int64_t H_kv, int64_t Nq, int64_t d, int format,
                      int64_t page_size, int64_t max_pages, int64_t* ws_bytes) {
    int64_t elems, bytes;
    if (!ws_bytes || !product({B, H, Nq, d}, &elems) || H_kv < 0 ||
        (H > 0 && (H_kv < 1 || H % H_kv != 0)))
        return FA_ERR_INVALID_ARG;
    if (elems == 0) {
        *ws_bytes = 0;
        return FA_OK;
    }
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if (H > INT32_MAX || Nq > (1 << 30)) return FA_ERR_INVALID_ARG;
    if (elems / d > INT32_MAX - 15) return FA_ERR_UNSUPPORTED;  // rows are counted in 32 bits
    const int st = pages_ok(nullptr, nullptr, format, 0, page_size,
                            reinterpret_cast<const int32_t*>(16), max_pages, B, H_kv, d, &bytes);
    if (st != FA_OK) return st;
    // a page of all heads is addressed in 32 bits
    if (H_kv * osm::kv_page_head_bytes(format, page_size, d) > INT32_MAX) return FA_ERR_UNSUPPORTED;
    int64_t dense;  // a sequence read out
    if (!product({H_kv, max_pages, page_size, 4 * d}, &dense) || dense > int64_t(1) << 50)
        return FA_ERR_UNSUPPORTED;
    *ws_bytes = osm::fa_paged_ws_bytes(B, H, H_kv, Nq, d, format, page_size, max_pages);
    return *ws_bytes < 0 ? FA_ERR_UNSUPPORTED : FA_OK;
}

int fa_fwd_paged(const void* Q, const void* k_pages, const void* v_pages, int format,
                 int64_t num_pages, int64_t page_size, const int32_t* page_table,
                 int64_t max_pages, const int32_t* kv_lens, const int32_t* q_lens, void* O,
                 float* LSE, int64_t B, int64_t H, int64_t H_kv, int64_t Nq, int64_t d,
                 float scale, int causal, void* ws, int64_t ws_bytes, void* stream) {
    int64_t need, rows, page_bytes;
    const int pst = fa_fwd_paged_plan(B, H, H_kv, Nq, d, format, page_size, max_pages, &need);
    if (pst != FA_OK) return pst;
    if (!product({B, H, Nq}, &rows)) return FA_ERR_INVALID_ARG;
    if (rows == 0) return FA_OK;
    const int st = pages_ok(k_pages, v_pages, format, num_pages, page_size, page_table, max_pages,
                            B, H_kv, d, &page_bytes);
    if (st != FA_OK) return st;
    if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
    if (!Q || !O || !aligned(Q, 16) || !aligned(O, 16) || (LSE && !aligned(LSE, 4)) || !kv_lens ||
        !aligned(kv_lens, 4) || (q_lens && !aligned(q_lens, 4)))
        return FA_ERR_INVALID_ARG;
    if (ws_bytes < need || (need > 0 && (!ws || !aligned(ws, 16)))) return FA_ERR_INVALID_ARG;
    const Span outs[3] = {span(O, rows * d * 2), span(LSE, LSE ? rows * 4 : 0), span(ws, need)};
    const Span ins[6] = {span(Q, rows * d * 2), span(k_pages, page_bytes),
                         span(v_pages, page_bytes), span(page_table, B * max_pages * 4),
                         span(kv_lens, B * 4), span(q_lens, q_lens ? B * 4 : 0)};
    if (!apart(outs, 3, ins, 6)) return FA_ERR_INVALID_ARG;
    const osm::KvPages pg = make_pages(k_pages, v_pages, format, num_pages, page_size, page_table,
                                       max_pages, H_kv, d);
    if (!pg.status) return FA_ERR_CUDA;
    return osm::fa_paged_launch(Q, O, LSE, pg, kv_lens, q_lens, B, H, Nq, d, scale, causal != 0,
                                ws, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
