// osm_pages.cu -- the pages of the paged cache as a pool that sequences share: osm_kv_grow,
// osm_kv_fork, osm_kv_free, osm_kv_compact.
//
// refs[p] counts the table entries that use page p; a page is free where it is 0 (or below).  What a
// call gives out are the lowest free pages in order, so that the result is the same on every run:
// page p is the r-th free one, r = the number of free pages below p, and the r-th entry that wants a
// page gets it.
//
// The counts are made by one cluster of kCtas CTAs, each over a run of the pool: every CTA counts its
// run, the counts meet at a cluster barrier, and each CTA goes through its run again and hands its free
// pages on.  So one launch does what would otherwise take a launch for each step of a scan, and at the
// usual sizes a launch costs more than the counting.  The copies and the table's entries, which are as
// many bytes as the cache's owner likes, follow in a kernel over all SMs.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "kv_cache.cuh"
#include "osm_internal.h"
#include "per_device.h"

namespace osm {
namespace {

namespace cg = cooperative_groups;

constexpr int kCtas = 8;  // of the cluster: the most that is portable
constexpr int kThreads = 1024;
constexpr int kPer = 4;  // consecutive pages a thread takes at a time
constexpr int kStep = kThreads * kPer;
constexpr int kNone = 0x7fffffff;
// Small calls are one launch without a workspace: up to kRowsHere rows, and pairs, a call's lists fit
// shared memory, and every CTA of the cluster makes them for itself (a call of 64 rows 23 us from
// Python, 28 with two launches and a workspace).  The cluster's eight SMs do the copies then too, so
// only where those are few: they take 3.6 us to fork 32 rows of 63 entries, 6.2 in two launches; but
// 20 and 8.5 for 79 rows of 2044, and 50 and 15 for 56 copies of two pages of up to 128 KB.
constexpr int kRowsHere = 2048;
constexpr int64_t kGrowCopies = 2 << 20;  // bytes, if every row copied a whole page
constexpr int64_t kForkEntries = 1 << 15;

__device__ __forceinline__ int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tokens of a row, within the table's room.
__device__ __forceinline__ int64_t tokens(int32_t len, int64_t room) {
    return len < 0 ? 0 : (len < room ? len : room);
}

// Sum of x over the threads before this one, and over all of them (1024 threads; s: 33 ints).
__device__ __forceinline__ int scan_block(int x, int* s, int* total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int inc = x;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, m);
        if (lane >= m) inc += o;
    }
    if (lane == 31) s[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int t = s[lane];
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, t, m);
            if (lane >= m) t += o;
        }
        s[lane] = t;
    }
    __syncthreads();
    *total = s[31];
    const int before = (warp ? s[warp - 1] : 0) + inc - x;
    __syncthreads();
    return before;
}

// The pages [lo, hi) of the cluster's CTA `rank`: whole steps.
struct Run {
    int64_t lo, hi;
};
__device__ __forceinline__ Run run_of(int64_t n, int rank) {
    const int64_t each = ceil_div(ceil_div(n, kCtas), kStep) * kStep;
    const int64_t lo = each * rank;
    return {lo < n ? lo : n, lo + each < n ? lo + each : n};
}

// This thread's kPer pages from `at` on, with bit i set where page at + i lies in the run and
// want(page, uses) holds.
template <typename Want>
__device__ __forceinline__ uint32_t marks(const int32_t* refs, int64_t at, int64_t hi,
                                          const Want& want) {
    int32_t r[kPer];
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) r[i] = at + i < hi ? refs[at + i] : 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (at + i < hi && want(at + i, r[i])) bits |= 1u << i;
    return bits;
}

template <typename Want>
__device__ __forceinline__ int count_run(const int32_t* refs, Run run, int* s, const Want& want) {
    int n = 0;
#pragma unroll 4
    for (int64_t at = run.lo + threadIdx.x * kPer; at < run.hi; at += kStep)
        n += __popc(marks(refs, at, run.hi, want));
    int total;
    scan_block(n, s, &total);
    return total;
}

// Calls use(page, rank) for every marked page of the run, in any order, with its rank, `base` the
// rank of the run's first; stops once all ranks are at or past `most`.
template <typename Want, typename Use>
__device__ __forceinline__ void rank_run(const int32_t* refs, Run run, int base, int most, int* s,
                                         const Want& want, const Use& use) {
    for (int64_t at = run.lo; at < run.hi && base < most; at += kStep) {
        const int64_t mine = at + threadIdx.x * kPer;
        const uint32_t bits = marks(refs, mine, run.hi, want);
        int total;
        int rank = base + scan_block(__popc(bits), s, &total);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (bits >> i & 1) {
                if (rank < most) use(mine + i, rank);
                ++rank;
            }
        base += total;
    }
}

// The cluster's counts (one a CTA), left in each CTA's shared memory: sum below `rank`, and of all.
__device__ __forceinline__ int gather_counts(cg::cluster_group& cl, int* mine, int* total) {
    int below = 0, all = 0;
    const int rank = static_cast<int>(cl.block_rank());
#pragma unroll
    for (int c = 0; c < kCtas; ++c) {
        const int n = *cl.map_shared_rank(mine, c);
        all += n;
        if (c < rank) below += n;
    }
    *total = all;
    return below;
}

struct PageParams {
    KvPages pg;        // fork and free: no page arrays
    int32_t* table;    // [rows, max_pages]
    int32_t* lens;     // [rows]
    int32_t* refs;     // [num_pages]
    int32_t* ws;
    int64_t rows;
    const int32_t *a, *b;  // grow: new_lens; fork: src, dst; free: rows or nullptr, keep or nullptr
    int32_t* out;          // grow: old_lens or nullptr; compact: page_map
    int32_t* used;         // compact
    int64_t n;             // fork: pairs; free: rows in the list
    int row_bytes;         // bytes of a token's values in a page head
};

__device__ __forceinline__ bool is_free(int64_t, int32_t r) { return r <= 0; }

// ------------------------------------------------------------------------------------------
// grow.  A row's entries that get pages are consecutive: those behind its last, and before them, where
// the last page is not full and has other uses, that page's own entry, which gets a copy.
// ------------------------------------------------------------------------------------------
struct GrowRow {
    int64_t old, now;
    int first, need, from, rest;  // its entries, the page to copy (-1: none) and the tokens of it
};
__device__ __forceinline__ GrowRow grow_row(const PageParams& p, int64_t r) {
    const int64_t room = p.pg.max_pages * p.pg.page;
    GrowRow g;
    g.old = tokens(p.lens[r], room);
    const int64_t more = p.a[r] < 0 ? 0 : p.a[r];
    g.now = g.old + more < room ? g.old + more : room;
    g.rest = static_cast<int>(g.old % p.pg.page);
    g.first = static_cast<int>(ceil_div(g.old, p.pg.page));
    g.from = -1;
    if (g.now > g.old && g.rest) {
        const int32_t e = p.table[r * p.pg.max_pages + g.first - 1];
        if (e >= 0 && e < p.pg.num_pages && p.refs[e] > 1) {
            g.from = e;
            --g.first;
        }
    }
    g.need = static_cast<int>(ceil_div(g.now, p.pg.page)) - g.first;
    return g;
}

// The `rest` tokens of page `from` into page `to`, every head's keys and values: threads tid, tid +
// all, ... of `all`.
__device__ __forceinline__ void copy_tokens(const PageParams& p, int from, int to, int rest, int tid,
                                            int all) {
    const int64_t src = static_cast<int64_t>(from) * p.pg.H_kv * p.pg.head_bytes;
    const int64_t dst = static_cast<int64_t>(to) * p.pg.H_kv * p.pg.head_bytes;
    const int chunks = rest * (p.row_bytes / 16), total = 2 * p.pg.H_kv * chunks;
#pragma unroll 4
    for (int u = tid; u < total; u += all) {
        const int h = u / chunks, c = u - h * chunks;
        uint8_t* pages = h < p.pg.H_kv ? p.pg.k : p.pg.v;
        const int64_t at = (h < p.pg.H_kv ? h : h - p.pg.H_kv) * p.pg.head_bytes + c * 16;
        *reinterpret_cast<uint4*>(pages + dst + at) =
            *reinterpret_cast<const uint4*>(pages + src + at);
    }
    if (p.pg.format != OSM_KV_INT4) return;
    // the words: row_bytes / 16 bytes a token (2 or 4)
    const int word = p.row_bytes / 16;
    for (int u = tid; u < 2 * p.pg.H_kv * rest; u += all) {
        const int h = u / rest, c = u - h * rest;
        uint8_t* pages = h < p.pg.H_kv ? p.pg.k : p.pg.v;
        const int64_t at = (h < p.pg.H_kv ? h : h - p.pg.H_kv) * p.pg.head_bytes +
                           static_cast<int64_t>(p.pg.page) * p.row_bytes + c * word;
        if (word == 4)
            *reinterpret_cast<uint32_t*>(pages + dst + at) =
                *reinterpret_cast<const uint32_t*>(pages + src + at);
        else
            *reinterpret_cast<uint16_t*>(pages + dst + at) =
                *reinterpret_cast<const uint16_t*>(pages + src + at);
    }
}

// The entry of the k-th page that is given out, before[r] of them to the rows before r.
__device__ __forceinline__ int32_t* entry_of(const PageParams& p, const int32_t* before,
                                             const int32_t* first, int k) {
    int64_t lo = 0, hi = p.rows - 1;  // the last row with before[row] <= k
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (before[mid] <= k) lo = mid;
        else hi = mid - 1;
    }
    return p.table + lo * p.pg.max_pages + first[lo] + (k - before[lo]);
}

// Hands out the run's free pages, once the counts of all CTAs are known: `base` free ones before it,
// `all` in the pool, `wanted` to give.
__device__ __forceinline__ void give_pages(const PageParams& p, Run run, int rank, int base, int all,
                                           int wanted, const int32_t* before, const int32_t* first,
                                           int* s) {
    rank_run(p.refs, run, base, wanted, s, is_free, [&](int64_t page, int k) {
        *entry_of(p, before, first, k) = static_cast<int32_t>(page);
        p.refs[page] = 1;
    });
    for (int64_t k = static_cast<int64_t>(all) + rank * kThreads + threadIdx.x; k < wanted;
         k += kCtas * kThreads) {
        *entry_of(p, before, first, static_cast<int>(k)) = -1;
        if (k == all) kv_bad_page(p.pg);
    }
}

// Up to kRowsHere rows: one launch.  Every CTA has the rows' lists; after the counts the pages are
// given out, and after that (another barrier) the cluster's warps make the copies.  The uses of copied
// pages go down last of all, when every CTA has seen the counts: a page whose rows all copy becomes
// free for the next call.
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    grow_kernel(const PageParams p) {
    __shared__ int s[33];
    __shared__ int s_count;
    __shared__ int32_t s_before[kRowsHere], s_first[kRowsHere];
    __shared__ int32_t s_copy[kRowsHere], s_rest[kRowsHere];  // of the rows that copy: row, tokens
    __shared__ int32_t s_from[kRowsHere];
    cg::cluster_group cl = cg::this_cluster();
    const int rank = static_cast<int>(cl.block_rank());
    const Run run = run_of(p.pg.num_pages, rank);
    int wanted = 0, copies = 0;
    int64_t old[kRowsHere / kThreads], now[kRowsHere / kThreads];
#pragma unroll
    for (int i = 0; i < kRowsHere / kThreads; ++i) {
        if (i * kThreads >= p.rows) break;
        const int64_t r = i * kThreads + threadIdx.x;
        GrowRow g{};
        g.from = -1;
        if (r < p.rows) g = grow_row(p, r);
        old[i] = g.old, now[i] = g.now;
        int total, copied;
        const int at = wanted + scan_block(g.need, s, &total);
        const int c = copies + scan_block(g.from >= 0, s, &copied);
        if (r < p.rows) {
            s_before[r] = at;
            s_first[r] = g.first;
        }
        if (g.from >= 0) {
            s_copy[c] = static_cast<int32_t>(r);
            s_from[c] = g.from;
            s_rest[c] = g.rest;
        }
        wanted += total;
        copies += copied;
    }
    const int n = count_run(p.refs, run, s, is_free);
    if (threadIdx.x == 0) s_count = n;
    cl.sync();  // the counts are there, and every CTA has read the lengths and the table
    if (rank == 0) {
#pragma unroll
        for (int i = 0; i < kRowsHere / kThreads; ++i) {
            const int64_t r = i * kThreads + threadIdx.x;
            if (r >= p.rows) break;
            p.lens[r] = static_cast<int32_t>(now[i]);
            if (p.out) p.out[r] = static_cast<int32_t>(old[i]);
        }
    }
    int all;
    const int base = gather_counts(cl, &s_count, &all);
    give_pages(p, run, rank, base, all, wanted, s_before, s_first, s);
    cl.sync();  // no CTA ends while another reads its count; and the pages are in the table
    const int warps = kCtas * kThreads / 32, warp = rank * (kThreads / 32) + threadIdx.x / 32;
    const int lane = threadIdx.x & 31, slices = max(1, warps / max(copies, 1));
    for (int u = warp; u < copies * slices; u += warps) {
        const int c = u / slices, slice = u - c * slices, r = s_copy[c];
        const int to = p.table[r * p.pg.max_pages + s_first[r]];
        if (slice == 0 && lane == 0) atomicSub(&p.refs[s_from[c]], 1);
        if (to >= 0) copy_tokens(p, s_from[c], to, s_rest[c], slice * 32 + lane, slices * 32);
    }
}

// Any number of rows, in two launches.  ws: before[rows + 1] (entries wanted by the rows before),
// first[rows] (the first of the row's), from[rows] (the page to copy, -1: none), rest[rows].
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    grow_plan_kernel(const PageParams p) {
    __shared__ int s[33];
    __shared__ int s_count;
    asm volatile("griddepcontrol.launch_dependents;");
    cg::cluster_group cl = cg::this_cluster();
    const int rank = static_cast<int>(cl.block_rank());
    int32_t* before = p.ws;
    int32_t* first = p.ws + p.rows + 1;
    const Run run = run_of(p.pg.num_pages, rank);
    if (rank == kCtas - 1) {  // the run that is shorter than the others, or empty
        int carry = 0;
        for (int64_t r0 = 0; r0 < p.rows; r0 += kThreads) {
            const int64_t r = r0 + threadIdx.x;
            GrowRow g{};
            if (r < p.rows) {
                g = grow_row(p, r);
                first[r] = g.first;
                first[p.rows + r] = g.from;
                first[2 * p.rows + r] = g.rest;
                p.lens[r] = static_cast<int32_t>(g.now);
                if (p.out) p.out[r] = static_cast<int32_t>(g.old);
            }
            int total;
            const int x = scan_block(g.need, s, &total);
            if (r < p.rows) before[r] = carry + x;
            carry += total;
        }
        if (threadIdx.x == 0) before[p.rows] = carry;
    }
    const int n = count_run(p.refs, run, s, is_free);
    if (threadIdx.x == 0) s_count = n;
    cl.sync();
    int all;
    const int base = gather_counts(cl, &s_count, &all);
    give_pages(p, run, rank, base, all, before[p.rows], before, first, s);
    cl.sync();  // no CTA ends while another reads its count
}

// CTA (x, r): slice x of the copy for row r, if it has one.
constexpr int kCopyThreads = 256;
__global__ void __launch_bounds__(kCopyThreads) grow_copy_kernel(const PageParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t* first = p.ws + p.rows + 1;
    for (int64_t r = blockIdx.y; r < p.rows; r += gridDim.y) {
        const int32_t from = first[p.rows + r];
        if (from < 0) continue;
        const int tid = blockIdx.x * kCopyThreads + threadIdx.x;
        if (tid == 0) atomicSub(&p.refs[from], 1);
        const int32_t to = p.table[r * p.pg.max_pages + first[r]];
        if (to >= 0)  // (a page was left)
            copy_tokens(p, from, to, first[2 * p.rows + r], tid, gridDim.x * kCopyThreads);
    }
}

// ------------------------------------------------------------------------------------------
// fork.  A pair is done if its rows are some, its destination is empty, and no earlier pair of the list
// has that destination; claim[row] is the first such pair.
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ bool fork_known(const PageParams& p, int64_t i) {
    return p.a[i] >= 0 && p.a[i] < p.rows && p.b[i] >= 0 && p.b[i] < p.rows && p.lens[p.b[i]] <= 0;
}

// Each pair's tokens in len (-1: nothing is done), by one block.
__device__ __forceinline__ void fork_plan(const PageParams& p, int32_t* claim, int32_t* len,
                                          bool report) {
    const int64_t room = p.pg.max_pages * p.pg.page;
    for (int64_t r = threadIdx.x; r < p.rows; r += kThreads) claim[r] = kNone;
    __syncthreads();
    for (int64_t i = threadIdx.x; i < p.n; i += kThreads)
        if (fork_known(p, i)) atomicMin(&claim[p.b[i]], static_cast<int>(i));
    __syncthreads();
    for (int64_t i = threadIdx.x; i < p.n; i += kThreads) {
        int64_t L = -1;
        if (fork_known(p, i) && claim[p.b[i]] == i)
            L = tokens(p.lens[p.a[i]], room);
        else if (report && p.a[i] >= 0 && p.b[i] >= 0)
            kv_bad_page(p.pg);  // no such row, or one that holds tokens or is taken
        len[i] = static_cast<int32_t>(L);
    }
}

// Slice `slice` of `slices` of pair i, by T threads.  (A row that is written holds no tokens before, so
// none of its entries is read.)
template <int T>
__device__ __forceinline__ void fork_row(const PageParams& p, int64_t i, int32_t L, int slice,
                                         int slices, int t) {
    const int32_t* from = p.table + p.a[i] * p.pg.max_pages;
    int32_t* to = p.table + p.b[i] * p.pg.max_pages;
    const int n = static_cast<int>(ceil_div(L, p.pg.page)), all = slices * T, tid = slice * T + t;
#pragma unroll 8
    for (int j = tid; j < n; j += all) {
        const int32_t e = from[j];
        to[j] = e;
        if (e >= 0 && e < p.pg.num_pages) atomicAdd(&p.refs[e], 1);
    }
    if (tid == 0) p.lens[p.b[i]] = L;
}

// Up to kRowsHere rows and pairs and kForkEntries entries: one launch.  Every CTA of the cluster makes
// the plan for itself; the lengths change when all have.
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    fork_kernel(const PageParams p) {
    __shared__ int32_t s_claim[kRowsHere], s_len[kRowsHere];
    cg::cluster_group cl = cg::this_cluster();
    const int rank = static_cast<int>(cl.block_rank());
    fork_plan(p, s_claim, s_len, rank == 0);
    cl.sync();
    const int warps = kCtas * kThreads / 32, warp = rank * (kThreads / 32) + threadIdx.x / 32;
    const int pairs = static_cast<int>(p.n), slices = max(1, warps / pairs);
    for (int u = warp; u < pairs * slices; u += warps) {
        const int i = u / slices;
        if (s_len[i] >= 0) fork_row<32>(p, i, s_len[i], u - i * slices, slices, threadIdx.x & 31);
    }
}

// Any number, in two launches.  ws: claim[rows], then each pair's tokens.
__global__ void __launch_bounds__(kThreads) fork_plan_kernel(const PageParams p) {
    asm volatile("griddepcontrol.launch_dependents;");
    fork_plan(p, p.ws, p.ws + p.rows, true);
}
// CTA (i, y): slice y of pair i.
__global__ void __launch_bounds__(kCopyThreads) fork_copy_kernel(const PageParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t i = blockIdx.x;
    const int32_t L = p.ws[p.rows + i];
    if (L >= 0) fork_row<kCopyThreads>(p, i, L, blockIdx.y, gridDim.y, threadIdx.x);
}

// ------------------------------------------------------------------------------------------
// free.  A CTA a row of the list.  The row's length goes down in one atomic step, so that a row
// listed twice gives each entry back once: whoever lowers the length from old to keep owns the
// entries between.  3.3 us for the last tokens of 64 rows, 7.5 for 64 rows of up to 2048 entries, both
// of them latency: the length, the entries, the counts.
// ------------------------------------------------------------------------------------------
constexpr int kFreeThreads = 512;
__global__ void __launch_bounds__(kFreeThreads) free_kernel(const PageParams p) {
    __shared__ int32_t s_old;
    const int64_t i = blockIdx.x;
    const int64_t row = p.a ? p.a[i] : i;
    if (row < 0) return;
    if (row >= p.rows) {
        if (threadIdx.x == 0) kv_bad_page(p.pg);
        return;
    }
    const int32_t keep = p.b && p.b[i] > 0 ? p.b[i] : 0;
    if (threadIdx.x == 0) s_old = atomicMin(&p.lens[row], keep);
    __syncthreads();
    const int64_t room = p.pg.max_pages * p.pg.page;
    const int64_t old = tokens(s_old, room);
    const int64_t j1 = ceil_div(old, p.pg.page);
    const int32_t* entries = p.table + row * p.pg.max_pages;
#pragma unroll 4
    for (int64_t j = ceil_div(keep, p.pg.page) + threadIdx.x; j < j1; j += kFreeThreads) {
        const int32_t e = entries[j];
        if (e < 0 || e >= p.pg.num_pages) continue;
        // never below 0: once the count is 0, every further step is taken back
        if (atomicSub(&p.refs[e], 1) <= 0) atomicAdd(&p.refs[e], 1);
    }
}

// ------------------------------------------------------------------------------------------
// compact.  ws: [0] the pages to move, then their places now and to come.
// ------------------------------------------------------------------------------------------
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    compact_plan_kernel(const PageParams p) {
    __shared__ int s[33];
    __shared__ int s_used, s_move, s_hole;
    asm volatile("griddepcontrol.launch_dependents;");
    cg::cluster_group cl = cg::this_cluster();
    const int rank = static_cast<int>(cl.block_rank());
    const Run run = run_of(p.pg.num_pages, rank);
    int32_t* from = p.ws + 1;
    int32_t* to = p.ws + 1 + p.pg.num_pages / 2;
    {
        const int n = count_run(p.refs, run, s, [](int64_t, int32_t r) { return r > 0; });
        if (threadIdx.x == 0) s_used = n;
    }
    cl.sync();
    int used;
    gather_counts(cl, &s_used, &used);
    // A run wholly below `used`, or wholly above it, knows its free pages to fill (holes) and its
    // pages to move from its first count; the one that `used` falls into counts again.
    auto hole = [=](int64_t page, int32_t r) { return page < used && r <= 0; };
    auto mover = [=](int64_t page, int32_t r) { return page >= used && r > 0; };
    int holes, movers;
    if (run.hi <= used) {
        holes = static_cast<int>(run.hi - run.lo) - s_used;
        movers = 0;
    } else if (run.lo >= used) {
        holes = 0;
        movers = s_used;
    } else {
        holes = count_run(p.refs, run, s, hole);
        movers = s_used - (used - static_cast<int>(run.lo) - holes);
    }
    if (threadIdx.x == 0) {
        s_hole = holes;
        s_move = movers;
    }
    cl.sync();
    int n_holes, n_moves;
    const int hole0 = gather_counts(cl, &s_hole, &n_holes);
    const int move0 = gather_counts(cl, &s_move, &n_moves);
    if (rank == 0 && threadIdx.x == 0) {
        p.ws[0] = n_moves;
        p.used[0] = used;
    }
    if (holes)
        rank_run(p.refs, run, hole0, kNone, s, hole,
                 [&](int64_t page, int k) { to[k] = static_cast<int32_t>(page); });
    if (movers)
        rank_run(p.refs, run, move0, kNone, s, mover,
                 [&](int64_t page, int k) { from[k] = static_cast<int32_t>(page); });
    for (int64_t at = run.lo + threadIdx.x; at < run.hi; at += kThreads) {
        const bool taken = p.refs[at] > 0;
        if (!taken || at < used) p.out[at] = taken ? static_cast<int32_t>(at) : -1;
    }
    cl.sync();
    for (int k = rank * kThreads + threadIdx.x; k < n_moves; k += kCtas * kThreads) {
        const int32_t a = from[k], b = to[k];
        p.out[a] = b;
        p.refs[b] = p.refs[a];
        p.refs[a] = 0;
    }
}

// A CTA copies pages (the keys or the values of one, all heads) in turn, and renames the entries of
// rows in turn.  Places now and to come are disjoint, so the copies need no order.  Half of 9551 pages
// of 128 KB and 128 KB in use, 626 MB to move: 188 us, 6.66 TB/s, 98 % of a copy's rate.
__global__ void __launch_bounds__(kCopyThreads) compact_copy_kernel(const PageParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t room = p.pg.max_pages * p.pg.page;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const int64_t n = ceil_div(tokens(p.lens[r], room), p.pg.page);
        int32_t* entries = p.table + r * p.pg.max_pages;
        for (int64_t j = threadIdx.x; j < n; j += kCopyThreads) {
            const int32_t e = entries[j];
            if (e < 0 || e >= p.pg.num_pages) continue;
            const int32_t now = p.out[e];
            if (now != e) entries[j] = now;
        }
    }
    const int moves = p.ws[0];
    const int32_t* from = p.ws + 1;
    const int32_t* to = p.ws + 1 + p.pg.num_pages / 2;
    const int64_t bytes = p.pg.head_bytes * p.pg.H_kv;
    const int chunks = static_cast<int>(bytes / 16);
    for (int64_t i = blockIdx.x; i < 2 * static_cast<int64_t>(moves); i += gridDim.x) {
        uint8_t* pages = i < moves ? p.pg.k : p.pg.v;
        const int k = static_cast<int>(i < moves ? i : i - moves);
        const uint4* a = reinterpret_cast<const uint4*>(pages + from[k] * bytes);
        uint4* b = reinterpret_cast<uint4*>(pages + to[k] * bytes);
        constexpr int U = 8;
        int c = threadIdx.x;
        for (; c + (U - 1) * kCopyThreads < chunks; c += U * kCopyThreads) {
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = __ldcs(a + c + u * kCopyThreads);
#pragma unroll
            for (int u = 0; u < U; ++u) __stcs(b + c + u * kCopyThreads, x[u]);
        }
        for (; c < chunks; c += kCopyThreads) b[c] = a[c];
    }
}

// The second kernel's launch overlaps the first (it waits for it on the device).
template <typename... Args>
int launch_after(void (*kernel)(Args...), dim3 grid, int threads, cudaStream_t stream,
                 const PageParams& p) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int launched() { return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

int sm_count() {
    const int n = device_sm_count();
    return n > 0 ? n : 152;
}

// One launch where the lists fit shared memory and a cluster's SMs are enough for the work.
bool grow_here(int64_t rows, int64_t page_bytes) {
    return rows <= kRowsHere && 2 * page_bytes <= kGrowCopies / (rows > 0 ? rows : 1);
}
bool fork_here(int64_t rows, int64_t pairs, int64_t max_pages) {
    return rows <= kRowsHere && pairs <= kRowsHere &&
           max_pages <= kForkEntries / (pairs > 0 ? pairs : 1);
}

int64_t round16(int64_t words) { return (4 * words + 15) / 16 * 16; }

}  // namespace

int64_t kv_grow_ws_bytes(int64_t rows, int64_t page_bytes) {
    return grow_here(rows, page_bytes) ? 0 : round16(4 * rows + 1);
}
int64_t kv_fork_ws_bytes(int64_t rows, int64_t pairs, int64_t max_pages) {
    return fork_here(rows, pairs, max_pages) ? 0 : round16(rows + pairs);
}
int64_t kv_compact_ws_bytes(int64_t num_pages) { return round16(1 + num_pages); }

int osm_kv_grow_launch(const KvPages& pg, int32_t* table, int32_t* lens, const int32_t* new_lens,
                       int32_t* old_lens, int32_t* refs, int64_t rows, int64_t d, void* ws,
                       cudaStream_t stream) {
    PageParams p{};
    p.pg = pg;
    p.table = table;
    p.lens = lens;
    p.refs = refs;
    p.ws = static_cast<int32_t*>(ws);
    p.rows = rows;
    p.a = new_lens;
    p.out = old_lens;
    p.row_bytes = static_cast<int>(pg.format == OSM_KV_BF16 ? 2 * d : d / 2);
    if (grow_here(rows, pg.head_bytes * pg.H_kv)) {
        grow_kernel<<<kCtas, kThreads, 0, stream>>>(p);
        return launched();
    }
    grow_plan_kernel<<<kCtas, kThreads, 0, stream>>>(p);
    const int st = launched();
    if (st != FA_OK) return st;
    // slices of a row: CTAs for two waves where every row copies
    int64_t x = (4 * sm_count() + rows - 1) / rows;
    x = x > 16 ? 16 : x;
    const int64_t y = rows < 65535 ? rows : 65535;
    return launch_after(grow_copy_kernel,
                        dim3(static_cast<unsigned>(x), static_cast<unsigned>(y)), kCopyThreads,
                        stream, p);
}

int osm_kv_fork_launch(const KvPages& pg, int32_t* table, int32_t* lens, int32_t* refs,
                       const int32_t* src, const int32_t* dst, int64_t rows, int64_t n, void* ws,
                       cudaStream_t stream) {
    PageParams p{};
    p.pg = pg;
    p.table = table;
    p.lens = lens;
    p.refs = refs;
    p.ws = static_cast<int32_t*>(ws);
    p.rows = rows;
    p.a = src;
    p.b = dst;
    p.n = n;
    if (fork_here(rows, n, pg.max_pages)) {
        fork_kernel<<<kCtas, kThreads, 0, stream>>>(p);
        return launched();
    }
    fork_plan_kernel<<<1, kThreads, 0, stream>>>(p);
    const int st = launched();
    if (st != FA_OK) return st;
    // slices of a pair: CTAs for two waves, and an entry a thread at least
    int64_t y = (4 * sm_count() + n - 1) / n;
    const int64_t most = (pg.max_pages + kCopyThreads - 1) / kCopyThreads;
    y = y > most ? most : y;
    y = y < 1 ? 1 : (y > 64 ? 64 : y);
    return launch_after(fork_copy_kernel, dim3(static_cast<unsigned>(n), static_cast<unsigned>(y)),
                        kCopyThreads, stream, p);
}

int osm_kv_free_launch(const KvPages& pg, int32_t* table, int32_t* lens, int32_t* refs,
                       const int32_t* list, const int32_t* keep, int64_t rows, int64_t n,
                       cudaStream_t stream) {
    PageParams p{};
    p.pg = pg;
    p.table = table;
    p.lens = lens;
    p.refs = refs;
    p.rows = rows;
    p.a = list;
    p.b = keep;
    p.n = n;
    free_kernel<<<static_cast<unsigned>(n), kFreeThreads, 0, stream>>>(p);
    return launched();
}

int osm_kv_compact_launch(const KvPages& pg, int32_t* table, int32_t* lens, int32_t* refs,
                          int32_t* page_map, int32_t* used, int64_t rows, void* ws,
                          cudaStream_t stream) {
    PageParams p{};
    p.pg = pg;
    p.table = table;
    p.lens = lens;
    p.refs = refs;
    p.ws = static_cast<int32_t*>(ws);
    p.rows = rows;
    p.out = page_map;
    p.used = used;
    compact_plan_kernel<<<kCtas, kThreads, 0, stream>>>(p);
    const int st = launched();
    if (st != FA_OK) return st;
    return launch_after(compact_copy_kernel, dim3(static_cast<unsigned>(8 * sm_count())),
                        kCopyThreads, stream, p);
}

}  // namespace osm
