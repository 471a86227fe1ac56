// fa_shared.cu -- attention over the paged cache for groups of sequences with a common prefix
// (fa_fwd_paged_shared).
//
// The computation is the online softmax of fa_fwd.cu with its two-worker merge ("How FlashAttention
// avoids storing the giant score table" (spicyshark.co, Online softmax lesson), "From softmax to
// attention"): a row's state over its group's common tokens and its state over its sequence's own
// tokens are made by different kernels and joined.  Four launches:
//   plan    finds what is common: for each sequence the leading entries of its table's row that are
//           those of its group's first one, and from these the groups' common tiles.
//   prefix  the common tokens, for all rows of a group at once: here, on tcgen05.
//   own     the tokens behind them, a sequence at a time: paged_kernel (fa_paged.cu).  It and the
//           prefix kernel share no data and run side by side, on SMs that the plan divides among them.
//   join    merges each row's states and writes O and LSE.
//
// Prefix kernel.  With m sequences of r query rows on a key/value head, each byte of the prefix meets
// m r rows instead of r, so that what bounds the work goes from memory to the tensor cores as m r
// grows: a tile of 128 tokens is 64 KB in bf16 (d = 128), about 2800 clocks of an SM's part of the
// memory, and 2500 clocks of products for 256 rows.  Hence blocks of 256 rows, two softmax groups of
// 128, so that one's exponentials run beside the other's products; with fewer rows the two groups
// take the tiles in turn.  Measured (d = 128, tiles of 128 tokens x 256 rows): bf16 1.7 us a tile, 5.9
// TB/s (87 % of a copy's rate), and 1.64 from the L2 (79 % of the tensor cores' rate); 4 bits 2.0, where
// the expansion's stores and the products share the shared memory, and 1.1 for up to 128 rows.  A CTA's
// start costs 15 us (the plan, then first reads of queries, table and pages), so that 64 sequences
// with 16384 common bf16 tokens take 32 us alone on all SMs, seven tiles a CTA (ncu; 68.8 MB read).  A
// CTA an SM, each with a piece of an item or an equal share of all (see the plan):
//   warps 0-3, 4-7  softmax group w, a row a thread: S from TMEM, the lazy running max of fa_fwd.cu,
//           exponentials, P in bf16 over S's own columns, O rescaled in TMEM when the max moves; at
//           an item's end O and (m, l) go to the workspace.  They load their rows' queries too.
//   warp 13         the key and value tiles in the order of their use, a lane the tokens that lie in
//           one page: bf16: TMA boxes into the ring of swizzled tiles; 4 bits: bulk copies of codes
//           and words as they are into a ring of their own.
//   warps 8-11      4 bits: expand them to bf16, swizzled as a TMA load would store them.
//   warp 12         tcgen05.mma.  Steps u = 0, 1, ... of each group, a tile each: S(0), then PV(u),
//           S(u + 1) of the groups in turn: P(u) lies in the columns of S(u), so S(u + 1) follows
//           PV(u), and the commit of S(u + 1) says that PV(u) is done, so that O may be rescaled
//           before PV(u + 1).  P comes in halves of 64 tokens, so that the first half's product runs
//           beside the second half's exponentials.  (Two buffers of S of half a tile each, so that
//           no product waits for a softmax: slower, 2.9 us a tile of 256 rows at d = 128 against 2.3
//           of whole tiles at the time, as products 64 columns wide read shared memory one and a half
//           times as much.)
// TMEM: S of group w at 128 w, its O at 256 + w d.
//
// 4 bits.  Eight codes of a word become four registers of bf16 pairs, values k and k + 4, by masking
// them over 0x4300 (128 + code), adding base - 128 and multiplying by the step: two exact steps and
// one rounding, as osm_kv_gather reads them out.  The pairs stay in that order: the queries are
// stored in the same order of d, and O's columns are put right as they are written.
//
// Every wait is bounded; one that gives up records FA_ERR_TIMEOUT, and the CTA drains its copies and
// products, frees its TMEM and ends.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cmath>
#include <utility>

#include "fa_shared.cuh"
#include "fa_shared_order.h"
#include "kv_cache.cuh"
#include "osm_internal.h"
#include "per_device.h"
#include "ptx_sm103.cuh"

namespace osm {
namespace {

namespace cg = cooperative_groups;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

// ------------------------------------------------------------------------------------------
// plan
// ------------------------------------------------------------------------------------------
// One cluster.  All its warps compare table entries, several warps a sequence while there are enough
// of them; then its first CTA turns what is common into groups.  That is a chain of short steps, each
// as long as a memory access: what they exchange lies in that CTA's shared memory (in the workspace
// for more than kPlanCap sequences), and each step walks over the sequences by as many threads as
// there are sequences for.  9.8 us for 64 sequences of 16384 common tokens; 38, 69 and 131 for 2048,
// 4096 and 8192 of 256 in one group.  (Through the workspace, and the run's lengths read again at each
// step: 11 to 14 us.  One warp for each step, and a search for each sequence's run: 9.7, and 97, 208
// and 500; with a first half that cannot share the call with 8192 took 1100 us, 487 now.)
constexpr int kPlanCtas = 8, kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
constexpr int kMostSlices = 8;  // warps that compare one sequence's entries
constexpr int kPlanCap = 1024;
constexpr int kNever = 0x7fffffff;
constexpr uint32_t kBarGroups = 1, kBarOwn = 2, kBarSplit = 3;
constexpr int kShLeast = 2;  // tiles of a piece or share: fewer leave more states than they save time
constexpr int kItemCost = 3;

// Each sequence's numbers, a list each: [kPlanCap] in shared memory or [B] in the workspace.
struct PlanLists {
    int32_t* base;
    int64_t each;
    __device__ __forceinline__ int32_t* list(int i) const { return base + i * each; }
    __device__ __forceinline__ int32_t& len(int b) const { return list(0)[b]; }  // tokens
    __device__ __forceinline__ int32_t& ql(int b) const { return list(1)[b]; }   // queries
    __device__ __forceinline__ int32_t& common(int b) const { return list(2)[b]; }  // tokens
    // its run's first sequence, and the run's first, up to itself, that can share (later the units of
    // the groups before, at a run's head)
    __device__ __forceinline__ int32_t& head(int b) const { return list(3)[b]; }
    __device__ __forceinline__ int32_t& lead(int b) const { return list(4)[b]; }
    // at a run's head: of its sequences with a tile or more in common, and the least number of tokens
    __device__ __forceinline__ int32_t& first(int b) const { return list(5)[b]; }
    __device__ __forceinline__ int32_t& last(int b) const { return list(6)[b]; }
    __device__ __forceinline__ int32_t& least(int b) const { return list(7)[b]; }
    // of the kernel over the own tokens, with none in common
    __device__ __forceinline__ int32_t& own_tiles(int b) const { return list(8)[b]; }
    __device__ __forceinline__ int32_t& own_items(int b) const { return list(9)[b]; }
    // [slices][B] leading common entries that a slice found
    __device__ __forceinline__ int32_t* same() const { return list(10); }
};
constexpr int kPlanLists = 10 + kMostSlices;  // [B] each, in the workspace

struct PlanParams {
    const int32_t *table, *kv_lens, *q_lens, *gid;
    int64_t num_pages, max_pages;
    int page, B, Nq, causal;
    int rows_per_seq, H_kv;
    int own_rows, own_tile, group;  // of the kernel over the sequences' own tokens
    int32_t* lists;
    ShHead* head;
    ShGroup* groups;
    ShSeq* seqs;
    int ctas, own_ctas;  // of the two kernels' launches
    int own_per_sm;
    int small_cost;  // tiles of a small block that cost as much as four of a large one
    int tile_ns, own_tile_ns, own_item_ns;  // see split_sms
};

__device__ __forceinline__ bool starts_run(const PlanParams& p, int b) {
    return b == 0 || (p.gid && p.gid[b] != p.gid[b - 1]);
}

// SMs for the prefix kernel, one a CTA; the others are the own tokens', which have `own` ns of work for
// one CTA.  Of all splits the one whose later kernel is done first (a whole warp).  A start of either
// kernel is a chain of first reads, which the other one's work covers: against one after the other on
// all SMs, us, replayed after an L2 flush, when this was made: 64 sequences of 16384 common bf16 tokens
// + up to 1000 of their own 82 and 88, + 20 62 and 62; 32 of 32768 + 512 in 4 bits with 3 queries 103
// and 112; 8 of 65536 + 20 in 4 bits 79 and 85; 64 of 8192 + 4000 134 and 140; four groups of 16 of 16384
// + 200 83 to 91 and 83.  (The first and the third 75 and 100 now, the last 81 back to back.)
constexpr float kStartNs = 6000.f;  // the prefix kernel's start takes this much longer
__device__ __forceinline__ int split_sms(const PlanParams& p, long long work, long long own) {
    if (work == 0 || own == 0) return p.ctas;
    const int lane = threadIdx.x & 31;
    float best = INFINITY;
    int at = p.ctas;
    for (int x = 1 + lane; x < p.ctas; x += 32) {
        const float tiles = ceilf(__fdividef(static_cast<float>(work), static_cast<float>(x)));
        const int ctas = min(p.own_ctas, (p.ctas - x) * p.own_per_sm);
        const float t = fmaxf(tiles * static_cast<float>(p.tile_ns) + kStartNs,
                              __fdividef(static_cast<float>(own), static_cast<float>(ctas)));
        if (t < best) best = t, at = x;
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        const float t = __shfl_xor_sync(0xffffffffu, best, m);
        const int x = __shfl_xor_sync(0xffffffffu, at, m);
        if (t < best || (t == best && x < at)) best = t, at = x;
    }
    return at;
}

// Some of a CTA's warps, that walk over the sequences together.  Few sequences take one warp, which
// need not wait for others (32 warps for any number: 2.4 us more for 64 sequences).
struct PlanTeam {
    int first, warps;     // its warps
    uint32_t bar;
    long long* s;         // [warps] in shared memory
    __device__ __forceinline__ int threads() const { return 32 * warps; }
    __device__ __forceinline__ int thread() const {
        return static_cast<int>(threadIdx.x) - 32 * first;
    }
    __device__ __forceinline__ bool has(int warp) const {
        return warp >= first && warp < first + warps;
    }
    __device__ __forceinline__ void sync() const {
        if (warps == 1) __syncwarp();
        else named_bar_sync(bar, 32 * warps);
    }
    // x of the threads before this one, summed, and of all threads
    struct Scan {
        long long before, total;
    };
    __device__ __forceinline__ Scan scan(long long x) const {
        const int warp = (threadIdx.x >> 5) - first, lane = threadIdx.x & 31;
        long long inc = x;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, inc, m);
            if (lane >= m) inc += o;
        }
        if (warps == 1) return {inc - x, __shfl_sync(0xffffffffu, inc, 31)};
        if (lane == 31) s[warp] = inc;
        sync();
        long long all = lane < warps ? s[lane] : 0;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, all, m);
            if (lane >= m) all += o;
        }
        const long long below = __shfl_sync(0xffffffffu, all, warp > 0 ? warp - 1 : 0);
        sync();  // s is free again
        return {inc - x + (warp > 0 ? below : 0), __shfl_sync(0xffffffffu, all, 31)};
    }
};
__device__ __forceinline__ long long low32(long long x) { return x & 0xffffffffll; }

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
    shared_plan_kernel(const PlanParams p) {
    __shared__ int32_t s_list[11][kPlanCap];
    __shared__ int32_t s_head[kPlanWarps], s_lead[kPlanWarps], s_pieces[kItemCost + 1], s_ctas, s_work;
    __shared__ long long s_scan[kPlanWarps], s_own;
    static_assert(kPlanWarps == 32, "a lane each");
    asm volatile("griddepcontrol.launch_dependents;");
    cg::cluster_group cl = cg::this_cluster();
    auto started = cl.barrier_arrive();  // (waited for before another CTA's shared memory is written)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, B = p.B;
    const bool small = B <= kPlanCap;
    const PlanLists x{small ? &s_list[0][0] : p.lists, small ? kPlanCap : B};
    const int64_t room = p.max_pages * p.page;
    const int slices = min(kMostSlices, max(1, kPlanCtas * kPlanWarps / B));
    const int first_unit = static_cast<int>(cl.block_rank()) * kPlanWarps + warp;
    {   // the rows on their way into the L2 while the lengths are read
        const int b = first_unit / slices, s = first_unit - b * slices;
        if (b < B)
            for (int64_t e = (s * 32 + lane) * 32; e < p.max_pages; e += slices * 1024)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p.table + b * p.max_pages + e));
    }
    if (threadIdx.x <= kItemCost) s_pieces[threadIdx.x] = 0;
    if (threadIdx.x == 0) s_work = 0;

    // ---- each sequence's run (its first sequence), and the first of the run, up to it, that can share.
    // (large: every CTA writes the same numbers)
    // Keys that every query of a sequence sees, less one, so that something is left of its own; below
    // 0: none, or no query.
    auto keys_seen = [&](int len, int ql) {
        return ql == 0 ? -1 : (p.causal ? len - ql : len - 1);
    };
    auto seen = [&](int b) { return keys_seen(x.len(b), x.ql(b)); };
    int run = -1, run_lead = -1;  // of the run that reaches into this step
    for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
        const int b = b0 + static_cast<int>(threadIdx.x), w0 = b - lane;
        bool start = false, can = false;
        if (b < B) {
            const int len = static_cast<int>(min(static_cast<int64_t>(max(p.kv_lens[b], 0)), room));
            const int ql = p.q_lens ? min(max(p.q_lens[b], 0), p.Nq) : p.Nq;
            x.len(b) = len;
            x.ql(b) = ql;
            x.own_tiles(b) = (len + p.own_tile - 1) / p.own_tile;
            x.own_items(b) = p.H_kv * ((ql * p.group + p.own_rows - 1) / p.own_rows);
            x.first(b) = kNever;
            x.last(b) = -1;
            x.least(b) = kNever;
            start = starts_run(p, b);
            can = keys_seen(len, ql) >= kShTile;
        }
        // within the warp: the last start up to this lane, the first that can share from there on
        const unsigned upto = 0xffffffffu >> (31 - lane);
        const unsigned starts = __ballot_sync(0xffffffffu, start) & upto;
        const int at = starts ? 31 - __clz(starts) : 0;
        const unsigned cans = __ballot_sync(0xffffffffu, can) & upto & (0xffffffffu << at);
        int head = starts ? w0 + at : -1, lead = cans ? w0 + __ffs(cans) - 1 : -1;
        if (lane == 31) {
            s_head[warp] = head;
            s_lead[warp] = lead;
        }
        __syncthreads();
        // what the warps before leave, `n` of them
        const int h = s_head[lane], l = s_lead[lane];
        const unsigned hs = __ballot_sync(0xffffffffu, h >= 0);
        const unsigned ls = __ballot_sync(0xffffffffu, l >= 0);
        auto reaches = [&](int n, int& r, int& r_lead) {
            const unsigned below = n == 32 ? 0xffffffffu : (1u << n) - 1u;
            const int k = hs & below ? 31 - __clz(hs & below) : 0;
            const unsigned from = ls & below & (0xffffffffu << k);
            const int hk = __shfl_sync(0xffffffffu, h, k);
            const int lk = __shfl_sync(0xffffffffu, l, from ? __ffs(from) - 1 : 0);
            if (hs & below) r = hk, r_lead = -1;
            if (r_lead < 0 && from) r_lead = lk;
        };
        int r = run, r_lead = run_lead;
        reaches(warp, r, r_lead);
        if (!starts) {
            head = r;
            if (r_lead >= 0) lead = r_lead;
        }
        if (b < B) {
            x.head(b) = head;
            x.lead(b) = lead;
        }
        if (b0 + kPlanThreads < B) {
            reaches(32, run, run_lead);
            __syncthreads();
        }
    }
    __syncthreads();

    // ---- the leading entries that a sequence has in common with that one
    cl.barrier_wait(std::move(started));
    int32_t* same_at = small ? cl.map_shared_rank(&s_list[10][0], 0) : x.same();
    for (int64_t u = first_unit; u < static_cast<int64_t>(B) * slices;
         u += kPlanCtas * kPlanWarps) {
        const int b = static_cast<int>(u / slices);
        const int s = static_cast<int>(u - static_cast<int64_t>(b) * slices);
        int32_t same = 0;
        if (seen(b) >= kShTile) {
            const int lead = x.lead(b);
            const int n = (min(seen(b), seen(lead)) + p.page - 1) / p.page;
            const int each = ((n + slices - 1) / slices + 31) & ~31;
            const int j0 = s * each, j1 = min(n, j0 + each);
            const int32_t* mine = p.table + b * p.max_pages;
            const int32_t* other = p.table + lead * p.max_pages;
            same = n;
            constexpr int U = 8;
            for (int j = j0; j < j1; j += 32 * U) {
                int32_t a[U], c[U];
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int k = j + 32 * i + lane;
                    a[i] = k < j1 ? mine[k] : 0;
                    c[i] = k < j1 ? other[k] : 0;
                }
                int first = kNever;
#pragma unroll
                for (int i = U - 1; i >= 0; --i) {
                    const int k = j + 32 * i + lane;
                    if (k < j1 && (a[i] != c[i] || a[i] < 0 || a[i] >= p.num_pages)) first = k;
                }
                first = __reduce_min_sync(0xffffffffu, first);
                if (first != kNever) {
                    same = first;
                    break;
                }
            }
        }
        if (lane == 0) same_at[static_cast<int64_t>(s) * B + b] = same;
    }
    cl.sync();
    if (cl.block_rank() != 0) return;

    // ---- the common tokens of each sequence, and what each run shares: the least of its sequences that
    // have a tile or more in common
    for (int w0 = warp * 32; w0 < B; w0 += kPlanThreads) {
        const int b = w0 + lane;
        int c = -1, h = 0;
        if (b < B) {
            int64_t e = p.max_pages;
            for (int s = 0; s < slices; ++s)
                e = min(e, static_cast<int64_t>(x.same()[static_cast<int64_t>(s) * B + b]));
            c = static_cast<int>(min(e * p.page, static_cast<int64_t>(seen(b))));
            x.common(b) = c;
            h = x.head(b);
        }
        const bool in = c >= kShTile;
        const unsigned who = __ballot_sync(0xffffffffu, in);
        if (!who) continue;
        const int h0 = __shfl_sync(0xffffffffu, h, __ffs(who) - 1);
        if (__all_sync(0xffffffffu, !in || h == h0)) {
            const int least = __reduce_min_sync(0xffffffffu, in ? c : kNever);
            if (lane == 0) {
                atomicMin(&x.first(h0), w0 + __ffs(who) - 1);
                atomicMax(&x.last(h0), w0 + 31 - __clz(who));
                atomicMin(&x.least(h0), least);
            }
        } else if (in) {
            atomicMin(&x.first(h), b);
            atomicMax(&x.last(h), b);
            atomicMin(&x.least(h), c);
        }
    }
    __syncthreads();
    // Common tiles of the run that begins with sequence h: there are two sequences at least.
    auto tiles_of = [&](int h) { return x.first(h) < x.last(h) ? x.least(h) / kShTile : 0; };

    // ---- the shared groups in order, and the units of the sequences' own tokens, by a team of warps
    // each, which meet to divide the SMs
    const int warps = B <= 128 ? 1 : min(kPlanWarps / 2, (B + 63) / 64);
    const PlanTeam groups{0, warps, kBarGroups, s_scan};
    const PlanTeam owns{kPlanWarps / 2, warps, kBarOwn, s_scan + kPlanWarps / 2};
    if (groups.has(warp)) {
        const int step = groups.threads();
        auto group_tiles = [&](int b) { return b < B && x.head(b) == b ? tiles_of(b) : 0; };
        auto cut_of = [&](int b, int tiles, int s, int small_s) {
            return sh_cut((x.last(b) - x.first(b) + 1) * p.rows_per_seq, tiles, s, small_s);
        };
        // Units of the run of sequence b for pieces of s tiles.
        auto units_of = [&](int b, int tiles, int s, int small_s) {
            return static_cast<long long>(p.H_kv) * cut_of(b, tiles, s, small_s).per;
        };
        auto small_of = [&](int s) { return s * p.small_cost / 4; };
        // The work in tiles of a large block (all of it below 2^31: see shares).
        uint32_t work = 0;
        for (int b = groups.thread(); b < B; b += step) {
            const int tiles = group_tiles(b);
            if (tiles == 0) continue;
            const ShCut c = cut_of(b, tiles, 1, 1);
            work += static_cast<uint32_t>(p.H_kv) *
                    static_cast<uint32_t>(c.big * tiles + c.small_units * 4 / p.small_cost);
        }
        work = __reduce_add_sync(0xffffffffu, work);
        if (lane == 0) atomicAdd(&s_work, static_cast<int32_t>(work));
        named_bar_sync(kBarSplit, 2 * step);
        const long long all = s_work;
        int ctas = 0;
        if (warp == 0) {
            ctas = split_sms(p, all, s_own);
            if (warps > 1 && lane == 0) s_ctas = ctas;
        }
        if (warps > 1) {
            groups.sync();
            ctas = s_ctas;
        }
        // Equal shares would end and begin within items, and an item more in a CTA costs it as much
        // as kItemCost tiles.  So the items are cut into pieces, one a CTA, where pieces of no more
        // than that over an equal share are few enough.
        const int equal = max(kShLeast, divide(all + ctas - 1, ctas));
        constexpr long long kMany = 1 << 20;  // (more than CTAs; 512 of them are below 2^31)
        int piece = 1, small_piece = 1;
#pragma unroll 1
        for (int i = 0; i <= kItemCost && piece == 1; ++i) {
            long long n = 0;
#pragma unroll 1
            for (int b = groups.thread(); b < B; b += step) {
                const int tiles = group_tiles(b);
                if (tiles > 0)
                    n = min(n + units_of(b, tiles, equal + i, small_of(equal + i)), kMany);
            }
            uint32_t pieces = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(n));
            if (warps > 1) {
                if (lane == 0) atomicAdd(&s_pieces[i], static_cast<int32_t>(pieces));
                groups.sync();
                pieces = static_cast<uint32_t>(s_pieces[i]);
            }
            if (pieces <= static_cast<uint32_t>(ctas)) piece = equal + i;
        }
        if (piece > 1) small_piece = small_of(piece);
        long long units = 0;  // and, above bit 32, groups
#pragma unroll 1
        for (int b0 = 0; b0 < B; b0 += step) {
            const int b = b0 + groups.thread(), tiles = group_tiles(b);
            const long long mine =
                tiles > 0 ? (1ll << 32) + units_of(b, tiles, piece, small_piece) : 0;
            if (warps == 1 && !__any_sync(0xffffffffu, tiles > 0)) continue;
            const PlanTeam::Scan scan = groups.scan(mine);
            if (tiles > 0) {
                const long long at = units + scan.before;
                ShGroup g{};
                g.unit0 = low32(at);
                g.first = x.first(b);
                g.count = x.last(b) - x.first(b) + 1;
                g.tiles = tiles;
                p.groups[at >> 32] = g;
                x.lead(b) = static_cast<int32_t>(low32(at));
            }
            units += scan.total;
        }
        if (groups.thread() == 0) {
            p.head->units = low32(units);
            p.head->groups = static_cast<int>(units >> 32);
            p.head->share = piece > 1 ? 1 : max(kShLeast, divide(low32(units) + ctas - 1, ctas));
            p.head->piece = piece;
            p.head->small_piece = small_piece;
        }
    } else if (owns.has(warp)) {
        const int step = owns.threads();
        long long own = 0;  // units (below 2^31: see shares), and, above bit 32, items
        for (int b0 = 0; b0 < B; b0 += step) {
            const int b = b0 + owns.thread();
            long long mine = 0;
            if (b < B) {
                const int skip = x.common(b) >= kShTile ? tiles_of(x.head(b)) : 0;
                const int tiles = x.own_tiles(b) - skip * (kShTile / p.own_tile);
                if (tiles > 0) mine = x.own_items(b) * ((1ll << 32) + tiles + kOwnItemUnits);
            }
            const PlanTeam::Scan scan = owns.scan(mine);
            if (b < B) p.seqs[b].own0 = low32(own + scan.before);
            own += scan.total;
        }
        const long long units = low32(own), items = own >> 32;
        const long long ns = (units - items * kOwnItemUnits) * p.own_tile_ns + items * p.own_item_ns;
        if (owns.thread() == 0) s_own = ns;
        named_bar_sync(kBarSplit, 2 * step);
        if (warp == owns.first) {
            const int ctas = split_sms(p, static_cast<long long>(s_work), ns);
            const int beside = (p.ctas - ctas) * p.own_per_sm;
            const int own_ctas = beside > 0 ? min(p.own_ctas, beside) : p.own_ctas;
            if (lane == 0) {
                p.head->own_units = units;
                p.head->own_share = max(1, divide(units + own_ctas - 1, own_ctas));
            }
        }
    }
    __syncthreads();
    for (int b = threadIdx.x; b < B; b += kPlanThreads) {
        const int h = x.head(b), tiles = x.common(b) >= kShTile ? tiles_of(h) : 0;
        ShSeq& s = p.seqs[b];
        s.skip = tiles * kShTile;
        if (tiles > 0) {
            s.unit0 = x.lead(h);
            s.first = x.first(h);
            s.count = x.last(h) - x.first(h) + 1;
        }
    }
}

// ------------------------------------------------------------------------------------------
// prefix
// ------------------------------------------------------------------------------------------
constexpr int kThreads = 512;
constexpr int kExpandWarp = 8;  // warps 8-11
constexpr int kMmaWarp = 12, kLoadWarp = 13;
constexpr int kHalfBytes = 128 * 128;  // 64 columns of a 128-row bf16 tile
constexpr float kMoveThreshold = 8.f, kMoveHeadroom = 24.f;  // log2 units, as in fa_fwd.cu
constexpr uint64_t kDrainNs = 1000000000ull;
constexpr uint32_t kBarTeardown = 1;  // TMEM no longer used: softmax warps and the MMA warp
constexpr uint32_t kTeardownThreads = 288;
constexpr int kMaxSlots = 10, kRaw = 6;

struct Bars {
    uint64_t full[kMaxSlots], empty[kMaxSlots];  // the ring of bf16 tiles
    uint64_t raw_full[kRaw], raw_empty[kRaw];    // 4 bits: the ring of tiles as they are stored
    uint64_t q_full[2];     // group w's queries are in shared memory (4 warps)
    uint64_t s_full[2];     // S of group w's step (tcgen05.commit)
    uint64_t p_full[2][2];  // a half of P stored, O rescaled if needed (4 warps)
    uint64_t o_full[2];     // the last P V of group w's item (tcgen05.commit)
    uint64_t done;       // every product of the CTA
    uint32_t tmem_base;
};

template <int D, int FMT>
struct Cfg {
    static constexpr bool kInt4 = FMT == OSM_KV_INT4;
    static constexpr int kHalves = D / 64;
    static constexpr int kTileBytes = kHalves * kHalfBytes;
    static constexpr int kG = D / kKvGroup;
    static constexpr int kRawRow = D / 2;                         // codes of a token
    static constexpr int kRawCodes = kShTile * kRawRow;
    static constexpr int kRawBytes = kRawCodes + kShTile * kG * 2;  // and the tokens' words
    // The ring: what the queries (two tiles) and the raw tiles leave.
    static constexpr int kSlots = sh_slots(D, kInt4);
    static constexpr int kQ = 0;
    static constexpr int kRing = kQ + 2 * kTileBytes;
    static constexpr int kRawAt = kRing + kSlots * kTileBytes;
    static constexpr int kBars = kRawAt + (kInt4 ? kRaw * kRawBytes : 0);
    static constexpr int kBytes = kBars + static_cast<int>(sizeof(Bars));
    static constexpr int kDyn = kBytes + 1024;  // slack for 1024-byte alignment
    static_assert(kDyn <= 227 * 1024, "shared memory budget");
    // Held at once: a K and a V of each group (tiles in turn), less the K whose product is done.
    static_assert(kSlots >= 3, "the ring holds what the products wait for together");
    static constexpr uint32_t kTmemO = 256;
    static_assert(kTmemO + 2 * D <= 512, "TMEM budget");
};
constexpr int kSoftRegs = 200, kExpandRegs = 72, kMmaRegs = 40;
static_assert(256 * kSoftRegs + 128 * kExpandRegs + 128 * kMmaRegs <= 65536, "register split");

struct PrefixParams {
    const __nv_bfloat16* Q;  // [B, H, Nq, D]
    KvPages pg;
    ShView v;
    int H, Nq, group;  // group: H / H_kv
    int64_t q_bytes;
    int box;               // tokens of a copy: they lie in one page
    uint32_t page_inv;     // 2^32 / (page / 16), rounded up; 0 for pages of 16
    uint32_t page_bytes;   // all heads of a page
    float scale_log2;
    unsigned long long timeout_ns;
};

// Page of a token: token / 16 is below 2^26 and page / 16 at most 64, so the product with the rounded
// inverse is off by less than 1 / 64 of a page's part of 2^32, and the quotient is exact.
__device__ __forceinline__ int page_of(const PrefixParams& p, int tok) {
    const uint32_t x = static_cast<uint32_t>(tok) >> 4;
    return static_cast<int>(p.page_inv ? __umulhi(x, p.page_inv) : x);
}

// A CTA's walk through the items of its share: tiles [t0, t1) of (group g, key/value head, block).
struct Walk {
    int j, first, tiles, group_rows;  // the group, its first sequence, tiles and rows
    int kvh, block, t0, t1;
    int left;  // units
    int piece, small_piece;

    __device__ __forceinline__ void load(const ShView& v) {
        const int2 seqs = __ldcg(reinterpret_cast<const int2*>(&v.groups[j].first));
        first = seqs.x;
        tiles = __ldcg(&v.groups[j].tiles);
        group_rows = seqs.y * v.rows_per_seq;
    }
    __device__ __forceinline__ void cut(int from) {  // from the item's unit `from` on
        const int size = halves() ? piece : small_piece, n = min(sh_units(tiles, size) - from, left);
        t0 = from * size;
        t1 = min(tiles, (from + n) * size);
        left -= n;
    }
    // (a whole warp: the first 32 groups are read, a lane each, beside the head, so that the walk starts
    // one read behind the plan)
    __device__ __forceinline__ void start(const ShView& v) {
        const int lane = threadIdx.x & 31;
        const ShGroup& mine = v.groups[min(lane, v.B - 1)];
        const long long at = __ldcg(&mine.unit0);
        const int2 seqs = __ldcg(reinterpret_cast<const int2*>(&mine.first));
        const int mine_tiles = __ldcg(&mine.tiles);
        const int n = __ldcg(&v.head->groups);
        const long long units = __ldcg(&v.head->units), share = __ldcg(&v.head->share);
        piece = __ldcg(&v.head->piece);
        small_piece = __ldcg(&v.head->small_piece);
        const long long u0 = share * blockIdx.x;
        left = static_cast<int>(max(min(units - u0, share), 0ll));
        t0 = t1 = 0;
        if (left == 0) return;
        // the last group with unit0 <= u0
        j = __popc(__ballot_sync(0xffffffffu, lane < n && at <= u0)) - 1;
        long long unit0 = __shfl_sync(0xffffffffu, at, j);
        first = __shfl_sync(0xffffffffu, seqs.x, j);
        group_rows = __shfl_sync(0xffffffffu, seqs.y, j) * v.rows_per_seq;
        tiles = __shfl_sync(0xffffffffu, mine_tiles, j);
        if (j == 31 && n > 32) {
            int hi = n - 1;
            while (j < hi) {
                const int mid = (j + hi + 1) >> 1;
                if (__ldcg(&v.groups[mid].unit0) <= u0) j = mid;
                else hi = mid - 1;
            }
            load(v);
            unit0 = __ldcg(&v.groups[j].unit0);
        }
        const long long r = u0 - unit0;
        const ShCut c = sh_cut(group_rows, tiles, piece, small_piece);
        kvh = divide(r, c.per);
        const int u = static_cast<int>(r - static_cast<long long>(kvh) * c.per);
        block = min(u / c.units, c.big);
        cut(u - block * c.units);
    }
    __device__ __forceinline__ bool done() const { return t1 == 0; }
    __device__ __forceinline__ void next(const ShView& v) {
        t0 = t1 = 0;
        if (left == 0) return;
        if (++block * kShRows >= group_rows) {
            block = 0;
            if (++kvh == v.H_kv) {
                kvh = 0;
                ++j;
                load(v);
            }
        }
        cut(0);
    }
    // Rows of the block; more than 128: each softmax group has its half and sees every tile.
    __device__ __forceinline__ int rows() const {
        return min(kShRows, group_rows - block * kShRows);
    }
    __device__ __forceinline__ bool halves() const { return rows() > kShHalf; }
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t timeout_ns,
                                          bool sleep) {
    const bool ok = mbar_wait(bar, parity, timeout_ns, sleep);
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void warp_arrive_tc(uint64_t* bar) {
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void bar_arrive(uint32_t id, uint32_t count) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const PrefixParams p) {
    using C = Cfg<D, FMT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    Bars* bars = reinterpret_cast<Bars*>(smem + C::kBars);
    const uint32_t ring = smem_u32(smem + C::kRing);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned long long timeout = p.timeout_ns;
    auto give_up = [&](int where) { atomicCAS(p.pg.status, 0, FA_ERR_TIMEOUT | (where << 8)); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(&bars->full[s], C::kInt4 ? 4 : 1);
            mbar_init(&bars->empty[s], 1);
        }
        for (int s = 0; s < kRaw; ++s) {
            mbar_init(&bars->raw_full[s], 1);
            mbar_init(&bars->raw_empty[s], 4);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(&bars->q_full[w], 4);
            mbar_init(&bars->s_full[w], 1);
            for (int b = 0; b < 2; ++b) mbar_init(&bars->p_full[w][b], 4);
            mbar_init(&bars->o_full[w], 1);
        }
        mbar_init(&bars->done, 1);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    // The queries come into the L2, and their addresses into the SM's translation, while the plan is
    // made: the first load from a place that has not been used for a while takes microseconds.
    if (warp < kExpandWarp) {
        const int64_t bytes = p.q_bytes, line = 128;
        for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kExpandWarp * 32 + threadIdx.x) * line;
             i < bytes; i += static_cast<int64_t>(gridDim.x) * kExpandWarp * 32 * line)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const uint8_t*>(p.Q) + i));
        asm volatile("prefetch.global.L1 [%0];" ::"l"(p.Q));
    }
    // It waits for the plan before it lets the kernel over the own tokens start, which then need not
    // (reads of the plan pass the L1 by).
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    Walk walk;
    walk.start(p.v);

    if (warp >= kMmaWarp) {
        setmaxnreg_dec<kMmaRegs>();
        if (warp == kMmaWarp) {
            // -------------------------------------------------------------- the products
            constexpr uint32_t idS = idesc_bf16_f32(kShHalf, kShTile, 0);
            constexpr uint32_t idO = idesc_bf16_f32(kShHalf, D, 1);
            constexpr uint32_t kHalfTile = kShTile / 2 * 128;  // bytes of 64 rows of 64 columns
            int slot = 0;                        // of the next tile
            int k0 = 0, k1 = 0, v0 = 0, v1 = 0;  // of the tile that group 0, 1 works on
            uint32_t phase = 0, q_phase = 0, p_phase = 0;  // a bit each group
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity, int where) {
                const bool good = issuer_wait<true>(bar, parity, timeout, true);
                if (!good && lane == 0) give_up(where);
                return good;
            };
            for (; ok && !walk.done(); walk.next(p.v)) {
                const bool halves = walk.halves();
                const int n = walk.t1 - walk.t0;
                ok = for_steps(n, halves, [&](auto x, int u, int, bool first, bool last) {
                    constexpr int w = decltype(x)::w;
                    constexpr bool pv = decltype(x)::pv;
                    int& at = pv ? (w ? v1 : v0) : (w ? k1 : k0);
                    const uint32_t tS = tmem + w * 128;
                    if constexpr (!pv) {
                        if (u == 0) {
                            if (!wait(&bars->q_full[w], q_phase >> w & 1, 30)) return false;
                            q_phase ^= 1u << w;
                        }
                    } else {
                        if (!wait(&bars->p_full[w][0], p_phase >> w & 1, 31)) return false;
                    }
                    if (first) {
                        if (!wait(&bars->full[slot], phase, 32)) return false;
                        at = slot;
                        if (halves) (pv ? v1 : k1) = slot;
                        if (++slot == C::kSlots) slot = 0, phase ^= 1;
                    }
                    tc_fence_after();
                    const uint32_t tile = ring + at * C::kTileBytes;
                    if constexpr (!pv) {
                        const uint32_t q = smem_u32(smem + C::kQ) + w * C::kTileBytes;
#pragma unroll
                        for (int h = 0; h < C::kHalves; ++h)
                            issue_ss_x4<true>(tS, smem_desc_sw128(q + h * kHalfBytes, 16, 1024),
                                              smem_desc_sw128(tile + h * kHalfBytes, 16, 1024), idS,
                                              h > 0 ? 1u : 0u);
                        issue_commit<true>(&bars->s_full[w]);
                    } else {
                        const uint32_t tO = tmem + C::kTmemO + w * D;
                        issue_ts_x4<true>(tO, tS, smem_desc_sw128(tile, kHalfBytes, 1024),
                                          2048 / 16, idO, u > 0 ? 1u : 0u);
                        if (!wait(&bars->p_full[w][1], p_phase >> w & 1, 31)) return false;
                        p_phase ^= 1u << w;
                        tc_fence_after();
                        issue_ts_x4<true>(tO, tS + 32,
                                          smem_desc_sw128(tile + kHalfTile, kHalfBytes, 1024),
                                          2048 / 16, idO, 1u);
                        if (u + 1 == steps_of(n, halves, w)) issue_commit<true>(&bars->o_full[w]);
                    }
                    if (last) issue_commit<true>(&bars->empty[at]);
                    return true;
                });
            }
            issue_commit<true>(&bars->done);
            issuer_wait<true>(&bars->done, 0, timeout > kDrainNs ? timeout : kDrainNs, true);
            __syncwarp();
            named_bar_sync(kBarTeardown, kTeardownThreads);
            tc_fence_after();
            tmem_dealloc(tmem, 512);
        } else if (warp == kLoadWarp) {
            // -------------------------------------------------------------- tiles from memory
            // A lane copies the tokens that lie in one page: bf16: a TMA box of one half of the
            // columns, into the ring; 4 bits: the codes, or the words, as they are, into the raw ring.
            constexpr int kStages = C::kInt4 ? kRaw : C::kSlots;
            uint64_t* full = C::kInt4 ? bars->raw_full : bars->full;
            uint64_t* empty = C::kInt4 ? bars->raw_empty : bars->empty;
            if (!C::kInt4 && lane == 0) {
                tma_prefetch_desc(&tmK);
                tma_prefetch_desc(&tmV);
            }
            const int boxes = kShTile / p.box;  // of a tile, for each half, or codes and words
            const int box = lane % boxes, half = lane / boxes;
            const bool mine = half < (C::kInt4 ? 2 : C::kHalves);
            int stage = 0, entry = 0;
            uint32_t phase = 1;
            bool ok = true;
            for (; ok && !walk.done(); walk.next(p.v)) {
                // The box's page and place in it for tiles base, base + 1 and base + 2: a tile's
                // serve its keys and its values, and the table is read two tiles ahead.
                const int32_t* row = p.pg.table + walk.first * p.pg.max_pages;
                int base = walk.t0, id[3], place[3];
                auto look = [&](int tile, int& i, int& at) {
                    const int tok = tile * kShTile + box * p.box, e = page_of(p, tok);
                    at = tok - e * p.pg.page;
                    i = mine && tile < walk.t1 ? row[e] : 0;
                };
#pragma unroll
                for (int x = 0; x < 3; ++x) look(base + x, id[x], place[x]);
                // The first values' addresses come into the translation while the keys do: the copies
                // themselves wait for one another there.
                if (mine) {
                    const int64_t at = static_cast<int64_t>(id[0]) * p.page_bytes +
                                       walk.kvh * p.pg.head_bytes;
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.pg.v + at));
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.pg.k + at));
                }
                ok = for_steps(walk.t1 - walk.t0, walk.halves(),
                               [&](auto x, int, int t, bool first, bool) {
                    if (!first) return true;
                    if (!warp_wait(&empty[stage], phase, timeout, true)) {
                        if (lane == 0) give_up(33);
                        return false;
                    }
                    if (lane == 0)
                        mbar_arrive_expect_tx(&full[stage],
                                              C::kInt4 ? C::kRawBytes : C::kTileBytes);
                    __syncwarp();
                    const int tile = walk.t0 + t;
                    if (tile > base + 1) {
                        id[0] = id[1], place[0] = place[1];
                        id[1] = id[2], place[1] = place[2];
                        ++base;
                        look(base + 2, id[2], place[2]);
                    }
                    const int page = tile > base ? id[1] : id[0];
                    const int at = tile > base ? place[1] : place[0];
                    if (mine) {
                        if constexpr (C::kInt4) {
                            const int per = half ? C::kG * 2 : C::kRawRow;  // bytes of a token
                            const uint8_t* src =
                                (decltype(x)::pv ? p.pg.v : p.pg.k) +
                                static_cast<uint64_t>(static_cast<uint32_t>(page)) * p.page_bytes +
                                static_cast<int64_t>(walk.kvh) * p.pg.head_bytes +
                                (half ? p.pg.page * C::kRawRow : 0) + at * per;
                            bulk_load(smem + C::kRawAt + stage * C::kRawBytes +
                                          (half ? C::kRawCodes : 0) + box * p.box * per,
                                      src, static_cast<uint32_t>(p.box * per), &full[stage]);
                        } else {
                            tma_load_4d(smem + C::kRing + stage * C::kTileBytes +
                                            half * kHalfBytes + box * p.box * 128,
                                        decltype(x)::pv ? &tmV : &tmK, &full[stage], half * 64, at,
                                        walk.kvh, page);
                        }
                    }
                    ++entry;
                    if (++stage == kStages) stage = 0, phase ^= 1;
                    return true;
                });
            }
            // what is on its way lands before the CTA ends
            const uint64_t drain = timeout > kDrainNs ? timeout : kDrainNs;
            for (int s = 0; s < kStages && s < entry; ++s) {
                const int last = s + (entry - 1 - s) / kStages * kStages;
                mbar_wait(&full[s], (last / kStages) & 1, drain, true);
            }
        }
    } else if (warp >= kExpandWarp) {
        setmaxnreg_dec<kExpandRegs>();
        if constexpr (C::kInt4) {
            // ------------------------------------------------------------ codes to bf16
            // Tile after tile (keys or values) from the raw ring into the ring, 16 bytes of codes a
            // lane at a time.
            constexpr int kChunks = C::kRawRow / 16, kRowsPer = 128 / kChunks;
            constexpr int kPasses = kShTile / kRowsPer;
            const int tid = threadIdx.x - kExpandWarp * 32;
            const int c = tid % kChunks, r0 = tid / kChunks;
            const uint32_t raw = smem_u32(smem + C::kRawAt);
            int slot = 0, stage = 0;
            uint32_t slot_phase = 1, stage_phase = 0;
            bool ok = true;
            for (; ok && !walk.done(); walk.next(p.v)) {
                for (int left = 2 * (walk.t1 - walk.t0); left > 0; --left) {
                    if (!warp_wait(&bars->raw_full[stage], stage_phase, timeout, true) ||
                        !warp_wait(&bars->empty[slot], slot_phase, timeout, true)) {
                        if (lane == 0) give_up(34);
                        ok = false;
                        break;
                    }
                    const uint32_t src = raw + stage * C::kRawBytes;
                    uint8_t* dst = smem + C::kRing + slot * C::kTileBytes + (c >> 1) * kHalfBytes;
                    uint32_t w[kPasses][4];
                    uint16_t word[kPasses];
#pragma unroll
                    for (int i = 0; i < kPasses; ++i) {
                        const int r = i * kRowsPer + r0;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                                     : "r"(src + r * C::kRawRow + c * 16)
                                     : "memory");
                        asm volatile("ld.shared.b16 %0, [%1];"
                                     : "=h"(word[i])
                                     : "r"(src + C::kRawCodes + (r * C::kG + c / 2) * 2)
                                     : "memory");
                    }
#pragma unroll
                    for (int i = 0; i < kPasses; ++i) {
                        const int r = i * kRowsPer + r0;
                        // step and base - 128 as pairs of bf16; both exact
                        const uint32_t s1 = (word[i] & 0xffc0u) >> 1;
                        const uint32_t step = s1 | s1 << 16;
                        const float base = static_cast<float>(kv4_word_base(word[i]) - 128);
                        const uint32_t shift = pack_bf16x2(base, base);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            // (the lanes of the second half in another order: no bank conflicts)
                            const uint32_t x = c & 2 ? w[i][j ^ 2] : w[i][j];
                            const int ch = (c & 1) * 4 + (j ^ (c & 2));
                            uint32_t y[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                y[k] = mul_bf16x2(
                                    add_bf16x2((x >> (4 * k) & 0x000f000fu) | 0x43004300u, shift),
                                    step);
                            *reinterpret_cast<uint4*>(dst + r * 128 + ((ch ^ (r & 7)) << 4)) =
                                make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bars->full[slot]);
                        mbar_arrive(&bars->raw_empty[stage]);
                    }
                    if (++slot == C::kSlots) slot = 0, slot_phase ^= 1;
                    if (++stage == kRaw) stage = 0, stage_phase ^= 1;
                }
            }
        }
    } else {
        setmaxnreg_inc<kSoftRegs>();
        // ------------------------------------------------------------------ softmax
        const int w = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lane_at = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_at + w * 128, tO = tmem + lane_at + C::kTmemO + w * D;
        uint8_t* sQ = smem + C::kQ + w * C::kTileBytes;
        const float scale = p.scale_log2;
        uint32_t s_phase = 0, o_phase = 0;
        bool ok = true;
        for (; ok && !walk.done(); walk.next(p.v)) {
            const int n = walk.t1 - walk.t0, rows = walk.rows();
            const bool halves = rows > kShHalf;
            const int steps = steps_of(n, halves, w);
            const int row = (halves ? w * kShHalf : 0) + r;  // of the block
            const int warp_row0 = row - lane;
            const bool real = row < rows;
            int64_t at = 0;  // the row's place in Q, O and LSE
            if (real) {
                const int R = walk.block * kShRows + row;
                const int b = R / p.v.rows_per_seq, x = R - b * p.v.rows_per_seq;
                const int i = x / p.group, h = walk.kvh * p.group + x - i * p.group;
                at = (static_cast<int64_t>(walk.first + b) * p.H + h) * p.Nq + i;
            }
            float m = -INFINITY, l = 0.f;
            if (steps > 0) {
                // The warp's 32 rows, whole rows at a time (a row a lane would touch 32 lines with
                // every load); the products with the last item's queries have been waited for.
                constexpr int kLanes = D / 8, kRowsAt = 32 / kLanes;  // lanes a row, rows at a time
                const int c = lane % kLanes;
                const uint4* q = reinterpret_cast<const uint4*>(p.Q) + c;
                uint4 x[kLanes];
#pragma unroll
                for (int i = 0; i < kLanes; ++i) {
                    const int src = i * kRowsAt + lane / kLanes;
                    const int64_t from = __shfl_sync(0xffffffffu, at, src);
                    x[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (warp_row0 + src < rows) x[i] = q[from * kLanes];
                }
#pragma unroll
                for (int i = 0; i < kLanes; ++i) {
                    const int rr = (warp & 3) * 32 + i * kRowsAt + lane / kLanes;
                    uint4 y = x[i];
                    if constexpr (C::kInt4) {  // values k and k + 4 side by side
                        y.x = __byte_perm(x[i].x, x[i].z, 0x5410);
                        y.y = __byte_perm(x[i].x, x[i].z, 0x7632);
                        y.z = __byte_perm(x[i].y, x[i].w, 0x5410);
                        y.w = __byte_perm(x[i].y, x[i].w, 0x7632);
                    }
                    *reinterpret_cast<uint4*>(sQ + (c >> 3) * kHalfBytes + rr * 128 +
                                              (((c & 7) ^ (rr & 7)) << 4)) = y;
                }
                fence_proxy_async_smem();
                warp_arrive_tc(&bars->q_full[w]);
            }
            for (int u = 0; u < steps; ++u) {
                if (!warp_wait(&bars->s_full[w], s_phase, timeout, true)) {
                    if (lane == 0) give_up(35);
                    ok = false;
                    break;
                }
                s_phase ^= 1;
                tc_fence_after();
                uint32_t sr[128];
                tmem_ld128_sync(tS, sr);
                float top[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) top[e] = __uint_as_float(sr[e]);
#pragma unroll
                for (int e = 16; e < 128; ++e)
                    top[e & 15] = fmaxf(top[e & 15], __uint_as_float(sr[e]));
#pragma unroll
                for (int x = 8; x >= 1; x >>= 1)
#pragma unroll
                    for (int e = 0; e < x; ++e) top[e] = fmaxf(top[e], top[e + x]);
                const float mx = top[0] * scale;
                const float m_new = mx - m > kMoveThreshold ? mx + kMoveHeadroom : m;
                const float alpha = m_new == m ? 1.f : ex2_approx(m - m_new);
                const float ref = m_new == -INFINITY ? 0.f : m_new;
                m = m_new;
                // O holds P V of the steps before: S of this one was committed after them
                if (u > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t o[16];
                        tmem_ld16_sync(tO + c * 16, o);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        uint32_t a[8], b[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) a[e] = o[e], b[e] = o[e + 8];
                        tmem_st8x2_sync(tO + c * 16, a, tO + c * 16 + 8, b);
                    }
                }
                float2 sum = make_float2(0.f, 0.f), sum2 = make_float2(0.f, 0.f);
                const float2 c2 = make_float2(scale, scale), n2 = make_float2(-ref, -ref);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pr[32];
#pragma unroll
                    for (int e = 0; e < 64; e += 4) {
                        const uint32_t* x = sr + 64 * h + e;
                        float2 x0 = ffma2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])),
                                          c2, n2);
                        float2 x1 = ffma2(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])),
                                          c2, n2);
                        x0.x = ex2_approx(x0.x);
                        x0.y = ex2_approx(x0.y);
                        x1.x = ex2_approx(x1.x);
                        x1.y = ex2_approx(x1.y);
                        sum = fadd2(sum, x0);
                        sum2 = fadd2(sum2, x1);
                        pr[e >> 1] = pack_bf16x2(x0.x, x0.y);
                        pr[(e >> 1) + 1] = pack_bf16x2(x1.x, x1.y);
                    }
                    tmem_st32_sync(tS + 32 * h, pr);
                    warp_arrive_tc(&bars->p_full[w][h]);
                }
                l = l * alpha + ((sum.x + sum.y) + (sum2.x + sum2.y));
            }
            if (ok && steps > 0) {
                if (!warp_wait(&bars->o_full[w], o_phase, timeout, true)) {
                    if (lane == 0) give_up(36);
                    ok = false;
                }
                o_phase ^= 1;
                tc_fence_after();
            }
            if (!ok) break;
            // ---------------------------------------------------------- the row's state
            const bool whole = walk.t0 == 0 && walk.t1 == walk.tiles;
            const int64_t place =
                whole ? 2 * at + (halves ? 0 : w)
                      : ((static_cast<int64_t>(blockIdx.x) * 2 + (walk.t0 == 0 ? 1 : 0)) * 2 + w) *
                                kShHalf + r;
            float* dst = whole ? p.v.row_o : p.v.edge_o;
            if (real) (whole ? p.v.row_ml : p.v.edge_ml)[place] = make_float2(m, l);
            if (steps == 0) continue;
            // 32 columns at a time through the warp's part of the queries' place (their last product
            // is done), so that a store writes whole lines.
            uint8_t* stage = sQ + (warp & 3) * 4096;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32_sync(tO + c * 32, o);
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint4 a, b;
                    if constexpr (C::kInt4) {  // columns 2 k and 2 k + 1 are values k and k + 4
                        a = make_uint4(o[e], o[e + 2], o[e + 4], o[e + 6]);
                        b = make_uint4(o[e + 1], o[e + 3], o[e + 5], o[e + 7]);
                    } else {
                        a = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                        b = make_uint4(o[e + 4], o[e + 5], o[e + 6], o[e + 7]);
                    }
                    *reinterpret_cast<uint4*>(stage + lane * 128 + ((e / 4 ^ (lane & 7)) << 4)) = a;
                    *reinterpret_cast<uint4*>(stage + lane * 128 +
                                              (((e / 4 + 1) ^ (lane & 7)) << 4)) = b;
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int src = 4 * i + lane / 8, ch = lane & 7;
                    const int64_t to = __shfl_sync(0xffffffffu, place, src);
                    const uint4 y = *reinterpret_cast<const uint4*>(stage + src * 128 +
                                                                    ((ch ^ (src & 7)) << 4));
                    if (warp_row0 + src < rows)
                        *reinterpret_cast<uint4*>(dst + to * D + c * 32 + ch * 4) = y;
                }
                __syncwarp();
            }
        }
        tc_fence_before();
        bar_arrive(kBarTeardown, kTeardownThreads);
    }
}

// ------------------------------------------------------------------------------------------
// join
// ------------------------------------------------------------------------------------------
struct JoinParams {
    __nv_bfloat16* O;
    float* LSE;
    const int32_t *kv_lens, *q_lens;
    ShView v;
    const float* own_edge;  // [ctas][2]: [rows][D], then m, l of the rows
    const float* own_o;     // [B * H * Nq][D]
    const float2* own_ml;
    int64_t room;
    int B, H, Nq, group, causal;
    int own_rows, own_tile;
};

__device__ __forceinline__ long long join64(int lo, int hi) {
    return static_cast<long long>(static_cast<unsigned long long>(static_cast<uint32_t>(hi)) << 32 |
                                  static_cast<uint32_t>(lo));
}

// W warps a row; the row's states in turn, two-worker merge.
constexpr int kJoinWarps = 8, kJoinCtasPerSm = 4;
template <int D, int W>
__global__ void __launch_bounds__(kJoinWarps * 32, kJoinCtasPerSm) join_kernel(const JoinParams p) {
    constexpr int E = D / 32, R = kJoinWarps / W;
    __shared__ float sM[kJoinWarps], sL[kJoinWarps], sO[kJoinWarps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * R + warp / W;
    const int64_t rows = static_cast<int64_t>(p.B) * p.H * p.Nq;
    float M = -INFINITY, L = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    bool sees = false;
    // Where the row's states are: from the plan, which is done (its reads pass the L1 by),
    // before the wait for the kernels that make them.
    int own_n = 0, pre_n = 0, pw = 1, g0 = 0, pr = 0, w0 = 0, c0 = 0, br = 0;
    bool whole = false, own_whole = false;
    if (at < rows) {
        const int64_t bh = at / p.Nq;
        const int i = static_cast<int>(at - bh * p.Nq);
        const int b = static_cast<int>(bh / p.H);
        const int h = static_cast<int>(bh - static_cast<int64_t>(b) * p.H);
        const int kvh = h / p.group;
        const int row = i * p.group + h - kvh * p.group;  // of the sequence and key/value head
        const int len = static_cast<int>(min(static_cast<int64_t>(max(p.kv_lens[b], 0)), p.room));
        const int ql = p.q_lens ? min(max(p.q_lens[b], 0), p.Nq) : p.Nq;
        const int4* rec = reinterpret_cast<const int4*>(p.v.seqs + b);
        const int4 at0 = __ldcg(rec), at1 = __ldcg(rec + 1);
        const int4* head = reinterpret_cast<const int4*>(p.v.head);
        const int4 h0 = __ldcg(head), h1 = __ldcg(head + 1);
        const long long unit0 = join64(at0.x, at0.y), share = join64(h1.x, h1.y);
        const int skip = at1.x;
        sees = i < ql && (p.causal ? len - ql + i : len - 1) >= 0;
        if (sees) {
            // the sequence's own tokens
            const int tiles = (len + p.own_tile - 1) / p.own_tile - skip / p.own_tile;
            const int blocks = (ql * p.group + p.own_rows - 1) / p.own_rows;
            const int block = row / p.own_rows;
            br = row - block * p.own_rows;
            const long long u = unit0 + kOwnItemUnits + (static_cast<long long>(kvh) * blocks + block) *
                                                         (tiles + kOwnItemUnits);
            c0 = divide(u, share);
            own_n = divide(u + tiles - 1, share) - c0 + 1;
            own_whole = own_n == 1;
            // the common ones
            if (skip > 0) {
                ShGroup g{};
                g.first = at1.y, g.count = at1.z;
                const long long ps = h0.w;
                const ShCut cut = sh_cut(g.count * p.v.rows_per_seq, skip / kShTile, h1.z, h1.w);
                const int RR = (b - g.first) * p.v.rows_per_seq + row;
                const int pb = RR / kShRows, rr = RR - pb * kShRows;
                const bool halves = min(kShRows, g.count * p.v.rows_per_seq - pb * kShRows) > kShHalf;
                const long long pu =
                    join64(at0.z, at0.w) + static_cast<long long>(kvh) * cut.per + pb * cut.units;
                g0 = divide(pu, ps);
                const int mine = pb < cut.big ? cut.units : cut.small_units;
                const int g1 = divide(pu + mine - 1, ps);
                whole = g0 == g1;
                pw = halves ? 1 : 2;
                w0 = halves && !whole ? rr / kShHalf : 0;
                pr = halves ? rr % kShHalf : rr;
                pre_n = (g1 - g0 + 1) * pw;
            }
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // 32 states at a time, a lane's m and l each; kAhead of their O in flight, the first of them beside
    // m and l.  (A state without a tile has m = -inf and l = 0, and its O is not one.)
    constexpr int kAhead = 4;
    const int states = own_n + pre_n;
    for (int k0 = warp % W; k0 < states; k0 += 32 * W) {
        const int k = k0 + lane * W;
        const float* src = p.own_o;
        float mk = -INFINITY, lk = 0.f;
        if (k < own_n && !own_whole) {
            const float* part = p.own_edge + (static_cast<int64_t>(c0 + k) * 2 + (k == 0 ? 1 : 0)) *
                                                 (p.own_rows * (D + 2));
            mk = part[p.own_rows * D + br];
            lk = part[p.own_rows * (D + 1) + br];
            src = part + br * D;
        } else if (k < states) {
            const int y = k - own_n, c = y / pw, w = y - c * pw + w0;
            const int64_t place =
                k < own_n ? at
                : whole   ? 2 * at + w
                          : ((static_cast<int64_t>(g0 + c) * 2 + (c == 0 ? 1 : 0)) * 2 + w) * kShHalf +
                                pr;
            const float2 ml = (k < own_n ? p.own_ml : whole ? p.v.row_ml : p.v.edge_ml)[place];
            mk = ml.x, lk = ml.y;
            src = (k < own_n ? p.own_o : whole ? p.v.row_o : p.v.edge_o) + place * D;
        }
        const int n = min(32, (states - k0 + W - 1) / W);
        float f = 0.f;
        unsigned some = 0;
        for (int x0 = 0; x0 < n; x0 += kAhead) {
            float v[kAhead][E];
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const float* at_x = reinterpret_cast<const float*>(__shfl_sync(
                    0xffffffffu, reinterpret_cast<unsigned long long>(src), x0 + x));
                if constexpr (E == 4) {
                    const float4 y = reinterpret_cast<const float4*>(at_x)[lane];
                    v[x][0] = y.x, v[x][1] = y.y, v[x][2] = y.z, v[x][3] = y.w;
                } else {
                    const float2 y = reinterpret_cast<const float2*>(at_x)[lane];
                    v[x][0] = y.x, v[x][1] = y.y;
                }
            }
            if (x0 == 0) {
                float mn = mk;
#pragma unroll
                for (int m = 16; m > 0; m >>= 1)
                    mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, m));
                mn = fmaxf(mn, M);
                const float ref = mn == -INFINITY ? 0.f : mn, a = ex2_approx(M - ref);
                M = mn;
                f = ex2_approx(mk - ref);
                L = L * a + lk * f;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] *= a;
                some = __ballot_sync(0xffffffffu, lk != 0.f || mk != -INFINITY);
            }
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const float fx = __shfl_sync(0xffffffffu, f, x0 + x);
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] += some >> (x0 + x) & 1 ? v[x][e] * fx : 0.f;
            }
        }
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) L += __shfl_xor_sync(0xffffffffu, L, m);
    if constexpr (W > 1) {
        if (lane == 0) {
            sM[warp] = M;
            sL[warp] = L;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) sO[warp][E * lane + e] = o[e];
        __syncthreads();
        if (warp % W != 0) return;
        float top = -INFINITY;
#pragma unroll
        for (int x = 0; x < W; ++x) top = fmaxf(top, sM[warp + x]);
        const float ref = top == -INFINITY ? 0.f : top;
        L = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll
        for (int x = 0; x < W; ++x) {
            const float f = ex2_approx(sM[warp + x] - ref);
            L += sL[warp + x] * f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] += sO[warp + x][E * lane + e] * f;
        }
        M = top;
    }
    if (at >= rows) return;
    const bool none = L == 0.f || !sees;
    const float inv = none ? 0.f : 1.f / L;
    if constexpr (E == 4) {
        uint2 y = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
        if (none) y = make_uint2(0u, 0u);
        reinterpret_cast<uint2*>(p.O + at * D)[lane] = y;
    } else {
        reinterpret_cast<uint32_t*>(p.O + at * D)[lane] =
            none ? 0u : pack_bf16x2(o[0] * inv, o[1] * inv);
    }
    if (lane == 0 && p.LSE) p.LSE[at] = none ? -INFINITY : (M + __log2f(L)) * kLn2;
}

// ------------------------------------------------------------------------------------------
// host
// ------------------------------------------------------------------------------------------
int sm_count() {
    const int n = device_sm_count();
    return n > 0 ? n : 152;
}

// Sharing costs two launches more, a plan and the states' way through memory, 8 to 13 us where there
// is nothing to share; what it saves at most are the reads of all sequences' tokens but one's, counted
// in values for each key/value head and block of rows.  fa_fwd_paged reads a 4-bit value faster, and
// has common pages from the L2.  Shared and not, us, sequences x common tokens + up to 200 of their
// own, in 2^20 reads of a head of 128:
//   bf16, 8 heads    8 x 8192 (0.45) 31 and 27; 64 x 1024 (0.59) 34 and 31; 8 x 16384 (0.89) 36 and 42;
//                    64 x 2048 (1.08) 33 and 45; 64 x 4096 (2.1) 39 and 74
//   4 bits, 8 heads  8 x 16384 (0.89) 41 and 37; 32 x 4096 (1.02) 35 and 39; 64 x 2048 (1.08) 37 and 43,
//                    with four queries 52 and 64; 8 x 32768 (1.76) 52 and 61; 64 x 4096 (2.1) 38 and 66,
//                    with four queries 65 and 99
//   4 heads of 64    64 x 4096 (0.52) bf16 29 and 27, 4 bits 29 and 29; 64 x 8192 (1.01) 31 and 43, 33
//                    and 46
// The tokens are what the table has room for: lengths are not known here.  Short rows in a table of 32768
// tokens, 8 heads of 128, shared and fa_fwd_paged:
//   64 x 1024 + up to 200   bf16 34 and 31, with nothing in common 65 and 54; 4 bits 33 and 31, 43 and 31
//   8 x 8192 + up to 200    bf16 31 and 27, 60 and 49; 4 bits 37 and 25, 37 and 25
//   64 x 100 + up to 20     bf16 25 and 17, 4 bits 27 and 15
constexpr int64_t kWorthBf16 = 7 << 24, kWorthInt4 = 10 << 24;

bool shares(int64_t B, int64_t H, int64_t H_kv, int64_t Nq, int64_t d, int format, int64_t page,
            int64_t max_pages, int64_t own_rows) {
    const int64_t rows = H / H_kv * Nq, blocks = (rows + own_rows - 1) / own_rows;
    if (fa_paged_takes_chunks(rows)) return false;
    const double tokens = static_cast<double>(max_pages * page), heads = static_cast<double>(H_kv);
    // (units of both kernels, of 16 tokens or more, are counted in 32 bits)
    const double units = static_cast<double>(B * blocks) * heads *
                         (tokens / 16 + 1 + kOwnItemUnits);
    return static_cast<double>((B - 1) * blocks) * tokens * heads * static_cast<double>(d) >=
               static_cast<double>(format == OSM_KV_INT4 ? kWorthInt4 : kWorthBf16) &&
           units < 2147483648.;
}

struct Workspace {
    int64_t lists, head, groups, seqs, edge_o, edge_ml, row_o, row_ml, own_edge, own_o, own_ml, bytes;
    int ctas;
    PagedOwn own;
};

Workspace workspace(int64_t B, int64_t H, int64_t H_kv, int64_t Nq, int64_t d, int format,
                    int64_t page, int64_t max_pages) {
    Workspace w{};
    auto part = [&](int64_t n) {
        const int64_t at = (w.bytes + 255) & ~int64_t(255);
        w.bytes = at + n;
        return at;
    };
    const int64_t rows = B * H * Nq;
    w.own = fa_paged_own(B, H, H_kv, Nq, d, format, page, max_pages);
    w.ctas = sm_count();
    w.lists = part(kPlanLists * B * 4);
    w.head = part(sizeof(ShHead));
    w.groups = part(B * static_cast<int64_t>(sizeof(ShGroup)));
    w.seqs = part(B * static_cast<int64_t>(sizeof(ShSeq)));
    w.edge_o = part(static_cast<int64_t>(w.ctas) * 4 * kShHalf * d * 4);
    w.edge_ml = part(static_cast<int64_t>(w.ctas) * 4 * kShHalf * 8);
    w.row_o = part(rows * 2 * d * 4);
    w.row_ml = part(rows * 2 * 8);
    w.own_edge = part(w.own.edge_bytes);
    w.own_o = part(rows * d * 4);
    w.own_ml = part(rows * 8);
    return w;
}

cudaLaunchConfig_t config(unsigned grid, int threads, int smem, cudaStream_t stream,
                          cudaLaunchAttribute* at) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    at->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at->val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cfg;
}

template <int D, int FMT>
int launch_prefix(const CUtensorMap& tk, const CUtensorMap& tv, const PrefixParams& p,
                  cudaStream_t stream) {
    using C = Cfg<D, FMT>;
    static PerDevice<bool> ready;
    if (!ready.get([](int) {
            return cudaFuncSetAttribute(prefix_kernel<D, FMT>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        C::kDyn) == cudaSuccess;
        }))
        return FA_ERR_CUDA;
    cudaLaunchAttribute at{};
    const cudaLaunchConfig_t cfg =
        config(static_cast<unsigned>(p.v.ctas), kThreads, C::kDyn, stream, &at);
    return cudaLaunchKernelEx(&cfg, prefix_kernel<D, FMT>, tk, tv, p) == cudaSuccess ? FA_OK
                                                                                     : FA_ERR_CUDA;
}

template <int D, int W>
int launch_join_w(const JoinParams& p, cudaStream_t stream) {
    const int64_t rows = static_cast<int64_t>(p.B) * p.H * p.Nq;
    constexpr int R = kJoinWarps / W;
    cudaLaunchAttribute at{};
    const cudaLaunchConfig_t cfg =
        config(static_cast<unsigned>((rows + R - 1) / R), kJoinWarps * 32, 0, stream, &at);
    return cudaLaunchKernelEx(&cfg, join_kernel<D, W>, p) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D>
int launch_join(const JoinParams& p, cudaStream_t stream) {
    const int64_t rows = static_cast<int64_t>(p.B) * p.H * p.Nq;
    // As many warps a row as are on the SMs at once: a second wave costs more than a warp's further
    // states (32 sequences of 32768 + 512 tokens with 3 queries, 32 heads: 112 us with one warp a row,
    // 116 with two in two waves).
    const int64_t warps = kJoinCtasPerSm * kJoinWarps * static_cast<int64_t>(sm_count());
    return 8 * rows <= warps   ? launch_join_w<D, 8>(p, stream)
           : 4 * rows <= warps ? launch_join_w<D, 4>(p, stream)
           : 2 * rows <= warps ? launch_join_w<D, 2>(p, stream)
                               : launch_join_w<D, 1>(p, stream);
}

}  // namespace

int64_t fa_shared_ws_bytes(int64_t B, int64_t H, int64_t H_kv, int64_t Nq, int64_t d, int format,
                           int64_t page, int64_t max_pages) {
    const int64_t need = fa_paged_ws_bytes(B, H, H_kv, Nq, d, format, page, max_pages);
    const PagedOwn own = fa_paged_own(B, H, H_kv, Nq, d, format, page, max_pages);
    if (need < 0 || !shares(B, H, H_kv, Nq, d, format, page, max_pages, own.rows)) return need;
    return workspace(B, H, H_kv, Nq, d, format, page, max_pages).bytes;
}

int fa_shared_launch(const void* Q, void* O, float* LSE, const KvPages& pg, const int32_t* kv_lens,
                     const int32_t* q_lens, const int32_t* groups, int64_t B, int64_t H, int64_t Nq,
                     int64_t d, float scale, bool causal, void* ws, cudaStream_t stream) {
    const int64_t rows = H / pg.H_kv * Nq;
    const PagedOwn own = fa_paged_own(B, H, pg.H_kv, Nq, d, pg.format, pg.page, pg.max_pages);
    if (!shares(B, H, pg.H_kv, Nq, d, pg.format, pg.page, pg.max_pages, own.rows) || pg.num_pages == 0)
        return fa_paged_launch(Q, O, LSE, pg, kv_lens, q_lens, B, H, Nq, d, scale, causal, ws,
                               stream);
    const Workspace w = workspace(B, H, pg.H_kv, Nq, d, pg.format, pg.page, pg.max_pages);
    uint8_t* base = static_cast<uint8_t*>(ws);
    PlanParams pl{};
    pl.table = pg.table;
    pl.kv_lens = kv_lens;
    pl.q_lens = q_lens;
    pl.gid = groups;
    pl.num_pages = pg.num_pages;
    pl.max_pages = pg.max_pages;
    pl.page = pg.page;
    pl.B = static_cast<int>(B);
    pl.Nq = static_cast<int>(Nq);
    pl.causal = causal ? 1 : 0;
    pl.rows_per_seq = static_cast<int>(rows);
    pl.H_kv = pg.H_kv;
    pl.own_rows = w.own.rows;
    pl.own_tile = w.own.tile;
    pl.own_ctas = w.own.ctas;
    pl.ctas = w.ctas;
    pl.own_per_sm = w.own.per_sm;
    // The prefix kernel's steady rates; for the own tokens, a CTA's time a tile with half of the SMs at
    // the memory, and an item's: with 2 tiles an item 4.8 us (4 bits 5.7).  Of 60 to 350 ns and 2 to 8 us
    // these are best over the cases above; too little for the own tokens costs most (4 bits, 3 queries:
    // 130 us with 3 us an item).
    pl.tile_ns = pg.format == OSM_KV_INT4 ? (d == 128 ? 2000 : 1500) : (d == 128 ? 1700 : 1400);
    pl.own_tile_ns = 150;
    pl.own_item_ns = 4500;
    // A tile of a block of up to 128 rows beside one of 256 (d = 128): in bf16, where the memory bounds
    // both, 1.6 us and 1.7; in 4 bits 1.1 and 2.0.
    pl.small_cost = pg.format == OSM_KV_INT4 ? 7 : 4;
    pl.group = static_cast<int>(H / pg.H_kv);
    pl.lists = reinterpret_cast<int32_t*>(base + w.lists);
    pl.head = reinterpret_cast<ShHead*>(base + w.head);
    pl.groups = reinterpret_cast<ShGroup*>(base + w.groups);
    pl.seqs = reinterpret_cast<ShSeq*>(base + w.seqs);

    ShView v{};
    v.head = pl.head;
    v.groups = pl.groups;
    v.seqs = pl.seqs;
    v.edge_o = reinterpret_cast<float*>(base + w.edge_o);
    v.edge_ml = reinterpret_cast<float2*>(base + w.edge_ml);
    v.row_o = reinterpret_cast<float*>(base + w.row_o);
    v.row_ml = reinterpret_cast<float2*>(base + w.row_ml);
    v.ctas = w.ctas;
    v.B = static_cast<int>(B);
    v.rows_per_seq = static_cast<int>(rows);
    v.H_kv = pg.H_kv;

    shared_plan_kernel<<<kPlanCtas, kPlanThreads, 0, stream>>>(pl);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;

    PrefixParams pp{};
    pp.Q = static_cast<const __nv_bfloat16*>(Q);
    pp.pg = pg;
    pp.v = v;
    pp.H = static_cast<int>(H);
    pp.Nq = static_cast<int>(Nq);
    pp.group = pl.group;
    pp.page_inv = static_cast<uint32_t>(((int64_t(1) << 32) + pg.page / 16 - 1) / (pg.page / 16));
    pp.page_bytes = static_cast<uint32_t>(pg.head_bytes * pg.H_kv);
    pp.scale_log2 = scale * kLog2e;
    pp.timeout_ns = fa_wait_timeout_ns();
    pp.q_bytes = B * H * Nq * d * 2;
    // the tokens of a copy: the most that divide both a tile and a page
    pp.box = 16;
    while (pp.box < kShTile && pg.page % (2 * pp.box) == 0) pp.box *= 2;
    CUtensorMap tk{}, tv{};
    if (pg.format == OSM_KV_BF16) {
        for (int i = 0; i < 2; ++i) {
            const int st = make_pages_tensor_map(i ? &tv : &tk, i ? pg.v : pg.k, pg.num_pages, pg.H_kv,
                                                 pg.page, d, pp.box);
            if (st != FA_OK) return st;
        }
    }
    JoinParams j{};
    j.own_o = reinterpret_cast<const float*>(base + w.own_o);
    j.own_ml = reinterpret_cast<const float2*>(base + w.own_ml);
    int st = pg.format == OSM_KV_INT4 ? (d == 64 ? launch_prefix<64, OSM_KV_INT4>(tk, tv, pp, stream)
                                                 : launch_prefix<128, OSM_KV_INT4>(tk, tv, pp, stream))
                                      : (d == 64 ? launch_prefix<64, OSM_KV_BF16>(tk, tv, pp, stream)
                                                 : launch_prefix<128, OSM_KV_BF16>(tk, tv, pp, stream));
    if (st != FA_OK) return st;
    st = fa_paged_own_launch(Q, pg, kv_lens, q_lens, B, H, Nq, d, scale, causal, w.own,
                             base + w.own_edge, v.seqs, v.head,
                             reinterpret_cast<float*>(base + w.own_o),
                             reinterpret_cast<float2*>(base + w.own_ml), stream);
    if (st != FA_OK) return st;

    j.O = static_cast<__nv_bfloat16*>(O);
    j.LSE = LSE;
    j.kv_lens = kv_lens;
    j.q_lens = q_lens;
    j.v = v;
    j.own_edge = reinterpret_cast<const float*>(base + w.own_edge);
    j.room = pg.max_pages * pg.page;
    j.B = static_cast<int>(B);
    j.H = static_cast<int>(H);
    j.Nq = static_cast<int>(Nq);
    j.group = pl.group;
    j.causal = pl.causal;
    j.own_rows = w.own.rows;
    j.own_tile = w.own.tile;
    return d == 64 ? launch_join<64>(j, stream) : launch_join<128>(j, stream);
}

}  // namespace osm
