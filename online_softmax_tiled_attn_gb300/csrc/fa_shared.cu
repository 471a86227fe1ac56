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
//   own     the tokens behind them, a sequence at a time: paged_kernel (fa_paged.cu).  It shares no
//           data with the prefix kernel, so its CTAs take the SMs that the prefix kernel leaves.
//   join    merges each row's states and writes O and LSE.
//
// Prefix kernel.  With m sequences of r query rows on a key/value head, each byte of the prefix meets
// m r rows instead of r, so that what bounds the work goes from memory to the tensor cores as m r
// grows: a tile of 128 tokens is 64 KB in bf16 (d = 128), about 2800 clocks of an SM's part of the
// memory, and 1024 clocks of products for 256 rows.  Hence blocks of 256 rows, two softmax groups of
// 128, so that one's exponentials run beside the other's products; with fewer rows the two groups
// take the tiles in turn.  A persistent CTA an SM takes an equal share of all tiles:
//   warps 0-3, 4-7  softmax group w, a row a thread: S from TMEM, the lazy running max of fa_fwd.cu,
//           exponentials, P in bf16 over S's own columns, O rescaled in TMEM when the max moves; at
//           an item's end O and (m, l) go to the workspace.  They load their rows' queries too.
//   warps 8-11      the ring of key and value tiles, in the order of their use.  bf16: one warp, TMA
//           boxes of the tokens that lie in one page, a box a lane.  4 bits: each lane copies
//           16 bytes of codes at a time into a ring of its own (asynchronously, three tiles
//           ahead), expands them to bf16 and stores them swizzled as a TMA load would.
//   warp 12         tcgen05.mma.  Steps s = (group, tile): S(0) S(1), then P V(s), S(s + 2) in turn:
//           P(s) lies in the columns of S(s), so S(s + 2) follows P V(s); and the commit of
//           S(s + 2) says that P V(s) is done, so that O may be rescaled before P V(s + 2).
// TMEM: S of group w [128 w, 128 w + 128), its O at 256 + w d.
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

#include "fa_shared.cuh"
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
constexpr int kPlanCtas = 8, kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
constexpr int kMostSlices = 8;  // warps that compare one sequence's entries

struct PlanParams {
    const int32_t *table, *kv_lens, *q_lens, *gid;
    int64_t num_pages, max_pages;
    int page, B, Nq, causal;
    int rows_per_seq, H_kv;
    int own_rows, own_tile, group;  // of the kernel over the sequences' own tokens
    int32_t* same;          // [slices][B] leading common entries seen by a slice
    int32_t* head;          // [B] shared group of a run's first sequence
    int32_t *run_first, *run_count, *run_tiles;  // [B] at a run's first sequence
    int32_t *skip, *group_of, *n;
    ShGroup* groups;
    long long* own0;        // [B + 1] units of the own tokens of the sequences before
};

// Keys that every query of sequence b sees, less one (so that something is left of its own); below 0:
// none, or no query.
__device__ __forceinline__ int64_t seen_by_all(const PlanParams& p, int b) {
    const int64_t room = p.max_pages * p.page;
    const int64_t len = min(static_cast<int64_t>(max(p.kv_lens[b], 0)), room);
    const int ql = p.q_lens ? min(max(p.q_lens[b], 0), p.Nq) : p.Nq;
    if (ql == 0) return -1;
    return (p.causal ? len - ql + 1 : len) - 1;
}
__device__ __forceinline__ bool joins(const PlanParams& p, int b) {
    return seen_by_all(p, b) >= kShTile;
}
__device__ __forceinline__ bool starts_run(const PlanParams& p, int b) {
    return b == 0 || (p.gid && p.gid[b] != p.gid[b - 1]);
}

// The whole warp: the first sequence of b's run that can join, -1 if that is none up to b.
__device__ __forceinline__ int lead_of(const PlanParams& p, int b) {
    const int lane = threadIdx.x & 31;
    int start = 0;
    for (int at = b; at >= 0 && p.gid; at -= 32) {
        const unsigned hit = __ballot_sync(0xffffffffu, at - lane >= 0 && starts_run(p, at - lane));
        if (hit) {
            start = at - (__ffs(hit) - 1);
            break;
        }
    }
    for (int at = start; at <= b; at += 32) {
        const unsigned hit = __ballot_sync(0xffffffffu, at + lane <= b && joins(p, at + lane));
        if (hit) return at + __ffs(hit) - 1;
    }
    return -1;
}

// What a run shares, from the slices' findings: the whole warp, `b` its first sequence.
struct RunInfo {
    int first, count, tiles, end;
};
__device__ __forceinline__ int64_t common_tokens(const PlanParams& p, int b, int slices) {
    int64_t e = p.max_pages;
    for (int s = 0; s < slices; ++s) e = min(e, static_cast<int64_t>(p.same[s * p.B + b]));
    return min(e * p.page, seen_by_all(p, b));
}
__device__ __forceinline__ RunInfo run_info(const PlanParams& p, int b, int slices) {
    const int lane = threadIdx.x & 31;
    RunInfo r{-1, 0, 0, p.B};
    int n = 0, last = -1;
    int least = 0x7fffffff;
    for (int at = b; at < p.B; at += 32) {
        const int i = at + lane;
        const unsigned out = __ballot_sync(0xffffffffu, i >= p.B || (i > b && starts_run(p, i)));
        const int end = out ? __ffs(out) - 1 : 32;
        int c = -1;
        if (lane < end) c = static_cast<int>(min(common_tokens(p, i, slices), int64_t(1) << 30));
        const unsigned in = __ballot_sync(0xffffffffu, c >= kShTile);
        least = min(least, __reduce_min_sync(0xffffffffu, c >= kShTile ? c : 0x7fffffff));
        if (in && r.first < 0) r.first = at + __ffs(in) - 1;
        if (in) last = at + 31 - __clz(in);
        n += __popc(in);
        if (out) {
            r.end = at + end;
            break;
        }
    }
    if (n >= 2) {
        r.count = last - r.first + 1;
        r.tiles = least / kShTile;
    }
    return r;
}

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
    shared_plan_kernel(const PlanParams p) {
    asm volatile("griddepcontrol.launch_dependents;");
    cg::cluster_group cl = cg::this_cluster();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // several warps a sequence while there are enough of them
    const int slices = min(kMostSlices, max(1, kPlanCtas * kPlanWarps / p.B));
    for (int64_t u = static_cast<int>(cl.block_rank()) * kPlanWarps + warp;
         u < static_cast<int64_t>(p.B) * slices; u += kPlanCtas * kPlanWarps) {
        const int b = static_cast<int>(u / slices);
        const int s = static_cast<int>(u - static_cast<int64_t>(b) * slices);
        int32_t same = 0;
        if (joins(p, b)) {
            const int lead = lead_of(p, b);
            const int64_t tokens = min(seen_by_all(p, b), seen_by_all(p, lead));
            const int n = static_cast<int>((tokens + p.page - 1) / p.page);
            const int each = ((n + slices - 1) / slices + 31) & ~31;
            const int j0 = s * each, j1 = min(n, j0 + each);
            const int32_t* x = p.table + b * p.max_pages;
            const int32_t* y = p.table + lead * p.max_pages;
            same = n;
            constexpr int U = 8;
            for (int j = j0; j < j1; j += 32 * U) {
                int32_t a[U], c[U];
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int k = j + 32 * i + lane;
                    a[i] = k < j1 ? x[k] : 0;
                    c[i] = k < j1 ? y[k] : 0;
                }
                int first = 0x7fffffff;
#pragma unroll
                for (int i = U - 1; i >= 0; --i) {
                    const int k = j + 32 * i + lane;
                    if (k < j1 && (a[i] != c[i] || a[i] < 0 || a[i] >= p.num_pages)) first = k;
                }
                first = __reduce_min_sync(0xffffffffu, first);
                if (first != 0x7fffffff) {
                    same = first;
                    break;
                }
            }
        }
        if (lane == 0) p.same[s * p.B + b] = same;
    }
    cl.sync();
    if (cl.block_rank() != 0) return;
    for (int b = warp; b < p.B; b += kPlanWarps) {
        RunInfo r{-1, 0, 0, 0};
        if (starts_run(p, b)) r = run_info(p, b, slices);
        if (lane == 0) {
            p.run_first[b] = r.first;
            p.run_count[b] = r.count;
            p.run_tiles[b] = r.tiles;
        }
    }
    __syncthreads();
    // the shared groups in order, and the own tokens' units (below)
    if (warp == 0) {
        int n = 0;
        long long units = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int b = b0 + lane;
            const int tiles = b < p.B ? p.run_tiles[b] : 0;
            const unsigned has = __ballot_sync(0xffffffffu, tiles > 0);
            ShGroup g{};
            long long mine = 0;
            if (tiles > 0) {
                g.first = p.run_first[b];
                g.count = p.run_count[b];
                g.tiles = tiles;
                const int blocks = (g.count * p.rows_per_seq + kShRows - 1) / kShRows;
                mine = static_cast<long long>(p.H_kv) * blocks * tiles;
            }
            long long inc = mine;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const long long o = __shfl_up_sync(0xffffffffu, inc, m);
                if (lane >= m) inc += o;
            }
            const int at = n + __popc(has & ((1u << lane) - 1u));
            if (tiles > 0) {
                g.unit0 = units + inc - mine;
                p.groups[at] = g;
            }
            if (b < p.B) p.head[b] = tiles > 0 ? at : -1;
            n += __popc(has);
            units += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) {
            ShGroup end{};
            end.unit0 = units;
            p.groups[n] = end;
            *p.n = n;
        }
    }
    __syncthreads();
    for (int b = warp; b < p.B; b += kPlanWarps) {
        if (!starts_run(p, b)) continue;
        const RunInfo r = run_info(p, b, slices);
        const int j = p.head[b];
        for (int i = b + lane; i < r.end; i += 32) {
            const bool in = j >= 0 && common_tokens(p, i, slices) >= kShTile;
            p.skip[i] = in ? r.tiles * kShTile : 0;
            p.group_of[i] = j;
        }
    }
    __syncthreads();
    if (warp == 0) {
        long long units = 0;
        const int64_t room = p.max_pages * p.page;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int b = b0 + lane;
            long long mine = 0;
            if (b < p.B) {
                const int64_t len = min(static_cast<int64_t>(max(p.kv_lens[b], 0)), room);
                const int ql = p.q_lens ? min(max(p.q_lens[b], 0), p.Nq) : p.Nq;
                mine = ((len + p.own_tile - 1) / p.own_tile - p.skip[b] / p.own_tile) * p.H_kv *
                       ((static_cast<int64_t>(ql) * p.group + p.own_rows - 1) / p.own_rows);
            }
            long long inc = mine;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const long long o = __shfl_up_sync(0xffffffffu, inc, m);
                if (lane >= m) inc += o;
            }
            if (b < p.B) p.own0[b] = units + inc - mine;
            units += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) p.own0[p.B] = units;
    }
}

// ------------------------------------------------------------------------------------------
// prefix
// ------------------------------------------------------------------------------------------
constexpr int kThreads = 512;
constexpr int kLoadWarp = 8;   // warps 8-11
constexpr int kMmaWarp = 12;
constexpr int kHalfBytes = 128 * 128;  // 64 columns of a 128-row bf16 tile
constexpr float kMoveThreshold = 8.f, kMoveHeadroom = 24.f;  // log2 units, as in fa_fwd.cu
constexpr uint64_t kDrainNs = 1000000000ull;
constexpr uint32_t kBarRaw = 1;       // the loading warps (4 bits)
constexpr uint32_t kBarTeardown = 2;  // TMEM no longer used: softmax warps and the MMA warp
constexpr uint32_t kTeardownThreads = 288;
constexpr int kMaxSlots = 10;

struct Bars {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t q_full[2];  // group w's queries are in shared memory (4 warps)
    uint64_t s_full[2];  // S of group w's step (tcgen05.commit)
    uint64_t p_full[2];  // P stored, O rescaled if needed (4 warps)
    uint64_t o_full[2];  // the last P V of group w's item (tcgen05.commit)
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
    static constexpr int kRaw = 3;                                // raw tiles on their way
    // The ring: what the queries (two tiles) and the raw tiles leave.
    static constexpr int kSlots = D == 128 ? (kInt4 ? 4 : 5) : (kInt4 ? 8 : 10);
    static constexpr int kQ = 0;
    static constexpr int kRing = kQ + 2 * kTileBytes;
    static constexpr int kRawAt = kRing + kSlots * kTileBytes;
    static constexpr int kBars = kRawAt + (kInt4 ? kRaw * kRawBytes : 0);
    static constexpr int kBytes = kBars + static_cast<int>(sizeof(Bars));
    static constexpr int kDyn = kBytes + 1024;  // slack for 1024-byte alignment
    static_assert(kDyn <= 227 * 1024, "shared memory budget");
    static constexpr uint32_t kTmemO = 256;
    static_assert(kTmemO + 2 * D <= 512, "TMEM budget");
};
constexpr int kSoftRegs = 200, kLoadRegs = 72, kMmaRegs = 40;
static_assert(256 * kSoftRegs + 128 * kLoadRegs + 128 * kMmaRegs <= 65536, "register split");

struct PrefixParams {
    const __nv_bfloat16* Q;  // [B, H, Nq, D]
    KvPages pg;
    ShView v;
    int H, Nq, group;  // group: H / H_kv
    int box;           // bf16: tokens of a TMA box
    float scale_log2;
    unsigned long long timeout_ns;
};

// A CTA's walk through the items of its share: tiles [t0, t1) of (group g, key/value head, block).
struct Walk {
    ShGroup g;
    int j, kvh, block, blocks, t0, t1;
    long long left;

    __device__ __forceinline__ void load(const ShView& v) {
        g = v.groups[j];
        blocks = sh_blocks(v, g);
    }
    __device__ __forceinline__ void start(const ShView& v) {
        const int n = *v.n;
        const long long units = v.groups[n].unit0;
        const long long share = sh_share(units, static_cast<int>(gridDim.x));
        const long long u0 = share * blockIdx.x;
        left = min(units, u0 + share) - u0;
        if (left <= 0) return;
        int lo = 0, hi = n - 1;  // the last group with unit0 <= u0
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (v.groups[mid].unit0 <= u0) lo = mid;
            else hi = mid - 1;
        }
        j = lo;
        load(v);
        const long long r = u0 - g.unit0;
        const int item = static_cast<int>(r / g.tiles);
        t0 = static_cast<int>(r - static_cast<long long>(item) * g.tiles);
        kvh = item / blocks;
        block = item - kvh * blocks;
        t1 = static_cast<int>(min(static_cast<long long>(g.tiles - t0), left)) + t0;
    }
    __device__ __forceinline__ bool done() const { return left <= 0; }
    __device__ __forceinline__ void next(const ShView& v) {
        left -= t1 - t0;
        if (left <= 0) return;
        if (++block == blocks) {
            block = 0;
            if (++kvh == v.H_kv) {
                kvh = 0;
                ++j;
                load(v);
            }
        }
        t0 = 0;
        t1 = static_cast<int>(min(static_cast<long long>(g.tiles), left));
    }
    // Rows of the block; more than 128: each softmax group has its half and sees every tile.
    __device__ __forceinline__ int rows(const ShView& v) const {
        return min(kShRows, g.count * v.rows_per_seq - block * kShRows);
    }
    __device__ __forceinline__ bool halves(const ShView& v) const { return rows(v) > kShHalf; }
};

// The steps of an item in the order of their products, load_k / load_v where a tile is first used.
// use(kind, step, tile, first use of the tile, last use of it) with kind 0: S, 1: P V.
template <typename Use>
__device__ __forceinline__ bool for_steps(int n, bool halves, const Use& use) {
    const int steps = halves ? 2 * n : n;
    auto call = [&](int kind, int s) {
        return halves ? use(kind, s, s >> 1, (s & 1) == 0, (s & 1) != 0)
                      : use(kind, s, s, true, true);
    };
    if (!call(0, 0)) return false;
    if (steps > 1 && !call(0, 1)) return false;
    for (int s = 0; s < steps; ++s) {
        if (!call(1, s)) return false;
        if (s + 2 < steps && !call(0, s + 2)) return false;
    }
    return true;
}

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
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
        for (int w = 0; w < 2; ++w) {
            mbar_init(&bars->q_full[w], 4);
            mbar_init(&bars->s_full[w], 1);
            mbar_init(&bars->p_full[w], 4);
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
            int entry = 0, k_slot = 0, v_slot = 0;
            uint32_t q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity, int where) {
                const bool good = issuer_wait<true>(bar, parity, timeout, true);
                if (!good && lane == 0) give_up(where);
                return good;
            };
            for (; ok && !walk.done(); walk.next(p.v)) {
                const int n = walk.t1 - walk.t0;
                const bool halves = walk.halves(p.v);
                const int steps = halves ? 2 * n : n;
                ok = for_steps(n, halves, [&](int kind, int s, int, bool first, bool last) {
                    const int w = s & 1;
                    int& slot = kind == 0 ? k_slot : v_slot;
                    if (kind == 0) {
                        if (s < 2) {
                            if (!wait(&bars->q_full[w], q_phase[w], 30)) return false;
                            q_phase[w] ^= 1;
                        }
                    } else {
                        if (!wait(&bars->p_full[w], p_phase[w], 31)) return false;
                        p_phase[w] ^= 1;
                    }
                    if (first) {
                        slot = entry % C::kSlots;
                        if (!wait(&bars->full[slot], (entry / C::kSlots) & 1, 32)) return false;
                        ++entry;
                    }
                    tc_fence_after();
                    const uint32_t tile = ring + slot * C::kTileBytes;
                    if (kind == 0) {
                        const uint32_t q = smem_u32(smem + C::kQ) + w * C::kTileBytes;
#pragma unroll
                        for (int h = 0; h < C::kHalves; ++h)
                            issue_ss_x4<true>(tmem + w * 128,
                                              smem_desc_sw128(q + h * kHalfBytes, 16, 1024),
                                              smem_desc_sw128(tile + h * kHalfBytes, 16, 1024), idS,
                                              h > 0 ? 1u : 0u);
                        issue_commit<true>(&bars->s_full[w]);
                    } else {
                        issue_ts_x8<true>(tmem + C::kTmemO + w * D, tmem + w * 128,
                                          smem_desc_sw128(tile, kHalfBytes, 1024), 2048 / 16, idO,
                                          s < 2 ? 0u : 1u);
                        if (s + 2 >= steps) issue_commit<true>(&bars->o_full[w]);
                    }
                    if (last) issue_commit<true>(&bars->empty[slot]);
                    return true;
                });
            }
            issue_commit<true>(&bars->done);
            issuer_wait<true>(&bars->done, 0, timeout > kDrainNs ? timeout : kDrainNs, true);
            __syncwarp();
            named_bar_sync(kBarTeardown, kTeardownThreads);
            tc_fence_after();
            tmem_dealloc(tmem, 512);
        }
    } else if (warp >= kLoadWarp) {
        setmaxnreg_dec<kLoadRegs>();
        if constexpr (!C::kInt4) {
            // ------------------------------------------------------------ bf16 tiles by TMA
            if (warp == kLoadWarp) {
                if (lane == 0) {
                    tma_prefetch_desc(&tmK);
                    tma_prefetch_desc(&tmV);
                }
                const int boxes = kShTile / p.box;  // of a tile, for each half: boxes * kHalves <= 16
                const int box = lane % boxes, half = lane / boxes;
                const bool mine = half < C::kHalves;
                int entry = 0;
                bool ok = true;
                for (; ok && !walk.done(); walk.next(p.v)) {
                    // The box's page and place in it for tiles base, base + 1 and base + 2: a tile's
                    // serve its keys and its values, and the table is read two tiles ahead.
                    const int32_t* row = p.pg.table + walk.g.first * p.pg.max_pages;
                    int base = walk.t0, id[3], place[3];
                    auto look = [&](int tile, int& i, int& at) {
                        const int tok = tile * kShTile + box * p.box, e = tok / p.pg.page;
                        at = tok - e * p.pg.page;
                        i = mine && tile < walk.t1 ? row[e] : 0;
                    };
#pragma unroll
                    for (int x = 0; x < 3; ++x) look(base + x, id[x], place[x]);
                    ok = for_steps(walk.t1 - walk.t0, walk.halves(p.v),
                                   [&](int kind, int, int t, bool first, bool) {
                        if (!first) return true;
                        const int slot = entry % C::kSlots;
                        if (entry >= C::kSlots &&
                            !warp_wait(&bars->empty[slot], ((entry / C::kSlots) - 1) & 1, timeout,
                                       true)) {
                            if (lane == 0) give_up(33);
                            return false;
                        }
                        ++entry;
                        if (lane == 0) mbar_arrive_expect_tx(&bars->full[slot], C::kTileBytes);
                        __syncwarp();
                        const int tile = walk.t0 + t;
                        if (tile > base + 1) {
                            id[0] = id[1], place[0] = place[1];
                            id[1] = id[2], place[1] = place[2];
                            ++base;
                            look(base + 2, id[2], place[2]);
                        }
                        const bool next = tile > base;
                        if (mine)
                            tma_load_4d(smem + C::kRing + slot * C::kTileBytes + half * kHalfBytes +
                                            box * p.box * 128,
                                        kind == 0 ? &tmK : &tmV, &bars->full[slot], half * 64,
                                        next ? place[1] : place[0], walk.kvh, next ? id[1] : id[0]);
                        return true;
                    });
                }
                // what is on its way lands before the CTA ends
                const uint64_t drain = timeout > kDrainNs ? timeout : kDrainNs;
                for (int s = 0; s < C::kSlots && s < entry; ++s) {
                    const int last = s + (entry - 1 - s) / C::kSlots * C::kSlots;
                    mbar_wait(&bars->full[s], (last / C::kSlots) & 1, drain, true);
                }
            }
        } else {
            // ------------------------------------------------------------ 4-bit tiles expanded
            // A walk of its own issues the raw copies, kRaw tiles (keys or values of 128 tokens)
            // ahead of the expansion; both go through the tiles in the order of their first use.
            // 16-byte chunks of codes: a row's, and the rows that the 128 threads take at a time
            constexpr int kChunks = C::kRawRow / 16, kRowsPer = 128 / kChunks;
            constexpr int kPasses = kShTile / kRowsPer;
            const int tid = threadIdx.x - kLoadWarp * 32;
            const int c = tid % kChunks, r0 = tid / kChunks;
            const uint32_t raw = smem_u32(smem + C::kRawAt);
            // order of first use: K(0) [K(1) when the groups take the tiles in turn] then V, K in turn
            struct Order {
                Walk w;
                int i, n;      // tile loads of the item so far, and in all
                bool halves;
                __device__ __forceinline__ void item(const ShView& v) {
                    i = 0;
                    n = w.done() ? 0 : 2 * (w.t1 - w.t0);
                    halves = !w.done() && w.halves(v);
                }
                // the load's tile and whether it is V
                __device__ __forceinline__ void at(int& tile, bool& is_v) const {
                    int x = i;
                    if (halves) {  // K0 V0 K1 V1 ...
                        is_v = x & 1;
                        tile = w.t0 + (x >> 1);
                        return;
                    }
                    // K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1)
                    const int tiles = n >> 1;
                    if (x == 0) is_v = false, tile = w.t0;
                    else if (x == n - 1) is_v = true, tile = w.t0 + tiles - 1;
                    else is_v = !(x & 1), tile = w.t0 + (is_v ? (x >> 1) - 1 : (x + 1) >> 1);
                }
                __device__ __forceinline__ bool done() const { return w.done(); }
                __device__ __forceinline__ void next(const ShView& v) {
                    if (++i == n) {
                        w.next(v);
                        item(v);
                    }
                }
            };
            Order ahead;
            ahead.w = walk;
            ahead.item(p.v);
            Order now = ahead;
            int fill = 0;
            // The pages and places of the next raw tile's rows and words, read a tile ahead.
            int32_t id[kPasses], w_id = 0;
            int place[kPasses], w_place = 0, tile = 0;
            bool is_v = false;
            constexpr int kPerChunk = 8 / C::kG;  // tokens whose words 16 bytes hold: of one page
            auto look = [&]() {
                if (ahead.done()) return;
                ahead.at(tile, is_v);
                const int32_t* row = p.pg.table + ahead.w.g.first * p.pg.max_pages;
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const int tok = tile * kShTile + i * kRowsPer + r0, e = tok / p.pg.page;
                    place[i] = tok - e * p.pg.page;
                    id[i] = row[e];
                }
                if (tid < kShTile / kPerChunk) {
                    const int tok = tile * kShTile + tid * kPerChunk, e = tok / p.pg.page;
                    w_place = tok - e * p.pg.page;
                    w_id = row[e];
                }
            };
            auto issue = [&]() {
                if (!ahead.done()) {
                    const uint8_t* pages = is_v ? p.pg.v : p.pg.k;
                    const uint32_t dst = raw + fill * C::kRawBytes;
#pragma unroll
                    for (int i = 0; i < kPasses; ++i)
                        copy16(dst + (i * kRowsPer + r0) * C::kRawRow + c * 16,
                               pages + kv_head_offset(p.pg, id[i], ahead.w.kvh) +
                                   place[i] * C::kRawRow + c * 16);
                    if (tid < kShTile / kPerChunk)
                        copy16(dst + C::kRawCodes + tid * 16,
                               pages + kv_head_offset(p.pg, w_id, ahead.w.kvh) +
                                   static_cast<int64_t>(p.pg.page) * C::kRawRow +
                                   w_place * (C::kG * 2));
                    ahead.next(p.v);
                    fill = fill == C::kRaw - 1 ? 0 : fill + 1;
                    look();
                }
                copies_commit();
            };
            look();
#pragma unroll
            for (int i = 0; i < C::kRaw - 1; ++i) issue();
            int entry = 0, take = 0;
            for (; !now.done(); now.next(p.v)) {
                const int slot = entry % C::kSlots;
                copies_wait<C::kRaw - 2>();
                bool good = true;
                if (entry >= C::kSlots)
                    good = warp_wait(&bars->empty[slot], ((entry / C::kSlots) - 1) & 1, timeout,
                                     true);
                if (!good && lane == 0) give_up(34);
                // all four warps see all words, and have done with the raw tile before this one
                if (!named_bar_and(kBarRaw, 128, good)) break;
                issue();
                const uint32_t src = raw + take * C::kRawBytes;
                uint8_t* dst = smem + C::kRing + slot * C::kTileBytes;
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const int r = i * kRowsPer + r0;
                    uint32_t w[4];
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                 : "r"(src + r * C::kRawRow + c * 16)
                                 : "memory");
                    uint16_t word;
                    asm volatile("ld.shared.b16 %0, [%1];"
                                 : "=h"(word)
                                 : "r"(src + C::kRawCodes + (r * C::kG + c / 2) * 2)
                                 : "memory");
                    // step and base - 128 as pairs of bf16; both exact
                    const uint32_t s1 = (word & 0xffc0u) >> 1;
                    const uint32_t step = s1 | s1 << 16;
                    const float base = static_cast<float>(kv4_word_base(word) - 128);
                    const uint32_t shift = pack_bf16x2(base, base);
                    uint8_t* half = dst + (c >> 1) * kHalfBytes + r * 128;
#pragma unroll
                    for (int jj = 0; jj < 4; ++jj) {
                        // (lanes of the second half in another order: no bank conflicts)
                        const int j = jj ^ (c & 2);
                        uint32_t x = jj == 0 ? w[0] : jj == 1 ? w[1] : jj == 2 ? w[2] : w[3];
                        if (c & 2) x = jj == 0 ? w[2] : jj == 1 ? w[3] : jj == 2 ? w[0] : w[1];
                        uint32_t y[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            y[k] = mul_bf16x2(
                                add_bf16x2((x >> (4 * k) & 0x000f000fu) | 0x43004300u, shift), step);
                        const int ch = (c & 1) * 4 + j;
                        *reinterpret_cast<uint4*>(half + ((ch ^ (r & 7)) << 4)) =
                            make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->full[slot]);
                ++entry;
                take = take == C::kRaw - 1 ? 0 : take + 1;
            }
            copies_wait<0>();
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
            const int n = walk.t1 - walk.t0, rows = walk.rows(p.v);
            const bool halves = rows > kShHalf;
            const int steps = halves ? n : (n + 1 - w) / 2;
            const int row = (halves ? w * kShHalf : 0) + r;  // of the block
            const bool real = row < rows;
            int64_t at = 0;  // the row's place in Q, O and LSE
            if (real) {
                const int R = walk.block * kShRows + row;
                const int b = R / p.v.rows_per_seq, x = R - b * p.v.rows_per_seq;
                const int i = x / p.group, h = walk.kvh * p.group + x - i * p.group;
                at = (static_cast<int64_t>(walk.g.first + b) * p.H + h) * p.Nq + i;
            }
            float m = -INFINITY, l = 0.f;
            if (steps > 0) {
                // the queries; the products with the last item's have all been waited for
                const uint4* q = reinterpret_cast<const uint4*>(p.Q + at * D);
#pragma unroll
                for (int c0 = 0; c0 < D / 8; c0 += 8) {
                    uint4 x[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        x[c] = real ? q[c0 + c] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        uint4 y = x[c];
                        if constexpr (C::kInt4) {  // values k and k + 4 side by side
                            y.x = __byte_perm(x[c].x, x[c].z, 0x5410);
                            y.y = __byte_perm(x[c].x, x[c].z, 0x7632);
                            y.z = __byte_perm(x[c].y, x[c].w, 0x5410);
                            y.w = __byte_perm(x[c].y, x[c].w, 0x7632);
                        }
                        *reinterpret_cast<uint4*>(sQ + (c0 / 8) * kHalfBytes + r * 128 +
                                                  ((c ^ (r & 7)) << 4)) = y;
                    }
                }
                fence_proxy_async_smem();
                warp_arrive_tc(&bars->q_full[w]);
            }
            for (int s = 0; s < steps; ++s) {
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
                for (int u = 0; u < 16; ++u) top[u] = __uint_as_float(sr[u]);
#pragma unroll
                for (int e = 16; e < 128; ++e)
                    top[e & 15] = fmaxf(top[e & 15], __uint_as_float(sr[e]));
#pragma unroll
                for (int x = 8; x >= 1; x >>= 1)
#pragma unroll
                    for (int u = 0; u < x; ++u) top[u] = fmaxf(top[u], top[u + x]);
                const float mx = top[0] * scale;
                const float m_new = mx - m > kMoveThreshold ? mx + kMoveHeadroom : m;
                const float alpha = m_new == m ? 1.f : ex2_approx(m - m_new);
                const float ref = m_new == -INFINITY ? 0.f : m_new;
                uint32_t pr[64];
                float2 sum = make_float2(0.f, 0.f), sum2 = make_float2(0.f, 0.f);
                const float2 c2 = make_float2(scale, scale), n2 = make_float2(-ref, -ref);
#pragma unroll
                for (int e = 0; e < 128; e += 4) {
                    float2 x0 = ffma2(
                        make_float2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), c2, n2);
                    float2 x1 = ffma2(
                        make_float2(__uint_as_float(sr[e + 2]), __uint_as_float(sr[e + 3])), c2, n2);
                    x0.x = ex2_approx(x0.x);
                    x0.y = ex2_approx(x0.y);
                    x1.x = ex2_approx(x1.x);
                    x1.y = ex2_approx(x1.y);
                    sum = fadd2(sum, x0);
                    sum2 = fadd2(sum2, x1);
                    pr[e >> 1] = pack_bf16x2(x0.x, x0.y);
                    pr[(e >> 1) + 1] = pack_bf16x2(x1.x, x1.y);
                }
                l = l * alpha + ((sum.x + sum.y) + (sum2.x + sum2.y));
                m = m_new;
                // O holds P V of the steps before: S of this one was committed after them
                if (s > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32_sync(tO + c * 32, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st32_sync(tO + c * 32, o);
                    }
                }
                tmem_st64_sync(tS, pr);
                warp_arrive_tc(&bars->p_full[w]);
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
            const bool whole = walk.t0 == 0 && walk.t1 == walk.g.tiles;
            const int64_t place =
                whole ? 2 * at + (halves ? 0 : w)
                      : ((static_cast<int64_t>(blockIdx.x) * 2 + (walk.t0 == 0 ? 1 : 0)) * 2 + w) *
                                kShHalf + r;
            float* dst = (whole ? p.v.row_o : p.v.edge_o) + place * D;
            if (real) (whole ? p.v.row_ml : p.v.edge_ml)[place] = make_float2(m, l);
            if (steps == 0) continue;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32_sync(tO + c * 32, o);
                if (!real) continue;
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    float4 a, b;
                    if constexpr (C::kInt4) {  // columns 2 k and 2 k + 1 are values k and k + 4
                        a = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 2]),
                                        __uint_as_float(o[e + 4]), __uint_as_float(o[e + 6]));
                        b = make_float4(__uint_as_float(o[e + 1]), __uint_as_float(o[e + 3]),
                                        __uint_as_float(o[e + 5]), __uint_as_float(o[e + 7]));
                    } else {
                        a = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                        __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
                        b = make_float4(__uint_as_float(o[e + 4]), __uint_as_float(o[e + 5]),
                                        __uint_as_float(o[e + 6]), __uint_as_float(o[e + 7]));
                    }
                    reinterpret_cast<float4*>(dst + c * 32 + e)[0] = a;
                    reinterpret_cast<float4*>(dst + c * 32 + e)[1] = b;
                }
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
    const long long* own0;
    const float* own_edge;  // [ctas][2]: [rows][D], then m, l of the rows
    const float* own_o;     // [B * H * Nq][D]
    const float2* own_ml;
    int64_t room;
    int B, H, Nq, group, causal;
    int own_rows, own_tile, own_ctas;
};

// W warps a row; the row's states in turn, two-worker merge.
constexpr int kJoinWarps = 8;
template <int D, int W>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const JoinParams p) {
    constexpr int E = D / 32, R = kJoinWarps / W;
    __shared__ float sM[kJoinWarps], sL[kJoinWarps], sO[kJoinWarps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * R + warp / W;
    const int64_t rows = static_cast<int64_t>(p.B) * p.H * p.Nq;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float M = -INFINITY, L = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    bool sees = false;
    if (at < rows) {
        const int64_t bh = at / p.Nq;
        const int i = static_cast<int>(at - bh * p.Nq);
        const int b = static_cast<int>(bh / p.H);
        const int h = static_cast<int>(bh - static_cast<int64_t>(b) * p.H);
        const int kvh = h / p.group;
        const int row = i * p.group + h - kvh * p.group;  // of the sequence and key/value head
        const int len = static_cast<int>(min(static_cast<int64_t>(max(p.kv_lens[b], 0)), p.room));
        const int ql = p.q_lens ? min(max(p.q_lens[b], 0), p.Nq) : p.Nq;
        sees = i < ql && (p.causal ? len - ql + i : len - 1) >= 0;
        if (sees) {
            // the sequence's own tokens
            const int skip = p.v.skip[b];
            const int tiles = (len + p.own_tile - 1) / p.own_tile - skip / p.own_tile;
            const int blocks = (ql * p.group + p.own_rows - 1) / p.own_rows;
            const int block = row / p.own_rows, br = row - block * p.own_rows;
            const long long units = p.own0[p.B];
            const long long share = own_share(units, p.own_ctas);
            const long long u =
                p.own0[b] + (static_cast<long long>(kvh) * blocks + block) * tiles;
            const int c0 = static_cast<int>(u / share);
            const int c1 = static_cast<int>((u + tiles - 1) / share);
            const int own_n = c0 == c1 ? 1 : c1 - c0 + 1;
            // the common ones
            int pre_n = 0, pw = 1, g0 = 0, pr = 0, w0 = 0;
            bool whole = false;
            if (skip > 0) {
                const ShGroup g = p.v.groups[p.v.group[b]];
                const int RR = (b - g.first) * p.v.rows_per_seq + row;
                const int pb = RR / kShRows, rr = RR - pb * kShRows;
                const bool halves = min(kShRows, g.count * p.v.rows_per_seq - pb * kShRows) > kShHalf;
                const long long all = p.v.groups[*p.v.n].unit0;
                const long long ps = sh_share(all, p.v.ctas);
                const long long pu =
                    g.unit0 + (static_cast<long long>(kvh) * sh_blocks(p.v, g) + pb) * g.tiles;
                g0 = static_cast<int>(pu / ps);
                const int g1 = static_cast<int>((pu + g.tiles - 1) / ps);
                whole = g0 == g1;
                pw = halves ? 1 : 2;
                w0 = halves && !whole ? rr / kShHalf : 0;
                pr = halves ? rr % kShHalf : rr;
                pre_n = (g1 - g0 + 1) * pw;
            }
#pragma unroll 4
            for (int k = warp % W; k < own_n + pre_n; k += W) {
                const float* src;
                float mk, lk;
                if (k < own_n) {
                    if (c0 == c1) {
                        const float2 ml = p.own_ml[at];
                        mk = ml.x, lk = ml.y;
                        src = p.own_o + at * D;
                    } else {
                        const float* part = p.own_edge + (static_cast<int64_t>(c0 + k) * 2 +
                                                          (k == 0 ? 1 : 0)) *
                                                             (p.own_rows * (D + 2));
                        mk = part[p.own_rows * D + br];
                        lk = part[p.own_rows * (D + 1) + br];
                        src = part + br * D;
                    }
                } else {
                    const int x = k - own_n, c = x / pw, w = x - c * pw + w0;
                    const int64_t place =
                        whole ? 2 * at + w
                              : ((static_cast<int64_t>(g0 + c) * 2 + (c == 0 ? 1 : 0)) * 2 + w) *
                                        kShHalf + pr;
                    const float2 ml = (whole ? p.v.row_ml : p.v.edge_ml)[place];
                    mk = ml.x, lk = ml.y;
                    src = (whole ? p.v.row_o : p.v.edge_o) + place * D;
                }
                // a state without a tile (l = 0, m = -inf) has no O
                const bool some = lk != 0.f || mk != -INFINITY;
                float v[E];
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = 0.f;
                if (some) {
                    if constexpr (E == 4) {
                        const float4 y = reinterpret_cast<const float4*>(src)[lane];
                        v[0] = y.x, v[1] = y.y, v[2] = y.z, v[3] = y.w;
                    } else {
                        const float2 y = reinterpret_cast<const float2*>(src)[lane];
                        v[0] = y.x, v[1] = y.y;
                    }
                }
                const float mn = fmaxf(M, mk), ref = mn == -INFINITY ? 0.f : mn;
                const float a = ex2_approx(M - ref), f = ex2_approx(mk - ref);
                M = mn;
                L = L * a + lk * f;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = o[e] * a + v[e] * f;
            }
        }
    }
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

struct Workspace {
    int64_t plan, own0, groups, edge_o, edge_ml, row_o, row_ml, own_edge, own_o, own_ml, bytes;
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
    w.plan = part((kMostSlices + 7) * B * 4 + 64);
    w.own0 = part((B + 1) * 8);
    w.groups = part((B + 1) * static_cast<int64_t>(sizeof(ShGroup)));
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
    return rows <= 16 * sm_count() ? launch_join_w<D, 8>(p, stream) : launch_join_w<D, 1>(p, stream);
}

}  // namespace

int64_t fa_shared_ws_bytes(int64_t B, int64_t H, int64_t H_kv, int64_t Nq, int64_t d, int format,
                           int64_t page, int64_t max_pages) {
    const int64_t need = fa_paged_ws_bytes(B, H, H_kv, Nq, d, format, page, max_pages);
    if (need < 0 || fa_paged_takes_chunks(H / H_kv * Nq)) return need;
    return workspace(B, H, H_kv, Nq, d, format, page, max_pages).bytes;
}

int fa_shared_launch(const void* Q, void* O, float* LSE, const KvPages& pg, const int32_t* kv_lens,
                     const int32_t* q_lens, const int32_t* groups, int64_t B, int64_t H, int64_t Nq,
                     int64_t d, float scale, bool causal, void* ws, cudaStream_t stream) {
    const int64_t rows = H / pg.H_kv * Nq;
    if (fa_paged_takes_chunks(rows) || pg.num_pages == 0)
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
    pl.group = static_cast<int>(H / pg.H_kv);
    int32_t* at = reinterpret_cast<int32_t*>(base + w.plan);
    pl.n = at;
    at += 16;
    for (int32_t** x : {&pl.head, &pl.run_first, &pl.run_count, &pl.run_tiles, &pl.skip,
                        &pl.group_of}) {
        *x = at;
        at += B;
    }
    pl.same = at;
    pl.groups = reinterpret_cast<ShGroup*>(base + w.groups);
    pl.own0 = reinterpret_cast<long long*>(base + w.own0);

    ShView v{};
    v.skip = pl.skip;
    v.group = pl.group_of;
    v.groups = pl.groups;
    v.n = pl.n;
    v.edge_o = reinterpret_cast<float*>(base + w.edge_o);
    v.edge_ml = reinterpret_cast<float2*>(base + w.edge_ml);
    v.row_o = reinterpret_cast<float*>(base + w.row_o);
    v.row_ml = reinterpret_cast<float2*>(base + w.row_ml);
    v.ctas = w.ctas;
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
    pp.scale_log2 = scale * kLog2e;
    pp.timeout_ns = fa_wait_timeout_ns();
    // the tokens of a box: the most that divide both a tile and a page
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
    int st = pg.format == OSM_KV_INT4
                 ? (d == 64 ? launch_prefix<64, OSM_KV_INT4>(tk, tv, pp, stream)
                            : launch_prefix<128, OSM_KV_INT4>(tk, tv, pp, stream))
                 : (d == 64 ? launch_prefix<64, OSM_KV_BF16>(tk, tv, pp, stream)
                            : launch_prefix<128, OSM_KV_BF16>(tk, tv, pp, stream));
    if (st != FA_OK) return st;

    JoinParams j{};
    j.own_o = reinterpret_cast<const float*>(base + w.own_o);
    j.own_ml = reinterpret_cast<const float2*>(base + w.own_ml);
    st = fa_paged_own_launch(Q, pg, kv_lens, q_lens, B, H, Nq, d, scale, causal, w.own,
                             base + w.own_edge, v.skip, reinterpret_cast<float*>(base + w.own_o),
                             reinterpret_cast<float2*>(base + w.own_ml), stream);
    if (st != FA_OK) return st;

    j.O = static_cast<__nv_bfloat16*>(O);
    j.LSE = LSE;
    j.kv_lens = kv_lens;
    j.q_lens = q_lens;
    j.v = v;
    j.own0 = pl.own0;
    j.own_edge = reinterpret_cast<const float*>(base + w.own_edge);
    j.room = pg.max_pages * pg.page;
    j.B = static_cast<int>(B);
    j.H = static_cast<int>(H);
    j.Nq = static_cast<int>(Nq);
    j.group = pl.group;
    j.causal = pl.causal;
    j.own_rows = w.own.rows;
    j.own_tile = w.own.tile;
    j.own_ctas = w.own.ctas;
    return d == 64 ? launch_join<64>(j, stream) : launch_join<128>(j, stream);
}

}  // namespace osm
