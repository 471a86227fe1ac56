// fa_paged.cu -- attention of a few queries over the paged key/value cache (fa_fwd_paged).
//
// Row i of sequence b sees the keys j <= kv_len - q_len + i (causal) or j < kv_len; rows at or past
// q_len see none (O = 0, LSE = -inf).  The computation is the online softmax of fa_fwd.cu; with few
// queries it is bound by reading the cache once, so the kernel is built around that stream.
//
// Rows.  The H / H_kv query heads of a key/value head times the Nq queries are one list of rows
// (row = query * (H / H_kv) + head), taken kRows = 8 or 16 at a time: an item is (sequence,
// key/value head, row block), and it reads the sequence's keys in tiles of kT tokens.
//
// Work.  All tiles of all items, in order, are cut into equal shares, one a CTA, so that sequences
// of very different lengths load the GPU evenly; lengths are read on the device.  A CTA goes
// through the items of its share; its four warps take an item's tiles in turn, each with its own
// running max, sum and accumulator, and merge them at the item's end (two-worker merge).  An item
// that lies within one share is written out; one that spans shares leaves a partial state for each
// in the workspace (at most two a CTA: its first and its last item), and the combine kernel merges
// them in a fixed order.
//
// Streams.  Each warp keeps its own ring of kStages tiles in shared memory, filled by its lanes'
// asynchronous 16-byte copies and running on from one item into the next; nothing but the warp
// itself waits for it.  (TMA boxes of a page's 16 rows in its place: 61 us on the bf16 case below,
// 46 with the copies at that stage: the box-by-box issue cost as many instructions as the rest of a
// tile.)  Rows are swizzled, chunk by chunk of 16 bytes, so that ldmatrix meets no bank conflict.
//
// Products (mma m16n8k16, fp32 out), with keys and values as the 16-row operand and the queries as
// the 8 columns, so that 8 query rows waste nothing:
//   S^T = K Q^T   16 tokens x 8 rows; ldmatrix gives lane (g, t) of K's operand token g's bytes
//   O^T += V^T P^T   16 of d x 8 rows; ldmatrix.trans gives it the token pair (2t, 2t + 1)
// (lane = 4 g + t).  P^T comes from S^T by a transpose within the warp (movmatrix).
//
// 4 bits.  What bounds the kernel there is the work on each value, not the memory: the integer pipe
// takes two warp instructions a cycle and an SM.  So a register of 8 codes goes into the product
// with as few as possible: masked with 0x000f000f and 0x00f000f0, and the same of the register
// shifted by 8, the codes are subnormal fp16 numbers, code * 2^-24 and code * 2^-20.  The tensor
// cores multiply them exactly, but align the 16 products of an instruction as if their exponents
// were -14 and drop what lies more than 25 bits below the largest: 2^-15 of code 1 times the
// largest other factor, far below the quantiser's half step.  (Codes ten bits higher would need a
// shift each.)
//   K: the queries' operand has the same order of d, and 1/16 of the odd values.  It is scaled by a
//   power of two a row so that bf16 queries fit fp16: values down to 2^-26 of the row's largest
//   are exact, those below are off by at most 2^-34 of it (rows of 2^116 and more overflow).  Per
//   group of 64 values S = s (sum q code + b sum q): step and base enter after the product.
//   V: the token's step multiplies its share (one set of P a group), O = sum (p s) code +
//   sum (p s) b; the second sum is one more product, with the bases as the rows, so that both have
//   the same rounded p s and an error in it counts with the value, not with the code.  p s is
//   rounded to fp16 relative to the largest step so far of the group's tokens that all rows see,
//   scaled to 2^7 (p <= 2^8): 2^-11 of itself down to 2^-20 of that step, 2^-31 of that step below.
//   (Larger steps of tokens that only some rows see: read_words.)
// Each lane takes one token's words a tile and leaves steps and bases in shared memory as the
// products want them.
//
// Measured (both kernels, inputs beyond L2): one query of 4 heads on each of 8 heads of 8 sequences
// of 32768 4-bit tokens, d = 128: 62.7 us, 4.5 TB/s (67 % of a copy's); 24 bf16 sequences of up to
// 8191, d = 64: 39.4 us, 5.2 TB/s (77 %).  At 4 bits a tile of 64 tokens x 8 rows costs 910 warp
// instructions, a third of them shifts and masks; the schedulers issue in 45 % of their cycles, with
// two warps each to choose from, waiting on the instruction before more than on memory.  Rows in
// blocks of 16 read and mask the tile anew for each block: 16 sequences of 40 rows on up to 6001
// tokens take 30 us, eight times what their bytes need.  (One tile for 64 rows, expanded to bf16 in
// shared memory once, 16 rows a warp: 43 to 51 us, with two barriers a tile and one chain of
// products a warp.)
#include <cuda_runtime.h>

#include <cmath>

#include "fa_shared.cuh"
#include "kv_cache.cuh"
#include "osm_internal.h"
#include "per_device.h"
#include "ptx_sm103.cuh"

namespace osm {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kMoveThreshold = 8.f;  // log2 units: the reference max moves only past this
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;

// Tokens a tile.  4 bits: 64 for 8 rows (62.8 us on the first case above, 68.7 at 32), 32 for 16 (64
// measured the same: 64 rows a head on 2 x 16384 tokens 52 us).  bf16: 16 at d = 128 and 32 at d = 64
// (39.1 us on the second case, 40.6 at 16); twice that does not fit shared memory with two CTAs an
// SM.
constexpr int tile_of(int64_t d, int format, int rows) {
    return format == OSM_KV_BF16 ? (d == 128 ? 16 : 32) : (rows == 8 ? 64 : 32);
}

constexpr int kCtasPerSm = 2;  // 8 warps an SM, up to 255 registers a thread

template <int D, int FMT, int NT>
struct Cfg {
    static constexpr bool kInt4 = FMT == OSM_KV_INT4;
    static constexpr int kRows = 8 * NT;
    static constexpr int kT = tile_of(D, FMT, kRows);          // tokens a tile
    static constexpr int kHalves = kT / 16;
    static constexpr int kG = kInt4 ? D / kKvGroup : 1;        // groups
    static constexpr int kRowBytes = kInt4 ? D / 2 : D * 2;
    static constexpr int kChunks = kRowBytes / 16;             // 16-byte chunks a row
    static constexpr int kRowsPer = 32 / kChunks;              // rows a warp-wide copy takes
    static constexpr int kBody = kT * kRowBytes;               // K or V of a tile
    static constexpr int kWord = kInt4 ? kT * kG * 2 : 0;      // words of K or V
    static constexpr int kStageBytes = 2 * kBody;
    // Two tiles on their way a warp cover the memory's latency with 8 warps an SM (three and four
    // measured the same).
    static constexpr int kStages = 2;
    // a tile's records, for each token and group: K's step and base and V's scaled step, each twice
    // (for arithmetic on pairs), then V's bases (fp16, token after token, group after group)
    static constexpr int kRecK = kInt4 ? kT * kG * 16 : 0;
    static constexpr int kRecV = kInt4 ? kT * kG * 8 : 0;
    static constexpr int kRec = kRecK + kRecV + (kInt4 ? kT * kG * 2 : 0);
    // shared memory: [warp][stage] bodies, [warp][stage] words, the warps' O for the merge (with
    // the warp's records in its place while it works), (m, l), the rows' places
    static constexpr int kWordAt = kWarps * kStages * kStageBytes;
    static constexpr int kOStride = D + 4;
    static constexpr int kOAt = kWordAt + kWarps * kStages * 2 * kWord;
    static constexpr int kOBytes =
        kRows * kOStride * 4 > kRec ? kRows * kOStride * 4 : kRec;
    static constexpr int kMlAt = kOAt + kWarps * kOBytes;
    static constexpr int kRowAt = kMlAt + 2 * kWarps * kRows * 4;
    // 4 bits: the tokens left out of the products (see read_words): for the item, each group and
    // token, the stamp of the item that set it; then the tokens' scores for the rows
    static constexpr int kAsideAt = kRowAt + 2 * kRows * 4;
    static constexpr int kAside = kInt4 ? 1 + kG * kRows : 0;
    static constexpr int kBytes = kAsideAt + (kInt4 ? (kAside + kRows * kRows) * 4 : 0);
    static constexpr int kDyn = kBytes + 128;  // slack for 128-byte alignment
    static_assert(kCtasPerSm * (kDyn + 1024) <= 228 * 1024, "shared memory budget");
};

struct PagedParams {
    const __nv_bfloat16* Q;  // [B, H, Nq, d]
    __nv_bfloat16* O;
    float* LSE;  // [B, H, Nq] or nullptr
    float* ws;   // [ctas][2][kRows][D + 2]: partial O, m, l
    const int32_t *kv_lens, *q_lens;
    int B, H, Nq, causal;
    int group;             // H / H_kv
    int rows, row_blocks;  // group * Nq rows a key/value head, in blocks of kRows
    const int32_t* only;  // or nullptr: the sequences to compute (the others' outputs stay)
    float scale_log2;
    int page_div, page_rem;  // kWarps tiles in pages and tokens
    uint32_t page_bytes;     // all heads of a page
    KvPages pg;
    // SHARED kernels: the sequences' common tokens, which the prefix kernel has taken, and where an
    // item within one share leaves its rows' states
    const ShSeq* seqs;
    float* row_o;      // [B * H * Nq][D]
    float2* row_ml;    // [B * H * Nq]
    const ShHead* head;
};

// ------------------------------------------------------------------------------------------
// PTX
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// 16 bytes from global to shared memory, or 16 zero bytes (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool real) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(real ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void lds64(uint32_t addr, uint32_t& a, uint32_t& b) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t a;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(a) : "r"(addr) : "memory");
    return a;
}
__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void sts_f4(uint32_t addr, float x, float y, float z, float w) {
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(x), "f"(y), "f"(z),
                 "f"(w)
                 : "memory");
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t x) {
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(static_cast<uint16_t>(x)) : "memory");
}
__device__ __forceinline__ void sts_f2(uint32_t addr, float x, float y) {
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ float2 lds_f2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
    uint16_t a;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(a) : "r"(addr) : "memory");
    return a;
}

// Step and base (as a float) of the lower (HI = false) or upper word of a register.
template <bool HI>
__device__ __forceinline__ float word_step(uint32_t w) {
    return __uint_as_float(HI ? (w & 0xffc00000u) >> 1 : (w & 0xffc0u) << 15);
}
template <bool HI>
__device__ __forceinline__ float word_base(uint32_t w) {
    const uint32_t x = HI ? w >> 16 : w;
    return __uint_as_float((x & 63u) ^ 0x4b000020u) - (8388608.f + 32.f);  // 2^23 + (base + 32)
}

// Steps below 2^(e - 126) (e: their largest biased exponent) times 2^(133 - e) are below 2^7.
__device__ __forceinline__ float step_scale(int e) {
    return __uint_as_float(static_cast<uint32_t>(min(260 - e, 227)) << 23);
}
__device__ __forceinline__ float step_unscale(int e) {  // 1 / step_scale(e)
    return __uint_as_float(static_cast<uint32_t>(254 - min(260 - e, 227)) << 23);
}

// Byte offset of 16-byte chunk c of row r of BYTES bytes: the chunk's place within 128 bytes is
// exchanged so that eight rows' chunks c lie in eight different groups of banks.
template <int BYTES>
__device__ __forceinline__ int swz(int r, int c) {
    if (BYTES >= 128) return r * BYTES + ((c ^ (r & 7)) << 4);
    if (BYTES == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    return r * 32 + ((c ^ ((r >> 2) & 1)) << 4);
}
// The same for row r0 + j * ROWS and a chunk, from the offset of row r0 < ROWS (ROWS rows are 512
// bytes).
template <int BYTES>
__device__ __forceinline__ uint32_t swz_step(uint32_t at, int j) {
    const int x = BYTES == 128 ? (j & 1) << 6 : (BYTES == 256 ? (j & 3) << 5 : 0);
    return (at + j * 512) ^ x;
}

// ------------------------------------------------------------------------------------------
// The shares
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ int seq_len(const PagedParams& p, int b) {
    if (p.only && !p.only[b]) return 0;
    const long long room = static_cast<long long>(p.pg.max_pages) * p.pg.page;
    return static_cast<int>(min(static_cast<long long>(max(p.kv_lens[b], 0)), room));
}

// Row blocks of a sequence that hold a query (the blocks of padding rows behind have no items).
template <int ROWS>
__device__ __forceinline__ int seq_blocks(const PagedParams& p, int b) {
    if (!p.q_lens) return p.row_blocks;
    const int ql = min(max(p.q_lens[b], 0), p.Nq);
    return (ql * p.group + ROWS - 1) / ROWS;
}

// E: units of an item in front of its tiles, 0 unless SHARED (see kOwnItemUnits in fa_shared.cuh).
// SHARED: the first tile of sequence b's own.  (Reads of the plan pass the L1 by: this kernel may start
// before the one in front of it, which has waited for the plan, ends.)
template <int T, int E>
__device__ __forceinline__ int seq_lo(const PagedParams& p, int b) {
    if constexpr (E > 0) return __ldcg(&p.seqs[b].skip) / T;
    else return 0;
}

// Units (a tile of an item is one) of sequence b.
template <int ROWS, int T, int E>
__device__ __forceinline__ long long seq_units(const PagedParams& p, int b) {
    const int tiles = (seq_len(p, b) + T - 1) / T - seq_lo<T, E>(p, b);
    return static_cast<long long>(tiles > 0 ? tiles + E : 0) * p.pg.H_kv *
           seq_blocks<ROWS>(p, b);
}

// The units of all sequences (a whole warp).
template <int ROWS, int T, int E>
__device__ __forceinline__ long long all_units(const PagedParams& p) {
    const int lane = threadIdx.x & 31;
    long long n = 0;
    for (int b = lane; b < p.B; b += 32) n += seq_units<ROWS, T, E>(p, b);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) n += __shfl_xor_sync(0xffffffffu, n, m);
    return n;
}

// Tiles that a CTA takes: at least one a warp.
__device__ __forceinline__ long long share_of(long long units, int ctas) {
    const long long s = (units + ctas - 1) / ctas;
    return s > kWarps ? s : kWarps;
}

// A CTA's walk through the items of its share.  An item is tiles [t0, t1) of item `it` (key/value
// head and row block) of sequence b, which has the tiles lo .. tiles - 1 (lo: 0 unless SHARED); all
// fields are the same in every thread.  A share may begin or end within the units in front of an
// item's tiles: the item is then the CTA's that has its first tile.
template <int ROWS, int T, int E>
struct Segment {
    int b, len, lo, tiles, blocks;  // sequence, its length, tiles and row blocks
    int kvh, block;             // the item's key/value head and row block
    int t0, t1;
    int left;  // units of the share from this segment's start on
    int took;  // of them this segment's (E > 0)

    // The segment from the item's unit `from` on.
    __device__ __forceinline__ void cut(int from) {
        took = min(tiles - lo + E - from, left);
        const int to = from + took;
        t0 = lo + max(from - E, 0);
        t1 = lo + max(to - E, 0);
        if (E > 0 && t1 == t0) left = 0;  // (the share ends in front of the item's tiles)
    }
    __device__ __forceinline__ void start(const PagedParams& p, long long u0, long long u1) {
        const int lane = threadIdx.x & 31;
        left = static_cast<int>(u1 - u0);
        b = p.B;
        kvh = block = t0 = t1 = lo = tiles = len = blocks = took = 0;
        if (left <= 0) return;
        // the sequence that holds unit u0: 32 sequences at a time
        long long base = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const long long n = b0 + lane < p.B ? seq_units<ROWS, T, E>(p, b0 + lane) : 0;
            long long inc = n;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const long long o = __shfl_up_sync(0xffffffffu, inc, m);
                if (lane >= m) inc += o;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, base + inc > u0);
            if (hit) {
                const int src = __ffs(hit) - 1;
                b = b0 + src;
                const long long before = __shfl_sync(0xffffffffu, base + inc - n, src);
                len = seq_len(p, b);
                lo = seq_lo<T, E>(p, b);
                tiles = (len + T - 1) / T;
                blocks = seq_blocks<ROWS>(p, b);
                const long long r = u0 - before;
                const int per = tiles - lo + E;
                const int it = static_cast<int>(r / per);
                kvh = it / blocks;
                block = it - kvh * blocks;
                cut(static_cast<int>(r - static_cast<long long>(it) * per));
                break;
            }
            base += __shfl_sync(0xffffffffu, inc, 31);
        }
    }
    __device__ __forceinline__ bool done() const { return left <= 0; }
    __device__ __forceinline__ void next(const PagedParams& p) {
        left -= E > 0 ? took : t1 - t0;
        if (left <= 0) return;
        if (++block == blocks) {
            block = 0;
            if (++kvh == p.pg.H_kv) {
                kvh = 0;
                do {
                    len = seq_len(p, ++b);
                    blocks = seq_blocks<ROWS>(p, b);
                } while (len == 0 || blocks == 0);
                lo = seq_lo<T, E>(p, b);
                tiles = (len + T - 1) / T;
            }
        }
        cut(0);
    }
};

// A row of an item's list: its query head and query, and the last key it sees (below 0: none; what
// the kernel computes for such a row is not used, and it masks no tile for its sake).
struct RowPlace {
    int head, i, last;
};
__device__ __forceinline__ RowPlace row_place(const PagedParams& p, int b, int kvh, int row,
                                              int len) {
    RowPlace r;
    r.i = row / p.group;
    r.head = kvh * p.group + row - r.i * p.group;
    const int ql = p.q_lens ? min(max(p.q_lens[b], 0), p.Nq) : p.Nq;
    r.last = p.causal ? len - ql + r.i : len - 1;
    if (row >= p.rows || r.i >= ql) r.last = -1;
    return r;
}

// SHARED: over the tokens behind each sequence's common ones; every item leaves its rows' states, and the
// kernel that joins them with the common tokens' writes O and LSE.
template <int D, int FMT, int NT, bool SHARED>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    paged_kernel(const PagedParams p) {
    using C = Cfg<D, FMT, NT>;
    constexpr int T = C::kT, RB = C::kRowBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStageBytes;
    const uint32_t words = smem_u32(smem) + C::kWordAt + warp * C::kStages * 2 * C::kWord;
    const uint32_t rec = smem_u32(smem) + C::kOAt + warp * C::kOBytes;
    float* sO = reinterpret_cast<float*>(smem + C::kOAt);
    float* sM = reinterpret_cast<float*>(smem + C::kMlAt);
    float* sL = sM + kWarps * C::kRows;
    int* sAt = reinterpret_cast<int*>(smem + C::kRowAt);  // the rows' places in O, whether they see a key
    int* sSees = sAt + C::kRows;
    // [0]: whether the item has tokens aside; [1 + group * kRows + i]: whether token min_last + 1 + i
    // is one.  An item's stamp is what is left of the share (at least 1, another for each item).
    int* sAside = reinterpret_cast<int*>(smem + C::kAsideAt);
    float* sScore = reinterpret_cast<float*>(sAside + C::kAside);  // [i][row], log2 units
    asm volatile("griddepcontrol.launch_dependents;");

    long long units, share;
    if constexpr (SHARED) {
        units = __ldcg(&p.head->own_units), share = __ldcg(&p.head->own_share);
    } else {
        units = all_units<C::kRows, T, 0>(p), share = share_of(units, gridDim.x);
    }
    const long long u0 = share * blockIdx.x;
    const long long u1 = min(units, u0 + share);

    // ------------------------------------------------------------------ the warp's ring
    // The issuing walk runs kStages tiles ahead of the consuming one; both visit, segment by
    // segment, the tiles t0 + warp, t0 + warp + 4, ...  A tile's 16-token halves ("boxes") each lie
    // in one page; the page ids are read one tile before they are needed.
    using Seg = Segment<C::kRows, T, SHARED ? kOwnItemUnits : 0>;
    Seg ahead;
    ahead.start(p, u0, u1);
    Seg seg = ahead;
    int ahead_t = ahead.t0 + warp;
    int at = 0;                      // place of the tile's first token in its page
    const int32_t* entry = nullptr;  // that page's entry of the table
    int32_t id[C::kHalves];          // pages of its boxes (-1: no tokens, or no page)
    uint32_t hides = 0;              // boxes without a page, a bit each, of the tiles in flight
    int in_flight = 0, fill = 0;
    const bool one_page = T == 16 || p.pg.page % T == 0;  // a tile never crosses pages
    const uint32_t num_pages = static_cast<uint32_t>(p.pg.num_pages);
    const int r0 = lane / C::kChunks;  // this lane's row and chunk of a warp-wide copy
    const uint32_t lane_dst = swz<RB>(r0, lane % C::kChunks);
    // Words: 16 bytes a lane, those of K by the first W lanes, of V by the next W; the first half
    // of them belongs to the first box.
    constexpr int W = C::kInt4 ? C::kWord / 16 : 2;
    const int64_t v_from_k = p.pg.v - p.pg.k;
    const uint8_t* src = nullptr;    // this lane's chunk of place 0 of the head's keys, page 0
    const uint8_t* w_src = nullptr;  // this lane's words of place 0 of the head, page 0

    // The page ids of the issuing walk's tile.
    auto read_ids = [&]() {
        if (one_page) {
            id[0] = entry[0];
#pragma unroll
            for (int h = 1; h < C::kHalves; ++h) id[h] = id[0];
            return;
        }
        const int rem = ahead.len - ahead_t * T;
        int a = at;
        const int32_t* e = entry;
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h) {
            id[h] = -1;
            if (16 * h < rem) id[h] = *e;
            a += 16;
            if (a >= p.pg.page) {
                a -= p.pg.page;
                ++e;
            }
        }
    };
    // The issuing walk is past its segment's last tile of this warp, or has just begun: on to the
    // next segment that has one.
    auto settle = [&]() {
        while (!ahead.done() && ahead_t >= ahead.t1) {
            ahead.next(p);
            ahead_t = ahead.t0 + warp;
        }
        if (ahead.done()) return;
        const int pi = ahead_t * T / p.pg.page;
        at = ahead_t * T - pi * p.pg.page;
        entry = p.pg.table + static_cast<int64_t>(ahead.b) * p.pg.max_pages + pi;
        const int64_t head = ahead.kvh * p.pg.head_bytes;
        src = p.pg.k + head + r0 * RB + lane % C::kChunks * 16;
        w_src = (lane < W ? p.pg.k : p.pg.v) + head +
                static_cast<int64_t>(p.pg.page) * (D / 2) + lane % W * 16;
        read_ids();
    };
    // Source of a box (its first token at `place` of page `i`) and of its words.
    auto page_at = [&](const uint8_t* base, int32_t i, int place, int bytes) {
        return base + static_cast<uint64_t>(static_cast<uint32_t>(i)) * p.page_bytes +
               place * bytes;
    };
    auto issue = [&]() {
        if (!ahead.done()) {
            const uint32_t dst = ring + fill * C::kStageBytes + lane_dst;
            const uint32_t w_dst = words + 2 * fill * C::kWord + lane * 16;
            const int rem = ahead.len - ahead_t * T;  // tokens of the tile, from its first
            int place[C::kHalves];
            place[0] = at;
            bool good = true;
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h) {
                if (h > 0) {
                    place[h] = place[h - 1] + 16;
                    if (!one_page && place[h] >= p.pg.page) place[h] -= p.pg.page;
                }
                good &= static_cast<uint32_t>(id[h]) < num_pages;
            }
            const uint8_t* from[C::kHalves];
            // this lane's words: those of box w_box, the first of which is lane w_box * kPer
            constexpr int kPer = C::kInt4 ? W / C::kHalves : 1;
            const int w_box = lane % W / kPer;
            int32_t w_id = id[0];
            int w_place = place[0];
#pragma unroll
            for (int h = 1; h < C::kHalves; ++h)
                if (w_box == h) {
                    w_id = id[h];
                    w_place = place[h] - 16 * h;
                }
            if (rem >= T && good) {
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h)
                    from[h] = one_page && h > 0 ? from[0] + 16 * h * RB
                                                : page_at(src, id[h], place[h], RB);
#pragma unroll
                for (int j = 0; j < T / C::kRowsPer; ++j) {
                    const int row = j * C::kRowsPer;
                    copy16(swz_step<RB>(dst, j), from[row / 16] + row % 16 * RB);
                    copy16(swz_step<RB>(dst + C::kBody, j),
                           from[row / 16] + v_from_k + row % 16 * RB);
                }
                if constexpr (C::kInt4) {
                    if (lane < 2 * W)
                        copy16(w_dst, page_at(w_src, one_page ? id[0] : w_id,
                                              one_page ? place[0] : w_place, C::kG * 2));
                }
            } else {
                // zeros for tokens behind the sequence and for boxes without a page
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h) {
                    const bool paged = static_cast<uint32_t>(id[h]) < num_pages;
                    from[h] = paged ? page_at(src, id[h], place[h], RB) : src;
                    if (!paged && 16 * h < rem) {
                        hides |= 1u << (C::kHalves * in_flight + h);
                        if (lane == 0) kv_bad_page(p.pg);
                    }
                }
#pragma unroll
                for (int j = 0; j < T / C::kRowsPer; ++j) {
                    const int row = j * C::kRowsPer;
                    const bool real =
                        static_cast<uint32_t>(id[row / 16]) < num_pages && row + r0 < rem;
                    const uint8_t* x = from[row / 16] + row % 16 * RB;
                    copy16_or_zero(swz_step<RB>(dst, j), x, real);
                    copy16_or_zero(swz_step<RB>(dst + C::kBody, j), x + v_from_k, real);
                }
                if constexpr (C::kInt4) {
                    if (lane < 2 * W) {
                        const bool real = static_cast<uint32_t>(w_id) < num_pages &&
                                          lane % W * (8 / C::kG) < rem;
                        copy16_or_zero(w_dst,
                                       real ? page_at(w_src, w_id, w_place, C::kG * 2) : w_src,
                                       real);
                    }
                }
            }
            ++in_flight;
            fill = fill == C::kStages - 1 ? 0 : fill + 1;
            // on to the warp's next tile
            ahead_t += kWarps;
            if (ahead_t >= ahead.t1) {
                settle();
            } else {
                entry += p.page_div;
                at += p.page_rem;
                if (at >= p.pg.page) {
                    at -= p.pg.page;
                    ++entry;
                }
                read_ids();
            }
        }
        copies_commit();
    };
    settle();
    for (int s = 0; s < C::kStages; ++s) issue();
    int slot = 0;  // the slot consumed next
    if constexpr (C::kInt4) {
        if (threadIdx.x < C::kAside) sAside[threadIdx.x] = 0;
        __syncthreads();
    }

    // ------------------------------------------------------------------ segment by segment
    for (; !seg.done(); seg.next(p)) {
        const int kvh = seg.kvh, row0 = seg.block * C::kRows;
        // The queries' operand, and (4 bits) the sums over each group of values and the factor
        // from the products to scores in log2 units.
        uint32_t qf[NT][D / 16][2];
        float qsum[NT][C::kG][2], cs[NT][2];
        int last[NT][2], min_last = 0x7fffffff;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = row0 + n * 8 + g;
            const RowPlace rp = row_place(p, seg.b, kvh, row, seg.len);
            const bool real = row < p.rows;
            const __nv_bfloat16* q =
                p.Q + ((static_cast<int64_t>(seg.b) * p.H + (real ? rp.head : 0)) * p.Nq +
                       (real ? rp.i : 0)) * D;
            if constexpr (C::kInt4) {
                uint4 x[D / 32];
                float top = 0.f;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    x[c] = make_uint4(0u, 0u, 0u, 0u);
                    if (real) x[c] = *reinterpret_cast<const uint4*>(q + c * 32 + t * 8);
                    const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        top = max_nan(top, max_nan(fabsf(__uint_as_float(w[e] << 16)),
                                                   fabsf(__uint_as_float(w[e] & 0xffff0000u))));
                }
                top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // 2^f brings the row's largest value into [2^13, 2^14)
                int f = 13 + 127 - static_cast<int>(__float_as_uint(top) >> 23);
                f = min(max(f, -100), 100);
                const float up = __uint_as_float(static_cast<uint32_t>(f + 127) << 23);
                float sum[C::kG] = {};
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[2 * e] = __uint_as_float(w[e] << 16) * up;
                        v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u) * up;
                        sum[c / 2] += v[2 * e] + v[2 * e + 1];
                    }
                    qf[n][2 * c][0] = pack_f16x2(v[0], v[4]);
                    qf[n][2 * c][1] = pack_f16x2(v[1] * 0.0625f, v[5] * 0.0625f);
                    qf[n][2 * c + 1][0] = pack_f16x2(v[2], v[6]);
                    qf[n][2 * c + 1][1] = pack_f16x2(v[3] * 0.0625f, v[7] * 0.0625f);
                }
#pragma unroll
                for (int k = 0; k < C::kG; ++k) {
                    float s = sum[k] * 5.9604644775390625e-8f;  // 2^-24, as the codes
                    s += __shfl_xor_sync(0xffffffffu, s, 1);
                    s += __shfl_xor_sync(0xffffffffu, s, 2);
                    qsum[n][k][0] = __shfl_sync(0xffffffffu, s, 8 * t);      // g = 2 t
                    qsum[n][k][1] = __shfl_sync(0xffffffffu, s, 8 * t + 4);  // g = 2 t + 1
                }
                const float down =
                    p.scale_log2 * __uint_as_float(static_cast<uint32_t>(24 - f + 127) << 23);
                cs[n][0] = __shfl_sync(0xffffffffu, down, 8 * t);
                cs[n][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
            } else {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    qf[n][k][0] = real ? *reinterpret_cast<const uint32_t*>(q + k * 16 + 2 * t) : 0u;
                    qf[n][k][1] =
                        real ? *reinterpret_cast<const uint32_t*>(q + k * 16 + 8 + 2 * t) : 0u;
                }
                cs[n][0] = cs[n][1] = p.scale_log2;
            }
            const int mine = rp.last;
            last[n][0] = __shfl_sync(0xffffffffu, mine, 8 * t);
            last[n][1] = __shfl_sync(0xffffffffu, mine, 8 * t + 4);
            if (mine >= 0) min_last = min(min_last, mine);
        }
        min_last = __reduce_min_sync(0xffffffffu, min_last);

        float acc[NT][D / 16][4], m[NT][2], l[NT][2];
        float side[NT][C::kG][4];  // 4 bits: sum of (p s) b, each row the same
        int top_e[C::kG];          // 4 bits: largest biased exponent of a step of V so far
        float scale[C::kG];        // its step_scale
#pragma unroll
        for (int k = 0; k < C::kG; ++k) {
            top_e[k] = 0;
            scale[k] = step_scale(0);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[n][k][e] = 0.f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int k = 0; k < C::kG; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) side[n][k][e] = 0.f;
        }

        // A tile's words, a token a lane, into the warp's records.  Behind the sequence they are
        // whatever the page holds: zeros in their place.
        // The scale of V's steps is shared by the rows, so a token that some rows do not see must
        // not raise it: its step may be any number of times those that they see (or NaN), and their
        // shares would round to nothing (or to NaN, a share of 0 too).  Where it would, its step is
        // taken out of the products, and the rows that see the token (fewer than kRows tokens lie
        // between the first and the last row's last key) get it value by value in the merge.
        auto read_words = [&](int tile, bool masked) {
            float v_step[(T + 31) / 32][C::kG];
            bool grows = false;
            auto exponent = [&](int i, int k) {
                return static_cast<int>(__float_as_uint(v_step[i][k]) >> 23);
            };
#pragma unroll
            for (int i = 0; i < T / 32; ++i) {
                const int at_lane = 32 * i + lane;
                const uint32_t w = words + 2 * slot * C::kWord + at_lane * (C::kG * 2);
                uint32_t wk = C::kG == 2 ? lds32(w) : lds16(w);
                uint32_t wv = C::kG == 2 ? lds32(w + C::kWord) : lds16(w + C::kWord);
                if (masked) {
                    const bool in = tile * T + at_lane < seg.len;
                    wk = in ? wk : 0u;
                    wv = in ? wv : 0u;
                }
                const uint32_t rk = rec + at_lane * (C::kG * 16);
                const uint32_t rb = rec + C::kRecK + C::kRecV + at_lane * 2;
                const float k0 = word_step<false>(wk), b0 = word_base<false>(wk);
                sts_f4(rk, k0, k0, b0, b0);
                v_step[i][0] = word_step<false>(wv);
                if constexpr (C::kG == 2) {
                    const float k1 = word_step<true>(wk), b1 = word_base<true>(wk);
                    sts_f4(rk + 16, k1, k1, b1, b1);
                    v_step[i][1] = word_step<true>(wv);
                    const uint32_t b2 = pack_f16x2(word_base<false>(wv), word_base<true>(wv));
                    sts16(rb, b2);
                    sts16(rb + T * 2, b2 >> 16);
                } else {
                    sts16(rb, pack_f16x2(word_base<false>(wv), 0.f));
                }
#pragma unroll
                for (int k = 0; k < C::kG; ++k)
                    grows |= exponent(i, k) > top_e[k];  // a NaN group (255) comes by here too
            }
            if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                for (int k = 0; k < C::kG; ++k) {
                    int e_top = 0;
#pragma unroll
                    for (int i = 0; i < T / 32; ++i)
                        if (exponent(i, k) != 255 && tile * T + 32 * i + lane <= min_last)
                            e_top = max(e_top, exponent(i, k));
                    const int up = max(top_e[k], __reduce_max_sync(0xffffffffu, e_top));
                    const float f = step_scale(up) * step_unscale(top_e[k]);
                    top_e[k] = up;
                    scale[k] = step_scale(up);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            side[n][k][x] *= f;
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[n][4 * k + i][x] *= f;
                        }
                }
                if (masked) {
                    int max_last = -1;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        max_last = max(max_last, max(last[n][0], last[n][1]));
                    max_last = __reduce_max_sync(0xffffffffu, max_last);
#pragma unroll
                    for (int i = 0; i < T / 32; ++i)
#pragma unroll
                        for (int k = 0; k < C::kG; ++k) {
                            const int tok = tile * T + 32 * i + lane;
                            if (tok <= min_last || exponent(i, k) <= top_e[k]) continue;
                            v_step[i][k] = 0.f;
                            if (tok > max_last) continue;
                            sAside[0] = seg.left;
                            sAside[1 + k * C::kRows + tok - min_last - 1] = seg.left;
                        }
                }
            }
#pragma unroll
            for (int i = 0; i < T / 32; ++i) {
                const uint32_t rv = rec + C::kRecK + (32 * i + lane) * (C::kG * 8);
                const float v0 = v_step[i][0] * scale[0];
                if constexpr (C::kG == 2) {
                    const float v1 = v_step[i][1] * scale[1];
                    sts_f4(rv, v0, v0, v1, v1);
                } else {
                    sts_f2(rv, v0, v0);
                }
            }
            __syncwarp();
        };
        // The products S of a tile with the queries: s[n][h][e] of tokens 16 h + g (e = 0, 1) and
        // 16 h + g + 8 (e = 2, 3), rows 2 t and 2 t + 1.
        auto products = [&](float (&s)[NT][C::kHalves][4]) {
            const uint32_t sk = ring + slot * C::kStageBytes;
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h) {
                if constexpr (C::kInt4) {
                    float part[C::kG][NT][4];
#pragma unroll
                    for (int k = 0; k < C::kG; ++k)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) part[k][n][e] = 0.f;
#pragma unroll
                    for (int c2 = 0; c2 < D / 64; ++c2) {
                        // matrices: chunk 2 c2 tokens 0-7, 8-15, chunk 2 c2 + 1 tokens 0-7, 8-15
                        uint32_t x[4];
                        const int row = 16 * h + (lane & 15), ch = 2 * c2 + (lane >> 4);
                        ldsm_x4(sk + swz<RB>(row, ch), x);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t lo = x[2 * j], hi = x[2 * j + 1];
                            const uint32_t l8 = lo >> 8, h8 = hi >> 8;
                            const int ks = 2 * (2 * c2 + j);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                mma_f16(part[c2][n], lo & 0x000f000fu, hi & 0x000f000fu,
                                        lo & 0x00f000f0u, hi & 0x00f000f0u, qf[n][ks][0],
                                        qf[n][ks][1]);
                                mma_f16(part[c2][n], l8 & 0x000f000fu, h8 & 0x000f000fu,
                                        l8 & 0x00f000f0u, h8 & 0x00f000f0u, qf[n][ks + 1][0],
                                        qf[n][ks + 1][1]);
                            }
                        }
                    }
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float4 rk[C::kG];  // step, step, base, base
#pragma unroll
                        for (int k = 0; k < C::kG; ++k)
                            rk[k] = lds_f4(rec + ((16 * h + g + 8 * r) * C::kG + k) * 16);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float2 x = make_float2(0.f, 0.f);
#pragma unroll
                            for (int k = 0; k < C::kG; ++k)
                                x = ffma2(make_float2(rk[k].x, rk[k].y),
                                          ffma2(make_float2(rk[k].z, rk[k].w),
                                                make_float2(qsum[n][k][0], qsum[n][k][1]),
                                                make_float2(part[k][n][2 * r],
                                                            part[k][n][2 * r + 1])),
                                          x);
                            s[n][h][2 * r] = x.x;
                            s[n][h][2 * r + 1] = x.y;
                        }
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[n][h][e] = 0.f;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {  // 16 values: chunks 2 k and 2 k + 1
                        uint32_t x[4];
                        const int row = 16 * h + (lane & 15), ch = 2 * k + (lane >> 4);
                        ldsm_x4(sk + swz<RB>(row, ch), x);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma16816(s[n][h], x[0], x[1], x[2], x[3], qf[n][k][0], qf[n][k][1]);
                    }
                }
            }
        };

        for (int tile = seg.t0 + warp; tile < seg.t1; tile += kWarps) {
            copies_wait<C::kStages - 1>();
            __syncwarp();
            const int tok0 = tile * T;
            const uint32_t hide = hides & ((1u << C::kHalves) - 1u);
            hides >>= C::kHalves;
            --in_flight;
            const bool masked = hide != 0 || tok0 + T - 1 > min_last;
            if constexpr (C::kInt4) read_words(tile, masked);
            float sc[NT][C::kHalves][4];
            products(sc);
            if (masked) {
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h) {
                    const bool gone = (hide >> h) & 1;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (gone || tok0 + 16 * h + g + 8 * (e >> 1) > last[n][e & 1])
                                sc[n][h][e] = -INFINITY;
                }
                if constexpr (C::kInt4) {
                    if (sAside[0] == seg.left) {  // by this warp's tile or another's
#pragma unroll
                        for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int i = tok0 + 16 * h + g + 8 * (e >> 1) - min_last - 1;
                                if (i < 0 || i >= C::kRows) continue;
#pragma unroll
                                for (int n = 0; n < NT; ++n)
                                    sScore[i * C::kRows + n * 8 + 2 * t + (e & 1)] =
                                        sc[n][h][e] * cs[n][e & 1];
                            }
                    }
                }
            }
            const uint32_t sv = ring + slot * C::kStageBytes + C::kBody;

            // ---- the reference max moves only when a score passes it by the threshold
            bool moves = false;
            float top[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(sc[n][0][e], sc[n][0][e + 2]);
#pragma unroll
                    for (int h = 1; h < C::kHalves; ++h)
                        x = fmaxf(x, fmaxf(sc[n][h][e], sc[n][h][e + 2]));
                    top[n][e] = x * cs[n][e];
                    moves |= top[n][e] - m[n][e] > kMoveThreshold;
                }
            if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = top[n][e];
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1)
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                        const float mn = fmaxf(m[n][e], x);
                        const float a = mn == m[n][e] ? 1.f : ex2_approx(m[n][e] - mn);
                        m[n][e] = mn;
                        l[n][e] *= a;
#pragma unroll
                        for (int k = 0; k < C::kG; ++k) side[n][k][e] *= a;
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            acc[n][k][e] *= a;
                            acc[n][k][e + 2] *= a;
                        }
                    }
            }
            // ---- shares
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 c2 = make_float2(cs[n][0], cs[n][1]);
                const float2 ref = make_float2(m[n][0] == -INFINITY ? 0.f : -m[n][0],
                                               m[n][1] == -INFINITY ? 0.f : -m[n][1]);
                float2 sum = make_float2(l[n][0], l[n][1]);
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float2 x = ffma2(make_float2(sc[n][h][2 * r], sc[n][h][2 * r + 1]), c2, ref);
                        x.x = ex2_approx(x.x);
                        x.y = ex2_approx(x.y);
                        sc[n][h][2 * r] = x.x;
                        sc[n][h][2 * r + 1] = x.y;
                        sum = fadd2(sum, x);
                    }
                l[n][0] = sum.x;
                l[n][1] = sum.y;
            }

            if constexpr (!C::kInt4) {
                if (masked) {
                    // A token that is hidden from some of the queries (causal) and holds a NaN or an
                    // infinity in its values is added for the queries that see it value by value,
                    // and cleared: in the product a share of 0 would make it NaN for the others.
                    // (Tokens behind the sequence were never copied: they are zeros.)
                    for (int j = max(0, min(min_last, tok0 + T) + 1 - tok0);
                         j < min(T, seg.len - tok0); ++j) {
                        constexpr int kMine = C::kChunks;  // chunks of the row, one a lane
                        const uint32_t place = sv + swz<RB>(j, lane % kMine);
                        bool wild = false;
                        if (lane < kMine) {
                            uint32_t v[4];
                            lds64(place, v[0], v[1]);
                            lds64(place + 8, v[2], v[3]);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                wild |= (v[e] & 0x7f80u) == 0x7f80u ||
                                        (v[e] & 0x7f800000u) == 0x7f800000u;
                        }
                        if (!__any_sync(0xffffffffu, wild)) continue;
                        const int hj = j >> 4, rj = (j >> 3) & 1, src = (j & 7) * 4 + t;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float share[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float x = 0.f;
#pragma unroll
                                for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
                                    for (int r = 0; r < 2; ++r)
                                        if (h == hj && r == rj) x = sc[n][h][e + 2 * r];
                                share[e] = __shfl_sync(0xffffffffu, x, src);
                            }
#pragma unroll
                            for (int k = 0; k < D / 8; ++k) {  // value 8 k + g
                                const float v =
                                    __uint_as_float(lds16(sv + swz<RB>(j, k) + 2 * g) << 16);
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (tok0 + j <= last[n][e])
                                        acc[n][k >> 1][2 * (k & 1) + e] += share[e] * v;
                            }
                        }
                        __syncwarp();
                        if (lane < kMine)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(place),
                                         "r"(0)
                                         : "memory");
                        __syncwarp();
                    }
                }
            }

            // ---- O^T += V^T P^T
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h) {
                if constexpr (C::kInt4) {
                    // shares times steps of the tokens g and g + 8, bases of the token pairs
                    uint32_t pf[C::kG][NT][2], base[C::kG][2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int row = 16 * h + g + 8 * r, pair = 16 * h + 2 * t + 8 * r;
                        float2 step[C::kG];  // twice the same
                        if constexpr (C::kG == 2) {
                            const float4 v = lds_f4(rec + C::kRecK + row * 16);
                            step[0] = make_float2(v.x, v.y);
                            step[1] = make_float2(v.z, v.w);
                        } else {
                            step[0] = lds_f2(rec + C::kRecK + row * 8);
                        }
#pragma unroll
                        for (int k = 0; k < C::kG; ++k)
                            base[k][r] = lds32(rec + C::kRecK + C::kRecV + (k * T + pair) * 2);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int k = 0; k < C::kG; ++k) {
                                const float2 x = fmul2(
                                    make_float2(sc[n][h][2 * r], sc[n][h][2 * r + 1]), step[k]);
                                pf[k][n][r] = transpose8x8(pack_f16x2(x.x, x.y));
                            }
                    }
#pragma unroll
                    for (int k = 0; k < C::kG; ++k)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma_f16(side[n][k], base[k][0], base[k][0], base[k][1], base[k][1],
                                    pf[k][n][0], pf[k][n][1]);
#pragma unroll
                    for (int c2 = 0; c2 < D / 64; ++c2) {
                        // matrices: chunk 2 c2 tokens 0-7, 8-15, chunk 2 c2 + 1 tokens 0-7, 8-15;
                        // a register holds values 4 g .. 4 g + 3 of the chunk's 32 for two tokens
                        uint32_t x[4];
                        const int row = 16 * h + (lane & 15), ch = 2 * c2 + (lane >> 4);
                        ldsm_x4_trans(sv + swz<RB>(row, ch), x);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t lo = x[2 * j], hi = x[2 * j + 1];
                            const uint32_t l8 = lo >> 8, h8 = hi >> 8;
                            const int mt = 2 * (2 * c2 + j);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                mma_f16(acc[n][mt], lo & 0x000f000fu, lo & 0x00f000f0u,
                                        hi & 0x000f000fu, hi & 0x00f000f0u, pf[c2][n][0],
                                        pf[c2][n][1]);
                                mma_f16(acc[n][mt + 1], l8 & 0x000f000fu, l8 & 0x00f000f0u,
                                        h8 & 0x000f000fu, h8 & 0x00f000f0u, pf[c2][n][0],
                                        pf[c2][n][1]);
                            }
                        }
                    }
                } else {
                    uint32_t pf[NT][2];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            pf[n][r] = transpose8x8(
                                pack_bf16x2(sc[n][h][2 * r], sc[n][h][2 * r + 1]));
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        // chunk 2 k tokens 0-7, chunk 2 k + 1 tokens 0-7, then tokens 8-15
                        uint32_t x[4];
                        const int row = 16 * h + (lane & 7) + 8 * (lane >> 4);
                        const int ch = 2 * k + ((lane >> 3) & 1);
                        ldsm_x4_trans(sv + swz<RB>(row, ch), x);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma16816(acc[n][k], x[0], x[1], x[2], x[3], pf[n][0], pf[n][1]);
                    }
                }
            }
            slot = slot == C::kStages - 1 ? 0 : slot + 1;
            __syncwarp();  // the slot has been read by every lane
            issue();
        }

        // ---------------------------------------------------------------- merge the four warps
        // Value of d that accumulator k's element pair `half` holds in this lane.
        auto value_of = [&](int k, int half) {
            return C::kInt4 ? (k >> 1) * 32 + 4 * g + 2 * (k & 1) + half : k * 16 + 8 * half + g;
        };
        const int active = min(kWarps, seg.t1 - seg.t0);  // warps that had a tile
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[n][e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                if (g == 0) {
                    sM[warp * C::kRows + n * 8 + 2 * t + e] = m[n][e];
                    sL[warp * C::kRows + n * 8 + 2 * t + e] = x;
                }
            }
        if constexpr (C::kInt4) {
            // back to units of the values: row g of an accumulator holds codes of weight 2^-24,
            // row g + 8 of weight 2^-20, both times the steps' scale
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < C::kG; ++k) {
                    const float un = step_unscale(top_e[k]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float* a = acc[n][4 * k + i];
                            a[e] = fmaf(a[e], 16777216.f, side[n][k][e]) * un;
                            a[e + 2] = fmaf(a[e + 2], 1048576.f, side[n][k][e]) * un;
                        }
                }
        }
        if (warp < active) {
            float* mine = sO + warp * (C::kOBytes / 4);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mine[(n * 8 + 2 * t + (e & 1)) * C::kOStride + value_of(k, e >> 1)] =
                            acc[n][k][e];
        }
        if (threadIdx.x < C::kRows) {
            const RowPlace rp = row_place(p, seg.b, kvh, row0 + threadIdx.x, seg.len);
            sAt[threadIdx.x] = (seg.b * p.H + rp.head) * p.Nq + rp.i;
            sSees[threadIdx.x] = rp.last >= 0;
        }
        __syncthreads();
        // ---------------------------------------------------------------- write out
        const bool whole = seg.t0 == seg.lo && seg.t1 == seg.tiles;
        float* part = p.ws + (static_cast<int64_t>(blockIdx.x) * 2 + (seg.t0 == seg.lo ? 1 : 0)) *
                                 (C::kRows * (D + 2));
        for (int i = threadIdx.x; i < C::kRows * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = i % (D / 4);
            if (row0 + r >= p.rows) break;
            float mw[kWarps], M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                mw[w] = w < active ? sM[w * C::kRows + r] : -INFINITY;
                M = fmaxf(M, mw[w]);
            }
            const float ref = M == -INFINITY ? 0.f : M;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w >= active) break;
                const float f = ex2_approx(mw[w] - ref);
                L += sL[w * C::kRows + r] * f;
                const float4 v = *reinterpret_cast<const float4*>(
                    sO + w * (C::kOBytes / 4) + r * C::kOStride + 4 * c);
                x.x += v.x * f;
                x.y += v.y * f;
                x.z += v.z * f;
                x.w += v.w * f;
            }
            if constexpr (C::kInt4) {
                if (sAside[0] == seg.left) {
                    const int k = 4 * c / kKvGroup;
                    for (int i = 0; i < C::kRows; ++i) {
                        const float score = sScore[i * C::kRows + r];
                        if (sAside[1 + k * C::kRows + i] != seg.left || score == -INFINITY) continue;
                        const int tok = min_last + 1 + i, pi = tok / p.pg.page;
                        const int place = tok - pi * p.pg.page;
                        const int32_t page =
                            p.pg.table[static_cast<int64_t>(seg.b) * p.pg.max_pages + pi];
                        const uint8_t* head = p.pg.v + kv_head_offset(p.pg, page, kvh);
                        const uint32_t codes = *reinterpret_cast<const uint16_t*>(
                            head + place * (D / 2) + 2 * c);
                        const uint32_t word = *reinterpret_cast<const uint16_t*>(
                            head + p.pg.page * (D / 2) + (place * C::kG + k) * 2);
                        const float f = ex2_approx(score - ref), s = kv4_word_step(word);
                        const int b = kv4_word_base(word);
                        x.x += f * static_cast<float>(b + static_cast<int>(codes & 15u)) * s;
                        x.y += f * static_cast<float>(b + static_cast<int>(codes >> 4 & 15u)) * s;
                        x.z += f * static_cast<float>(b + static_cast<int>(codes >> 8 & 15u)) * s;
                        x.w += f * static_cast<float>(b + static_cast<int>(codes >> 12)) * s;
                    }
                }
            }
            if (!whole) {
                *reinterpret_cast<float4*>(part + r * D + 4 * c) = x;
                if (c == 0) {
                    part[C::kRows * D + r] = M;
                    part[C::kRows * (D + 1) + r] = L;
                }
                continue;
            }
            const int64_t at = sAt[r];
            if constexpr (SHARED) {
                *reinterpret_cast<float4*>(p.row_o + at * D + 4 * c) = x;
                if (c == 0) p.row_ml[at] = make_float2(M, L);
                continue;
            }
            const bool none = L == 0.f || !sSees[r];
            const float inv = none ? 0.f : 1.f / L;
            uint2 o = make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
            if (none) o = make_uint2(0u, 0u);
            *reinterpret_cast<uint2*>(p.O + at * D + 4 * c) = o;
            if (c == 0 && p.LSE) p.LSE[at] = none ? -INFINITY : (M + __log2f(L)) * kLn2;
        }
        __syncthreads();  // the merge's shared memory is free for the next item
    }
    copies_wait<0>();
    if constexpr (SHARED) {
        // The kernel that joins the states waits for this one, and with it for the prefix kernel.  (It
        // looks after the other rows too.)  One CTA is enough for that; the others leave their SMs.
        if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }

    // Rows without an item: those of sequences without a key, blocks of padding rows.
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (p.only && !p.only[b]) continue;
        const int first = seq_len(p, b) == 0 ? 0 : seq_blocks<C::kRows>(p, b) * C::kRows;
        const int64_t missing = p.rows - first;
        for (int64_t i = threadIdx.x; i < missing * p.pg.H_kv * (D / 8); i += kThreads) {
            const int64_t r = i / (D / 8);
            const int h = static_cast<int>(r / missing);
            const RowPlace rp = row_place(p, b, h, static_cast<int>(first + r - h * missing), 0);
            const int64_t at = (static_cast<int64_t>(b) * p.H + rp.head) * p.Nq + rp.i;
            reinterpret_cast<uint4*>(p.O + at * D)[i % (D / 8)] = make_uint4(0u, 0u, 0u, 0u);
            if (p.LSE && i % (D / 8) == 0) p.LSE[at] = -INFINITY;
        }
    }
}

// Merges the partial states of the items that span shares.  CTA (c, r): 8 rows of the item that
// begins within share c and goes on past its end, if there is one; its warps take the shares in
// turn.  All that does not depend on the states happens before the wait for the kernel that makes
// them.
constexpr int kCombineRows = 8;

template <int D, int ROWS, int T, int W>
__global__ void __launch_bounds__(W * 32) paged_combine_kernel(const PagedParams p, int ctas) {
    constexpr int R = kCombineRows, E = D / 32;
    __shared__ float sM[W][R], sL[W][R];
    __shared__ float4 sO[W][R][D / 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = blockIdx.x / (ROWS / R), r0 = blockIdx.x % (ROWS / R) * R;
    if (r0 >= p.rows) return;
    const long long units = all_units<ROWS, T, 0>(p);
    const long long share = share_of(units, ctas);
    const long long u1 = share * (c0 + 1);
    Segment<ROWS, T, 0> seg;
    seg.start(p, u1 - 1, min(u1, units));
    const bool mine = !seg.done() && seg.t0 + 1 < seg.tiles && seg.t0 < share &&
                      seg.block * ROWS + r0 < p.rows;
    const int row0 = mine ? seg.block * ROWS + r0 : 0;
    const int n = min(R, p.rows - row0);
    const long long c1 = mine ? (u1 - 1 - seg.t0 + seg.tiles - 1) / share : c0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!mine) return;
    // lane i (and i + 8, i + 16, i + 24) holds the state of row i
    float M = -INFINITY, L = 0.f, o[R][E];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) o[i][e] = 0.f;
#pragma unroll 2
    for (long long c = c0 + warp; c <= c1; c += W) {
        const float* part = p.ws + (c * 2 + (c == c0 ? 1 : 0)) * (ROWS * (D + 2));
        const float mc = part[ROWS * D + r0 + lane % R], lc = part[ROWS * (D + 1) + r0 + lane % R];
        float v[R][E];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float* x = part + (r0 + i) * D + E * lane;
#pragma unroll
            for (int e = 0; e < E; ++e) v[i][e] = 0.f;
            if (i < n) {
                if constexpr (E == 4) {
                    const float4 y = *reinterpret_cast<const float4*>(x);
                    v[i][0] = y.x, v[i][1] = y.y, v[i][2] = y.z, v[i][3] = y.w;
                } else {
                    const float2 y = *reinterpret_cast<const float2*>(x);
                    v[i][0] = y.x, v[i][1] = y.y;
                }
            }
        }
        const float mn = fmaxf(M, mc), ref = mn == -INFINITY ? 0.f : mn;
        const float a = ex2_approx(M - ref), w = ex2_approx(mc - ref);
        M = mn;
        L = L * a + lc * w;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float ai = __shfl_sync(0xffffffffu, a, i), wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
            for (int e = 0; e < E; ++e) o[i][e] = o[i][e] * ai + v[i][e] * wi;
        }
    }
    if (lane < R) {
        sM[warp][lane] = M;
        sL[warp][lane] = L;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        float* x = reinterpret_cast<float*>(sO[warp][i]) + E * lane;
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = o[i][e];
    }
    __syncthreads();
    constexpr int kPer = W * 32 / R;  // threads a row
    const int i = threadIdx.x / kPer, u = threadIdx.x % kPer;
    if (i >= n) return;
    M = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, sM[w][i]);
    const float ref = M == -INFINITY ? 0.f : M;
    float f[W];
    L = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        f[w] = ex2_approx(sM[w][i] - ref);
        L += sL[w][i] * f[w];
    }
    const RowPlace rp = row_place(p, seg.b, seg.kvh, row0 + i, seg.len);
    const int64_t at = (static_cast<int64_t>(seg.b) * p.H + rp.head) * p.Nq + rp.i;
    const bool none = L == 0.f || rp.last < 0;
    const float inv = none ? 0.f : 1.f / L;
#pragma unroll
    for (int q = u; q < D / 4; q += kPer) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float4 v = sO[w][i][q];
            x.x += v.x * f[w];
            x.y += v.y * f[w];
            x.z += v.z * f[w];
            x.w += v.w * f[w];
        }
        uint2 y = make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
        if (none) y = make_uint2(0u, 0u);
        reinterpret_cast<uint2*>(p.O + at * D)[q] = y;
    }
    if (u == 0 && p.LSE) p.LSE[at] = none ? -INFINITY : (M + __log2f(L)) * kLn2;
}

int sm_count() {
    const int n = device_sm_count();
    return n > 0 ? n : 152;
}

// 8 rows an item where the query rows of a key/value head fit, else blocks of 16.
int rows_of(int64_t rows) { return rows <= 8 ? 8 : 16; }

// CTAs: those that the GPU runs at once (kCtasPerSm an SM), and no more than a tile a warp at the
// longest lengths.
int64_t ctas_of(int64_t B, int64_t H_kv, int64_t rows, int64_t d, int format, int64_t page,
                int64_t max_pages) {
    const int64_t T = tile_of(d, format, rows_of(rows));
    const int64_t tiles = (max_pages * page + T - 1) / T;
    const int64_t items = B * H_kv * ((rows + rows_of(rows) - 1) / rows_of(rows));
    const int64_t most = static_cast<int64_t>(sm_count()) * kCtasPerSm;
    if (tiles == 0) return 1;
    if (items > most * kWarps / tiles) return most;
    const int64_t n = (items * tiles + kWarps - 1) / kWarps;
    return n < most ? n : most;
}

// The combine kernel's launch overlaps the kernel before it (it waits for it on the device).
template <int D, int ROWS, int T, int W>
int launch_combine(const PagedParams& p, int ctas, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas * (ROWS / kCombineRows)));
    cfg.blockDim = dim3(W * 32);
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_combine_kernel<D, ROWS, T, W>, p, ctas) == cudaSuccess
               ? FA_OK
               : FA_ERR_CUDA;
}

template <int D, int FMT, int NT, bool SHARED>
int launch(const PagedParams& p, int ctas, cudaStream_t stream) {
    using C = Cfg<D, FMT, NT>;
    static PerDevice<bool> ready;
    if (!ready.get([](int) {
            return cudaFuncSetAttribute(paged_kernel<D, FMT, NT, SHARED>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        C::kDyn) == cudaSuccess;
        }))
        return FA_ERR_CUDA;
    if constexpr (SHARED) {
        // its launch overlaps the kernel in front of it
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(static_cast<unsigned>(ctas));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = C::kDyn;
        cfg.stream = stream;
        cudaLaunchAttribute at{};
        at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, paged_kernel<D, FMT, NT, true>, p) == cudaSuccess
                   ? FA_OK
                   : FA_ERR_CUDA;
    }
    paged_kernel<D, FMT, NT, SHARED><<<ctas, kThreads, C::kDyn, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
    // The merge: 8 warps where an item may span many shares (one item of 30000 tokens: 24.2 us, 35.4
    // with 4), and for items of 8 rows; else 4, of which more run at once (16 sequences of 40 rows a
    // head: 30.2 us, 32.1 with 8).
    if constexpr (NT > 1) {
        const int64_t items = static_cast<int64_t>(p.B) * p.pg.H_kv * p.row_blocks;
        if (ctas <= 32 * items) return launch_combine<D, C::kRows, C::kT, 4>(p, ctas, stream);
    }
    return launch_combine<D, C::kRows, C::kT, 8>(p, ctas, stream);
}

template <int D, int FMT, bool SHARED>
int launch_rows(const PagedParams& p, int ctas, cudaStream_t stream) {
    return rows_of(p.rows) == 8 ? launch<D, FMT, 1, SHARED>(p, ctas, stream)
                                : launch<D, FMT, 2, SHARED>(p, ctas, stream);
}

template <bool SHARED>
int launch_kind(const PagedParams& p, int64_t d, int ctas, cudaStream_t stream) {
    if (p.pg.format == OSM_KV_INT4)
        return d == 64 ? launch_rows<64, OSM_KV_INT4, SHARED>(p, ctas, stream)
                       : launch_rows<128, OSM_KV_INT4, SHARED>(p, ctas, stream);
    return d == 64 ? launch_rows<64, OSM_KV_BF16, SHARED>(p, ctas, stream)
                   : launch_rows<128, OSM_KV_BF16, SHARED>(p, ctas, stream);
}

// The kernel's parameters, `ws` its workspace.
PagedParams make_params(const void* Q, void* O, float* LSE, const KvPages& pg,
                        const int32_t* kv_lens, const int32_t* q_lens, int64_t B, int64_t H,
                        int64_t Nq, int64_t d, float scale, bool causal, void* ws) {
    PagedParams p{};
    p.Q = static_cast<const __nv_bfloat16*>(Q);
    p.O = static_cast<__nv_bfloat16*>(O);
    p.LSE = LSE;
    p.ws = static_cast<float*>(ws);
    p.kv_lens = kv_lens;
    p.q_lens = q_lens;
    p.B = static_cast<int>(B);
    p.H = static_cast<int>(H);
    p.Nq = static_cast<int>(Nq);
    p.causal = causal ? 1 : 0;
    p.group = static_cast<int>(H / pg.H_kv);
    p.rows = static_cast<int>(H / pg.H_kv * Nq);
    p.row_blocks = (p.rows + rows_of(p.rows) - 1) / rows_of(p.rows);
    p.scale_log2 = scale * kLog2e;
    p.pg = pg;
    const int step = kWarps * tile_of(d, pg.format, rows_of(p.rows));
    p.page_bytes = static_cast<uint32_t>(pg.head_bytes * pg.H_kv);
    p.page_div = step / pg.page;
    p.page_rem = step % pg.page;
    if (pg.num_pages == 0) p.pg.k = p.pg.v = static_cast<uint8_t*>(ws);  // no page is read
    return p;
}

}  // namespace

namespace {

// Where the workspace's parts begin, in bytes, and the sizes they were made for.  The partial
// states of the kernel above come first; a chunk call (see chunked) adds the flags of irregular
// sequences, dense keys and values of `seqs` sequences at a time, and the split-key attention's
// partial states.
struct Workspace {
    int64_t ctas, flags, k, v, o, lse, bytes;
    int64_t seqs, splits, tokens;
    bool chunk;
};

// Chunks of a prompt: from 256 query rows a key/value head on, the pages are read out dense, by
// kv_gather_for_attention, and the tcgen05 attention of fa_fwd.cu runs over them.  Kernel above
// (mma.sync, 16 rows at a time) against this, us at 128, 256 and 512 rows a head: 8 heads on 2 x 16384
// 4-bit keys 89 / 88, 164 / 104, 316 / 124; on 1 x 4000 24 / 31, 32 / 33, 52 / 43; 8 heads on 16 x 2000
// bf16 keys 107 / 102, 191 / 105, 383 / 147; 4 heads of 64 on 4 x 8000 31 / 40, 50 / 43, 90 / 56.
// Sequences whose pages hold what a dense attention cannot leave out (a page that is none, a NaN
// that only some queries see) are flagged and left to the kernel above.
bool chunked(int64_t rows) { return rows >= 256; }

Workspace workspace(int64_t B, int64_t H, int64_t H_kv, int64_t Nq, int64_t d, int format,
                    int64_t page, int64_t max_pages) {
    const int64_t rows = H / H_kv * Nq;
    Workspace w{};
    w.ctas = ctas_of(B, H_kv, rows, d, format, page, max_pages);
    w.bytes = w.ctas * 2 * rows_of(rows) * (d + 2) * 4;
    w.tokens = max_pages * page;
    w.chunk = chunked(rows) && w.tokens > 0;
    if (!w.chunk) return w;
    auto part = [&](int64_t n) {
        const int64_t at = (w.bytes + 255) & ~int64_t(255);
        w.bytes = at + n;
        return at;
    };
    w.flags = part(B * 4);
    // as many sequences at a time as 1 GB of dense keys and values holds, at least one
    const int64_t one = H_kv * w.tokens * d * 2;
    w.seqs = (int64_t(1) << 29) / one;
    w.seqs = w.seqs < 1 ? 1 : (w.seqs > B ? B : w.seqs);
    w.k = part(w.seqs * one);
    w.v = part(w.seqs * one);
    // Key ranges: none where the row tiles fill the SMs, else two waves of four key tiles or more.
    const int64_t items = w.seqs * H_kv * ((rows + 127) / 128), tiles = (w.tokens + 127) / 128;
    int64_t want = items >= sm_count() ? 1 : 2 * sm_count() / items;
    if (want > tiles / 4) want = tiles / 4;
    if (want > 64) want = 64;
    w.splits = splitkv_choose_splits(w.seqs * H_kv, rows, w.tokens, want < 1 ? 1 : want);
    if (w.splits > 1) {
        w.o = part(w.splits * w.seqs * H * Nq * d * 4);
        w.lse = part(w.splits * w.seqs * H * Nq * 4);
    }
    return w;
}

}  // namespace

int64_t fa_paged_ws_bytes(int64_t B, int64_t H, int64_t H_kv, int64_t Nq, int64_t d, int format,
                          int64_t page, int64_t max_pages) {
    const int64_t rows = H / H_kv * Nq, block = rows_of(rows);
    const int64_t T = tile_of(d, format, rows_of(rows));
    const int64_t units = B * H_kv * ((rows + block - 1) / block) * ((max_pages * page + T - 1) / T);
    const Workspace w = workspace(B, H, H_kv, Nq, d, format, page, max_pages);
    return units / w.ctas >= INT32_MAX - 1 ? -1 : w.bytes;  // a share is counted in 32 bits
}

int fa_paged_launch(const void* Q, void* O, float* LSE, const KvPages& pg,
                    const int32_t* kv_lens, const int32_t* q_lens, int64_t B, int64_t H,
                    int64_t Nq, int64_t d, float scale, bool causal, void* ws,
                    cudaStream_t stream) {
    const Workspace w = workspace(B, H, pg.H_kv, Nq, d, pg.format, pg.page, pg.max_pages);
    uint8_t* base = static_cast<uint8_t*>(ws);
    int32_t* flags = nullptr;
    if (w.chunk) {
        flags = reinterpret_cast<int32_t*>(base + w.flags);
        if (cudaMemsetAsync(flags, 0, B * 4, stream) != cudaSuccess) return FA_ERR_CUDA;
        for (int64_t b0 = 0; b0 < B; b0 += w.seqs) {
            const int64_t n = b0 + w.seqs < B ? w.seqs : B - b0;
            KvPages part = pg;
            part.table += b0 * pg.max_pages;
            const int32_t* ql = q_lens ? q_lens + b0 : nullptr;
            int st = kv_gather_for_attention(part, kv_lens + b0, ql, Nq, causal, flags + b0,
                                             base + w.k, base + w.v, n, w.tokens, d, stream);
            if (st != FA_OK) return st;
            AttnShape sh{n, H, pg.H_kv, Nq, w.tokens, d, kv_lens + b0, 0};
            sh.seq = true;
            sh.q_lens = ql;
            const int64_t row0 = b0 * H * Nq;
            st = fa_fwd_splitkv_launch(
                static_cast<const __nv_bfloat16*>(Q) + row0 * d, base + w.k, base + w.v,
                static_cast<__nv_bfloat16*>(O) + row0 * d, LSE ? LSE + row0 : nullptr, sh, scale,
                causal, w.splits, reinterpret_cast<float*>(base + w.o),
                reinterpret_cast<float*>(base + w.lse), stream);
            if (st != FA_OK) return st;
        }
    }
    PagedParams p = make_params(Q, O, LSE, pg, kv_lens, q_lens, B, H, Nq, d, scale, causal, ws);
    p.only = flags;
    return launch_kind<false>(p, d, static_cast<int>(w.ctas), stream);
}

bool fa_paged_takes_chunks(int64_t rows) { return chunked(rows); }

PagedOwn fa_paged_own(int64_t B, int64_t H, int64_t H_kv, int64_t Nq, int64_t d, int format,
                      int64_t page, int64_t max_pages) {
    const int64_t rows = H / H_kv * Nq;
    PagedOwn o{};
    o.rows = static_cast<int>(rows_of(rows));
    o.tile = tile_of(d, format, o.rows);
    o.ctas = static_cast<int>(ctas_of(B, H_kv, rows, d, format, page, max_pages));
    o.per_sm = kCtasPerSm;
    o.edge_bytes = static_cast<int64_t>(o.ctas) * 2 * o.rows * (d + 2) * 4;
    return o;
}

int fa_paged_own_launch(const void* Q, const KvPages& pg, const int32_t* kv_lens,
                        const int32_t* q_lens, int64_t B, int64_t H, int64_t Nq, int64_t d,
                        float scale, bool causal, const PagedOwn& own, void* edge,
                        const ShSeq* seqs, const ShHead* head, float* row_o, float2* row_ml,
                        cudaStream_t stream) {
    PagedParams p = make_params(Q, nullptr, nullptr, pg, kv_lens, q_lens, B, H, Nq, d, scale, causal,
                                edge);
    p.seqs = seqs;
    p.row_o = row_o;
    p.row_ml = row_ml;
    p.head = head;
    return launch_kind<true>(p, d, own.ctas, stream);
}

}  // namespace osm
