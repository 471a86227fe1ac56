// osm_internal.h -- declarations shared by the translation units of libosmattn.so.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "osm_attn.h"

namespace osm {

// Tiled TMA descriptor over a [BH, N, d] bf16 tensor (d innermost): a box of 64 columns x 128
// rows of one (b, h), 128-byte swizzle, zero fill outside [0, N) x [0, d).
int make_bhnd_tensor_map(CUtensorMap* map, const void* base, int64_t BH, int64_t N, int64_t d);

// Tiled TMA descriptor over an array of bf16 pages [num_pages, H_kv, page, d]: a box of 64 columns x
// `tokens` rows (a divisor of page) of one head of one page, 128-byte swizzle.
int make_pages_tensor_map(CUtensorMap* map, const void* base, int64_t num_pages, int64_t H_kv,
                          int64_t page, int64_t d, int64_t tokens);

// Tiled TMA descriptor over an explicit mask: uint32 words [Bm, Hm, Nq, W] with the given
// strides in words between heads and sequences (used where Hm, Bm > 1); a box of 4 words
// (one key tile) x 128 query rows, no swizzle, zero fill past Nq.
int make_mask_tensor_map(CUtensorMap* map, const uint32_t* mask, int64_t W, int64_t Nq,
                         int64_t Hm, int64_t Bm, int64_t mask_hs, int64_t mask_bs);

// Deadline of every bounded mbarrier wait in the attention kernel.
unsigned long long fa_wait_timeout_ns();

// Shape of one attention call: Q, O [B, H, Nq, d]; K, V [B, H_kv, Nk, d] (H_kv divides H;
// query head h reads key/value head h / (H / H_kv)); kv_lens, if not null, a device array of
// the B valid key counts (clamped to [0, Nk] in the kernel).  q_pos = 0 means Nq; otherwise
// the rows are packed query heads (see pack_query_heads) with q_pos positions each.
struct AttnShape {
    int64_t B, H, H_kv, Nq, Nk, d;
    const int32_t* kv_lens;
    int64_t q_pos;
    // Optional explicit mask: uint32 words, row i of query head (b, h) at
    // mask + b * mask_bs + h * mask_hs + i * 4 * ceil(Nk / 128); bit j % 32 of word j / 32 set =
    // key j allowed.  Not combined with packed query heads.
    const uint32_t* mask = nullptr;
    int64_t mask_bs = 0, mask_hs = 0;
    // Optional device buffer for the mask's tile map (mask_tile_map_words words): filled by a
    // pre-pass, then key tiles with no allowed key for a whole query tile are skipped.
    uint32_t* tile_map = nullptr;
    // seq: causal positions count from each sequence's own end, query i of sequence b being token
    // kv_lens[b] - q_lens[b] + i; rows at or past q_lens[b] (device, nullptr: Nq) see no key.  Not
    // combined with an explicit mask.
    bool seq = false;
    const int32_t* q_lens = nullptr;
};

// Words of the tile map of an explicit mask: one row of ceil(ceil(Nk / 128) / 32) words per
// 128-row query tile and mask instance (B instances when mask_bs != 0, times H when
// mask_hs != 0).
int64_t mask_tile_map_words(int64_t B, int64_t H, int64_t Nq, int64_t Nk, int64_t mask_bs,
                            int64_t mask_hs);

// The same call with the H / H_kv query heads that share a key/value head packed into one row
// block of (H / H_kv) * Nq rows: the [B, H, Nq, d] memory of Q, O and LSE read as
// [B, H_kv, (H / H_kv) * Nq, d].  Each key/value tile is then loaded once per block instead of
// once per query head, and short query blocks (decoding) fill the 128-row tiles.
AttnShape pack_query_heads(const AttnShape& sh);

int fa_fwd_launch(const void* Q, const void* K, const void* V, void* O, float* LSE, int64_t BH,
                  int64_t N, int64_t d, float scale, bool causal, cudaStream_t stream);
int fa_fwd_shape_launch(const void* Q, const void* K, const void* V, void* O, float* LSE,
                        const AttnShape& sh, float scale, bool causal, cudaStream_t stream);
// Number of key ranges the split-key path uses for `requested` (<= 0: chosen from the shape and
// the SM count); 0 when there is no key.
int64_t splitkv_choose_splits(int64_t BH, int64_t Nq, int64_t Nk, int64_t requested);
int fa_fwd_splitkv_launch(const void* Q, const void* K, const void* V, void* O, float* LSE,
                          const AttnShape& sh, float scale, bool causal, int64_t n_splits,
                          float* ws_O, float* ws_LSE, cudaStream_t stream);
int fa_read_device_status(cudaStream_t stream, int* status);
// Device address of the status word the kernels' bounded waits report to (null on failure).
int* device_status_word();
// Q, O, dO, dQ [B, H, N, d]; K, V, dK, dV [B, H_kv, N, d]; LSE, ws_D [B, H, N]; kv_lens null or
// a device int32 [B] of valid keys per sequence.
int fa_bwd_launch(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                  const float* LSE, void* dQ, void* dK, void* dV, float* ws_D, int64_t B,
                  int64_t H, int64_t H_kv, int64_t N, int64_t d, const int32_t* kv_lens,
                  float scale, bool causal, cudaStream_t stream);
int selftest_wait_launch(long long timeout_us, cudaStream_t stream);

int osm_softmax_launch(const float* x, float* y, int64_t rows, int64_t cols, float* lse,
                       cudaStream_t stream);
int osm_softmax_topk_launch(const float* x, int64_t rows, int64_t cols, int64_t k, float* vals,
                            int32_t* idx, float* lse, cudaStream_t stream);

struct KvPages;  // kv_cache.cuh
int osm_rope_launch(const void* x, void* y, int dtype, int64_t B, int64_t H, int64_t N, int64_t d,
                    const int64_t* xs, const int64_t* ys, const int32_t* positions,
                    int64_t pos_bs, const int64_t* table, int64_t rot, int layout,
                    float amplitude, bool inverse, cudaStream_t stream);
int osm_kv_append_launch(const void* k, const void* v, const int64_t* ks, const int64_t* vs,
                         const KvPages& pg, const int32_t* cache_lens, const int32_t* new_lens,
                         const int64_t* table, int64_t rot, int layout, float amplitude,
                         const void* q, void* q_out, const int64_t* qs, int64_t B, int64_t H,
                         int64_t N, int64_t d, cudaStream_t stream);
int osm_kv_gather_launch(const KvPages& pg, const int32_t* kv_lens, void* K, void* V, int64_t B,
                         int64_t N, int64_t d, cudaStream_t stream);
// osm_kv_gather for an attention that follows: rows behind a sequence are zeroed up to the next
// multiple of 128 only, and irregular[b] is set where the dense attention would go wrong: a page
// that is none, or a value (V) that is not finite and that some row must not see (with causal, the
// last q_lens[b] tokens', Nq where q_lens is nullptr; any, where there are padding rows).
int kv_gather_for_attention(const KvPages& pg, const int32_t* kv_lens, const int32_t* q_lens,
                            int64_t Nq, bool causal, int32_t* irregular, void* K, void* V,
                            int64_t B, int64_t N, int64_t d, cudaStream_t stream);
// Workspace bytes; page_bytes: of all heads of a page.
int64_t kv_grow_ws_bytes(int64_t rows, int64_t page_bytes);
int64_t kv_fork_ws_bytes(int64_t rows, int64_t pairs, int64_t max_pages);
int64_t kv_compact_ws_bytes(int64_t num_pages);
int osm_kv_grow_launch(const KvPages& pg, int32_t* table, int32_t* lens, const int32_t* new_lens,
                       int32_t* old_lens, int32_t* refs, int64_t rows, int64_t d, void* ws,
                       cudaStream_t stream);
int osm_kv_fork_launch(const KvPages& pg, int32_t* table, int32_t* lens, int32_t* refs,
                       const int32_t* src, const int32_t* dst, int64_t rows, int64_t n, void* ws,
                       cudaStream_t stream);
int osm_kv_free_launch(const KvPages& pg, int32_t* table, int32_t* lens, int32_t* refs,
                       const int32_t* list, const int32_t* keep, int64_t rows, int64_t n,
                       cudaStream_t stream);
int osm_kv_compact_launch(const KvPages& pg, int32_t* table, int32_t* lens, int32_t* refs,
                          int32_t* page_map, int32_t* used, int64_t rows, void* ws,
                          cudaStream_t stream);
// Bytes of fa_fwd_paged's workspace; -1: too much work for one launch.
int64_t fa_paged_ws_bytes(int64_t B, int64_t H, int64_t H_kv, int64_t Nq, int64_t d, int format,
                          int64_t page, int64_t max_pages);
int fa_paged_launch(const void* Q, void* O, float* LSE, const KvPages& pg,
                    const int32_t* kv_lens, const int32_t* q_lens, int64_t B, int64_t H,
                    int64_t Nq, int64_t d, float scale, bool causal, void* ws,
                    cudaStream_t stream);

// fa_fwd_paged from this many rows a key/value head on takes the pages read out dense.
bool fa_paged_takes_chunks(int64_t rows);
struct ShSeq;  // fa_shared.cuh
struct ShHead;
// The kernel of fa_fwd_paged over the tokens of each sequence from seqs[b].skip on, leaving the rows' states
// for another to join: items of `rows` rows over tiles of `tile` tokens, all tiles in equal shares of
// head->own_share over the first CTAs of `ctas`, `per_sm` of which an SM holds; a partial state is
// [rows][d] of O, then m and l of the rows.  Launched behind the prefix kernel.
struct PagedOwn {
    int rows, tile, ctas, per_sm;
    int64_t edge_bytes;
};
PagedOwn fa_paged_own(int64_t B, int64_t H, int64_t H_kv, int64_t Nq, int64_t d, int format,
                      int64_t page, int64_t max_pages);
int fa_paged_own_launch(const void* Q, const KvPages& pg, const int32_t* kv_lens,
                        const int32_t* q_lens, int64_t B, int64_t H, int64_t Nq, int64_t d,
                        float scale, bool causal, const PagedOwn& own, void* edge,
                        const ShSeq* seqs, const ShHead* head, float* row_o, float2* row_ml,
                        cudaStream_t stream);
// fa_fwd_paged_shared's workspace (-1: too much work for one launch), and the call.
int64_t fa_shared_ws_bytes(int64_t B, int64_t H, int64_t H_kv, int64_t Nq, int64_t d, int format,
                           int64_t page, int64_t max_pages);
int fa_shared_launch(const void* Q, void* O, float* LSE, const KvPages& pg, const int32_t* kv_lens,
                     const int32_t* q_lens, const int32_t* groups, int64_t B, int64_t H, int64_t Nq,
                     int64_t d, float scale, bool causal, void* ws, cudaStream_t stream);

}  // namespace osm
