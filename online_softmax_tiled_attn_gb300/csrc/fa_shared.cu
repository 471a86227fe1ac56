// fa_shared.cu -- attention over the paged cache for groups of sequences with a common prefix
// (fa_fwd_paged_shared): the sequences one by one, as fa_fwd_paged reads them.
#include <cuda_runtime.h>

#include "kv_cache.cuh"
#include "osm_internal.h"

namespace osm {

int64_t fa_shared_ws_bytes(int64_t B, int64_t H, int64_t H_kv, int64_t Nq, int64_t d, int format,
                           int64_t page, int64_t max_pages) {
    return fa_paged_ws_bytes(B, H, H_kv, Nq, d, format, page, max_pages);
}

int fa_shared_launch(const void* Q, void* O, float* LSE, const KvPages& pg, const int32_t* kv_lens,
                     const int32_t* q_lens, const int32_t*, int64_t B, int64_t H, int64_t Nq,
                     int64_t d, float scale, bool causal, void* ws, cudaStream_t stream) {
    return fa_paged_launch(Q, O, LSE, pg, kv_lens, q_lens, B, H, Nq, d, scale, causal, ws, stream);
}

}  // namespace osm
