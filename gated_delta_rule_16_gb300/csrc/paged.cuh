// paged.cuh -- shared declarations of the decode-step operators over a paged
// key-value cache (block tables, cache writes, one-token attention) and of the
// sampling step (not part of the ABI).
#pragma once

#include <cuda_fp8.h>

#include "gdn_internal.cuh"

namespace gdn {

struct TablesArgs {
    int B, page, max_pages, n_free, n_slots;
    const int32_t *cached_lens, *new_lens, *free_pages;  // cached_lens may be NULL
    int32_t *block_table, *seq_lens, *cu_new, *positions, *counts;
    int64_t *slots;
};

struct AppendArgs {
    gdn_kv_cache c;
    int n;
    gdn_dtype dtype;
    const void *k, *v;
    int64_t k_tok, k_head, v_tok, v_head;  // strides in elements
    const int64_t *slots;
};

struct AttendArgs {
    gdn_kv_cache c;
    int B, Hq;
    const void *q;
    int64_t q_req, q_head;  // strides in elements
    const int32_t *table;
    int64_t table_stride;
    int max_pages, window;
    const int32_t *lens;
    float scale;
    void *o;
    float *lse;  // may be NULL
    void *ws;
};

struct SampleArgs {
    int B, V;
    gdn_dtype dtype;
    const void *logits;
    int64_t logits_stride;
    const float *noise;
    int64_t noise_stride;
    const float *temperature, *top_p, *min_p;  // each may be NULL
    const int32_t *top_k;                      // may be NULL
    int32_t *tokens;
    float *logprobs;  // may be NULL
};

cudaError_t launch_page_tables(const TablesArgs &a, cudaStream_t stream);
cudaError_t launch_kv_append(const AppendArgs &a, cudaStream_t stream);
size_t paged_decode_workspace_bytes(const gdn_kv_cache &c, int Hq);
cudaError_t launch_paged_decode(const AttendArgs &a, cudaStream_t stream);
cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream);

}  // namespace gdn
