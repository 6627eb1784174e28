// paged.cuh -- shared declarations of the decode-step operators over a paged
// key-value cache (block tables, cache writes, one-token attention), of the
// sampling step, and of the prompt chunks' operators (not part of the ABI).
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

struct RopeArgs {
    int n, Hq, Hkv, d;
    gdn_dtype dtype;
    const void *q, *k;
    void *q_out, *k_out;
    int64_t q_tok, q_head, k_tok, k_head, qo_tok, qo_head, ko_tok, ko_head;  // strides in elements
    const int32_t *positions;
    const double *freqs;
    int pairs, interleaved;
    float mscale, eps;
    const float *q_weight, *k_weight;  // each may be NULL
    int heads_per_cta;                 // set by the launch
};

// n / by for 0 <= n < 2^31, with l = ceil(log2 by): (n mul) >> (31 + l), mul = ceil(2^(31 + l) / by).
struct Divisor {
    uint32_t by, mul, shift;
#ifdef __CUDACC__
    __device__ __forceinline__ int quotient(int n) const { return (int)((uint64_t)(uint32_t)n * mul >> shift); }
    __device__ __forceinline__ int quotient(int n, int &rest) const {
        const int q = quotient(n);
        rest = n - q * (int)by;
        return q;
    }
#endif
};
inline Divisor divisor(uint32_t by) {
    uint32_t l = 0;
    while ((uint64_t)1 << l < by) ++l;
    return {by, (uint32_t)((((uint64_t)1 << (31 + l)) + by - 1) / by), 31 + l};
}

struct PrefillArgs {
    gdn_kv_cache c;
    int B, n, Hq;
    const void *q;
    int64_t q_tok, q_head;  // strides in elements
    const int32_t *table;
    int64_t table_stride;
    int max_pages, window;
    const int32_t *lens, *cu;
    float scale;
    void *o;
    float *lse;  // may be NULL
    void *ws;
    Divisor group, page;  // set by the launch
    uint32_t lost_ns;     // self-test of waits, not 0: after 128 keys a CTA's copies wait so long for what never comes
};

struct LogprobArgs {
    int B, V, top;
    gdn_dtype dtype;
    const void *logits;
    int64_t stride;
    const int32_t *tokens;
    float *logprobs, *entropy;  // entropy may be NULL
    int32_t *top_tokens;        // NULL where top is 0
    float *top_logprobs;
};

cudaError_t launch_page_tables(const TablesArgs &a, cudaStream_t stream);
cudaError_t launch_kv_append(const AppendArgs &a, cudaStream_t stream);
size_t paged_decode_workspace_bytes(const gdn_kv_cache &c, int Hq);
cudaError_t launch_paged_decode(const AttendArgs &a, cudaStream_t stream);
cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream);
cudaError_t launch_qk_rope(const RopeArgs &a, cudaStream_t stream);
size_t paged_prefill_workspace_bytes(const gdn_kv_cache &c, int B, int n, int Hq);
cudaError_t launch_paged_prefill(const PrefillArgs &a, cudaStream_t stream);
cudaError_t launch_logprobs(const LogprobArgs &a, cudaStream_t stream);

}  // namespace gdn
