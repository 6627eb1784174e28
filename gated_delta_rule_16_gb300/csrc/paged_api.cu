// paged_api.cu -- the extern "C" entry points of the decode-step operators (declared in
// include/gdn.h): argument validation and launches.  No allocation, no synchronisation
// except in the status query.
#include "paged.cuh"

namespace gdn {
namespace {

constexpr size_t kWsAlign = 256;

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

int bytes_of(gdn_dtype t) { return t == GDN_E4M3 ? 1 : (t == GDN_BF16 ? 2 : 4); }

// A stride that keeps 16-byte pieces aligned.
bool stride_ok(int64_t s, gdn_dtype t) { return s >= 0 && s * bytes_of(t) % 16 == 0; }

// Everything about a cache but its pointers.
gdn_status check_cache_sizes(const gdn_kv_cache *c) {
    if (!c) return GDN_ERR_NULL;
    if (c->dtype != GDN_BF16 && c->dtype != GDN_F32 && c->dtype != GDN_E4M3) return GDN_ERR_DTYPE;
    if (c->Hkv <= 0 || c->page <= 0 || c->pages < 0 || c->pages > INT32_MAX) return GDN_ERR_SHAPE;
    if (c->d != 64 && c->d != 128 && c->d != 256) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status check_cache(const gdn_kv_cache *c) {
    const gdn_status st = check_cache_sizes(c);
    if (st != GDN_OK) return st;
    if (!c->k || !c->v) return GDN_ERR_NULL;
    if (c->dtype == GDN_E4M3 && (!c->k_scale || !c->v_scale)) return GDN_ERR_NULL;
    if (c->dtype != GDN_E4M3 && (c->k_scale || c->v_scale)) return GDN_ERR_UNSUPPORTED;
    if (!aligned16(c->k) || !aligned16(c->v)) return GDN_ERR_ALIGN;
    if (((uintptr_t)c->k_scale | (uintptr_t)c->v_scale) & 3u) return GDN_ERR_ALIGN;
    if (!stride_ok(c->stride_page, c->dtype) || !stride_ok(c->stride_token, c->dtype) ||
        !stride_ok(c->stride_head, c->dtype))
        return GDN_ERR_ALIGN;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_page_tables(int32_t B, int32_t page, int32_t max_pages, const int32_t *cached_lens,
                           const int32_t *new_lens, const int32_t *free_pages, int32_t n_free, int32_t *block_table,
                           int32_t *seq_lens, int32_t *cu_new, int64_t *slots, int32_t *positions, int32_t n_slots,
                           int32_t *counts, void *stream) {
    if (B < 0 || page <= 0 || max_pages < 0 || n_free < 0 || n_slots < 0) return GDN_ERR_SHAPE;
    if (!cu_new || !counts) return GDN_ERR_NULL;
    if (B > 0 && (!new_lens || !seq_lens)) return GDN_ERR_NULL;
    if (B > 0 && max_pages > 0 && !block_table) return GDN_ERR_NULL;
    if (n_free > 0 && !free_pages) return GDN_ERR_NULL;
    if (n_slots > 0 && (!slots || !positions)) return GDN_ERR_NULL;
    const void *words[] = {cached_lens, new_lens, free_pages, block_table, seq_lens, cu_new, positions, counts};
    for (const void *p : words)
        if ((uintptr_t)p & 3u) return GDN_ERR_ALIGN;
    if ((uintptr_t)slots & 7u) return GDN_ERR_ALIGN;
    if (!device_ok()) return GDN_ERR_DEVICE;
    // Every CTA reads all lengths, and one of them writes the results: in place a CTA would read what another has written.
    struct Range { const void *p; int64_t bytes; };
    const Range in[] = {{cached_lens, 4ll * B}, {new_lens, 4ll * B}, {free_pages, 4ll * n_free}};
    const Range out[] = {{block_table, 4ll * B * max_pages}, {seq_lens, 4ll * B}, {cu_new, 4ll * (B + 1ll)}, {slots, 8ll * n_slots},
                         {positions, 4ll * n_slots}, {counts, 16}};
    for (const Range &x : in)
        for (const Range &y : out)
            if (x.p && x.bytes > 0 && y.bytes > 0 && (uintptr_t)x.p < (uintptr_t)y.p + y.bytes && (uintptr_t)y.p < (uintptr_t)x.p + x.bytes)
                return GDN_ERR_UNSUPPORTED;
    const TablesArgs a = {B, page, max_pages, n_free, n_slots, cached_lens, new_lens, free_pages,
                          block_table, seq_lens, cu_new, positions, counts, slots};
    return launch_page_tables(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_page_tables_status(const int32_t *counts, void *stream) {
    if (!counts) return GDN_ERR_NULL;
    int32_t host[4] = {0, 0, 0, 0};
    if (cudaMemcpyAsync(host, counts, sizeof(host), cudaMemcpyDeviceToHost, (cudaStream_t)stream) != cudaSuccess ||
        cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess)
        return GDN_ERR_CUDA;
    return host[2] ? GDN_ERR_CAPACITY : GDN_OK;
}

gdn_status gdn_kv_append(const gdn_kv_cache *cache, int32_t n, gdn_dtype dtype, const void *k, int64_t k_stride_token,
                         int64_t k_stride_head, const void *v, int64_t v_stride_token, int64_t v_stride_head,
                         const int64_t *slots, void *stream) {
    gdn_status st = check_cache_sizes(cache);
    if (st != GDN_OK) return st;
    if (n < 0) return GDN_ERR_SHAPE;
    if (dtype != GDN_BF16 && dtype != GDN_F32) return GDN_ERR_DTYPE;
    if (cache->dtype != GDN_E4M3 && cache->dtype != dtype) return GDN_ERR_DTYPE;
    if (n == 0 || cache->pages == 0) return GDN_OK;
    if ((st = check_cache(cache)) != GDN_OK) return st;
    if (!k || !v || !slots) return GDN_ERR_NULL;
    if (!aligned16(k) || !aligned16(v) || ((uintptr_t)slots & 7u)) return GDN_ERR_ALIGN;
    if (!stride_ok(k_stride_token, dtype) || !stride_ok(k_stride_head, dtype) || !stride_ok(v_stride_token, dtype) ||
        !stride_ok(v_stride_head, dtype))
        return GDN_ERR_ALIGN;
    if (!device_ok()) return GDN_ERR_DEVICE;
    const AppendArgs a = {*cache, n, dtype, k, v, k_stride_token, k_stride_head, v_stride_token, v_stride_head, slots};
    return launch_kv_append(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_paged_decode_workspace_bytes(const gdn_kv_cache *cache, int32_t Hq) {
    if (check_cache_sizes(cache) != GDN_OK || Hq <= 0 || Hq % cache->Hkv) return 0;
    return paged_decode_workspace_bytes(*cache, Hq) + kWsAlign;
}

gdn_status gdn_paged_decode(const gdn_kv_cache *cache, int32_t B, int32_t Hq, gdn_dtype dtype, const void *q,
                            int64_t q_stride_request, int64_t q_stride_head, const int32_t *block_table,
                            int64_t table_stride, int32_t max_pages, const int32_t *seq_lens, int32_t window,
                            float scale, void *o, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    gdn_status st = check_cache_sizes(cache);
    if (st != GDN_OK) return st;
    if (B < 0 || Hq <= 0 || Hq % cache->Hkv || max_pages < 0 || window < 0 || table_stride < 0) return GDN_ERR_SHAPE;
    if (dtype != (cache->dtype == GDN_E4M3 ? GDN_BF16 : cache->dtype)) return GDN_ERR_DTYPE;
    if ((int64_t)B * Hq > INT32_MAX) return GDN_ERR_SHAPE;
    if ((int64_t)max_pages * cache->page > INT32_MAX - 127) return GDN_ERR_UNSUPPORTED;  // token positions are int32
    if (B == 0) return GDN_OK;
    // with no page in the pool or no column in the table every request is empty, but o and lse are still written
    if (cache->pages > 0 && max_pages > 0) {
        if ((st = check_cache(cache)) != GDN_OK) return st;
        if (!block_table) return GDN_ERR_NULL;
    }
    if (!q || !seq_lens || !o || !workspace) return GDN_ERR_NULL;
    if (!aligned16(q) || !aligned16(o) || !stride_ok(q_stride_request, dtype) || !stride_ok(q_stride_head, dtype) ||
        (((uintptr_t)block_table | (uintptr_t)seq_lens | (uintptr_t)lse) & 3u) || (uintptr_t)workspace % kWsAlign)
        return GDN_ERR_ALIGN;
    if (workspace_bytes < gdn_paged_decode_workspace_bytes(cache, Hq)) return GDN_ERR_WORKSPACE;
    if (!device_ok()) return GDN_ERR_DEVICE;
    AttendArgs a = {*cache, B, Hq, q, q_stride_request, q_stride_head, block_table, table_stride,
                    cache->pages > 0 ? max_pages : 0, window, seq_lens, scale, o, lse, workspace};
    if (a.max_pages == 0) a.c.k_scale = a.c.v_scale = nullptr;
    return launch_paged_decode(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_sample(int32_t B, int32_t V, gdn_dtype dtype, const void *logits, int64_t logits_stride,
                      const float *noise, int64_t noise_stride, const float *temperature, const int32_t *top_k,
                      const float *top_p, const float *min_p, int32_t *tokens, float *logprobs, void *stream) {
    if (dtype != GDN_BF16 && dtype != GDN_F32) return GDN_ERR_DTYPE;
    if (B < 0 || V <= 0 || logits_stride < 0 || noise_stride < 0) return GDN_ERR_SHAPE;
    if (V > (1 << 22)) return GDN_ERR_UNSUPPORTED;  // 2^22 weights of at most 2^40 units: sums stay below 2^63
    if (B == 0) return GDN_OK;
    if (!logits || !noise || !tokens) return GDN_ERR_NULL;
    if ((uintptr_t)logits % (unsigned)bytes_of(dtype) ||
        (((uintptr_t)noise | (uintptr_t)temperature | (uintptr_t)top_k | (uintptr_t)top_p | (uintptr_t)min_p |
          (uintptr_t)tokens | (uintptr_t)logprobs) & 3u))
        return GDN_ERR_ALIGN;
    if (!device_ok()) return GDN_ERR_DEVICE;
    const SampleArgs a = {B, V, dtype, logits, logits_stride, noise, noise_stride, temperature, top_p, min_p, top_k,
                          tokens, logprobs};
    return launch_sample(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
