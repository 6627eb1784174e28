// k_page_tables.cu -- block tables and slot maps of a step from the requests' lengths.
//
// Two running sums over the requests, of the new tokens and of the new pages,
// place everything: request b's tokens fill slots [cu[b], cu[b+1]) and its new
// pages are the free list's entries [f[b], f[b+1]).  A few bytes per request, 12 B
// per token: bound by the launch and the scan's latency, so every CTA repeats the
// scan (one or two loads per request) and no second launch passes it on.  Rows of
// the block table and ranges of tokens are dealt to the CTAs in turn; a token
// finds its request by bisection in the scan kept in shared memory.  A new
// token's page comes from the free list or from a table entry below `old`, never
// from an entry that this launch writes, so the CTAs need no order.
#include "paged.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 512;  // requests per scan step

struct Req {
    int64_t cached, len;
    int old_pages, need_pages;
};

__device__ __forceinline__ Req request(const TablesArgs &a, int b) {
    Req r;
    const int c = a.cached_lens ? a.cached_lens[b] : 0, n = a.new_lens[b];
    r.cached = max(c, 0);
    r.len = r.cached + max(n, 0);
    r.old_pages = (int)((r.cached + a.page - 1) / a.page);
    r.need_pages = (int)min((r.len + a.page - 1) / a.page, (int64_t)a.max_pages);
    return r;
}

__global__ void __launch_bounds__(kThreads) page_tables_kernel(TablesArgs a) {
    __shared__ int64_t cu[kThreads + 1], fr[kThreads + 1];  // running sums of this step's requests
    __shared__ int64_t warp_tok[kThreads / 32], warp_page[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t tok0 = 0, page0 = 0, longest = 0;  // sums over the steps before
    int status = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int nb = min(kThreads, a.B - b0), b = b0 + tid;
        Req r = {0, 0, 0, 0};
        if (tid < nb) r = request(a, b);
        const int64_t n_tok = r.len - r.cached, n_page = max(r.need_pages - r.old_pages, 0);
        int64_t st = n_tok, sp = n_page;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, st, off), y = __shfl_up_sync(0xffffffffu, sp, off);
            if (lane >= off) st += x, sp += y;
        }
        __syncthreads();  // the step before has read cu, fr and the warp sums
        if (lane == 31) warp_tok[warp] = st, warp_page[warp] = sp;
        __syncthreads();
        int64_t wt = tok0, wp = page0;
        for (int w = 0; w < warp; ++w) wt += warp_tok[w], wp += warp_page[w];
        cu[tid + 1] = wt + st;
        fr[tid + 1] = wp + sp;
        if (tid == 0) cu[0] = tok0, fr[0] = page0;
        __syncthreads();
        longest = max(longest, r.len);
        if ((r.len + a.page - 1) / a.page > a.max_pages) status |= 2;
        if (blockIdx.x == 0 && tid < nb) {
            a.seq_lens[b] = (int32_t)min(r.len, (int64_t)INT32_MAX);
            a.cu_new[b + 1] = (int32_t)min(cu[tid + 1], (int64_t)INT32_MAX);
        }
        // table rows of this step's requests: entries from `old` on
        for (int i = blockIdx.x; i < nb; i += gridDim.x) {
            const Req q = request(a, b0 + i);
            int32_t *row = a.block_table + (int64_t)(b0 + i) * a.max_pages;
            for (int64_t j = (int64_t)q.old_pages + tid; j < a.max_pages; j += kThreads) {
                const int64_t at = fr[i] + j - q.old_pages;
                row[j] = j < q.need_pages && at < a.n_free ? a.free_pages[at] : -1;
            }
        }
        // slots of this step's tokens
        const int64_t t1 = min(cu[nb], (int64_t)a.n_slots);
        for (int64_t t = cu[0] + (int64_t)blockIdx.x * kThreads + tid; t < t1; t += (int64_t)gridDim.x * kThreads) {
            int lo = 0, hi = nb;  // the last i with cu[i] <= t
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= t) lo = mid; else hi = mid;
            }
            const Req q = request(a, b0 + lo);
            const int64_t pos = q.cached + t - cu[lo], cell = pos / a.page;
            int64_t id = -1;
            if (cell < a.max_pages) {
                const int64_t at = fr[lo] + cell - q.old_pages;
                if (cell < q.old_pages) id = a.block_table[(int64_t)(b0 + lo) * a.max_pages + cell];
                else if (at < a.n_free) id = a.free_pages[at];
            }
            a.slots[t] = id < 0 ? -1 : id * a.page + pos % a.page;
            a.positions[t] = (int32_t)min(pos, (int64_t)INT32_MAX);
        }
        tok0 = cu[nb];
        page0 = fr[nb];
    }
    for (int64_t t = tok0 + (int64_t)blockIdx.x * kThreads + tid; t < a.n_slots; t += (int64_t)gridDim.x * kThreads) {
        a.slots[t] = -1;
        a.positions[t] = 0;
    }
    if (blockIdx.x != 0) return;
    if (page0 > a.n_free) status |= 1;
    if (tok0 > a.n_slots) status |= 4;
    status = __syncthreads_or(status & 1) * 1 | (__syncthreads_or(status & 2) ? 2 : 0) | (__syncthreads_or(status & 4) ? 4 : 0);
    for (int off = 16; off; off >>= 1) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, off));
    if (lane == 0) warp_tok[warp] = longest;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kThreads / 32; ++w) longest = max(longest, warp_tok[w]);
        a.cu_new[0] = 0;
        a.counts[0] = (int32_t)min(tok0, (int64_t)INT32_MAX);
        a.counts[1] = (int32_t)min(page0, (int64_t)a.n_free);
        a.counts[2] = status;
        a.counts[3] = (int32_t)min(longest, (int64_t)INT32_MAX);
    }
}

}  // namespace

cudaError_t launch_page_tables(const TablesArgs &a, cudaStream_t stream) {
    // one CTA per 4096 slots or per two table rows, one wave at most
    const int64_t want = max((int64_t)a.n_slots / 4096, (int64_t)a.B / 2) + 1;
    page_tables_kernel<<<(unsigned)min(want, (int64_t)152), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
