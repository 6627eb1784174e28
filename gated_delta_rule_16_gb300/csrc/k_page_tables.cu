// k_page_tables.cu -- block tables and slot maps of a step from the requests' lengths.
//
// Two running sums over the requests, of the new tokens and of the new pages,
// place everything: request b's tokens fill slots [cu[b], cu[b+1]) and its new
// pages are the free list's entries [f[b], f[b+1]).  A few bytes per request, 12 B
// per token: bound by the launch and the scan's latency, so every CTA repeats the
// scan (two loads per request, two requests per thread and step) and no second launch
// passes it on.  Rows of the block table and ranges of tokens are dealt to the CTAs
// in turn; a token finds its request by bisection in the scan kept in shared
// memory.  A new token's page comes from the free list or from a table entry below
// `old`, never from an entry that this launch writes, so the CTAs need no order.
// A length is below 2^32 (two int32 added), running sums are 64 bits wide and are
// kept saturated at 2^31 - 1, which no slot and no free page passes.  64 requests with a token each
// take 4.1 us, 1021 with 521731 slots 7.9 us (an empty launch: 2 us).
#include "paged.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 512, kEach = 2, kStep = kThreads * kEach;  // requests per scan step

struct Scan {
    int cu[kStep + 1], fr[kStep + 1];        // running sums of new tokens and new pages
    uint32_t cached[kStep], old_pages[kStep], need_pages[kStep];
    int64_t warp_tok[kThreads / 32], warp_page[kThreads / 32];
};

__device__ __forceinline__ int saturated(int64_t x) { return (int)min(x, (int64_t)INT32_MAX); }

__global__ void __launch_bounds__(kThreads) page_tables_kernel(TablesArgs a) {
    __shared__ Scan s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool pow2 = (a.page & (a.page - 1)) == 0;
    const int shift = 31 - __clz(a.page);
    auto page_of = [&](uint32_t pos) { return pow2 ? pos >> shift : pos / (uint32_t)a.page; };
    auto pages_for = [&](uint32_t n) { return n == 0 ? 0u : page_of(n - 1) + 1; };
    int64_t tok0 = 0, page0 = 0;  // sums over the steps before
    uint32_t longest = 0;
    int status = 0;
    for (int b0 = 0; b0 < a.B; b0 += kStep) {
        const int nb = min(kStep, a.B - b0);
        int64_t n_tok[kEach], n_page[kEach], st = 0, sp = 0;
        uint32_t len[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = tid * kEach + e, b = b0 + i;
            const int c = i < nb && a.cached_lens ? a.cached_lens[b] : 0, n = i < nb ? a.new_lens[b] : 0;
            const uint32_t cached = (uint32_t)max(c, 0);
            len[e] = cached + (uint32_t)max(n, 0);
            const uint32_t old = pages_for(cached), all = pages_for(len[e]), need = min(all, (uint32_t)a.max_pages);
            if (i < nb) s.cached[i] = cached, s.old_pages[i] = old, s.need_pages[i] = need;
            longest = max(longest, len[e]);
            if (all > (uint32_t)a.max_pages) status |= 2;
            n_tok[e] = len[e] - cached;
            n_page[e] = need > old ? need - old : 0;
            st += n_tok[e], sp += n_page[e];
        }
        int64_t it = st, ip = sp;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, it, off), y = __shfl_up_sync(0xffffffffu, ip, off);
            if (lane >= off) it += x, ip += y;
        }
        if (lane == 31) s.warp_tok[warp] = it, s.warp_page[warp] = ip;
        __syncthreads();
        int64_t wt = tok0 + it - st, wp = page0 + ip - sp, all_tok = tok0, all_page = page0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) wt += s.warp_tok[w], wp += s.warp_page[w];
            all_tok += s.warp_tok[w], all_page += s.warp_page[w];
        }
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = tid * kEach + e;
            s.cu[i] = saturated(wt), s.fr[i] = saturated(wp);
            wt += n_tok[e], wp += n_page[e];
            if (blockIdx.x == 0 && i < nb) {
                a.seq_lens[b0 + i] = saturated(len[e]);
                a.cu_new[b0 + i + 1] = saturated(wt);
            }
        }
        if (tid == kThreads - 1) s.cu[kStep] = saturated(wt), s.fr[kStep] = saturated(wp);
        __syncthreads();
        // table rows of this step's requests: entries from `old` on
        for (int i = blockIdx.x; i < nb; i += gridDim.x) {
            int32_t *row = a.block_table + (int64_t)(b0 + i) * a.max_pages;
            const uint32_t old = s.old_pages[i], need = s.need_pages[i];
            const int64_t first = s.fr[i];
            for (uint32_t j = old + tid; j < (uint32_t)a.max_pages; j += kThreads) {
                const int64_t at = first + (j - old);
                row[j] = j < need && at < a.n_free ? a.free_pages[at] : -1;
            }
        }
        // slots of this step's tokens
        const int t1 = min(s.cu[nb], a.n_slots);
        for (int64_t t = s.cu[0] + (int64_t)blockIdx.x * kThreads + tid; t < t1; t += (int64_t)gridDim.x * kThreads) {
            int lo = 0, hi = nb;  // the last i with cu[i] <= t
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s.cu[mid] <= t) lo = mid; else hi = mid;
            }
            const uint32_t pos = s.cached[lo] + (uint32_t)(t - s.cu[lo]), cell = page_of(pos), old = s.old_pages[lo];
            int64_t id = -1;
            if (cell < (uint32_t)a.max_pages) {
                const int64_t at = (int64_t)s.fr[lo] + cell - old;
                if (cell < old) id = a.block_table[(int64_t)(b0 + lo) * a.max_pages + cell];
                else if (at < a.n_free) id = a.free_pages[at];
            }
            a.slots[t] = id < 0 ? -1 : id * a.page + (pos - cell * (uint32_t)a.page);
            a.positions[t] = saturated(pos);
        }
        tok0 = all_tok;
        page0 = all_page;
        if (b0 + kStep < a.B) __syncthreads();  // the next step overwrites the scan
    }
    for (int64_t t = tok0 + (int64_t)blockIdx.x * kThreads + tid; t < a.n_slots; t += (int64_t)gridDim.x * kThreads) {
        a.slots[t] = -1;
        a.positions[t] = 0;
    }
    if (blockIdx.x != 0) return;
    if (page0 > a.n_free) status |= 1;
    if (tok0 > a.n_slots) status |= 4;
    status = __reduce_or_sync(0xffffffffu, status);
    longest = __reduce_max_sync(0xffffffffu, longest);
    __syncthreads();
    if (lane == 0) s.warp_tok[warp] = longest, s.warp_page[warp] = status;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kThreads / 32; ++w) {
            longest = max(longest, (uint32_t)s.warp_tok[w]);
            status |= (int)s.warp_page[w];
        }
        a.cu_new[0] = 0;
        a.counts[0] = saturated(tok0);
        a.counts[1] = (int32_t)min(page0, (int64_t)a.n_free);
        a.counts[2] = status;
        a.counts[3] = saturated(longest);
    }
}

}  // namespace

cudaError_t launch_page_tables(const TablesArgs &a, cudaStream_t stream) {
    // one CTA per 2048 slots or per two table rows, one wave at most
    const int64_t want = max((int64_t)a.n_slots / 2048, (int64_t)a.B / 2) + 1;
    page_tables_kernel<<<(unsigned)min(want, (int64_t)152), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
