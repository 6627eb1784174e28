// k_logprobs.cu -- log probabilities of given tokens, the distribution's entropy and its likeliest tokens, of every row of logits.
//
// With m = max x, Z = sum e^(x - m) and H = sum e^(x - m) (x - m):  log p_i = x_i - m - log Z,  entropy = log Z - H / Z.  One pass:
// every thread keeps a running (m, Z, H) of what it met, rescaled when its maximum grows (H gets (m - m') Z besides), and the
// triples of a row are joined in a fixed order.
//
// The likeliest tokens come from the same pass.  A token's place is a 64-bit key, its logit's ordered bits above the complement of
// its index, so that no two are alike and ties go to the lowest index.  A CTA keeps a threshold T that at least `top` of its keys
// reach: first the top-th largest of the threads' maxima over the first batch, later the top-th of what was gathered.  Tokens that reach T
// are gathered in shared memory, some tens to hundreds in a row, and cut back to `top` by comparing all with all when there are
// many.  A batch whose maximum, which the sums need anyway, is below T costs nothing more.  If a batch (rising logits, say)
// brings more than fits, T is raised from that batch's own maxima and what found no place is gathered again.
//
// What bounds it: the row is read once from HBM, at 4 bytes for some 10 instructions per logit.  One row takes a cluster of CTAs where rows
// are few, as many as the GPU has room for, each with a share of every batch.
#include <cooperative_groups.h>

#include "paged.cuh"

namespace gdn {
namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;    // per row: the largest cluster that every GPU of this kind can place
constexpr int kMaxTop = 32;
constexpr int kList = 1024;    // keys gathered
constexpr int kMany = 256;     // keys from which they are cut back
constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp_fast(float x) {  // 2^-21 relative near 0; below the normal range 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * kLog2e));
    return y;
}
// Larger is likelier; 0 is no token.  -0 counts as 0, NaN comes last.
__device__ __forceinline__ u64 key_of(float x, int i) {
    uint32_t b = __float_as_uint(x + 0.f);
    b = b & 0x80000000u ? ~b : b | 0x80000000u;
    if (x != x) b = 1;
    return (u64)b << 32 | (0xffffffffu - (uint32_t)i);
}
__device__ __forceinline__ float logit_of(u64 key) {
    const uint32_t b = (uint32_t)(key >> 32);
    return b <= 1 ? -INFINITY : __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}
__device__ __forceinline__ int token_of(u64 key) { return (int)(0xffffffffu - (uint32_t)key); }

// m = -FLT_MAX, z = h = 0: nothing met.  The differences are bounded so that a weight of 0 does not meet an infinity.
struct Sums {
    float m, z, h;
    __device__ __forceinline__ void raise(float to) {
        const float d = fmaxf(m - to, -1e4f), f = exp_fast(d);
        h = f * (h + d * z);
        z *= f;
        m = to;
    }
    __device__ __forceinline__ void join(Sums o) {
        const float top = fmaxf(m, o.m);
        raise(top);
        o.raise(top);
        z += o.z;
        h += o.h;
    }
};

template <typename T> __device__ __forceinline__ float element(const uint4 &u, int j);
template <> __device__ __forceinline__ float element<float>(const uint4 &u, int j) {
    return __uint_as_float(j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w);
}
template <> __device__ __forceinline__ float element<__nv_bfloat16>(const uint4 &u, int j) {
    const uint32_t w = j < 2 ? u.x : j < 4 ? u.y : j < 6 ? u.z : u.w;
    return __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
}

struct Shared {
    u64 list[kList];
    u64 best[kMaxTop];    // the largest keys after a cut, descending
    u64 maxima[kThreads];
    u64 threshold;
    int count;
    Sums part[kWarps];
    Sums sums;            // of this CTA
};

// The largest keys of s.list, to s.best and back to the list; T rises to the top-th.
__device__ void cut(Shared &s, int top) {
    const int tid = threadIdx.x, n = min(s.count, kList);
    if (tid < kMaxTop) s.best[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        const u64 mine = s.list[i];
        int above = 0;
        for (int j = 0; j < n; ++j) above += s.list[j] > mine;
        if (above < top) s.best[above] = mine;
    }
    __syncthreads();
    if (tid < top) s.list[tid] = s.best[tid];
    if (tid == 0) {
        s.count = min(n, top);
        s.threshold = max(s.threshold, s.best[top - 1]);
    }
    __syncthreads();
}

// T rises to the top-th largest of the threads' keys (0 where fewer threads have one).
__device__ void raise_threshold(Shared &s, int top, u64 mine) {
    const int tid = threadIdx.x;
    s.maxima[tid] = mine;
    __syncthreads();
    int above = 0;
#pragma unroll 8
    for (int j = 0; j < kThreads; ++j) above += s.maxima[j] > mine;
    if (above == top - 1 && mine > s.threshold) s.threshold = mine;
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) logprobs_kernel(LogprobArgs a, int ctas) {
    constexpr int N = 16 / sizeof(T), kVecs = 4, kBatch = kVecs * kThreads;
    __shared__ Shared s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x % ctas, row = blockIdx.x / ctas;
    const T *x = (const T *)a.logits + (int64_t)row * a.stride;
    const int head = min(a.V, (int)((16 - ((uintptr_t)x & 15)) & 15) / (int)sizeof(T));
    const int vecs = (a.V - head) / N, tail = head + vecs * N;  // whole 16 bytes; elements [0, head) and [tail, V) are read one by one
    const int batches = (vecs + kBatch * ctas - 1) / (kBatch * ctas);
    const uint4 *xv = reinterpret_cast<const uint4 *>(x + head);
    if (tid == 0) s.count = 0, s.threshold = 0;
    __syncthreads();

    Sums sums = {kLowest, 0.f, 0.f};
    // What a thread has of a batch: 4 x 16 bytes, and which of them are real.
    constexpr uint32_t kNone = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;  // -inf, which has no weight
    const uint4 none = make_uint4(kNone, kNone, kNone, kNone);
    uint4 in[kVecs];
    auto load = [&](int batch, uint4 (&to)[kVecs]) {
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int64_t i = ((int64_t)batch * ctas + cta) * kBatch + v * kThreads + tid;
            to[v] = i < vecs ? __ldcs(xv + i) : none;
        }
    };
    load(0, in);
    // batch `batches` is the row's ends, an element to a thread, which the first CTA has
    const int rounds = batches + (cta == 0 && (head > 0 || tail < a.V));
    bool first = true;
    for (int batch = 0; batch < rounds; ++batch) {
        uint32_t real = 0;
        int at[kVecs];  // index of a piece's first element
        uint4 next[kVecs];
        if (batch < batches) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                const int64_t i = ((int64_t)batch * ctas + cta) * kBatch + v * kThreads + tid;
                at[v] = head + (int)i * N;
                if (i < vecs) real |= ((1u << N) - 1) << (v * N);
            }
            if (batch + 1 < batches) load(batch + 1, next);
        } else {
            const int i = tid < head ? tid : tail + tid - head;
#pragma unroll
            for (int v = 0; v < kVecs; ++v) at[v] = i, in[v] = none;
            if (i < a.V) {
                real = 1;
                if constexpr (sizeof(T) == 4) in[0].x = __float_as_uint(x[i]);
                else in[0].x = 0xff800000u | *reinterpret_cast<const uint16_t *>(x + i);
            }
        }
        float most = -INFINITY;
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
            for (int j = 0; j < N; ++j) most = fmaxf(most, element<T>(in[v], j));
        if (most > sums.m) sums.raise(most);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            float z = 0.f, h = 0.f;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float y = element<T>(in[v], j) - sums.m, e = exp_fast(y);
                z += e;
                h += e * fmaxf(y, -200.f);  // -inf has e = 0
            }
            sums.z += z;
            sums.h += h;
        }
        if (a.top > 0) {
            auto largest = [&] {
                u64 key = 0;
#pragma unroll
                for (int v = 0; v < kVecs; ++v)
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        if (real >> (v * N + j) & 1) key = max(key, key_of(element<T>(in[v], j), at[v] + j));
                return key;
            };
            if (first) raise_threshold(s, a.top, largest());
            first = false;
            uint32_t left = 0;  // elements that found no place
            bool many = false;
            auto gather = [&](uint32_t which, u64 threshold) {
                left = 0;
                many = false;
#pragma unroll
                for (int v = 0; v < kVecs; ++v)
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        if (which >> (v * N + j) & 1) {
                            const u64 key = key_of(element<T>(in[v], j), at[v] + j);
                            if (key >= threshold) {
                                const int to = atomicAdd(&s.count, 1);
                                if (to < kList) s.list[to] = key;
                                else left |= 1u << (v * N + j);
                                many |= to >= kMany;
                            }
                        }
            };
            // nobody writes the threshold between here and the next barrier
            const u64 threshold = s.threshold;
            if (most >= logit_of(threshold)) gather(real, threshold);
            // rounds are few: after the first, T is at least the top-th of the threads' maxima of this very batch
            while (__syncthreads_or(many)) {
                if (__syncthreads_or(left != 0)) raise_threshold(s, a.top, largest());
                cut(s, a.top);
                many = false;
                if (left) gather(left, s.threshold);
            }
        }
        if (batch + 1 < batches) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v) in[v] = next[v];
        }
    }

    // ---- the CTA's sums and keys, then the row's
#pragma unroll
    for (int off = 16; off; off >>= 1)
        sums.join({__shfl_xor_sync(0xffffffffu, sums.m, off), __shfl_xor_sync(0xffffffffu, sums.z, off), __shfl_xor_sync(0xffffffffu, sums.h, off)});
    if (lane == 0) s.part[warp] = sums;
    __syncthreads();
    if (a.top > 0) cut(s, a.top);
    if (tid == 0) {
        Sums all = s.part[0];
        for (int w = 1; w < kWarps; ++w) all.join(s.part[w]);
        s.sums = all;
    }
    if (ctas > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        if (cta == 0) {
            if (a.top > 0 && tid < ctas * kMaxTop) s.list[tid] = cluster.map_shared_rank(&s, tid / kMaxTop)->best[tid % kMaxTop];
            if (tid == 0) {
                Sums all = s.sums;
                for (int c = 1; c < ctas; ++c) all.join(cluster.map_shared_rank(&s, c)->sums);
                s.sums = all;
                s.count = ctas * kMaxTop;
            }
        }
        cluster.sync();
        if (cta != 0) return;
        if (a.top > 0) cut(s, a.top);
    }
    __syncthreads();
    const Sums all = s.sums;
    const float log_z = logf(all.z);
    auto logprob = [&](float v) { return all.z == 0.f ? -INFINITY : v - all.m - log_z; };
    if (tid == 0) {
        const int token = a.tokens[row];
        float lp = 0.f;
        if (token >= 0 && token < a.V) {
            if constexpr (sizeof(T) == 4) lp = logprob(x[token]);
            else lp = logprob(__bfloat162float(x[token]));
        }
        a.logprobs[row] = lp;
        if (a.entropy) a.entropy[row] = all.z == 0.f ? 0.f : log_z - all.h / all.z;
    }
    if (tid < a.top) {
        const u64 key = s.best[tid];
        a.top_tokens[(int64_t)row * a.top + tid] = token_of(key);
        a.top_logprobs[(int64_t)row * a.top + tid] = logprob(logit_of(key));
    }
}

template <typename T>
cudaError_t launch(const LogprobArgs &a, cudaStream_t stream) {
    // CTAs to a row: doubled while all of them fit the GPU at once and each has a batch of its own
    const int64_t batch = (int64_t)4 * kThreads * (16 / sizeof(T));
    int ctas = 1;
    while (ctas < kMaxCtas && (int64_t)a.B * ctas * 2 <= 4 * 152 && batch * ctas < a.V) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.B * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, a, ctas);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs &a, cudaStream_t stream) {
    return a.dtype == GDN_BF16 ? launch<__nv_bfloat16>(a, stream) : launch<float>(a, stream);
}

}  // namespace gdn
