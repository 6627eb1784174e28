// k_logprobs.cu -- log probabilities of given tokens, the distribution's entropy and its likeliest tokens, of every row of logits.
//
// With m = max x, Z = sum e^(x - m) and H = sum e^(x - m) (x - m):  log p_i = x_i - m - log Z,  entropy = log Z - H / Z.  One pass:
// every thread keeps a running (m, Z, H) of what it met, rescaled when its maximum grows (H gets (m - m') Z besides), and the
// triples of a row are joined in a fixed order.
//
// The likeliest tokens come from the same pass.  A token's place is a 64-bit key, its logit's ordered bits above the complement of
// its index, so that no two are alike and ties go to the lowest index.  A CTA keeps a threshold T that at least `top` of its keys
// reach: first, of the threads' maxima over the first batch, the least of the eight warps' (top / 8)-th largest, and the top-th of what reaches
// that; then, whenever 64 more keys that reach T have been gathered in shared memory, the warp that brought the last of them takes the
// top-th of these 64.  So 100 to 200 of 100000 logits are gathered, no barrier is met on the way (one per batch cost more
// than all else together), and a batch whose maximum, which the sums need
// anyway, is below T costs nothing more.  At the end the list is cut by comparing all with all.  If more were brought than it holds (rising
// logits, say, or some 1500 of them in bf16, of which not all threads have one to start T from), the CTA goes over its share again with
// barriers: T is raised from the maxima of each part that brings too many.
//
// What bounds it: the row is read once from HBM, at 4 bytes for some 8 instructions per logit.  A thread copies its own 64 bytes of a batch to
// shared memory by cp.async, three batches ahead, and reads them back when it gets there: no barrier, no registers held by loads on their
// way, and a logit that the gathering wants is looked up by its number.  One row takes a cluster of CTAs where rows
// are few, as many as the GPU has room for, each with a share of every batch.  2047 rows of 100003 fp32 logits: 122 us without top tokens (6.7 TB/s, 99 %
// of a copy), 130 with 5, 146 with 20 (84 %), 178 with 32: what is gathered takes some 70 instructions each, in warps of their own, and the list's
// cuts; in bf16 71, 112, 130 and 149 us (409 MB), as the instructions per logit count more.  4 rows of 131072 bf16 logits with 5: 11 us, half of it
// the clusters' two joins and the cuts.
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
constexpr int kBlock = 64;     // keys from which a threshold is taken
constexpr int kMore = 224;     // keys over `top` from which a list is cut back in the second go
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

// Two sums (products) at once
__device__ __forceinline__ u64 pair(float lo, float hi) {
    u64 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(u64 x, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x)); }
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
    u64 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
    u64 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
    u64 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The pairs of 16 bytes: two of fp32, four of bf16
template <typename T> __device__ __forceinline__ void pairs_of(const uint4 &u, u64 (&x)[8 / sizeof(T)]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8 / (int)sizeof(T); ++i) {
        if constexpr (sizeof(T) == 4) x[i] = pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else x[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
}
__device__ __forceinline__ float value(const float *p) { return *p; }
__device__ __forceinline__ float value(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void cp16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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
    const u64 threshold = s.threshold;  // `top` keys at least reach it
    for (int i = tid; i < n; i += kThreads) {
        const u64 mine = s.list[i];
        if (mine < threshold) continue;
        int above = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) above += s.list[j] > mine;
        if (above < top) s.best[above] = mine;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) s.list[i] = i < top ? s.best[i] : 0;  // no key stands in the list twice
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

// T from the threads' largest keys: each warp's (top / 8)-th largest, of these the least.
__device__ void first_threshold(Shared &s, int top, u64 mine) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t high = 0, low = 0;
    for (int i = 0; i < (top + kWarps - 1) / kWarps; ++i) {
        high = __reduce_max_sync(0xffffffffu, (uint32_t)(mine >> 32));
        low = __reduce_max_sync(0xffffffffu, (uint32_t)(mine >> 32) == high ? (uint32_t)mine : 0u);
        if (mine == ((u64)high << 32 | low)) mine = 0;  // keys are all different
    }
    if (lane == 0) s.maxima[warp] = (u64)high << 32 | low;
    __syncthreads();
    if (threadIdx.x == 0) {
        u64 least = s.maxima[0];
        for (int w = 1; w < kWarps; ++w) least = min(least, s.maxima[w]);
        s.threshold = least;
    }
    __syncthreads();
}

// T rises to the top-th of 64 keys of the list, by one warp.  Keys that are not written yet count as none.
__device__ void raise_from_block(Shared &s, int top, int block) {
    const volatile u64 *keys = s.list + block * kBlock;
    const u64 a = keys[threadIdx.x & 31], b = keys[32 + (threadIdx.x & 31)];
    int above_a = 0, above_b = 0;
#pragma unroll 8
    for (int j = 0; j < kBlock; ++j) {
        const u64 x = keys[j];
        above_a += x > a;
        above_b += x > b;
    }
    if (above_a == top - 1 && a) atomicMax(&s.threshold, a);
    if (above_b == top - 1 && b) atomicMax(&s.threshold, b);
}

constexpr int kVecs = 4, kAhead = 4, kBatch = kVecs * kThreads;  // 16-byte pieces of a thread's batch; batches on their way or worked on
constexpr int kSmem = kAhead * kBatch * 16;

// The list once more, with barriers: parts of 16 logits per thread whose keys are gathered until there are too many, then cut.  The parts
// are those of this CTA's batches and no others: the row's other CTAs may have come through with theirs.
template <typename T> __device__ __noinline__ void gather_again(Shared &s, const LogprobArgs &a, const T *x, int ctas, int cta, int head, int vecs) {
    constexpr int N = 16 / sizeof(T), kEach = 16, kParts = kVecs * N / kEach;  // of a batch
    const int tid = threadIdx.x, tail = head + vecs * N, parts = (vecs + kBatch * ctas - 1) / (kBatch * ctas) * kParts;
    __syncthreads();
    if (tid == 0) s.count = 0;
    __syncthreads();
    for (int part = 0; part < parts + (cta == 0); ++part) {  // the last has the row's ends, in the first CTA
        auto index = [&](int i) {  // a.V or more: none
            if (part == parts) return i > 0 ? a.V : tid < head ? tid : tail + tid - head;
            const int vec = (part / kParts * ctas + cta) * kBatch + (part % kParts * (kEach / N) + i / N) * kThreads + tid;
            return vec < vecs ? head + vec * N + i % N : a.V;
        };
        uint32_t left = 0;  // those that found no place
        bool many = false;
        auto gather = [&](uint32_t which) {
            const u64 threshold = s.threshold;  // which nobody writes between here and the next barrier
            left = 0;
            many = false;
            for (int i = 0; i < kEach; ++i) {
                if (!(which >> i & 1) || index(i) >= a.V) continue;
                const u64 key = key_of(value(x + index(i)), index(i));
                if (key < threshold) continue;
                const int to = atomicAdd(&s.count, 1);
                if (to < kList) s.list[to] = key;
                else left |= 1u << i;
                many |= to >= a.top + kMore;
            }
        };
        gather(~0u);
        // rounds are few: after the first, T is at least the top-th of the threads' maxima of this very part
        while (__syncthreads_or(many)) {
            if (__syncthreads_or(left != 0)) {
                u64 key = 0;
                for (int i = 0; i < kEach; ++i)
                    if (index(i) < a.V) key = max(key, key_of(value(x + index(i)), index(i)));
                raise_threshold(s, a.top, key);
            }
            cut(s, a.top);
            many = false;
            if (left) gather(left);
        }
    }
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) logprobs_kernel(LogprobArgs a, int ctas) {
    constexpr int N = 16 / sizeof(T), kEach = kVecs * N;
    extern __shared__ __align__(16) uint4 slots[];  // [kAhead][kVecs][kThreads]: a thread's own
    __shared__ Shared s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x % ctas, row = blockIdx.x / ctas;
    const T *x = (const T *)a.logits + (int64_t)row * a.stride;
    const int head = min(a.V, (int)((16 - ((uintptr_t)x & 15)) & 15) / (int)sizeof(T));
    const int vecs = (a.V - head) / N, tail = head + vecs * N;  // whole 16 bytes; elements [0, head) and [tail, V) are read one by one
    const int batches = (vecs + kBatch * ctas - 1) / (kBatch * ctas);
    const uint4 *xv = reinterpret_cast<const uint4 *>(x + head);
    if (tid == 0) s.count = 0, s.threshold = 0;
    for (int i = tid; i < kList; i += kThreads) s.list[i] = 0;
    __syncthreads();

    Sums sums = {kLowest, 0.f, 0.f};
    constexpr uint32_t kNone = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;  // -inf, which has no weight
    const uint4 none = make_uint4(kNone, kNone, kNone, kNone);
    auto vec_at = [&](int batch, int v) { return (batch * ctas + cta) * kBatch + v * kThreads + tid; };  // below 2^30
    auto slot_of = [&](int batch, int v) -> uint4 & { return slots[((batch & (kAhead - 1)) * kVecs + v) * kThreads + tid]; };
    auto copy = [&](int batch) {
        if (batch < batches) {
            const int first = (batch * ctas + cta) * kBatch;
            if (first + kBatch <= vecs) {
#pragma unroll
                for (int v = 0; v < kVecs; ++v) cp16(&slot_of(batch, v), xv + first + tid + v * kThreads);
            } else {
#pragma unroll
                for (int v = 0; v < kVecs; ++v)
                    if (vec_at(batch, v) < vecs) cp16(&slot_of(batch, v), xv + vec_at(batch, v));
                    else slot_of(batch, v) = none;
            }
        }
        cp_commit();
    };
#pragma unroll
    for (int b = 0; b < kAhead - 1; ++b) copy(b);
    // batch `batches` is the row's ends, an element to a thread, which the first CTA has
    const int rounds = batches + (cta == 0 && (head > 0 || tail < a.V));
#pragma unroll 1
    for (int batch = 0; batch < rounds; ++batch) {
        cp_wait<kAhead - 2>();
        if (batch == batches) {
            const int i = tid < head ? tid : tail + tid - head;
            uint4 one = none;
            if (i < a.V) {
                if constexpr (sizeof(T) == 4) one.x = __float_as_uint(x[i]);
                else one.x = 0xff800000u | *reinterpret_cast<const uint16_t *>(x + i);
            }
            slot_of(batch, 0) = one;
#pragma unroll
            for (int v = 1; v < kVecs; ++v) slot_of(batch, v) = none;
        }
        copy(batch + kAhead - 1);  // over the batch before this one
        float most = -INFINITY;
        u64 in[kVecs][N / 2];
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            pairs_of<T>(slot_of(batch, v), in[v]);
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                float lo, hi;
                unpair(in[v][j], lo, hi);
                most = fmaxf(most, fmaxf(lo, hi));
            }
        }
        if (most > sums.m) sums.raise(most);
        const u64 minus = pair(-sums.m, -sums.m), scale = pair(kLog2e, kLog2e);
        u64 z = 0, h = 0;
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                const u64 y = add2(in[v][j], minus);
                float lo, hi, y0, y1;
                unpair(mul2(y, scale), lo, hi);
                unpair(y, y0, y1);
                const u64 e = pair(ex2(lo), ex2(hi));
                z = add2(z, e);
                h = fma2(e, pair(fmaxf(y0, -200.f), fmaxf(y1, -200.f)), h);  // -inf has e = 0
            }
        float lo, hi;
        unpair(z, lo, hi);
        sums.z += lo + hi;
        unpair(h, lo, hi);
        sums.h += lo + hi;
        if (a.top > 0) {
            // logit i of the thread's kEach, and its index
            const int from = batch == batches ? (tid < head ? tid : tail + tid - head) : head + ((batch * ctas + cta) * kBatch + tid) * N;
            auto key_at = [&](int i) { return key_of(value((const T *)&slot_of(batch, i / N) + i % N), from + i / N * (kThreads * N) + i % N); };
            auto real_of = [&] {
                uint32_t real = 0;
                if (batch == batches) real = from < a.V;
                else
#pragma unroll
                    for (int v = 0; v < kVecs; ++v) real |= vec_at(batch, v) < vecs ? ((1u << N) - 1) << (v * N) : 0u;
                return real;
            };
            if (batch == 0) {
                const uint32_t real = real_of();
                int at = -1;
                float best = 0.f;
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    float pr[2];
                    unpair(in[i / N][i % N / 2], pr[0], pr[1]);
                    if ((real >> i & 1) && (at < 0 || pr[i & 1] > best)) at = i, best = pr[i & 1];
                }
                first_threshold(s, a.top, at < 0 ? 0 : key_at(at));
            }
            const u64 threshold = *(volatile u64 *)&s.threshold;
            const float least = logit_of(threshold);
            int full = -1;  // a block of the list that this thread completed
            if (most >= least) {
                uint32_t which = 0;
#pragma unroll
                for (int v = 0; v < kVecs; ++v)
#pragma unroll
                    for (int j = 0; j < N / 2; ++j) {
                        float lo, hi;
                        unpair(in[v][j], lo, hi);
                        which |= (lo < least ? 0u : 1u << (v * N + 2 * j)) | (hi < least ? 0u : 2u << (v * N + 2 * j));  // NaN is looked at too
                    }
                which &= real_of();
#pragma unroll 1
                while (which) {
                    const int i = __ffs(which) - 1;
                    which &= which - 1;
                    const u64 key = key_at(i);
                    if (key < threshold) continue;
                    const int to = atomicAdd(&s.count, 1);
                    if (to < kList) *(volatile u64 *)&s.list[to] = key;
                    if (to < kList && to % kBlock == kBlock - 1) full = to / kBlock;
                }
            }
            // (of two blocks completed by one warp at once the later)
            if (__any_sync(0xffffffffu, full >= 0)) raise_from_block(s, a.top, (int)__reduce_max_sync(0xffffffffu, (unsigned)(full + 1)) - 1);
            if (batch == 0) {
                __syncthreads();
                if (s.count <= kList) cut(s, a.top);
            }
        }
    }
    cp_wait<0>();

    // ---- the CTA's sums and keys, then the row's
#pragma unroll
    for (int off = 16; off; off >>= 1)
        sums.join({__shfl_xor_sync(0xffffffffu, sums.m, off), __shfl_xor_sync(0xffffffffu, sums.z, off), __shfl_xor_sync(0xffffffffu, sums.h, off)});
    if (lane == 0) s.part[warp] = sums;
    __syncthreads();
    if (a.top > 0) {
        if (s.count > kList) gather_again(s, a, x, ctas, cta, head, vecs);
        cut(s, a.top);
    }
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
    const cudaError_t e = cudaFuncSetAttribute(logprobs_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    // CTAs to a row: doubled while all of them fit the GPU at once and each has a batch of its own
    const int64_t batch = (int64_t)kBatch * 16 / sizeof(T);
    int ctas = 1;
    while (ctas < kMaxCtas && (int64_t)a.B * ctas * 2 <= 3 * 152 && batch * ctas < a.V) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.B * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
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
