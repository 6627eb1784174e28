// k_sample.cu -- the next token of every row of logits.
//
// With y = (x - max x) / T and w = exp(y): the top_k largest w stay (ties by index),
// of them the shortest prefix in descending order that holds top_p of their mass,
// of it what is at least min_p of the largest w.  The token is the largest
// y + Gumbel(u) over what stays; -log(-log u) of a uniform u is a Gumbel variable, and
// the maximum over the tokens is distributed as a draw from w (normalised).  The race
// needs no running sum over the kept tokens, so its result does not hang on the
// rounding of one.
//
// What bounds it: the row is read once from HBM; everything after works on few tokens, or on the
// row in L2, where instructions per token count (about 10 to 20 in each pass below).  A
// cluster of CTAs shares a row, as many as fill the GPU, each with a slice:
//   1. one pass for the maximum, the minimum, the sum of weights and every thread's own maximum;
//   2. a threshold that no kept token is below.  For top_k: among the threads' maxima, the ceil(k / CTAs)-th largest of
//      every CTA, and the least of those (k tokens at least are as large).  For top_p: tokens below (1 - p) M / V hold
//      (1 - p) M together at most, so the prefix of mass p M ends above it.  What passes the threshold, a few hundred
//      tokens as a rule, is gathered, sorted and cut in the first CTA's shared memory;
//   3. if it is more than fits (flat rows, large k), a histogram of 2048 bins over y, of counts and of what the
//      weights lack to their bin's upper edge (32-bit atomics both), finds the bins where the cut falls: one, or
//      a few where sums of mass leave it open.  Only their tokens are gathered, with the exact mass above them;
//   4. if even those are more than fit (thousands of equal logits), the first CTA finds the cut digit by digit of the
//      sorting key, a pass over the row each;
//   5. the race.  The largest token is always kept and its Gumbel is above -3.2, no Gumbel is above 16.7:
//      tokens with y < -20 cannot win, and their noise is not read.  The others race on approximate scores, and
//      only those within 10^-3 of a thread's best are decided on exact ones.
//
// Masses are whole numbers in units of 2^-40 of the largest weight, summed in 64 bits: exact
// sums, whatever order the atomics come in.  The weights in masses are 2^x approximations
// (2^-21); w >= min_p and the race are decided in IEEE fp32 with accurate exp and log.
#include <cooperative_groups.h>

#include "paged.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;   // per row: the largest cluster every GPU of this kind can place
constexpr int kList = 2048;   // gathered tokens
constexpr int kBins = 2048;
constexpr float kUnit = 1099511627776.f;  // 2^40
constexpr float kReach = 28.f;            // in y: 40 ln 2, below which a mass rounds to 0
constexpr float kLack = 131072.f;         // 2^17: resolution of a weight's lack relative to its bin's upper edge
using u64 = unsigned long long;

__device__ __forceinline__ float clean(float x) {  // NaN is -inf, +inf is the largest number
    return fminf(fmaxf(x, -INFINITY), 3.402823466e38f);
}
// Ordered: larger floats have larger keys; -0 and 0 have one.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
// The sorting key of a token: its logit's ordered bits, then the complement of its index.
__device__ __forceinline__ u64 full_key(float v, int i) { return (u64)key_of(v) << 32 | (uint32_t)~i; }
__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

struct Best { float v; int i; };
__device__ __forceinline__ Best better(Best a, Best b) {
    return b.v > a.v || (b.v == a.v && (unsigned)b.i < (unsigned)a.i) ? b : a;
}

struct Shared {
    u64 list[kList];
    u64 mass[kBins];
    uint32_t count[kBins], lack[kBins];
    u64 sums[kWarps];
    Best bests[kWarps];
    float parts[kWarps];
    int n, found;          // tokens gathered; bin or rank found
    u64 before, digit;
    // read by the row's other CTAs, each written once between two barriers of the cluster
    struct {
        Best top, won;
        float low, sum, least;
        int gathered;      // tokens gathered, or more than kList
        u64 mass;          // of the tokens above the gathered bins
        int lo, hi;        // the first CTA's: bins to gather next; lo < 0: none, race
        u64 cut;           // the first CTA's: the smallest key that top_k and top_p keep
    } x;
};

__device__ Best block_best(Best x, Shared &s) {
    for (int off = 16; off; off >>= 1)
        x = better(x, {__shfl_xor_sync(0xffffffffu, x.v, off), __shfl_xor_sync(0xffffffffu, x.i, off)});
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.bests[threadIdx.x >> 5] = x;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) x = better(x, s.bests[w]);
    return x;
}
template <typename F>
__device__ float block_fold(float x, Shared &s, F f) {
    for (int off = 16; off; off >>= 1) x = f(x, __shfl_xor_sync(0xffffffffu, x, off));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.parts[threadIdx.x >> 5] = x;
    __syncthreads();
    x = s.parts[0];
    for (int w = 1; w < kWarps; ++w) x = f(x, s.parts[w]);
    return x;
}
// Sum over the threads before this one; `all` gets the sum over the block.
__device__ u64 block_before(u64 x, u64 &all, Shared &s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 incl = x;
    for (int off = 1; off < 32; off <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
    }
    __syncthreads();
    if (lane == 31) s.sums[warp] = incl;
    __syncthreads();
    u64 base = 0;
    all = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) base += s.sums[w];
        all += s.sums[w];
    }
    return base + incl - x;
}

// f(logits, how many, index of the first) for the tokens [from, to) of a row, in pieces of 16 bytes, four of which are
// in flight per thread; a thread meets its tokens in ascending order.  f returns false to end the thread's pass.
template <typename T, typename F>
__device__ __forceinline__ void each_piece(const T *row, int from, int to, F f) {
    constexpr int kPer = 16 / sizeof(T);
    const int tid = threadIdx.x;
    const T *x = row + from;
    const int n = to - from;
    const int head = min(n, (int)((16 - ((uintptr_t)x & 15)) & 15) / (int)sizeof(T)), pieces = (n - head) / kPer;
    float v[kPer];
    if (tid < head) {
        v[0] = clean(io<T>::ld(x + tid));
        if (!f(v, 1, from + tid)) return;
    }
    const uint4 *p = (const uint4 *)(x + head);
    for (int i0 = tid; i0 < pieces; i0 += 4 * kThreads) {
        uint4 w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i0 + u * kThreads < pieces) w[u] = p[i0 + u * kThreads];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (i0 + u * kThreads >= pieces) break;
            const uint32_t q[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                if constexpr (sizeof(T) == 2) v[e] = clean(__uint_as_float(e & 1 ? q[e / 2] & 0xffff0000u : q[e / 2] << 16));
                else v[e] = clean(__uint_as_float(q[e]));
            }
            if (!f(v, kPer, from + head + (i0 + u * kThreads) * kPer)) return;
        }
    }
    const int t = head + pieces * kPer + tid;
    if (t < n) {
        v[0] = clean(io<T>::ld(x + t));
        f(v, 1, from + t);
    }
}
// f(logit, index), token by token.
template <typename T, typename F>
__device__ __forceinline__ void each(const T *row, int from, int to, F f) {
    constexpr int kPer = 16 / sizeof(T);
    each_piece(row, from, to, [&](const float (&v)[kPer], int n, int at) {
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            if (e < n && !f(v[e], at + e)) return false;
        return true;
    });
}

// Appends to the list (or only counts, past its room); false once it has overflowed.
__device__ __forceinline__ bool gather(Shared &s, u64 key) {
    const unsigned peers = __activemask();
    const int lane = threadIdx.x & 31, first = __ffs(peers) - 1;
    int at = 0;
    if (lane == first) at = atomicAdd(&s.n, __popc(peers));
    at = __shfl_sync(peers, at, first) + __popc(peers & ((1u << lane) - 1));
    if (at < kList) s.list[at] = key;
    return at < kList;
}

// Sorts the s.n gathered keys in descending order.
__device__ void sort_list(Shared &s) {
    int size = 2;
    while (size < s.n) size <<= 1;
    for (int i = s.n + threadIdx.x; i < size; i += kThreads) s.list[i] = 0;
    for (int run = 2; run <= size; run <<= 1)
        for (int gap = run >> 1; gap; gap >>= 1) {
            __syncthreads();
            for (int p = threadIdx.x; p < size / 2; p += kThreads) {
                const int i = 2 * p - (p & (gap - 1)), j = i + gap;
                const u64 x = s.list[i], y = s.list[j];
                if ((x < y) == ((i & run) == 0)) s.list[i] = y, s.list[j] = x;
            }
        }
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(SampleArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared &s = *(Shared *)raw;
    constexpr int kPer = 16 / sizeof(T);
    auto cluster = cooperative_groups::this_cluster();
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
    auto peer = [&](int r) -> const Shared & { return *cluster.map_shared_rank(&s, r); };
    const int b = blockIdx.x / ctas, tid = threadIdx.x;
    const T *x = (const T *)a.logits + b * a.logits_stride;
    const float *u = a.noise + b * a.noise_stride;
    const int share = (a.V + ctas * kPer - 1) / (ctas * kPer) * kPer;
    const int from = min(a.V, rank * share), to = min(a.V, from + share);
    const float t = a.temperature ? a.temperature[b] : 1.f;
    const bool greedy = !(t > 0.f);
    const int k = a.top_k ? a.top_k[b] : 0;
    const float p = a.top_p ? a.top_p[b] : 1.f, min_p = a.min_p ? a.min_p[b] : 0.f;
    const bool by_k = !greedy && k > 0 && k < a.V, by_p = !greedy && p < 1.f;
    // y log2(e) per unit of x, kept off 0 and infinity: 0 and infinite differences stay what they are
    auto bounded = [](float f) { return fmaxf(fminf(f, 1e30f), 1e-37f); };
    const float rate = bounded(1.4426950408889634f / t);

    // 1. maximum, minimum, sum of weights
    Best top = {-INFINITY, -1};
    float sum = 0.f, low = INFINITY;
    each_piece(x, from, to, [&](const float (&v)[kPer], int n, int at) {
        float m = v[0];
#pragma unroll
        for (int e = 1; e < kPer; ++e)
            if (e < n) m = fmaxf(m, v[e]);
        if (m > top.v) {
            sum *= ex2((top.v - m) * rate);
            top.v = m;
            int i = 0;
#pragma unroll
            for (int e = kPer - 1; e >= 0; --e)
                if (e < n && v[e] == m) i = e;
            top.i = at + i;
        }
        if (!greedy && top.i >= 0) {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (e < n) {
                    sum += ex2((v[e] - top.v) * rate);
                    low = fminf(low, v[e] > -INFINITY ? v[e] : INFINITY);
                }
        }
        return true;
    });
    const float mine = top.v;
    top = block_best(top, s);
    if (!greedy) {
        sum = block_fold(mine > -INFINITY ? sum * ex2((mine - top.v) * rate) : 0.f, s, [](float y, float z) { return y + z; });
        low = block_fold(low, s, [](float y, float z) { return fminf(y, z); });
    }
    float least = -INFINITY;  // a logit that no kept token is below
    if (by_k) {
        const int need = (k + ctas - 1) / ctas;
        if (need <= kThreads) {
            const uint32_t own = mine > -INFINITY ? key_of(mine) : 0u;
            uint32_t key = 0;
#pragma unroll 1
            for (int bit = 31; bit >= (sizeof(T) == 2 ? 16 : 0); --bit) {
                const uint32_t next = key | 1u << bit;
                if (__syncthreads_count(own >= next) >= need) key = next;
            }
            if (key) least = value_of(key);
        }
    }
    if (tid == 0) s.x.top = top, s.x.sum = sum, s.x.low = low, s.x.least = least;
    cluster.sync();
    for (int r = 0; r < ctas; ++r) {
        top = better(top, peer(r).x.top);
        low = fminf(low, peer(r).x.low);
        least = fminf(least, peer(r).x.least);
    }
    float total = 0.f;
    for (int r = 0; r < ctas; ++r)
        if (peer(r).x.top.i >= 0) total += peer(r).x.sum * ex2((peer(r).x.top.v - top.v) * rate);

    auto finish = [&](Best won) {  // thread 0 of the first CTA
        if (won.i < 0) won = top;  // min_p above 1 leaves nothing: the largest stays
        a.tokens[b] = won.i;
        if (a.logprobs) a.logprobs[b] = won.i < 0 ? -INFINITY : greedy ? 0.f : (clean(io<T>::ld(x + won.i)) - top.v) / t - logf(total);
    };
    if (top.i < 0 || greedy) {
        if (rank == 0 && tid == 0) finish(top);
        cluster.sync();  // no CTA leaves while another may read its shared memory
        return;
    }

    auto mass = [&](float v) { return (u64)(ex2((v - top.v) * rate) * kUnit + 0.5f); };
    // a logit below (side -1) or above (side 1) which w < f (w >= f), with room for every rounding on the way
    auto logit_of = [&](float f, float side) {
        const float d = t * logf(f);
        return top.v + d + side * (1e-5f * (fabsf(top.v) + fabsf(d)) + 1e-3f * t);
    };
    const float min_logit = min_p > 0.f ? logit_of(fminf(min_p, 1.f), -1.f) : -INFINITY;
    auto goal_of = [&](double m) {  // p of mass m, at least one unit: the largest token always stays
        const double g = ceil((double)fmaxf(p, 0.f) * m);
        return g < 1.0 ? 1ull : (u64)g;
    };
    // exact score of a token, {-inf, -1} if min_p or a weight of 0 rules it out
    auto score = [&](float v, int i) -> Best {
        const float y = (v - top.v) / t, w = expf(y);
        if (!(w > 0.f) || w < min_p) return {-INFINITY, -1};
        const float r = fminf(fmaxf(u[i], 2.3283064365386963e-10f), 0.999999940395355f);
        return {y - logf(-logf(r)), i};
    };
    // the first CTA takes over the tokens that the others have gathered; false if they are too many
    auto collect = [&]() {
        int n = 0;
        for (int r = 0; r < ctas; ++r) n += peer(r).x.gathered;
        if (n > kList) return false;
        int at = s.x.gathered;
        for (int r = 1; r < ctas; ++r) {
            const int m = peer(r).x.gathered;
            for (int i = tid; i < m; i += kThreads) s.list[at + i] = peer(r).list[i];
            at += m;
        }
        __syncthreads();
        if (tid == 0) s.n = n;
        __syncthreads();
        sort_list(s);
        return true;
    };
    // Over the first `limit` tokens of the sorted list, with the mass `start` before them: s.found = the first rank whose
    // running mass reaches goal (kList: none).  Returns the mass at the end.
    auto in_list = [&](int limit, u64 start, u64 goal) {
        constexpr int kEach = kList / kThreads;
        u64 own = 0, all, m[kEach];
        for (int e = 0; e < kEach; ++e) {
            const int r = tid * kEach + e;
            m[e] = r < limit ? mass(value_of((uint32_t)(s.list[r] >> 32))) : 0;
            own += m[e];
        }
        u64 at = start + block_before(own, all, s);
        if (tid == 0) s.found = kList;
        __syncthreads();
        for (int e = 0; e < kEach; ++e) {
            if (at < goal && at + m[e] >= goal) s.found = tid * kEach + e;
            at += m[e];
        }
        __syncthreads();
        return start + all;
    };

    u64 cut = 0;  // the smallest key that top_k and top_p keep
    if (by_k || by_p) {
        // 2. gather what passes the threshold
        if (!(by_k && by_p)) least = fmaxf(least, min_logit);  // with both, all of K counts in its mass
        if (by_p && !by_k) least = fmaxf(least, logit_of((1.f - fmaxf(p, 0.f)) * total / (float)a.V, -1.f));
        if (tid == 0) s.n = 0;
        __syncthreads();
        each(x, from, to, [&](float v, int i) { return v >= least && v > -INFINITY ? gather(s, full_key(v, i)) : true; });
        __syncthreads();
        if (tid == 0) s.x.gathered = min(s.n, kList + 1);
        cluster.sync();
        int n = 0;
        for (int r = 0; r < ctas; ++r) n += peer(r).x.gathered;
        if (n <= kList) {
            if (rank == 0) {
                collect();
                const int limit = by_k ? min(n, k) : n;
                int keep = limit;
                if (by_p) {
                    const double m = by_k ? (double)in_list(limit, 0, ~0ull) : (double)total * (double)kUnit;
                    in_list(limit, 0, goal_of(m));
                    keep = min(limit, s.found + 1);
                }
                Best won = {-INFINITY, -1};
                for (int r = tid; r < keep; r += kThreads) {
                    const u64 key = s.list[r];
                    won = better(won, score(value_of((uint32_t)(key >> 32)), (int)~(uint32_t)key));
                }
                won = block_best(won, s);
                if (tid == 0) finish(won);
            }
            cluster.sync();
            return;
        }
        // 3. histogram over y, from the largest logit down to where no cut can be below
        const float bottom = fmaxf(fmaxf(top.v - kReach * t, low), by_p && !by_k ? least : -INFINITY);
        const float scale = bounded((float)kBins / (top.v - bottom));
        const float width = (top.v - bottom) / (t * kBins);  // of a bin, in y
        auto bin_of = [&](float v) { return (int)fminf((top.v - v) * scale, (float)(kBins - 1)); };
        for (int i = tid; i < kBins; i += kThreads) s.count[i] = s.lack[i] = 0;
        __syncthreads();
        each(x, from, to, [&](float v, int i) {
            if (v > -INFINITY && (by_k || v >= least)) {
                const float d = fminf((top.v - v) * scale, (float)(kBins - 1));
                const int bin = (int)d;
                const float f = (d - (float)bin) * width;
                atomicAdd(&s.count[bin], 1u);
                if (by_p) atomicAdd(&s.lack[bin], (uint32_t)((f - 0.5f * f * f) * kLack));  // 1 - exp(-f)
            }
            return true;
        });
        cluster.sync();
        // the first bin whose running sum reaches `goal` (s.found, with the sum before it in s.before), or kBins
        auto find_bin = [&](u64 goal, bool of_mass) {
            constexpr int kEach = kBins / kThreads;
            u64 own = 0, all;
            for (int e = 0; e < kEach; ++e) own += of_mass ? s.mass[tid * kEach + e] : s.count[tid * kEach + e];
            u64 at = block_before(own, all, s);
            if (tid == 0 && all < goal) s.found = kBins;
            if (at < goal && at + own >= goal) {
                int e = 0;
                for (;; ++e) {
                    const u64 y = of_mass ? s.mass[tid * kEach + e] : s.count[tid * kEach + e];
                    if (at + y >= goal) break;
                    at += y;
                }
                s.found = tid * kEach + e;
                s.before = at;
            }
            __syncthreads();
        };
        // the first CTA's decisions
        int bin_k = kBins, rank_k = 0;
        bool want_p = false, slow = false;
        u64 goal = 0;
        auto set_plan = [&](int lo, int hi) {
            if (tid == 0) s.x.lo = lo, s.x.hi = hi, s.x.cut = cut;
        };
        auto plan_p = [&](int limit) {  // the bins that may hold the end of the mass `goal`: sums are good to 2^-15 and V units
            find_bin(max((u64)((double)goal * (1.0 - 1.0 / 8192)), 1ull), true);
            const int lo = s.found;
            __syncthreads();
            find_bin((u64)((double)goal * (1.0 + 1.0 / 8192)) + 1, true);
            const int hi = min(min(s.found, kBins - 1), limit);
            __syncthreads();
            want_p = true;
            if (lo > hi) set_plan(-1, 0);  // less mass than that in all: everything stays
            else set_plan(lo, hi);
        };
        if (rank == 0) {
            for (int i = tid; i < kBins; i += kThreads) {
                uint32_t c = 0, l = 0;
                for (int r = 0; r < ctas; ++r) c += peer(r).count[i], l += peer(r).lack[i];
                s.count[i] = c;
                const double edge = (double)ex2(-(float)i * width * 1.4426950408889634f) * (double)kUnit;
                s.mass[i] = (u64)(edge * ((double)c - (double)l / (double)kLack));
            }
            __syncthreads();
            if (by_k) {
                find_bin((u64)k, false);
                bin_k = s.found;
                rank_k = k - (int)s.before;
                __syncthreads();
            }
            if (bin_k < kBins) set_plan(bin_k, bin_k);
            else if (by_p) goal = goal_of((double)total * (double)kUnit), plan_p(kBins - 1);
            else set_plan(-1, 0);  // fewer than k finite logits
        }
        for (;;) {
            cluster.sync();
            const int lo = peer(0).x.lo, hi = peer(0).x.hi;
            cut = peer(0).x.cut;
            if (lo < 0) break;
            u64 above = 0;
            if (tid == 0) s.n = 0;
            __syncthreads();
            each(x, from, to, [&](float v, int i) {
                if (!(v > -INFINITY)) return true;
                const int bin = bin_of(v);
                if (by_p && bin < lo) above += mass(v);
                if (bin >= lo && bin <= hi) gather(s, full_key(v, i));
                return true;
            });
            u64 all = 0;
            block_before(above, all, s);
            if (tid == 0) s.x.gathered = min(s.n, kList + 1), s.x.mass = all;
            cluster.sync();
            if (rank != 0) continue;
            above = 0;
            for (int r = 0; r < ctas; ++r) above += peer(r).x.mass;
            if (!collect()) {
                slow = true;
            } else if (!want_p) {
                cut = s.list[rank_k - 1];
                if (!by_p) {
                    set_plan(-1, 0);
                } else {
                    goal = goal_of((double)in_list(rank_k, above, ~0ull));
                    if (goal > above) {
                        in_list(rank_k, above, goal);
                        cut = s.list[min(s.found, rank_k - 1)];
                        set_plan(-1, 0);
                    } else {
                        plan_p(bin_k - 1);
                    }
                }
            } else {
                const u64 end = in_list(s.n, above, goal);
                // outside what the bins' sums allow for (a bin of over 2^21 tokens, say): settle it exactly
                if (above >= goal || s.n == 0 || (end < goal && hi < min(kBins, bin_k) - 1)) slow = true;
                else cut = s.list[min(s.found, s.n - 1)];
                set_plan(-1, 0);
            }
            if (slow) {
                // 4. digit by digit: the key of the last token of the shortest descending prefix, among keys >= floor, whose
                // measure (tokens, or mass) reaches goal
                auto descend = [&](u64 goal, bool of_mass, u64 floor) {
                    u64 prefix = 0, before = 0;
                    for (int shift = 56; shift >= 0; shift -= 8) {
                        __syncthreads();
                        if (tid < 256) s.mass[tid] = 0;
                        __syncthreads();
                        each(x, 0, a.V, [&](float v, int i) {
                            const u64 key = full_key(v, i);
                            if (v > -INFINITY && key >= floor && (shift == 56 || (key >> (shift + 8)) == prefix))
                                atomicAdd(&s.mass[(key >> shift) & 255], of_mass ? mass(v) : 1ull);
                            return true;
                        });
                        __syncthreads();
                        if (tid == 0) {
                            u64 at = before;
                            int d = 255;
                            for (; d > 0 && at + s.mass[d] < goal; --d) at += s.mass[d];
                            s.digit = d;
                            s.before = at;
                        }
                        __syncthreads();
                        prefix = prefix << 8 | s.digit;
                        before = s.before;
                    }
                    return prefix;
                };
                cut = bin_k < kBins ? descend((u64)k, false, 0) : 0;
                if (by_p) {
                    u64 own = 0;
                    each(x, 0, a.V, [&](float v, int i) {
                        if (v > -INFINITY && full_key(v, i) >= cut) own += mass(v);
                        return true;
                    });
                    block_before(own, all, s);
                    const u64 c = descend(min(goal_of((double)all), all), true, cut);
                    cut = c > cut ? c : cut;
                }
                set_plan(-1, 0);
            }
        }
    }

    // 5. the race over the row
    const float cut_v = cut ? value_of((uint32_t)(cut >> 32)) : -INFINITY;
    const int cut_i = (int)~(uint32_t)cut;
    const float floor = fmaxf(fmaxf(fmaxf(min_logit, top.v - 20.f * t - 1e-5f * fabsf(top.v)), cut_v), -3.402823466e38f);
    const float sure = min_p > 0.f ? logit_of(fminf(min_p, 1.f), 1.f) : -INFINITY;  // w >= min_p for certain, if min_p <= 1
    const bool near_only = min_p > 1.f;
    Best lead = {-INFINITY, -1}, won = {-INFINITY, -1};
    constexpr int kAhead = 8;
    for (int i0 = from + tid; i0 < to; i0 += kAhead * kThreads) {
        float v[kAhead], r[kAhead];
        bool in[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            const int i = i0 + e * kThreads;
            v[e] = i < to ? clean(io<T>::ld(x + i)) : -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            const int i = i0 + e * kThreads;
            in[e] = v[e] >= floor && (v[e] > cut_v || i <= cut_i);
            r[e] = in[e] ? u[i] : 0.5f;
        }
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            const int i = i0 + e * kThreads;
            if (!in[e]) continue;
            const float c = fminf(fmaxf(r[e], 2.3283064365386963e-10f), 0.999999940395355f), d = 1.f - c;
            // -log u: by its series near 1, where the approximate logarithm has no digits left
            const float clock = c > 0.99f ? d + 0.5f * d * d : lg2(c) * -0.6931471805599453f;
            const float rough = ((v[e] - top.v) * rate - lg2(clock)) * 0.6931471805599453f;  // good to 10^-4
            if (rough < lead.v - 1e-3f) continue;
            if (v[e] < sure || near_only) {
                if (score(v[e], i).i < 0) continue;
            }
            if (rough <= lead.v + 1e-3f) {  // too near to tell
                won = better(won, score(v[e], i));
                if (rough > lead.v) {
                    won = better(won, score(clean(io<T>::ld(x + lead.i)), lead.i));
                    lead = {rough, i};
                }
            } else {
                lead = {rough, i};
            }
        }
    }
    if (lead.i >= 0) won = better(won, score(clean(io<T>::ld(x + lead.i)), lead.i));
    won = block_best(won, s);
    if (tid == 0) s.x.won = won;
    cluster.sync();
    if (rank == 0 && tid == 0) {
        for (int r = 1; r < ctas; ++r) won = better(won, peer(r).x.won);
        finish(won);
    }
    cluster.sync();
}

}  // namespace

size_t sample_workspace_bytes(int, int) { return 0; }

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream) {
    // CTAs per row: double while the GPU (152 SMs, two CTAs each) is not full and a CTA has 4096 tokens left
    int ctas = 1;
    while (ctas < kMaxCtas && (int64_t)a.B * ctas * 2 <= 608 && a.V / (2 * ctas) >= 4096) ctas *= 2;
    auto go = [&](auto kern) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)a.B * ctas);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = sizeof(Shared);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kern, a);
    };
    return a.dtype == GDN_BF16 ? go(sample_kernel<__nv_bfloat16>) : go(sample_kernel<float>);
}

}  // namespace gdn
