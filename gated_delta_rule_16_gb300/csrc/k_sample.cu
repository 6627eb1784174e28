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
// row in L2, where instructions per token count (about 10 to 20 in each pass below).  Greedy rows, one
// pass, take 21 us at 256 rows of 100003 fp32 logits (4.9 TB/s), with top_k 50 and top_p 0.9 47 us, unfiltered ones 71 us with
// their noise read; one row of 131072 in bf16 4.8, 14.4 and 11.3 us.  A cluster of CTAs shares a row, as many as fill the
// GPU, each with a slice:
//   1. one pass for the maximum, the sum of weights and every thread's own maximum;
//   2. a threshold that no kept token is below.  For top_k: among the threads' maxima, the ceil(k / CTAs)-th largest of
//      every CTA, and the least of those (k tokens at least are as large).  For top_p: tokens below (1 - p) M / V hold
//      (1 - p) M together at most, so the prefix of mass p M ends above it.  What passes the threshold, a few hundred
//      tokens as a rule, is gathered and cut in the first CTA's shared memory;
//   3. if it is more than fits (flat rows, large k), the k-th largest logit is bracketed by a histogram of every 8th load
//      (of every one if that fails, or k is too large for it), the bracket gathered, with the number and mass
//      of the tokens above it from the same pass; thousands of equal logits leave the first CTA to descend the
//      sorting key digit by digit, a pass over the row each.  The end of top_p's prefix is not looked for: the race is run
//      over all of K, and its winner's mass above says whether it was kept.  If not, nothing below it is either, and the race
//      is run again above it: 1 + log(1 / top_p) times as a rule, or until what is left can be gathered;
//   4. the race.  The largest token is always kept, so its score bounds the winner's from the start: no Gumbel is above
//      16.64, and a token whose logit cannot make up for it has its noise not read; of the others one comparison of
//      1 - u with a multiple of w leaves a few per warp whose score is worked out.
//
// Masses are summed as whole numbers in units of 2^-40 of the largest weight, of a token or of what one thread met of a
// row, so that no sum depends on the order of atomics.  The weights in masses are 2^x approximations (2^-21); w >= min_p
// and the race are decided in IEEE fp32 with accurate exp and log.
#include <cooperative_groups.h>

#include "paged.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;   // per row: the largest cluster every GPU of this kind can place
constexpr int kList = 2048;   // gathered tokens
constexpr int kBins = 2048;
constexpr int kRounds = 24;   // races and probes before the end of top_p's prefix is looked for
constexpr float kUnit = 1099511627776.f;  // 2^40
constexpr float kReach = 28.f;            // in y: 40 ln 2, below which a mass rounds to 0
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
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The weight of a logit in units of 2^-40.
__device__ __forceinline__ u64 mass_of(float v, float top, float rate) { return (u64)(ex2((v - top) * rate) * kUnit + 0.5f); }

struct Best { float v; int i; };
__device__ __forceinline__ Best better(Best a, Best b) {
    return b.v > a.v || (b.v == a.v && (unsigned)b.i < (unsigned)a.i) ? b : a;
}

struct Shared {
    u64 list[kList];
    uint32_t count[kBins];  // of this CTA's tokens; the first CTA has the row's in list
    u64 digit_sum[256];
    uint32_t digit_count[256];
    u64 sums[kWarps];
    Best bests[kWarps];
    float parts[2][kWarps];
    int n, found;           // tokens gathered; bin or rank found
    u64 before;
    bool whole;
    // read by the row's other CTAs, each written once between two barriers of the cluster
    struct {
        Best top, won;
        float low, sum, least;
        int gathered;      // tokens gathered, or more than kList
        int above[2];      // tokens above those, or above a race's winner, and their mass: by turns, so that a round's are
        u64 mass[2];       // written while others may still read the last's
        int lo, hi;        // the first CTA's: bins to gather
        bool settled;      // the first CTA's: whether cut is the key of the k-th token (0: K is all that matters), and mass_k
        u64 cut, mass_k;   // the mass of K
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

template <int N> struct Count { static constexpr int value = N; };

// f(logits, how many, index of the first) for the tokens [from, to) of a row, in pieces of 16 bytes (or single tokens
// before and after them), four of which are in flight per thread; a thread meets its tokens in ascending order.  The
// logits are as stored.  f returns false to end the thread's pass.
template <typename T, typename F>
__device__ __forceinline__ void each_piece(const T *row, int from, int to, F f) {
    constexpr int kPer = 16 / sizeof(T);
    const int tid = threadIdx.x;
    const T *x = row + from;
    const int n = to - from;
    const int head = min(n, (int)((16 - ((uintptr_t)x & 15)) & 15) / (int)sizeof(T)), pieces = (n - head) / kPer;
    float v[kPer];
    if (tid < head) {
        v[0] = io<T>::ld(x + tid);
        if (!f(v, Count<1>(), from + tid)) return;
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
                if constexpr (sizeof(T) == 2) v[e] = __uint_as_float(e & 1 ? q[e / 2] & 0xffff0000u : q[e / 2] << 16);
                else v[e] = __uint_as_float(q[e]);
            }
            if (!f(v, Count<kPer>(), from + head + (i0 + u * kThreads) * kPer)) return;
        }
    }
    const int t = head + pieces * kPer + tid;
    if (t < n) {
        v[0] = io<T>::ld(x + t);
        f(v, Count<1>(), from + t);
    }
}
template <int N>
__device__ __forceinline__ float largest(const float *v) {  // NaN aside
    float m = v[0];
#pragma unroll
    for (int e = 1; e < N; ++e) m = fmaxf(m, v[e]);
    return m;
}
// f(clean logit, index) for the tokens whose logit is at least `least` and above -inf.
template <typename T, typename F>
__device__ __forceinline__ void each(const T *row, int from, int to, float least, F f) {
    each_piece(row, from, to, [&](const float *v, auto n, int at) {
        constexpr int N = decltype(n)::value;
        const float m = largest<N>(v);
        if (!(m >= least) || m == -INFINITY) return true;
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (v[e] >= least && v[e] > -INFINITY && !f(clean(v[e]), at + e)) return false;
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

// Of the n gathered keys that are `floor` or more: a key that divides off the shortest descending prefix whose measure
// (tokens, or mass) reaches goal; 0 if all of it does not.  By 8 bits of the key at a time, from the first that differ.
__device__ __noinline__ u64 select(Shared &s, int n, u64 goal, bool of_mass, u64 floor, float top, float rate) {
    constexpr int kEach = kList / kThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    u64 key[kEach], measure[kEach];
    uint32_t most = 0, least = ~0u;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int i = e * kThreads + tid;
        key[e] = i < n ? s.list[i] : 0;
        if (key[e] < floor) key[e] = 0;
        measure[e] = of_mass ? mass_of(value_of((uint32_t)(key[e] >> 32)), top, rate) : 1;
        if (key[e]) {
            most = max(most, (uint32_t)(key[e] >> 32));
            least = min(least, (uint32_t)(key[e] >> 32));
        }
    }
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    __syncthreads();
    if (lane == 0) s.sums[warp] = (u64)most << 32 | least;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        most = max(most, (uint32_t)(s.sums[w] >> 32));
        least = min(least, (uint32_t)s.sums[w]);
    }
    if (most == 0) return 0;
    int above = most == least ? 32 : 64 - __clz(most ^ least);  // bits below `above` may differ
    u64 prefix = above == 64 ? 0 : ((u64)most << 32) >> above, before = 0;
    for (;;) {
        const int shift = max(above - 8, 0), bits = above - shift;
        __syncthreads();
        if (tid < 256) s.digit_sum[tid] = 0, s.digit_count[tid] = 0;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            if (key[e] && (above == 64 || key[e] >> above == prefix)) {
                const int d = (int)(key[e] >> shift) & ((1 << bits) - 1);
                atomicAdd(&s.digit_count[d], 1u);
                if (of_mass) atomicAdd(&s.digit_sum[d], measure[e]);
            }
        __syncthreads();
        if (warp == 0) {
            // lane l has the digits 255 - 8 l down to 248 - 8 l
            u64 m[8], own = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int d = 255 - 8 * lane - j;
                m[j] = of_mass ? s.digit_sum[d] : s.digit_count[d];
                own += m[j];
            }
            u64 incl = own;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const u64 y = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += y;
            }
            u64 at = before + incl - own;
            if (lane == 31 && before + incl < goal) s.found = -1;
            if (at < goal && at + own >= goal) {
                int j = 0;
                for (; at + m[j] < goal; ++j) at += m[j];
                s.found = 255 - 8 * lane - j;
                s.before = at;
                // the prefix ends with this digit if it takes all of it, or its only token
                s.whole = at + m[j] == goal || s.digit_count[s.found] == 1;
            }
        }
        __syncthreads();
        if (s.found < 0) return 0;
        prefix = prefix << bits | (u64)s.found;
        before = s.before;
        above = shift;
        if (s.whole || above == 0) return prefix << above;
    }
}

// Exact score of a token, {-inf, -1} if min_p or a weight of 0 rules it out.  A call: few tokens need it, and inlined in
// several loops it crowds the instruction cache.
__device__ __noinline__ Best exact_score(float v, int i, float top, float t, float min_p, const float *u) {
    const float y = (v - top) / t, w = expf(y);
    if (!(w > 0.f) || w < min_p) return {-INFINITY, -1};
    const float r = fminf(fmaxf(u[i], 2.3283064365386963e-10f), 0.999999940395355f);
    return {y - logf(-logf(r)), i};
}

// ---- passes over a slice [from, to) of a row.  Calls, so that each has the registers to itself.

// 16-byte pieces of a row for whole warps: f(how many, logits as stored or NaN, index of the first) for kAhead pieces at a time,
// with every lane in every step; every stride-th piece only.  Single tokens before and after the pieces come one to a lane.
template <int kAhead, typename T, typename F>
__device__ __forceinline__ void each_together(const T *x, int from, int to, int stride, F f) {
    constexpr int kPer = 16 / sizeof(T);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T *row = x + from;
    const int head = min(to - from, (int)((16 - ((uintptr_t)row & 15)) & 15) / (int)sizeof(T)), pieces = (to - from - head) / kPer;
    const uint4 *p4 = (const uint4 *)(row + head);
    for (int i0 = warp * 32; i0 * stride < pieces; i0 += kAhead * kThreads) {
        uint4 w[kAhead];
        float v[kAhead][kPer];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const int i = (i0 + q * kThreads + lane) * stride;
            w[q] = i < pieces ? p4[i] : make_uint4(~0u, ~0u, ~0u, ~0u);  // NaN in either type
        }
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const uint32_t y[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                if constexpr (sizeof(T) == 2) v[q][e] = __uint_as_float(e & 1 ? y[e / 2] & 0xffff0000u : y[e / 2] << 16);
                else v[q][e] = __uint_as_float(y[e]);
            }
        }
        f(Count<kAhead>(), Count<kPer>(), &v[0][0], from + head + (i0 + lane) * stride * kPer, stride * kThreads * kPer);
    }
    if (warp == 0) {
        const int tail = head + pieces * kPer, i = lane < 16 ? lane : tail + lane - 16;
        const bool have = lane < 16 ? lane < head : i < to - from;
        const float v = have ? io<T>::ld(row + i) : __uint_as_float(~0u);
        f(Count<1>(), Count<1>(), &v, have ? from + i : 0, 0);
    }
}

// Gathers the tokens from `least` up and above the key `under`.
template <typename T>
__device__ __noinline__ void gather_pass(const T *x, int from, int to, float least, u64 under, Shared &s) {
    each(x, from, to, least, [&](float v, int i) {
        const u64 key = full_key(v, i);
        return key > under ? gather(s, key) : true;
    });
}

__device__ __forceinline__ int bin_of(float v, float top, float scale) { return (int)fminf((top - v) * scale, (float)(kBins - 1)); }

// Counts by bin of every stride-th load.
template <typename T>
__device__ __noinline__ void count_pass(const T *x, int from, int to, int stride, float top, float scale, Shared &s) {
    each_together<2>(x, from, to, stride, [&](auto q, auto n, const float *w, int, int) {
#pragma unroll
        for (int e = 0; e < decltype(q)::value * decltype(n)::value; ++e)
            if (w[e] > -INFINITY) atomicAdd(&s.count[bin_of(clean(w[e]), top, scale)], 1u);
    });
}

// Gathers the tokens of the bins [lo, hi]; number and mass (in weights) of those above.
struct Above { int n; float mass; };
template <typename T>
__device__ __noinline__ Above bracket_pass(const T *x, int from, int to, int lo, int hi, float top, float scale, float rate, Shared &s) {
    Above a = {0, 0.f};
    each_together<2>(x, from, to, 1, [&](auto q, auto n, const float *w, int at, int step) {
        constexpr int N = decltype(n)::value;
        uint32_t mine = 0;
#pragma unroll
        for (int e = 0; e < decltype(q)::value * N; ++e) {
            const float v = clean(w[e]);
            const int bin = bin_of(v, top, scale);  // of -inf: the last
            if (bin < lo) {
                a.mass += ex2((v - top) * rate);
                ++a.n;
            }
            mine |= (uint32_t)(bin >= lo && bin <= hi && v > -INFINITY) << e;
        }
        while (mine) {  // few: read again
            const int e = __ffs(mine) - 1, i = at + e / N * step + e % N;
            mine &= mine - 1;
            gather(s, full_key(clean(io<T>::ld(x + i)), i));
        }
    });
    return a;
}

// Number and mass (in weights) of the tokens before one of logit `mark` and index i, in descending order.
template <typename T>
__device__ __noinline__ Above mass_pass(const T *x, int from, int to, float mark, uint32_t i, float top, float rate) {
    Above a = {0, 0.f};
    each_piece(x, from, to, [&](const float *w, auto n, int at) {
        constexpr int N = decltype(n)::value;
        if (!(largest<N>(w) >= mark)) return true;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float v = clean(w[e]);
            if (v > mark || (v == mark && (uint32_t)(at + e) < i)) {
                a.mass += ex2((v - top) * rate);
                ++a.n;
            }
        }
        return true;
    });
    return a;
}

// By one CTA over a whole row, digit by digit: the key of the k-th token.
template <typename T>
__device__ __noinline__ u64 kth_key(const T *x, int V, int k, Shared &s) {
    u64 prefix = 0, before = 0;
    for (int shift = 56; shift >= 0; shift -= 8) {
        __syncthreads();
        for (int d = threadIdx.x; d < 256; d += kThreads) s.digit_count[d] = 0;
        __syncthreads();
        each(x, 0, V, -INFINITY, [&](float v, int i) {
            const u64 key = full_key(v, i);
            if (shift == 56 || (key >> (shift + 8)) == prefix) atomicAdd(&s.digit_count[(key >> shift) & 255], 1u);
            return true;
        });
        __syncthreads();
        if (threadIdx.x == 0) {
            int d = 255;
            u64 at = before;
            for (; d > 0 && at + s.digit_count[d] < (u64)k; --d) at += s.digit_count[d];
            s.found = d;
            s.before = at;
        }
        __syncthreads();
        prefix = prefix << 8 | (u64)s.found;
        before = s.before;
    }
    return prefix;
}

// The race.  A token beats the score `best` only if -log u <= w exp(-best), and 1 - u <= -log u: one comparison, with room
// for its rounding, leaves a handful of tokens per warp for exact scores once the best is shared in the warp.
struct Track {
    const float *u;
    float top, t, rate, min_p;
    float floor, reach;  // logits below cannot be kept or cannot win; exp(-best)
    u64 cut;             // keys below are not kept
};
template <typename T>
__device__ __noinline__ Best race_pass(const T *x, int from, int to, const Track &track, Best won) {
    const float *u = track.u;
    const float top = track.top, rate = track.rate, floor = track.floor;
    float reach = track.reach;
    each_together<sizeof(T)>(x, from, to, 1, [&](auto q, auto n, const float *w, int at, int step) {
        constexpr int N = decltype(n)::value, Q = decltype(q)::value;
        if (!__any_sync(0xffffffffu, largest<Q * N>(w) >= floor)) return;
        float r[Q * N];
        uint32_t hit = 0;
#pragma unroll
        for (int e = 0; e < Q * N; ++e) r[e] = w[e] >= floor ? u[at + e / N * step + e % N] : -1.f;
#pragma unroll
        for (int e = 0; e < Q * N; ++e) {
            const float weight = ex2((fminf(w[e], 3.402823466e38f) - top) * rate);  // of NaN: where r = -1
            hit |= (uint32_t)(1.f - fminf(r[e], 0.999999940395355f) < weight * reach && r[e] >= 0.f) << e;
        }
        if (!__any_sync(0xffffffffu, hit != 0)) return;
        while (hit) {
            const int e = __ffs(hit) - 1, i = at + e / N * step + e % N;
            hit &= hit - 1;
            const float v = clean(io<T>::ld(x + i));
            if (full_key(v, i) >= track.cut) won = better(won, exact_score(v, i, top, track.t, track.min_p, u));
        }
        float best = won.v;
#pragma unroll
        for (int off = 16; off; off >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, off));
        reach = fminf(reach, 1.01f * ex2(best * -1.4426950408889634f));
    });
    return won;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) sample_kernel(SampleArgs a) {
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

    // 1. maximum, sum of weights, and how low logits go (one token of each load: a sample is enough for the bins below).
    // No branch on a new maximum: some lane of a warp has one at nearly every load.
    float most = -INFINITY, sum = 0.f, low = INFINITY;
    int at_most = 0;
    each_piece(x, from, to, [&](const float *w, auto n, int at) {
        constexpr int N = decltype(n)::value;
        float v[N];
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = clean(w[e]);
        const float m = largest<N>(v);
        at_most = m > most ? at : at_most;
        const float now = fmaxf(most, m);
        if (!greedy) {
            const float ref = now == -INFINITY ? 0.f : now;
            sum *= ex2((most - ref) * rate);
            float y = 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) y += ex2((v[e] - ref) * rate);
            sum += y;
            low = fminf(low, v[0] > -INFINITY ? v[0] : INFINITY);
        }
        most = now;
        return true;
    });
    const float mine = most;
    // the index of the load stands for the token's until the end: loads do not overlap
    Best top = {most, most > -INFINITY ? at_most : -1};
    {
#pragma unroll
        for (int off = 16; off; off >>= 1) {
            top = better(top, {__shfl_xor_sync(0xffffffffu, top.v, off), __shfl_xor_sync(0xffffffffu, top.i, off)});
            low = fminf(low, __shfl_xor_sync(0xffffffffu, low, off));
        }
        sum = mine > -INFINITY ? sum * ex2((mine - top.v) * rate) : 0.f;
#pragma unroll
        for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if ((tid & 31) == 0) s.bests[tid >> 5] = top, s.parts[0][tid >> 5] = sum, s.parts[1][tid >> 5] = low;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) top = better(top, s.bests[w]), low = fminf(low, s.parts[1][w]);
        sum = 0.f;
        for (int w = 0; w < kWarps; ++w)
            if (s.bests[w].i >= 0) sum += s.parts[0][w] * ex2((s.bests[w].v - top.v) * rate);
    }
    float least = -INFINITY;  // a logit that no kept token is below
    if (by_k) {
        const int need = (k + ctas - 1) / ctas;
        if (need <= kThreads) {
            const uint32_t own = mine > -INFINITY ? key_of(mine) : 0u;
            uint32_t key = 0;
#pragma unroll 1
            for (int bit = 31; bit >= 16; --bit) {  // the leading bits will do: a little lower, a few tokens more
                const uint32_t next = key | 1u << bit;
                if (__syncthreads_count(own >= next) >= need) key = next;
            }
            if (key) least = value_of(key);
        }
    }
    if (tid == 0) s.x.top = top, s.x.sum = sum, s.x.low = low, s.x.least = least;
    cluster.sync();
    // Lane r of every warp reads CTA r's values: a loop over the CTAs would wait for each in turn.
    const int lane = tid & 31, warp = tid >> 5;
    const bool reads = lane < ctas;
    auto best_of = [&](Best mine) {  // over the lanes that read
        if (!reads) mine = {-INFINITY, -1};
#pragma unroll
        for (int off = kMaxCtas / 2; off; off >>= 1)
            mine = better(mine, {__shfl_xor_sync(0xffffffffu, mine.v, off), __shfl_xor_sync(0xffffffffu, mine.i, off)});
        return Best{__shfl_sync(0xffffffffu, mine.v, 0), __shfl_sync(0xffffffffu, mine.i, 0)};
    };
    auto sum_of = [&](auto mine) {
        if (!reads) mine = 0;
#pragma unroll
        for (int off = kMaxCtas / 2; off; off >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, off);
        return __shfl_sync(0xffffffffu, mine, 0);
    };
    auto least_of = [&](float mine) {
        if (!reads) mine = INFINITY;
#pragma unroll
        for (int off = kMaxCtas / 2; off; off >>= 1) mine = fminf(mine, __shfl_xor_sync(0xffffffffu, mine, off));
        return __shfl_sync(0xffffffffu, mine, 0);
    };
    const Shared &from_peer = peer(reads ? lane : 0);
    const Best its_top = from_peer.x.top;
    const float its_sum = from_peer.x.sum, its_low = from_peer.x.low, its_least = from_peer.x.least;
    top = best_of(its_top);
    low = least_of(its_low);
    least = least_of(its_least);
    const float total = sum_of(its_top.i >= 0 ? its_sum * ex2((its_top.v - top.v) * rate) : 0.f);

    auto finish = [&](Best won) {  // thread 0 of the first CTA
        if (won.i < 0 && top.i >= 0) {  // greedy, or min_p above 1 leaves nothing: the largest
            won = top;
            for (int e = kPer - 1; e >= 0; --e)  // within its load
                if (top.i + e < a.V && clean(io<T>::ld(x + top.i + e)) == top.v) won.i = top.i + e;
        }
        a.tokens[b] = won.i;
        if (a.logprobs) a.logprobs[b] = won.i < 0 ? -INFINITY : greedy ? 0.f : (clean(io<T>::ld(x + won.i)) - top.v) / t - logf(total);
    };
    if (top.i < 0 || greedy || min_p > 1.f) {
        cluster.sync();  // no CTA leaves while another may read its shared memory
        if (rank == 0 && tid == 0) finish({-INFINITY, -1});
        return;
    }

    // a logit below which w < f, with room for every rounding on the way
    auto logit_of = [&](float f) {
        const float d = t * logf(f);
        return top.v + d - (1e-5f * (fabsf(top.v) + fabsf(d)) + 1e-3f * t);
    };
    const float min_logit = min_p > 0.f ? logit_of(min_p) : -INFINITY;
    auto goal_of = [&](double m) {  // p of mass m, at least one unit: the largest token always stays
        const double g = ceil((double)fmaxf(p, 0.f) * m);
        return g < 1.0 ? 1ull : (u64)g;
    };
    auto score = [&](float v, int i) { return exact_score(v, i, top.v, t, min_p, u); };
    // the first CTA takes over the tokens that the others have gathered; false if they are too many
    auto collect = [&]() {
        const int its_n = from_peer.x.gathered, n = sum_of(its_n);
        if (n > kList) return false;
        for (int r = 1 + warp % (kWarps / 2); r < ctas; r += kWarps / 2) {  // two warps to a CTA
            int at = 0;
            for (int q = 0; q < r; ++q) at += __shfl_sync(0xffffffffu, its_n, q);
            const int m = __shfl_sync(0xffffffffu, its_n, r);
            for (int i = lane + 32 * (warp / (kWarps / 2)); i < m; i += 64) s.list[at + i] = peer(r).list[i];
        }
        __syncthreads();
        return true;
    };
    auto mass_from = [&](int n, u64 key) {  // of the list's keys
        u64 own = 0, all;
        for (int i = tid; i < n; i += kThreads) own += s.list[i] >= key ? mass_of(value_of((uint32_t)(s.list[i] >> 32)), top.v, rate) : 0;
        block_before(own, all, s);
        return all;
    };

    Best won = {-INFINITY, -1};
    // Gathers the tokens from `least` up (and above the key `under`); if they fit, the first CTA cuts the list at rank k and at
    // mass `goal` (0: at top_p of the list's first k), races what is left and writes the result.
    auto settle_in_list = [&](float least, u64 under, u64 goal) {
        if (tid == 0) s.n = 0;
        __syncthreads();
        gather_pass(x, from, to, least, under, s);
        __syncthreads();
        if (tid == 0) s.x.gathered = min(s.n, kList + 1);
        cluster.sync();
        const int n = sum_of(from_peer.x.gathered);
        if (n > kList) return false;
        if (rank == 0) collect();
        cluster.sync();  // the others are done
        if (rank == 0) {
            if (n <= 256) {
                // every key against every other: rank and mass before it, by the kThreads / 2^m threads of a key together
                int per = kThreads / 32;
                while (kThreads / per < n) per /= 2;
                if (tid < n) s.digit_sum[tid] = mass_of(value_of((uint32_t)(s.list[tid] >> 32)), top.v, rate);
                __syncthreads();
                const int i = tid / per;
                const u64 key = i < n ? s.list[i] : 0;
                int ahead = 0;
                u64 before = 0, all;
                for (int j = tid % per; j < n; j += per)
                    if (s.list[j] > key) ++ahead, before += s.digit_sum[j];
                for (int off = per / 2; off; off >>= 1) {
                    ahead += __shfl_xor_sync(0xffffffffu, ahead, off);
                    before += __shfl_xor_sync(0xffffffffu, before, off);
                }
                bool keep = tid % per == 0 && i < n && !(by_k && ahead >= k);
                if (by_p) {
                    if (goal == 0) {
                        block_before(keep ? s.digit_sum[i] : 0, all, s);
                        goal = goal_of((double)all);
                    }
                    keep = keep && before < goal;
                }
                if (keep) won = score(value_of((uint32_t)(key >> 32)), (int)~(uint32_t)key);
            } else {
                u64 from_key = by_k && n > k ? select(s, n, (u64)k, false, 0, top.v, rate) : 0;
                if (by_p) {
                    if (goal == 0) goal = goal_of((double)mass_from(n, from_key));
                    from_key = max(from_key, select(s, n, goal, true, from_key, top.v, rate));
                }
                for (int i = tid; i < n; i += kThreads) {
                    const u64 key = s.list[i];
                    if (key >= from_key) won = better(won, score(value_of((uint32_t)(key >> 32)), (int)~(uint32_t)key));
                }
            }
            won = block_best(won, s);
            if (tid == 0) finish(won);
        }
        return true;
    };

    u64 cut = 0;  // the key of the k-th token
    u64 goal = by_p && !by_k ? goal_of((double)total * (double)kUnit) : 0;
    if (by_k || by_p) {
        // 2. what passes the threshold
        if (!(by_k && by_p)) least = fmaxf(least, min_logit);  // with both, all of K counts in its mass
        if (by_p && !by_k) least = fmaxf(least, logit_of((1.f - fmaxf(p, 0.f)) * total / (float)a.V));
        if (settle_in_list(least, 0, goal)) return;
    }
    if (by_k) {
        // 3. the k-th token, from a histogram over the logits
        const float bottom = fmaxf(top.v - kReach * t, low);
        const bool deep = bottom == top.v - kReach * t;  // the last bin's tokens have no mass and cannot win
        const float scale = bounded((float)kBins / (top.v - bottom));
        // of every `stride`-th load, as long as 3 standard deviations either way stay well below the list's room
        int stride = 8;
        while (stride > 1 && (int64_t)stride * k > 54000) stride /= 2;
        for (;; stride = 1) {
            for (int i = tid; i < kBins; i += kThreads) s.count[i] = 0;
            __syncthreads();
            count_pass(x, from, to, stride, top.v, scale, s);
            cluster.sync();
            {
                // each CTA adds up a range of bins for the first one
                const int step = kBins / ctas;
                uint32_t *counts = (uint32_t *)cluster.map_shared_rank(s.list, 0);
                for (int i = rank * step + tid; i < (rank + 1) * step; i += kThreads) {
                    uint32_t c = 0;
#pragma unroll
                    for (int r = 0; r < kMaxCtas; ++r)
                        if (r < ctas) c += peer(r).count[i];
                    counts[i] = c;
                }
            }
            cluster.sync();
            if (rank == 0) {
                // the first bin whose running count reaches `nth`, or the last
                auto find_bin = [&](u64 nth) {
                    constexpr int kEach = kBins / kThreads;
                    const uint32_t *counts = (const uint32_t *)s.list;
                    u64 own = 0, all;
                    for (int e = 0; e < kEach; ++e) own += counts[tid * kEach + e];
                    u64 at = block_before(own, all, s);
                    if (tid == 0) s.found = kBins - 1;
                    __syncthreads();
                    if (at < nth && at + own >= nth) {
                        int e = 0;
                        while ((at += counts[tid * kEach + e]) < nth) ++e;
                        s.found = tid * kEach + e;
                    }
                    __syncthreads();
                    const int bin = s.found;
                    __syncthreads();
                    return bin;
                };
                const float mid = (float)k / (float)stride, off = stride > 1 ? 3.2f * sqrtf(mid) + 2.f : 0.f;
                const int lo = find_bin((u64)fmaxf(stride > 1 ? mid - off : (float)k, 1.f)), hi = stride > 1 ? find_bin((u64)(mid + off)) : lo;
                if (tid == 0) s.x.lo = lo, s.x.hi = hi;
            }
            cluster.sync();
            const int lo = peer(0).x.lo, hi = peer(0).x.hi;
            if (tid == 0) s.n = 0;
            __syncthreads();
            const Above above = bracket_pass(x, from, to, lo, deep ? min(hi, kBins - 2) : hi, top.v, scale, rate, s);
            u64 all_mass, all_above;
            block_before((u64)(above.mass * kUnit + 0.5f), all_mass, s);
            block_before((u64)above.n, all_above, s);
            if (tid == 0) s.x.gathered = min(s.n, kList + 1), s.x.mass[0] = all_mass, s.x.above[0] = (int)all_above;
            cluster.sync();
            if (rank == 0) {
                const int before = sum_of(from_peer.x.above[0]), n = sum_of(from_peer.x.gathered);
                const u64 mass_before = sum_of(from_peer.x.mass[0]);
                bool settled = true;
                u64 mass_k = (u64)((double)total * (double)kUnit);
                if (before < k && hi == kBins - 1 && n <= kList && before + n < k) {
                    // K is every finite logit, or ends among those of no mass: all that matters is in it
                } else if (before < k && n <= kList && before + n >= k) {
                    collect();
                    cut = select(s, n, (u64)(k - before), false, 0, top.v, rate);
                    mass_k = mass_before + mass_from(n, cut);
                } else if (stride > 1) {
                    settled = false;  // outside the bracket, or too many in it
                } else {
                    cut = kth_key(x, a.V, k, s);
                    u64 own = 0;
                    each(x, 0, a.V, -INFINITY, [&](float v, int i) {
                        if (full_key(v, i) >= cut) own += mass_of(v, top.v, rate);
                        return true;
                    });
                    block_before(own, mass_k, s);
                }
                if (tid == 0) s.x.settled = settled, s.x.cut = cut, s.x.mass_k = mass_k;
            }
            cluster.sync();
            if (!peer(0).x.settled) continue;
            cut = peer(0).x.cut;
            if (by_p) goal = goal_of((double)peer(0).x.mass_k);
            break;
        }
    }
    // 4. the race over K, until its winner is in top_p's prefix
    // from the largest token, which is always kept, on
    const uint32_t same = __ballot_sync(0xffffffffu, lane < kPer && top.i + lane < a.V && clean(io<T>::ld(x + top.i + lane)) == top.v);
    const Best first = score(top.v, top.i + __ffs(same) - 1);
    // A rejected winner with well over the goal's mass above it leaves another race a poor chance: two probes between it and
    // the largest, a pass for the mass each, come first.  Noise that goes with the logits' order could have winner after
    // winner rejected: from round kRounds on the keys between are halved, 64 times at most, and the race is run once more from
    // the end of the prefix.
    bool verify = by_p;
    int probes = 0;
    u64 kept = full_key(top.v, 0);  // keys from here on are kept
    for (int round = 0;; ++round) {
        const bool racing = probes == 0 && (round < kRounds || !verify);
        u64 probe = cut + (kept - cut) / 2;
        if (probes > 0) {
            const u64 middle = (u64)key_of(0.5f * (value_of((uint32_t)(cut >> 32)) + value_of((uint32_t)(kept >> 32)))) << 32;
            if (middle > cut && middle < kept) probe = middle;
        }
        if (racing) {
            // no Gumbel is above 16.64
            const float floor = fmaxf(fmaxf(min_logit, top.v + t * (first.v - 16.7f) - 1e-5f * fabsf(top.v)), cut ? value_of((uint32_t)(cut >> 32)) : -INFINITY);
            const Track track = {u, top.v, t, rate, min_p, fmaxf(floor, -3.402823466e38f), 1.01f * ex2(first.v * -1.4426950408889634f), cut};
            won = race_pass(x, from, to, track, first);
            won = block_best(won, s);
            if (tid == 0) s.x.won = won;
            cluster.sync();
            won = best_of(from_peer.x.won);
            if (!verify || won.i < 0) break;
            probe = full_key(clean(io<T>::ld(x + won.i)), won.i);
        }
        const Above above = mass_pass(x, from, to, value_of((uint32_t)(probe >> 32)), ~(uint32_t)probe, top.v, rate);
        u64 all_mass, all_above;
        block_before((u64)(above.mass * kUnit + 0.5f), all_mass, s);
        block_before((u64)above.n, all_above, s);
        if (tid == 0) s.x.mass[round & 1] = all_mass, s.x.above[round & 1] = (int)all_above;
        cluster.sync();
        const u64 mass = sum_of(from_peer.x.mass[round & 1]);
        const int before = sum_of(from_peer.x.above[round & 1]);
        if (probes > 0) --probes;
        if (mass < goal) {
            if (racing) break;
            kept = probe;
        } else {
            cut = probe + 1;  // the probe and what is below it are not kept
            won = {-INFINITY, -1};
            if (before <= kList && settle_in_list(value_of((uint32_t)(probe >> 32)), probe, goal)) return;
            if (mass < goal + goal / 4) probes = 0;
            else if (racing) probes = 2;
        }
        if (!racing && cut >= kept) {
            cut = kept;
            verify = false;
            probes = 0;
        }
    }
    cluster.sync();
    if (rank == 0 && tid == 0) finish(won);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream) {
    // CTAs per row: double while all rows' CTAs make two waves at most (152 SMs, four CTAs each) and a CTA has 4096 tokens
    // left.  At 256 rows of 100003, on one, two, four and eight CTAs each: rows alike, with top_k 50 and top_p 0.9, take 53, 39,
    // 47 and 77 us, rows of mixed settings 317, 202, 134 and 121 us, where the few flat rows' CTAs run on alone.  Four of 256
    // threads to an SM against two of 512: 32 rows of 131072 take 17.8 us against 20.1.  (One wave, with the rows that step 2 does
    // not settle left to a second launch of eight CTAs each, took 156 us for the mixed rows: the worst row's own time remains.)
    int ctas = 1;
    while (ctas < kMaxCtas && (int64_t)a.B * ctas * 2 <= 1216 && a.V / (2 * ctas) >= 4096) ctas *= 2;
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
