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
// What bounds it: the row is read once from HBM; everything after works on few tokens, or on the row in L2, where
// instructions per token (about 10 in each pass below) and barriers of the cluster count.  A pass handles 16 tokens per
// thread at a time without a branch between them, as few warps are there to hide their latency: one branch per token made the
// passes for masses twice as long.  Greedy rows, one pass, take 26 us at 256 rows of 100003 fp32 logits (3.9 TB/s), with
// top_k 50 and top_p 0.9 50 us, unfiltered ones 66 us with their noise read; one row of 131072 in bf16 5.5, 14.3 and 11 us.
// A cluster of CTAs shares a row, as many as fill the GPU, each with a slice:
//   1. one pass for the maximum, the sum of weights and every thread's own maximum;
//   2. a threshold that no kept token is below.  For top_k: among the threads' maxima, the ceil(k / CTAs)-th largest of
//      every CTA, and the least of those (k tokens at least are as large).  For top_p: tokens below (1 - p) M / V hold
//      (1 - p) M together at most, so the prefix of mass p M ends above it.  What passes the threshold, a few hundred
//      tokens as a rule, is gathered and cut in the first CTA's shared memory.  (If the largest token alone holds p M, it is
//      taken at once.)
//   3. if it is more than fits (flat rows, large k), the k-th largest logit is bracketed by a histogram of every 8th load
//      (of every one if that fails, or k is too large for it), the bracket gathered, with the number and mass
//      of the tokens above it from the same pass; every CTA finds the k-th in it for itself, which costs less than to wait
//      for one that does.  Thousands of equal logits leave them to descend the sorting key digit by digit, a pass over the
//      row each.  The end of top_p's prefix is not looked for: the race is run over all of K, and its winner's mass above
//      says whether it was kept.  If not, nothing below it is either, and the race is run again above it:
//      1 + log(1 / top_p) times as a rule.  As soon as each CTA's part of K, or of what lies above a rejected winner, is
//      short enough, it is held in shared memory, and races and masses take it from there;
//   4. the race.  The largest token is always kept, so its score bounds the winner's from the start: no Gumbel is above
//      16.64, and a token whose logit cannot make up for it has its noise not read; of the others one comparison of
//      1 - u with a multiple of w leaves a few per warp whose score is worked out.
//
// Masses are summed as whole numbers in units of 2^-40 of the largest weight, of a token or of what one thread met of a
// row (in fp32, in the order of its tokens), and the sum of all weights in fp32 by thread, warp and CTA in turn: no sum depends on
// the order of atomics, but its last bits do on how many CTAs share the row.  The weights in masses are 2^x approximations (2^-21); w >= min_p
// and the race are decided in IEEE fp32 with accurate exp and log.
#include <cooperative_groups.h>

#include "paged.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;   // per row: the largest cluster every GPU of this kind can place
constexpr int kList = 2048;   // gathered tokens
constexpr int kRanked = 256;  // of them ranked by comparing all with all
constexpr int kBins = 2048;
// Tokens that a CTA holds for races.  With twice as many, four CTAs' shared memory leaves an SM 28 KB of L1, and greedy rows take
// 33 us instead of 26 (256 x 100003); with none held, rows with top_k 5000 and top_p 0.5 take 188 us instead of 157.
constexpr int kHeld = 1472;
constexpr int kRounds = 24;   // races before the end of top_p's prefix is looked for
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
    u64 held[kHeld];        // this CTA's tokens that may yet win
    uint32_t count[kBins];  // of this CTA's tokens
    u64 digit_sum[256];
    uint32_t digit_count[256];
    u64 sums[kWarps];
    Best bests[kWarps];
    float parts[2][kWarps];
    uint32_t leasts[kWarps];
    int n, held_n, found;   // tokens gathered, held; digit found
    int lo, hi;             // bins found
    u64 before;
    bool whole;
    // read by the row's other CTAs, each written once between two barriers of the cluster
    struct {
        Best top, won;
        float low, sum, least;
        int gathered;      // tokens gathered, or more than kList
        int above[2];      // tokens above those, or above a race's winner, and their mass: by turns, so that a round's are
        u64 mass[2];       // written while others may still read the last's
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
__device__ __noinline__ Best exact_score(float v, int i, float top, float t, float min_p, float u) {
    const float y = (v - top) / t, w = expf(y);
    if (!(w > 0.f) || w < min_p) return {-INFINITY, -1};
    const float r = fminf(fmaxf(u, 2.3283064365386963e-10f), 0.999999940395355f);
    return {y - logf(-logf(r)), i};
}

// ---- passes over a slice [from, to) of a row.  Calls, so that each has the registers to itself.

// 16-byte pieces of a row for whole warps: f(how many, logits as stored or NaN, index of the first) for kAhead pieces at a time,
// with every lane in every step; every stride-th piece only.  Single tokens before and after the pieces come one to a lane.
// f returns false, in the whole warp, to end the warp's pass.
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
        if (!f(Count<kAhead>(), Count<kPer>(), &v[0][0], from + head + (i0 + lane) * stride * kPer, stride * kThreads * kPer)) return;
    }
    if (warp == 0) {
        const int tail = head + pieces * kPer, i = lane < 16 ? lane : tail + lane - 16;
        const bool have = lane < 16 ? lane < head : i < to - from;
        const float v = have ? io<T>::ld(row + i) : __uint_as_float(~0u);
        f(Count<1>(), Count<1>(), &v, have ? from + i : 0, 0);
    }
}

// Gathers the tokens with logits from `least` up, of logit `least` only those up to index `last`, in list[0, room) and their
// number in n; a warp ends its pass once they are too many.
template <typename T>
__device__ __noinline__ void gather_pass(const T *x, int from, int to, float least, uint32_t last, u64 *list, int room, int *n) {
    const int lane = threadIdx.x & 31;
    least = fmaxf(least, -3.402823466e38f);
    each_together<sizeof(T)>(x, from, to, 1, [&](auto q, auto per, const float *w, int at, int step) {
        constexpr int N = decltype(per)::value, Q = decltype(q)::value;
        if (!__any_sync(0xffffffffu, largest<Q * N>(w) >= least)) return true;
        uint32_t mine = 0;
#pragma unroll
        for (int e = 0; e < Q * N; ++e)  // NaN is not in
            mine |= (uint32_t)(w[e] >= least && (fminf(w[e], 3.402823466e38f) > least || (uint32_t)(at + e / N * step + e % N) <= last)) << e;
        int end = 0;
        for (unsigned peers; (peers = __ballot_sync(0xffffffffu, mine != 0)) != 0;) {
            int place = 0;
            if (lane == 0) place = atomicAdd(n, __popc(peers));
            place = __shfl_sync(0xffffffffu, place, 0);
            end = place + __popc(peers);
            place += __popc(peers & ((1u << lane) - 1));
            if (mine) {
                const int e = __ffs(mine) - 1, i = at + e / N * step + e % N;
                mine &= mine - 1;
                if (place < room) list[place] = full_key(clean(io<T>::ld(x + i)), i);
            }
        }
        return end <= room;
    });
}

// Gathers the tokens with logits in [least, upto); a warp ends its pass once they are too many.  Those from upto up are held, as
// far as there is room, and counted; their mass (in weights).
template <typename T>
__device__ __noinline__ float bracket_pass(const T *x, int from, int to, float least, float upto, float top, float rate, Shared &s) {
    const int lane = threadIdx.x & 31;
    float mass = 0.f;
    least = fmaxf(least, -3.402823466e38f);
    each_together<sizeof(T)>(x, from, to, 1, [&](auto q, auto per, const float *w, int at, int step) {
        constexpr int N = decltype(per)::value, Q = decltype(q)::value;
        if (!__any_sync(0xffffffffu, largest<Q * N>(w) >= least)) return true;
        uint32_t in = 0, above = 0;
#pragma unroll
        for (int e = 0; e < Q * N; ++e) {  // no branches: the tokens' latencies overlap
            const float v = fminf(w[e], 3.402823466e38f);
            const bool over = w[e] >= least && v >= upto;  // NaN is not
            mass += ex2(((over ? v : -INFINITY) - top) * rate);
            above |= (uint32_t)over << e;
            in |= (uint32_t)(w[e] >= least && !over) << e;
        }
        // places of both kinds from one sum over the warp
        const uint32_t own = __popc(in) | __popc(above) << 16;
        uint32_t upto_here = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, upto_here, off);
            if (lane >= off) upto_here += y;
        }
        int place = 0, held = 0;
        if (lane == 31) {
            place = atomicAdd(&s.n, (int)(upto_here & 0xffff));
            held = atomicAdd(&s.held_n, (int)(upto_here >> 16));
        }
        const int end = __shfl_sync(0xffffffffu, place + (int)(upto_here & 0xffff), 31);
        place = __shfl_sync(0xffffffffu, place, 31) + (int)(upto_here - own & 0xffff);
        held = __shfl_sync(0xffffffffu, held, 31) + (int)(upto_here - own >> 16);
        for (uint32_t left = in | above; left; left &= left - 1) {
            const int e = __ffs(left) - 1, i = at + e / N * step + e % N;
            const u64 key = full_key(clean(io<T>::ld(x + i)), i);
            if (above >> e & 1) {
                if (held < kHeld) s.held[held] = key;
                ++held;
            } else {
                if (place < kList) s.list[place] = key;
                ++place;
            }
        }
        return end <= kList;
    });
    return mass;
}

__device__ __forceinline__ int bin_of(float v, float top, float scale) { return (int)fminf((top - v) * scale, (float)(kBins - 1)); }

// Counts by bin of every stride-th load.
template <typename T>
__device__ __noinline__ void count_pass(const T *x, int from, int to, int stride, float top, float scale, Shared &s) {
    each_together<2>(x, from, to, stride, [&](auto q, auto n, const float *w, int, int) {
#pragma unroll
        for (int e = 0; e < decltype(q)::value * decltype(n)::value; ++e)
            if (w[e] > -INFINITY) atomicAdd(&s.count[bin_of(clean(w[e]), top, scale)], 1u);
        return true;
    });
}

// The smallest logit whose bin is `bin` or before it; by a whole warp.
__device__ float edge_of(int bin, float top, float scale) {
    const uint32_t lane = threadIdx.x & 31;
    uint32_t lo = key_of(-3.402823466e38f), hi = key_of(top);
    while (lo < hi) {
        const uint32_t step = (hi - lo) / 32 + 1;
        const unsigned in = __ballot_sync(0xffffffffu, bin_of(value_of(min(lo + lane * step, hi)), top, scale) <= bin);
        const uint32_t first = in ? __ffs(in) - 1 : 32;
        if (first < 32) hi = min(lo + first * step, hi);
        if (first > 0) lo = min(lo + (first - 1) * step + 1, hi);
    }
    return value_of(hi);
}

struct Above { int n; float mass; };
// Number and mass (in weights) of the tokens before one of logit `mark` and index i, in descending order.
template <typename T>
__device__ __noinline__ Above mass_pass(const T *x, int from, int to, float mark, uint32_t i, float top, float rate) {
    Above a = {0, 0.f};
    each_together<sizeof(T)>(x, from, to, 1, [&](auto q, auto n, const float *w, int at, int step) {
        constexpr int N = decltype(n)::value, Q = decltype(q)::value;
        if (!__any_sync(0xffffffffu, largest<Q * N>(w) >= mark)) return true;
#pragma unroll
        for (int e = 0; e < Q * N; ++e) {
            const float v = fminf(w[e], 3.402823466e38f);
            const bool in = w[e] >= mark && (v > mark || (uint32_t)(at + e / N * step + e % N) < i);  // NaN is not
            a.mass += ex2(((in ? v : -INFINITY) - top) * rate);
            a.n += in;
        }
        return true;
    });
    return a;
}

// Over a whole row, digit by digit: the key of the k-th token.
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
    float floor, reach;  // logits below cannot be kept or cannot win; log2 exp(-best), with room
    u64 cut;             // keys below are not kept
};
__device__ __forceinline__ float reach_of(float best) { return fmaf(best, -1.4426950408889634f, 0.015f); }
template <typename T>
__device__ __noinline__ Best race_pass(const T *x, int from, int to, const Track &track, Best won) {
    const float *u = track.u;
    const float top = track.top, rate = track.rate, floor = track.floor;
    float reach = track.reach;
    each_together<sizeof(T)>(x, from, to, 1, [&](auto q, auto n, const float *w, int at, int step) {
        constexpr int N = decltype(n)::value, Q = decltype(q)::value;
        if (!__any_sync(0xffffffffu, largest<Q * N>(w) >= floor)) return true;
        float r[Q * N];
        if (N >= 4 && ((uintptr_t)(u + at) & 15) == 0) {  // the same for all pieces
#pragma unroll
            for (int e = 0; e < Q * N; e += N < 4 ? 1 : 4) {
                constexpr int M = N < 4 ? 1 : 4;
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                if (largest<M>(w + e) >= floor) y = *(const float4 *)(u + at + e / N * step + e % N);
                const float z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int j = 0; j < M; ++j) r[e + j] = z[j];
            }
        } else {
#pragma unroll
            for (int e = 0; e < Q * N; ++e) r[e] = w[e] >= floor ? u[at + e / N * step + e % N] : 0.f;
        }
        uint32_t hit = 0;
#pragma unroll
        for (int e = 0; e < Q * N; ++e) hit |= (uint32_t)(w[e] >= floor && !(1.f - r[e] >= ex2(fmaf(w[e] - top, rate, reach)))) << e;
        if (!__any_sync(0xffffffffu, hit != 0)) return true;
        while (hit) {
            const int e = __ffs(hit) - 1, i = at + e / N * step + e % N;
            hit &= hit - 1;
            const float v = clean(io<T>::ld(x + i));
            if (full_key(v, i) >= track.cut) won = better(won, exact_score(v, i, top, track.t, track.min_p, u[i]));
        }
        float best = won.v;
#pragma unroll
        for (int off = 16; off; off >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, off));
        reach = fminf(reach, reach_of(best));
        return true;
    });
    return won;
}

// The same among the tokens held.
__device__ __noinline__ Best race_held(const Track &track, Best won, Shared &s) {
    constexpr int kStep = 4;
    const int n = s.held_n;
    float reach = track.reach;
    for (int i0 = threadIdx.x; i0 < n; i0 += kStep * kThreads) {
        u64 key[kStep];
        float r[kStep];
#pragma unroll
        for (int j = 0; j < kStep; ++j) key[j] = i0 + j * kThreads < n ? s.held[i0 + j * kThreads] : 0;
#pragma unroll
        for (int j = 0; j < kStep; ++j) r[j] = key[j] >= track.cut && key[j] ? track.u[~(uint32_t)key[j]] : 0.f;
#pragma unroll
        for (int j = 0; j < kStep; ++j) {
            const float v = value_of((uint32_t)(key[j] >> 32));
            if (key[j] < track.cut || !key[j] || 1.f - r[j] >= ex2(fmaf(v - track.top, track.rate, reach))) continue;
            won = better(won, exact_score(v, (int)~(uint32_t)key[j], track.top, track.t, track.min_p, r[j]));
            reach = fminf(reach, reach_of(won.v));
        }
    }
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
        const uint32_t own = mine > -INFINITY ? key_of(mine) : 0u, least_own = __reduce_min_sync(0xffffffffu, own);
        if ((tid & 31) == 0) s.leasts[tid >> 5] = least_own, s.bests[tid >> 5] = top, s.parts[0][tid >> 5] = sum, s.parts[1][tid >> 5] = low;
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
            // between the least and the largest of them, to 1 / 256 of what is between: a little low, a few tokens more
            uint32_t lo = s.leasts[0], hi = key_of(top.v);
            for (int w = 1; w < kWarps; ++w) lo = min(lo, s.leasts[w]);
#pragma unroll 1
            for (int bit = 0; bit < 8; ++bit) {
                const uint32_t mid = lo + (hi - lo) / 2 + 1;
                if (__syncthreads_count(own >= mid) >= need) lo = mid;
                else hi = mid - 1;
            }
            // lo starts at 0 where a thread met no finite token, and keys below the lowest finite number's are no numbers: no threshold
            if (lo >= key_of(-3.402823466e38f)) least = value_of(lo);
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

    auto write = [&](int i, float v) {
        a.tokens[b] = i;
        if (a.logprobs) a.logprobs[b] = i < 0 ? -INFINITY : greedy ? 0.f : (v - top.v) / t - logf(total);
    };
    auto finish = [&](Best won) {  // thread 0 of the first CTA
        if (won.i < 0 && top.i >= 0) {  // the largest
            won = top;
            for (int e = kPer - 1; e >= 0; --e)  // within its load
                if (top.i + e < a.V && clean(io<T>::ld(x + top.i + e)) == top.v) won.i = top.i + e;
        }
        write(won.i, won.i < 0 ? -INFINITY : clean(io<T>::ld(x + won.i)));
    };
    // whatever the noise: also if the largest token alone holds top_p of the mass
    if (top.i < 0 || greedy || min_p > 1.f || (by_p && (double)fmaxf(p, 0.f) * (double)total <= 1.0)) {
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
    auto score = [&](float v, int i, float r) { return exact_score(v, i, top.v, t, min_p, r); };
    // takes over the tokens that the row's other CTAs have gathered
    auto collect = [&](int its_n) {  // the lanes' counts of the CTAs that they read
        for (int q = 1 + warp % (kWarps / 2); q < ctas; q += kWarps / 2) {  // two warps to a CTA
            int at = 0;  // behind this CTA's own, which others may be reading
            for (int j = 0; j < q; ++j) at += __shfl_sync(0xffffffffu, its_n, (rank + j) % ctas);
            const int r = (rank + q) % ctas, m = __shfl_sync(0xffffffffu, its_n, r);
            for (int i = lane + 32 * (warp / (kWarps / 2)); i < m; i += 64) s.list[at + i] = peer(r).list[i];
        }
        __syncthreads();
    };
    auto mass_from = [&](int n, u64 key) {  // of the list's keys
        u64 own = 0, all;
        for (int i = tid; i < n; i += kThreads) own += s.list[i] >= key ? mass_of(value_of((uint32_t)(s.list[i] >> 32)), top.v, rate) : 0;
        block_before(own, all, s);
        return all;
    };

    Best won = {-INFINITY, -1};
    // Gathers the tokens from `least` up; if they fit, the first CTA cuts the list at rank k and at mass `goal` (0: at top_p of the list's first k), races what is left and writes the result.
    auto settle_in_list = [&](float least, u64 goal) {
        if (tid == 0) s.n = 0;
        // if every thread has some in a long slice, they are too many
        const int passing = __syncthreads_count(mine >= least);
        if (passing == kThreads && to - from > 2 * kList) {
            if (tid == 0) s.n = kList + 1;
        } else {
            gather_pass(x, from, to, least, ~0u, s.list, kList, &s.n);
        }
        __syncthreads();
        if (tid == 0) s.x.gathered = min(s.n, kList + 1);
        cluster.sync();
        const int its_n = from_peer.x.gathered, n = sum_of(its_n);
        if (n > kList) return false;
        if (rank == 0) collect(its_n);
        cluster.sync();
        if (rank == 0) {
            float won_at = 0.f;
            if (n <= kRanked) {
                // every key against every other: rank and mass before it, by the kThreads / 2^m threads of a key together
                int per = kThreads / 32;
                while (kThreads / per < n) per /= 2;
                if (tid < n) s.digit_sum[tid] = mass_of(value_of((uint32_t)(s.list[tid] >> 32)), top.v, rate);
                __syncthreads();
                const int i = tid / per;
                const u64 key = i < n ? s.list[i] : 0;
                const float r = i < n ? u[~(uint32_t)key] : 0.f;  // on its way while the keys are ranked
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
                won_at = value_of((uint32_t)(key >> 32));
                if (keep) won = score(won_at, (int)~(uint32_t)key, r);
            } else {
                u64 from_key = by_k && n > k ? select(s, n, (u64)k, false, 0, top.v, rate) : 0;
                if (by_p) {
                    if (goal == 0) goal = goal_of((double)mass_from(n, from_key));
                    from_key = max(from_key, select(s, n, goal, true, from_key, top.v, rate));
                }
                for (int i = tid; i < n; i += kThreads) {
                    const u64 key = s.list[i];
                    if (key < from_key) continue;
                    const Best now = better(won, score(value_of((uint32_t)(key >> 32)), (int)~(uint32_t)key, u[~(uint32_t)key]));
                    if (now.i != won.i) won_at = value_of((uint32_t)(key >> 32));
                    won = now;
                }
            }
            const Best all = block_best(won, s);
            if (won.i >= 0 && won.i == all.i) write(won.i, won_at);
            if (all.i < 0 && tid == 0) finish(all);
        }
        return true;
    };

    u64 cut = 0;  // the key of the k-th token
    bool held = false;  // whether what may yet win is held by the CTAs
    // whether all CTAs of the row have room for what they count
    auto fits = [&](int its_n) { return (int)__reduce_max_sync(0xffffffffu, reads ? its_n : 0) <= kHeld; };
    u64 goal = by_p && !by_k ? goal_of((double)total * (double)kUnit) : 0;
    if (by_k || by_p) {
        // 2. what passes the threshold
        if (!(by_k && by_p)) least = fmaxf(least, min_logit);  // with both, all of K counts in its mass
        if (by_p && !by_k) least = fmaxf(least, logit_of((1.f - fmaxf(p, 0.f)) * total / (float)a.V));
        if ((least > -INFINITY || a.V <= kList) && settle_in_list(least, goal)) return;
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
            // the row's counts: each thread has 8 bins of all CTAs
            constexpr int kEach = kBins / kThreads;
            uint32_t counts[kEach] = {};
#pragma unroll 1
            for (int r = 0; r < ctas; ++r) {
                const uint4 *c = (const uint4 *)(peer(r).count + tid * kEach);
#pragma unroll
                for (int e = 0; e < kEach; e += 4) {
                    const uint4 y = c[e / 4];
                    counts[e] += y.x, counts[e + 1] += y.y, counts[e + 2] += y.z, counts[e + 3] += y.w;
                }
            }
            u64 own = 0, all;
#pragma unroll
            for (int e = 0; e < kEach; ++e) own += counts[e];
            const u64 at = block_before(own, all, s);
            // the first bin whose running count reaches `nth`, or the last
            auto find_bin = [&](u64 nth, int &bin) {
                if (at < nth && at + own >= nth) {
                    u64 running = at;
                    int e = 0;
#pragma unroll
                    for (; e < kEach - 1 && (running += counts[e]) < nth; ++e) {}
                    bin = tid * kEach + e;
                }
            };
            const float mid = (float)k / (float)stride, off = stride > 1 ? 3.2f * sqrtf(mid) + 2.f : 0.f;
            if (tid == 0) s.lo = s.hi = kBins - 1;
            __syncthreads();
            find_bin((u64)fmaxf(stride > 1 ? mid - off : (float)k, 1.f), s.lo);
            find_bin((u64)fmaxf(stride > 1 ? mid + off : (float)k, 1.f), s.hi);
            __syncthreads();
            const int lo = s.lo, hi = s.hi;
            const float gather_from = edge_of(deep ? min(hi, kBins - 2) : hi, top.v, scale), gather_upto = lo > 0 ? edge_of(lo - 1, top.v, scale) : INFINITY;
            if (tid == 0) s.n = s.held_n = 0;
            __syncthreads();
            const float mass_above = bracket_pass(x, from, to, gather_from, gather_upto, top.v, rate, s);
            u64 all_mass;
            block_before((u64)(mass_above * kUnit + 0.5f), all_mass, s);
            if (tid == 0) s.x.gathered = min(s.n, kList + 1), s.x.mass[0] = all_mass, s.x.above[0] = s.held_n;
            cluster.sync();
            const int its_n = from_peer.x.gathered, its_above = from_peer.x.above[0];
            const u64 its_mass = from_peer.x.mass[0], mass_before = sum_of(its_mass);
            const int before = sum_of(its_above), n = sum_of(its_n);
            // every CTA settles it for itself
            u64 mass_k = (u64)((double)total * (double)kUnit);
            if (before < k && hi == kBins - 1 && n <= kList && before + n < k) {
                // K is every finite logit, or ends among those of no mass: all that matters is in it
            } else if (before < k && n <= kList && before + n >= k) {
                collect(its_n);
                cut = select(s, n, (u64)(k - before), false, 0, top.v, rate);
                mass_k = mass_before + mass_from(n, cut);
                held = fits(its_above + its_n);
                if (held) {
                    const int own_n = s.n;
                    for (int i = tid; i < own_n; i += kThreads)
                        if (s.list[i] >= cut) s.held[atomicAdd(&s.held_n, 1)] = s.list[i];
                    __syncthreads();
                }
            } else if (stride > 1) {
                cluster.sync();  // others may still read what the next turn writes
                continue;        // outside the bracket, or too many in it
            } else {
                cut = kth_key(x, a.V, k, s);
                u64 own_mass = 0;
                each(x, 0, a.V, -INFINITY, [&](float v, int i) {
                    if (full_key(v, i) >= cut) own_mass += mass_of(v, top.v, rate);
                    return true;
                });
                block_before(own_mass, mass_k, s);
            }
            if (by_p) goal = goal_of((double)mass_k);
            break;
        }
    }
    // 4. the race over K, until its winner is in top_p's prefix
    // from the largest token, which is always kept, on
    const uint32_t same = __ballot_sync(0xffffffffu, lane < kPer && top.i + lane < a.V && clean(io<T>::ld(x + top.i + lane)) == top.v);
    const int first_i = top.i + __ffs(same) - 1;
    const Best first = score(top.v, first_i, u[first_i]);
    // Noise that goes with the logits' order could have winner after winner rejected: from round kRounds on the keys between
    // the last one and the lowest known to be kept are halved, 64 times at most, and the race is run once more from the end of
    // the prefix.
    bool verify = by_p;
    u64 kept = full_key(top.v, 0);  // keys from here on are kept
    for (int round = 0;; ++round) {
        const bool racing = round < kRounds || !verify;
        u64 probe = cut + (kept - cut) / 2;
        if (racing) {
            // no Gumbel is above 16.64
            const float floor = fmaxf(fmaxf(min_logit, top.v + t * (first.v - 16.7f) - 1e-5f * fabsf(top.v)), cut ? value_of((uint32_t)(cut >> 32)) : -INFINITY);
            const Track track = {u, top.v, t, rate, min_p, fmaxf(floor, -3.402823466e38f), reach_of(first.v), cut};
            won = held ? race_held(track, first, s) : race_pass(x, from, to, track, first);
            won = block_best(won, s);
            if (tid == 0) s.x.won = won;
            cluster.sync();
            won = best_of(from_peer.x.won);
            if (!verify || won.i < 0) break;
            probe = full_key(clean(io<T>::ld(x + won.i)), won.i);
        }
        u64 own_mass = 0, own_above = 0, all_mass, all_above;
        if (held) {
            const int n = s.held_n;
            for (int i = tid; i < n; i += kThreads)
                if (s.held[i] > probe) own_mass += mass_of(value_of((uint32_t)(s.held[i] >> 32)), top.v, rate);
        } else {
            const Above above = mass_pass(x, from, to, value_of((uint32_t)(probe >> 32)), ~(uint32_t)probe, top.v, rate);
            own_mass = (u64)(above.mass * kUnit + 0.5f);
            own_above = (u64)above.n;
        }
        block_before(own_mass, all_mass, s);
        block_before(own_above, all_above, s);
        const int slot = round & 1;
        if (tid == 0) s.x.mass[slot] = all_mass, s.x.above[slot] = (int)all_above;
        cluster.sync();
        const u64 mass = sum_of(from_peer.x.mass[slot]);
        const int its_above = from_peer.x.above[slot];
        if (mass < goal) {
            if (racing) break;
            kept = probe;
        } else {
            cut = probe + 1;  // the probe and what is below it are not kept
            won = {-INFINITY, -1};
            if (!held && fits(its_above)) {  // what is left: those above the probe
                held = true;
                if (tid == 0) s.held_n = 0;
                __syncthreads();
                gather_pass(x, from, to, value_of((uint32_t)(cut >> 32)), ~(uint32_t)cut, s.held, kHeld, &s.held_n);
                __syncthreads();
            }
        }
        if (!racing && cut >= kept) {
            cut = kept;
            verify = false;
        }
    }
    cluster.sync();
    if (rank == 0 && tid == 0) finish(won);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream) {
    // CTAs per row: double while all rows' CTAs make two waves at most (152 SMs, four CTAs each) and a CTA has 4096 tokens
    // left.  At 256 rows of 100003, on one, two, four and eight CTAs each: rows alike, with top_k 50 and top_p 0.9, take 58, 45,
    // 50 and 72 us, greedy ones 27, 22, 26 and 37, rows of mixed settings (six draws of them) 160 to 197, 108 to 117, 80 to 93 and 95
    // to 107 us, where the few flat rows' CTAs run on alone.  Four of 256 threads to an SM against three: greedy rows 26 us and 32,
    // rows with top_k 50 and top_p 0.9 50 and 60, mixed ones 80 to 93 and 84 to 95.
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
