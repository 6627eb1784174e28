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
//   3. if it is more than fits (flat rows, large k), a histogram of 2048 bins over y, of counts for top_k and of the
//      weights relative to their bin's upper edge for top_p (32-bit atomics), finds the bins where the cut falls: one,
//      or a few where sums of mass leave it open.  Only their tokens are gathered, with the exact mass above them;
//   4. if even those are more than fit (thousands of equal logits), the first CTA finds the cut digit by digit of the
//      sorting key, a pass over the row each;
//   5. the race.  The largest token is always kept and its Gumbel is above -3.2, no Gumbel is above 16.7:
//      tokens with y < -20 cannot win, and their noise is not read.  The others race on approximate scores, and
//      only those within 10^-3 of a thread's best are decided on exact ones.
//
// Masses are whole numbers in units of 2^-40 of the largest weight, of a token or of the up to 8 tokens of one load,
// summed in 64 bits: the sums do not depend on the order the atomics come in.  The weights in masses are 2^x approximations
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
    u64 mass[kBins];       // of the whole row's bins; before that, the warps' queues of the race
    uint32_t count[kBins], part[kBins];  // of this CTA's tokens
    u64 sums[kWarps];
    Best bests[kWarps];
    float parts[2][kWarps];
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

// Sorts the s.n gathered keys in descending order (bitonic).  Key i lies with thread i % kThreads: keys kThreads and more
// apart meet in a thread, less than 32 apart by shuffles, and only the distances between go through shared memory.
__device__ void sort_list(Shared &s) {
    constexpr int kEach = kList / kThreads;
    const int tid = threadIdx.x, n = s.n;
    int size = 32;
    while (size < n) size <<= 1;
    u64 r[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int i = e * kThreads + tid;
        r[e] = i < n ? s.list[i] : 0;
    }
    auto keep = [](u64 mine, u64 other, bool larger) { return (mine < other) == larger ? other : mine; };
    for (int run = 2; run <= size; run <<= 1)
        for (int gap = run >> 1; gap; gap >>= 1) {
            if (gap >= kThreads) {
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    const int f = e ^ (gap / kThreads);
                    if (f > e && f < kEach) {
                        const bool down = ((e * kThreads + tid) & run) == 0;
                        const u64 x = r[e], y = r[f];
                        r[e] = keep(x, y, down);
                        r[f] = keep(y, x, !down);
                    }
                }
            } else if (gap >= 32) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < kEach; ++e)
                    if (e * kThreads < size) s.list[e * kThreads + tid] = r[e];
                __syncthreads();
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    const int i = e * kThreads + tid;
                    if (e * kThreads < size) r[e] = keep(r[e], s.list[i ^ gap], ((i & run) == 0) == ((i & gap) == 0));
                }
            } else {
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    const int i = e * kThreads + tid;
                    if (e * kThreads < size)
                        r[e] = keep(r[e], __shfl_xor_sync(0xffffffffu, r[e], gap), ((i & run) == 0) == ((i & gap) == 0));
                }
            }
        }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kEach; ++e)
        if (e * kThreads < size) s.list[e * kThreads + tid] = r[e];
    __syncthreads();
}

// Exact score of a token, {-inf, -1} if min_p or a weight of 0 rules it out.  A call: few tokens need it, and inlined in
// several loops it crowds the instruction cache.
__device__ __noinline__ Best exact_score(float v, int i, float top, float t, float min_p, const float *u) {
    const float y = (v - top) / t, w = expf(y);
    if (!(w > 0.f) || w < min_p) return {-INFINITY, -1};
    const float r = fminf(fmaxf(u[i], 2.3283064365386963e-10f), 0.999999940395355f);
    return {y - logf(-logf(r)), i};
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
            while (clean(io<T>::ld(x + won.i)) != top.v) ++won.i;  // within its load
        }
        a.tokens[b] = won.i;
        if (a.logprobs) a.logprobs[b] = won.i < 0 ? -INFINITY : greedy ? 0.f : (clean(io<T>::ld(x + won.i)) - top.v) / t - logf(total);
    };
    if (top.i < 0 || greedy) {
        if (rank == 0 && tid == 0) finish({-INFINITY, -1});
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

    // 5. the race.  Tokens that may win wait in a queue per warp until four per lane are there: all lanes work, on loads that
    // overlap.  Where most tokens may win they are taken as they come.
    Best lead = {-INFINITY, -1}, won = {-INFINITY, -1};
    float cut_v = -INFINITY, floor = 0.f;  // set by race_from: what is below cannot be kept, or cannot win
    int cut_i = -1;
    const float sure = min_p > 1.f ? INFINITY : min_p > 0.f ? logit_of(min_p, 1.f) : -INFINITY;  // w >= min_p from here on
    auto race_from = [&](u64 key) {
        cut_v = key ? value_of((uint32_t)(key >> 32)) : -INFINITY;
        cut_i = (int)~(uint32_t)key;
        floor = fmaxf(fmaxf(fmaxf(min_logit, top.v - 20.f * t - 1e-5f * fabsf(top.v)), cut_v), -3.402823466e38f);
        lead = won = {-INFINITY, -1};
    };
    auto enter = [&](float v, int i, float r) {  // v = -inf: no token
        const float c = fminf(fmaxf(r, 2.3283064365386963e-10f), 0.999999940395355f), d = 1.f - c;
        // -log u: by its series near 1, where the approximate logarithm has no digits left
        const float clock = c > 0.99f ? d + 0.5f * d * d : lg2(c) * -0.6931471805599453f;
        const float rough = ((v - top.v) * rate - lg2(clock)) * 0.6931471805599453f;  // good to 10^-4
        const bool clear = rough > lead.v + 1e-3f && v >= sure;
        if (!clear && rough >= lead.v - 1e-3f && v > -INFINITY) {  // too near to tell, or min_p in doubt
            const Best exact = score(v, i);
            if (exact.i >= 0) {
                won = better(won, exact);
                if (rough > lead.v) {
                    if (lead.i >= 0) won = better(won, score(clean(io<T>::ld(x + lead.i)), lead.i));
                    lead = {rough, i};
                }
            }
        }
        lead.v = clear ? rough : lead.v;
        lead.i = clear ? i : lead.i;
    };
    constexpr int kBatch = 128, kRoom = kBatch + 32;
    static_assert(kWarps * kRoom <= kList + kBins, "the queues lie over list and mass");
    auto race_tokens = [&]() {
        u64 *queue = s.list + warp * kRoom;
        int waiting = 0;
        auto run_batch = [&](int n) {
            float v[4], r[4];
            int i[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool have = lane + 32 * e < n;
                const u64 q = have ? queue[lane + 32 * e] : 0;
                v[e] = have ? __uint_as_float((uint32_t)(q >> 32)) : -INFINITY;
                i[e] = (int)(uint32_t)q;
                r[e] = u[i[e]];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) enter(v[e], i[e], r[e]);
        };
        // N tokens from `at` on per lane, -inf where there is none
        auto take = [&](auto count, const float *w, int at) {
            constexpr int N = decltype(count)::value;
            float v[N];
            uint32_t mask[N];
            int some = 0;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float y = clean(w[e]);
                const bool in = y >= floor && !(y == cut_v && at + e > cut_i);
                v[e] = in ? y : -INFINITY;
                mask[e] = __ballot_sync(0xffffffffu, in);
                some += __popc(mask[e]);
            }
            if (some >= 16 * N) {
                float r[N];
#pragma unroll
                for (int e = 0; e < N; ++e) r[e] = v[e] > -INFINITY ? u[at + e] : 0.5f;
#pragma unroll
                for (int e = 0; e < N; ++e) enter(v[e], at + e, r[e]);
                return;
            }
            if (some == 0) return;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                if (mask[e] == 0) continue;
                if (v[e] > -INFINITY)
                    queue[waiting + __popc(mask[e] & ((1u << lane) - 1))] = (u64)__float_as_uint(v[e]) << 32 | (uint32_t)(at + e);
                waiting += __popc(mask[e]);
                __syncwarp();
                if (waiting >= kBatch) {
                    run_batch(kBatch);
                    waiting -= kBatch;
                    const u64 rest = lane < waiting ? queue[kBatch + lane] : 0;
                    __syncwarp();
                    if (lane < waiting) queue[lane] = rest;
                    __syncwarp();
                }
            }
        };
        // as each_piece, but every lane of a warp takes part in every step
        const T *row = x + from;
        const int head = min(to - from, (int)((16 - ((uintptr_t)row & 15)) & 15) / (int)sizeof(T)), pieces = (to - from - head) / kPer;
        const uint4 *p4 = (const uint4 *)(row + head);
        for (int i0 = warp * 32; i0 < pieces; i0 += 4 * kThreads) {
            uint4 w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = i0 + q * kThreads + lane;
                // all ones: NaN in either type, never kept
                w[q] = i < pieces ? p4[i] : make_uint4(~0u, ~0u, ~0u, ~0u);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (i0 + q * kThreads >= pieces) break;
                const uint32_t b[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
                float v[kPer];
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    if constexpr (sizeof(T) == 2) v[e] = __uint_as_float(e & 1 ? b[e / 2] & 0xffff0000u : b[e / 2] << 16);
                    else v[e] = __uint_as_float(b[e]);
                }
                take(Count<kPer>(), v, from + head + (i0 + q * kThreads + lane) * kPer);
            }
        }
        if (warp == 0) {  // the single tokens before and after
            const int tail = head + pieces * kPer, i = lane < 16 ? lane : tail + lane - 16;
            const bool have = lane < 16 ? lane < head : i < to - from;
            const float v = have ? io<T>::ld(row + i) : -INFINITY;
            take(Count<1>(), &v, have ? from + i : 0);
        }
        run_batch(waiting);
    };

    bool raced = false;
    u64 cut = 0;  // the smallest key that top_k and top_p keep
    if (by_k || by_p) {
        // 2. gather what passes the threshold
        if (!(by_k && by_p)) least = fmaxf(least, min_logit);  // with both, all of K counts in its mass
        if (by_p && !by_k) least = fmaxf(least, logit_of((1.f - fmaxf(p, 0.f)) * total / (float)a.V, -1.f));
        if (tid == 0) s.n = 0;
        __syncthreads();
        each(x, from, to, least, [&](float v, int i) { return gather(s, full_key(v, i)); });
        __syncthreads();
        if (tid == 0) s.x.gathered = min(s.n, kList + 1);
        cluster.sync();
        const int n = sum_of(from_peer.x.gathered);
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
        const bool deep = bottom == top.v - kReach * t;  // the last bin's tokens have no mass and cannot win
        const float scale = bounded((float)kBins / (top.v - bottom));
        const float width = (top.v - bottom) / (t * kBins);  // of a bin, in y
        auto bin_of = [&](float v) { return (int)fminf((top.v - v) * scale, (float)(kBins - 1)); };
        // sums of weights relative to their bin's upper edge, in units that the CTA's tokens cannot overflow together
        const float unit = (float)(1u << min(20, 31 - (32 - __clz(share))));
        for (int i = tid; i < kBins; i += kThreads) s.count[i] = s.part[i] = 0;
        __syncthreads();
        each(x, from, to, by_k ? -INFINITY : least, [&](float v, int) {
            const float d = fminf((top.v - v) * scale, (float)(kBins - 1));
            const int bin = (int)d;
            const float f = (d - (float)bin) * width;
            if (by_k) atomicAdd(&s.count[bin], 1u);
            if (by_p) atomicAdd(&s.part[bin], (uint32_t)((1.f - f + 0.5f * f * f) * unit + 0.5f));  // exp(-f)
            return true;
        });
        cluster.sync();
        {
            // each CTA joins a range of bins for the first one: counts into its list, masses into its mass
            const int step = kBins / ctas;
            uint32_t *counts = (uint32_t *)cluster.map_shared_rank(s.list, 0);
            u64 *masses = cluster.map_shared_rank(s.mass, 0);
            for (int i = rank * step + tid; i < (rank + 1) * step; i += kThreads) {
                uint32_t c = 0;
                u64 m = 0;
#pragma unroll
                for (int r = 0; r < kMaxCtas; ++r)
                    if (r < ctas) c += peer(r).count[i], m += peer(r).part[i];
                counts[i] = c;
                masses[i] = (u64)(ex2(-(float)i * width * 1.4426950408889634f) * (kUnit / unit) * (float)m);
            }
        }
        cluster.sync();
        // the first bin whose running sum reaches `goal` (s.found, with the sum before it in s.before), or kBins
        auto find_bin = [&](u64 goal, bool of_mass) {
            constexpr int kEach = kBins / kThreads;
            u64 own = 0, all;
            const uint32_t *counts = (const uint32_t *)s.list;
            for (int e = 0; e < kEach; ++e) own += of_mass ? s.mass[tid * kEach + e] : counts[tid * kEach + e];
            u64 at = block_before(own, all, s);
            if (tid == 0 && all < goal) s.found = kBins;
            if (at < goal && at + own >= goal) {
                int e = 0;
                for (;; ++e) {
                    const u64 y = of_mass ? s.mass[tid * kEach + e] : counts[tid * kEach + e];
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
        auto plan_p = [&](int limit) {  // the bins that may hold the end of the mass `goal`: sums are good to 2^-16
            find_bin(max((u64)((double)goal * (1.0 - 1.0 / 32768)), 1ull), true);
            const int lo = s.found;
            __syncthreads();
            find_bin((u64)((double)goal * (1.0 + 1.0 / 32768)) + 1, true);
            const int hi = min(min(s.found, kBins - 1), limit);
            __syncthreads();
            want_p = true;
            if (lo > hi) set_plan(-1, 0);  // less mass than that in all: everything stays
            else set_plan(lo, hi);
        };
        if (rank == 0) {
            if (by_k) {
                find_bin((u64)k, false);
                bin_k = s.found;
                rank_k = k - (int)s.before;
                if (deep && bin_k == kBins - 1) bin_k = kBins;  // all that matters is in K
                __syncthreads();
            }
            if (bin_k < kBins) set_plan(bin_k, bin_k);
            else if (by_p) goal = goal_of((double)total * (double)kUnit), plan_p(kBins - 1 - deep);
            else set_plan(-1, 0);  // K is every token that can win
        }
        for (;;) {
            cluster.sync();
            const int lo = peer(0).x.lo, hi = peer(0).x.hi;
            cut = peer(0).x.cut;
            if (lo < 0) break;
            u64 above = 0;
            if (tid == 0) s.n = 0;
            __syncthreads();
            each_piece(x, from, to, [&](const float *w, auto n, int at) {
                constexpr int N = decltype(n)::value;
                float y = 0.f;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float v = clean(w[e]);
                    const int bin = bin_of(v);  // of -inf: the last
                    if (bin < lo) y += ex2((v - top.v) * rate);
                    else if (bin <= hi && v > -INFINITY) gather(s, full_key(v, at + e));
                }
                if (by_p) above += (u64)(y * kUnit + 0.5f);
                return true;
            });
            u64 all = 0;
            block_before(above, all, s);
            if (tid == 0) s.x.gathered = min(s.n, kList + 1), s.x.mass = all;
            cluster.sync();
            if (rank != 0) continue;
            above = sum_of(from_peer.x.mass);
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
                if (above >= goal || s.n == 0 || (end < goal && hi < min(kBins - deep, bin_k) - 1)) slow = true;
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
                        each(x, 0, a.V, -INFINITY, [&](float v, int i) {
                            const u64 key = full_key(v, i);
                            if (key >= floor && (shift == 56 || (key >> (shift + 8)) == prefix))
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
                    each(x, 0, a.V, -INFINITY, [&](float v, int i) {
                        if (full_key(v, i) >= cut) own += mass(v);
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
    if (!raced) {
        race_from(cut);
        __syncthreads();  // list and mass are free
        race_tokens();
    }
    if (lead.i >= 0) won = better(won, score(clean(io<T>::ld(x + lead.i)), lead.i));
    won = block_best(won, s);
    if (tid == 0) s.x.won = won;
    cluster.sync();
    if (rank == 0 && warp == 0) {
        won = best_of(from_peer.x.won);
        if (tid == 0) finish(won);
    }
    cluster.sync();
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream) {
    // CTAs per row: double while all rows' CTAs fit the GPU at once (152 SMs, two CTAs each) and a CTA has 4096 tokens
    // left.  Past one wave it costs: 256 rows of 100003 with top_k 50 and top_p 0.9 take 43 us on one CTA each, 59 on
    // two; 32 rows of 131072 take 24 us on eight.
    int ctas = 1;
    while (ctas < kMaxCtas && (int64_t)a.B * ctas * 2 <= 304 && a.V / (2 * ctas) >= 4096) ctas *= 2;
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
