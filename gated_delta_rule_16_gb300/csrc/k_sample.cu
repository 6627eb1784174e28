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
// What bounds it: the row is read once from HBM; everything after works on few tokens or
// on the row in L2.  One CTA per row:
//   1. one pass for the maximum, the sum of weights and every thread's own maximum;
//   2. a threshold that no kept token is below.  For top_k: the k-th largest of the threads' maxima (k
//      tokens at least are as large).  For top_p: tokens below (1 - p) M / V hold (1 - p) M
//      together at most, so the prefix of mass p M ends above it.  What passes the
//      threshold, a few hundred tokens as a rule, is gathered, sorted and cut in shared memory;
//   3. if it is more than fits (flat rows, large k), a histogram of 2048 bins over y finds
//      the bin where the cut falls, and only that bin's tokens are sorted;
//   4. if even one bin is more than fits (thousands of equal logits), the cut is found digit by
//      digit of the sorting key, a pass over the row each;
//   5. the race.  The largest token is always kept and its Gumbel is above -3.2, no Gumbel
//      is above 16.7: tokens with y < -20 cannot win, and their noise is not read.
//
// Masses are whole numbers in units of 2^-40 of the largest weight, summed in 64 bits: exact
// sums, whatever order the atomics come in.  The weights in masses are 2^x approximations
// (2^-21); w > 0, w >= min_p and the race are decided in IEEE fp32 with accurate exp and log.
#include "paged.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kList = 2048;  // gathered tokens
constexpr int kBins = 2048;  // of width 1/73 in y: 28 = 40 ln 2, below which a mass rounds to 0
constexpr float kUnit = 1099511627776.f;  // 2^40
using u64 = unsigned long long;

__device__ __forceinline__ float clean(float x) {  // NaN never wins, +inf is the largest number, -0 is 0
    return x != x ? -INFINITY : fminf(x, 3.402823466e38f) + 0.f;
}
// Ordered: larger floats have larger keys.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x);
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

struct Best { float v; int i; };
__device__ __forceinline__ Best better(Best a, Best b) {
    return b.v > a.v || (b.v == a.v && (unsigned)b.i < (unsigned)a.i) ? b : a;
}

struct Shared {
    u64 list[kList];
    u64 mass[kBins];
    uint32_t count[kBins];
    u64 sums[kWarps];
    Best bests[kWarps];
    float parts[kWarps];
    int n, found;          // tokens gathered; bin or rank found
    u64 before, digit;
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
__device__ float block_sum(float x, Shared &s) {
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.parts[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += s.parts[w];
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

// f(logit, index) for every token of a row, in 16-byte loads four of which are in flight per thread;
// a thread meets its tokens in ascending order.  f returns false to end the thread's pass.
template <typename T, typename F>
__device__ __forceinline__ void each(const T *x, int V, F f) {
    constexpr int kPer = 16 / sizeof(T);
    const int tid = threadIdx.x;
    const int head = min(V, (int)((16 - ((uintptr_t)x & 15)) & 15) / (int)sizeof(T)), pieces = (V - head) / kPer;
    if (tid < head && !f(io<T>::ld(x + tid), tid)) return;
    const uint4 *p = (const uint4 *)(x + head);
    for (int i0 = tid; i0 < pieces; i0 += 4 * kThreads) {
        uint4 w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i0 + u * kThreads < pieces) w[u] = p[i0 + u * kThreads];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (i0 + u * kThreads >= pieces) break;
            const int at = head + (i0 + u * kThreads) * kPer;
            const uint32_t q[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                float v;
                if constexpr (sizeof(T) == 2) v = __uint_as_float(e & 1 ? q[e / 2] & 0xffff0000u : q[e / 2] << 16);
                else v = __uint_as_float(q[e]);
                if (!f(v, at + e)) return;
            }
        }
    }
    const int t = head + pieces * kPer + tid;
    if (t < V) f(io<T>::ld(x + t), t);
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
__global__ void __launch_bounds__(kThreads) sample_kernel(SampleArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared &s = *(Shared *)raw;
    const int b = blockIdx.x, tid = threadIdx.x;
    const T *x = (const T *)a.logits + b * a.logits_stride;
    const float *u = a.noise + b * a.noise_stride;
    const float t = a.temperature ? a.temperature[b] : 1.f;
    const bool greedy = !(t > 0.f);
    // y log2(e) per unit of x, kept off 0 and infinity: 0 and infinite differences stay what they are
    auto bounded = [](float f) { return fmaxf(fminf(f, 1e30f), 1e-37f); };
    const float rate = bounded(1.4426950408889634f / t);

    // 1. maximum, sum of weights
    Best top = {-INFINITY, -1};
    float sum = 0.f;
    if (greedy) {
        each(x, a.V, [&](float v, int i) {
            v = clean(v);
            if (v > top.v) top = {v, i};
            return true;
        });
    } else {
        each(x, a.V, [&](float v, int i) {
            v = clean(v);
            if (v > top.v) {
                sum = sum * ex2((top.v - v) * rate) + 1.f;
                top = {v, i};
            } else if (v > -INFINITY) {
                sum += ex2((v - top.v) * rate);
            }
            return true;
        });
    }
    const float mine = top.v;
    top = block_best(top, s);
    if (top.i < 0 || greedy) {
        if (tid == 0) {
            a.tokens[b] = top.i;
            if (a.logprobs) a.logprobs[b] = top.i < 0 ? -INFINITY : 0.f;
        }
        return;
    }
    const float total = block_sum(mine > -INFINITY ? sum * ex2((mine - top.v) * rate) : 0.f, s);

    auto tempered = [&](float v) { return (v - top.v) / t; };
    auto mass = [&](float v) { return (u64)(ex2((v - top.v) * rate) * kUnit + 0.5f); };
    const int k = a.top_k ? a.top_k[b] : 0;
    const float p = a.top_p ? a.top_p[b] : 1.f, min_p = a.min_p ? a.min_p[b] : 0.f;
    const bool by_k = k > 0 && k < a.V, by_p = p < 1.f;
    // a logit below which w < f, with room for every rounding on the way
    auto logit_of = [&](float f) {
        const float d = t * logf(f);
        return top.v + d - (1e-5f * (fabsf(top.v) + fabsf(d)) + 1e-3f * t);
    };
    const float min_logit = min_p > 0.f ? logit_of(fminf(min_p, 1.f)) : -INFINITY;
    auto goal_of = [&](double m) {  // p of mass m, at least one unit: the largest token always stays
        const double g = ceil((double)fmaxf(p, 0.f) * m);
        return g < 1.0 ? 1ull : (u64)g;
    };

    Best won = {-INFINITY, -1};
    // exact conditions and score of one token whose key passes the cut
    auto race = [&](float v, int i) {
        const float y = tempered(v), w = expf(y);
        if (!(w > 0.f) || w < min_p) return;
        const float r = fminf(fmaxf(u[i], 2.3283064365386963e-10f), 0.999999940395355f);
        won = better(won, {y - logf(-logf(r)), i});
    };

    u64 cut = 0;  // the smallest key that top_k and top_p keep
    bool done = false;
    if (by_k || by_p) {
        // 2. gather what passes the threshold
        float least = -INFINITY;
        if (by_k && k <= kThreads) {
            const uint32_t own = mine > -INFINITY ? key_of(mine) : 0u;
            uint32_t key = 0;
#pragma unroll 1
            for (int bit = 31; bit >= (sizeof(T) == 2 ? 16 : 0); --bit) {
                const uint32_t next = key | 1u << bit;
                if (__syncthreads_count(own >= next) >= k) key = next;
            }
            if (key) least = value_of(key);
        }
        if (!(by_k && by_p)) least = fmaxf(least, min_logit);  // with both, all of K counts in its mass
        if (by_p && !by_k) least = fmaxf(least, logit_of((1.f - fmaxf(p, 0.f)) * total / (float)a.V));
        if (tid == 0) s.n = 0;
        __syncthreads();
        each(x, a.V, [&](float v, int i) {
            v = clean(v);
            return v >= least && v > -INFINITY ? gather(s, full_key(v, i)) : true;
        });
        __syncthreads();
        if (s.n <= kList) {
            const int n = s.n;
            sort_list(s);
            constexpr int kEach = kList / kThreads;
            u64 own = 0, all, m[kEach];
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int r = tid * kEach + e;
                m[e] = r < n && !(by_k && r >= k) ? mass(value_of((uint32_t)(s.list[r] >> 32))) : 0;
                own += m[e];
            }
            u64 before = block_before(own, all, s);
            const u64 goal = by_p ? goal_of(by_k ? (double)all : (double)total * (double)kUnit) : ~0ull;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int r = tid * kEach + e;
                if (r < n && !(by_k && r >= k) && before < goal) {
                    const u64 key = s.list[r];
                    race(value_of((uint32_t)(key >> 32)), (int)~(uint32_t)key);
                }
                before += m[e];
            }
            done = true;
        } else {
            // 3. histogram over y
            const float scale = bounded(73.f / t);
            auto bin_of = [&](float v) { return (int)fminf((top.v - v) * scale, (float)(kBins - 1)); };
            __syncthreads();
            for (int i = tid; i < kBins; i += kThreads) s.count[i] = 0, s.mass[i] = 0;
            __syncthreads();
            each(x, a.V, [&](float v, int i) {
                v = clean(v);
                if (v > -INFINITY) {
                    const int bin = bin_of(v);
                    atomicAdd(&s.count[bin], 1u);
                    if (by_p) atomicAdd(&s.mass[bin], mass(v));
                }
                return true;
            });
            __syncthreads();
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
            auto gather_bin = [&](int bin) {  // sorted; false if there are too many
                if (tid == 0) s.n = 0;
                __syncthreads();
                each(x, a.V, [&](float v, int i) {
                    v = clean(v);
                    return v > -INFINITY && bin_of(v) == bin ? gather(s, full_key(v, i)) : true;
                });
                __syncthreads();
                if (s.n > kList) return false;
                sort_list(s);
                return true;
            };
            // mass before rank r of the sorted list, if r >= 0; else the first rank whose running mass reaches goal,
            // in s.found (kList: none)
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
            bool fits = true;
            int bin_k = kBins, rank_k = 0;
            u64 above_k = 0, mass_k = 0;  // masses of the bins above the k-th token's, and of K
            if (by_k) {
                find_bin((u64)k, false);
                bin_k = s.found;
                if (bin_k < kBins) {
                    rank_k = k - (int)s.before;
                    fits = gather_bin(bin_k);
                    if (fits) {
                        cut = s.list[rank_k - 1];
                        if (by_p) {
                            u64 own = 0;
                            for (int i = tid; i < bin_k; i += kThreads) own += s.mass[i];
                            block_before(own, above_k, s);
                            mass_k = in_list(rank_k, above_k, ~0ull);
                        }
                    }
                }  // else fewer than k finite logits: all of them are in K
            }
            if (by_p && fits) {
                const bool all_of = bin_k == kBins;  // K is every finite logit
                const u64 goal = goal_of(all_of ? (double)total * (double)kUnit : (double)mass_k);
                if (!all_of && goal > above_k) {
                    in_list(rank_k, above_k, goal);
                    if (s.found < rank_k) cut = s.list[s.found];
                } else {
                    find_bin(goal, true);
                    const int bin = s.found;
                    const u64 before = s.before;
                    if (bin < kBins) {
                        fits = gather_bin(bin);
                        if (fits) {
                            in_list(s.n, before, goal);
                            cut = s.list[s.found];
                        }
                    }
                }
            }
            if (!fits) {
                // 4. digit by digit: the key of the last token of the shortest descending prefix, among keys >= floor, whose
                // measure (tokens, or mass) reaches goal
                auto descend = [&](u64 goal, bool of_mass, u64 floor) {
                    u64 prefix = 0, before = 0;
                    for (int shift = 56; shift >= 0; shift -= 8) {
                        __syncthreads();
                        if (tid < 256) s.mass[tid] = 0;
                        __syncthreads();
                        each(x, a.V, [&](float v, int i) {
                            v = clean(v);
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
                cut = by_k && bin_k < kBins ? descend((u64)k, false, 0) : 0;
                if (by_p) {
                    u64 own = 0, all;
                    each(x, a.V, [&](float v, int i) {
                        v = clean(v);
                        if (v > -INFINITY && full_key(v, i) >= cut) own += mass(v);
                        return true;
                    });
                    block_before(own, all, s);
                    const u64 c = descend(min(goal_of((double)all), all), true, cut);
                    cut = c > cut ? c : cut;
                }
            }
        }
    }
    // 5. the race over the row
    if (!done) {
        const float floor = fmaxf(fmaxf(min_logit, top.v - 20.f * t - 1e-5f * fabsf(top.v)),
                                  cut ? value_of((uint32_t)(cut >> 32)) : -INFINITY);
        each(x, a.V, [&](float v, int i) {
            v = clean(v);
            if (v >= floor && v > -INFINITY && full_key(v, i) >= cut) race(v, i);
            return true;
        });
    }
    won = block_best(won, s);
    if (won.i < 0) won = top;  // min_p above 1 leaves nothing: the largest stays
    if (tid == 0) {
        a.tokens[b] = won.i;
        if (a.logprobs) a.logprobs[b] = tempered(clean(io<T>::ld(x + won.i))) - logf(total);
    }
}

}  // namespace

size_t sample_workspace_bytes(int, int) { return 0; }

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream) {
    auto go = [&](auto kern) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
        if (e != cudaSuccess) return e;
        kern<<<a.B, kThreads, sizeof(Shared), stream>>>(a);
        return cudaGetLastError();
    };
    return a.dtype == GDN_BF16 ? go(sample_kernel<__nv_bfloat16>) : go(sample_kernel<float>);
}

}  // namespace gdn
