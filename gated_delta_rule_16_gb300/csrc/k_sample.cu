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
// Masses are whole numbers in units of 2^-40 of the largest weight, summed in 64
// bits: exact sums, whatever order the atomics come in.
//
// First form: one CTA per row; top_k and top_p find their cut by descending the digits of
// the sorting key (the logit's ordered bits, then the index), one pass over the row each.
#include "paged.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 1024;
constexpr float kUnit = 1099511627776.f;  // 2^40

__device__ __forceinline__ float clean(float x) {  // NaN never wins, +inf is the largest number, -0 is 0
    return x != x ? -INFINITY : fminf(x, 3.402823466e38f) + 0.f;
}
// Ordered: larger floats have larger keys.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Best { float v; int i; };
__device__ __forceinline__ Best better(Best a, Best b) {
    return b.v > a.v || (b.v == a.v && (unsigned)b.i < (unsigned)a.i) ? b : a;
}
__device__ Best block_best(Best x, Best *buf) {
    for (int off = 16; off; off >>= 1)
        x = better(x, {__shfl_xor_sync(0xffffffffu, x.v, off), __shfl_xor_sync(0xffffffffu, x.i, off)});
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) x = better(x, buf[w]);
    return x;
}
__device__ unsigned long long block_sum(unsigned long long x, unsigned long long *buf) {
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0;
    for (int w = 0; w < kThreads / 32; ++w) x += buf[w];
    return x;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(SampleArgs a) {
    __shared__ unsigned long long hist[256], sums[kThreads / 32];
    __shared__ Best bests[kThreads / 32];
    __shared__ unsigned long long chosen_digit, chosen_before;
    const int b = blockIdx.x, tid = threadIdx.x;
    const T *x = (const T *)a.logits + b * a.logits_stride;
    const float *u = a.noise + b * a.noise_stride;
    const float t = a.temperature ? a.temperature[b] : 1.f;

    Best top = {-INFINITY, -1};
    for (int i = tid; i < a.V; i += kThreads) {
        const float v = clean(io<T>::ld(x + i));
        if (v > -INFINITY) top = better(top, {v, i});
    }
    top = block_best(top, bests);
    if (top.i < 0 || !(t > 0.f)) {
        if (tid == 0) {
            a.tokens[b] = top.i;
            if (a.logprobs) a.logprobs[b] = top.i < 0 ? -INFINITY : 0.f;
        }
        return;
    }
    auto tempered = [&](float v) { return (v - top.v) / t; };
    auto mass = [&](float w) { return w > 0.f ? (unsigned long long)(w * kUnit + 0.5f) : 0ull; };
    unsigned long long total = 0;
    for (int i = tid; i < a.V; i += kThreads) total += mass(expf(tempered(clean(io<T>::ld(x + i)))));
    total = block_sum(total, sums);

    // The sorting key of a token: ordered logit bits, then the complement of the index.
    auto full_key = [&](float v, int i) { return (unsigned long long)key_of(v) << 32 | (uint32_t)~i; };
    // The key of the last token of the shortest descending prefix, among keys >= least, of measure >= target.
    auto cut = [&](unsigned long long target, bool by_mass, unsigned long long least) {
        unsigned long long prefix = 0, before = 0;
        for (int shift = 56; shift >= 0; shift -= 8) {
            __syncthreads();
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int i = tid; i < a.V; i += kThreads) {
                const float v = clean(io<T>::ld(x + i));
                const unsigned long long k = full_key(v, i);
                if (k < least || (shift < 56 && (k >> (shift + 8)) != prefix)) continue;
                atomicAdd(&hist[(k >> shift) & 255], by_mass ? mass(expf(tempered(v))) : 1ull);
            }
            __syncthreads();
            if (tid == 0) {
                unsigned long long cum = before;
                int d = 255;
                for (; d > 0 && cum + hist[d] < target; --d) cum += hist[d];
                chosen_digit = d;
                chosen_before = cum;
            }
            __syncthreads();
            prefix = prefix << 8 | chosen_digit;
            before = chosen_before;
        }
        return prefix;
    };
    unsigned long long least = 0;
    const int k = a.top_k ? a.top_k[b] : 0;
    if (k > 0 && k < a.V) least = cut((unsigned long long)k, false, 0);
    const float p = a.top_p ? a.top_p[b] : 1.f;
    if (p < 1.f) {
        unsigned long long m = 0;
        for (int i = tid; i < a.V; i += kThreads) {
            const float v = clean(io<T>::ld(x + i));
            if (full_key(v, i) >= least) m += mass(expf(tempered(v)));
        }
        m = block_sum(m, sums);
        const double target = ceil((double)fmaxf(p, 0.f) * (double)m);
        const unsigned long long goal = target < 1.0 ? 1ull : (unsigned long long)target;
        const unsigned long long c = cut(goal, true, least);
        least = c > least ? c : least;
    }
    const float min_p = a.min_p ? a.min_p[b] : 0.f;
    Best won = {-INFINITY, -1};
    for (int i = tid; i < a.V; i += kThreads) {
        const float v = clean(io<T>::ld(x + i)), y = tempered(v), w = expf(y);
        if (!(w > 0.f) || w < min_p || full_key(v, i) < least) continue;
        const float r = fminf(fmaxf(u[i], 2.3283064365386963e-10f), 0.999999940395355f);
        won = better(won, {y - logf(-logf(r)), i});
    }
    won = block_best(won, bests);
    if (tid == 0) {
        if (won.i < 0) won = top;  // min_p above 1 leaves nothing: the largest stays
        a.tokens[b] = won.i;
        if (a.logprobs) {
            const float y = tempered(clean(io<T>::ld(x + won.i)));
            a.logprobs[b] = y - logf((float)((double)total / (double)kUnit));
        }
    }
}

}  // namespace

size_t sample_workspace_bytes(int, int) { return 0; }

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream) {
    if (a.dtype == GDN_BF16) sample_kernel<__nv_bfloat16><<<a.B, kThreads, 0, stream>>>(a);
    else sample_kernel<float><<<a.B, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
