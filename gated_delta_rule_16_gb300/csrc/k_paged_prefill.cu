// k_paged_prefill.cu -- softmax attention of new tokens over the paged cache: the simple form.
//
// One CTA per (token, query head) goes over the row's keys 128 at a time with a running maximum and sum in fp32.
#include "paged.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;

template <typename T> __device__ __forceinline__ float value(const T *p) { return io<T>::ld(p); }
template <> __device__ __forceinline__ float value(const __nv_fp8_e4m3 *p) { return (float)*p; }

// Maximum (of numbers: NaN is left out) or sum over the CTA.
template <bool MAX> __device__ float reduce(float x, float *buf) {
    for (int off = 16; off; off >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, off);
        x = MAX ? fmaxf(x, y) : x + y;
    }
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    x = buf[0];
    for (int w = 1; w < kThreads / 32; ++w) x = MAX ? fmaxf(x, buf[w]) : x + buf[w];
    __syncthreads();
    return x;
}

template <typename C, typename T>
__global__ void __launch_bounds__(kThreads) prefill_simple(PrefillArgs a) {
    __shared__ float q[256], p[kThreads], buf[kThreads / 32];
    __shared__ int64_t at[kThreads];
    const int tid = threadIdx.x, t = blockIdx.x, h = blockIdx.y, d = a.c.d, kv = h / (a.Hq / a.c.Hkv);
    int lo = 0, hi = a.B;  // the last request that begins at or before t
    while (lo + 1 < hi) {
        const int mid = (lo + hi) / 2;
        if (a.cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    if (t < a.cu[lo] || t >= a.cu[lo + 1]) return;
    const int64_t pos = (int64_t)a.lens[lo] - a.cu[lo + 1] + t, room = (int64_t)a.max_pages * a.c.page;
    const int64_t first = a.window > 0 ? max((int64_t)0, pos - a.window + 1) : 0, last = min(pos + 1, room);
    const float ks = a.c.k_scale ? a.c.k_scale[kv] : 1.f, vs = a.c.v_scale ? a.c.v_scale[kv] : 1.f;
    for (int i = tid; i < d; i += kThreads) q[i] = value((const T *)a.q + t * a.q_tok + h * a.q_head + i);
    float m = -INFINITY, l = 0.f, o[2] = {0.f, 0.f};
    __syncthreads();
    for (int64_t j0 = first; j0 < last; j0 += kThreads) {
        const int64_t j = j0 + tid;
        const int page = j < last ? a.table[lo * a.table_stride + j / a.c.page] : -1;
        const bool real = page >= 0 && page < a.c.pages;
        at[tid] = real ? page * a.c.stride_page + j % a.c.page * a.c.stride_token + kv * a.c.stride_head : -1;
        float z = -INFINITY;
        if (real) {
            z = 0.f;
            for (int i = 0; i < d; ++i) z += q[i] * value((const C *)a.c.k + at[tid] + i);
            z *= ks * a.scale;
        }
        const float top = fmaxf(m, reduce<true>(z, buf)), ref = top == -INFINITY ? 0.f : top, f = expf(m - ref);
        p[tid] = expf(z - ref);
        l = l * f + reduce<false>(p[tid], buf);
        o[0] *= f, o[1] *= f;
        m = top;
        for (int k = 0; k < kThreads; ++k)
            if (at[k] >= 0)
                for (int e = 0; e < 2; ++e)
                    if (tid + e * kThreads < d) o[e] += p[k] * value((const C *)a.c.v + at[k] + tid + e * kThreads);
        __syncthreads();
    }
    const int64_t row = (int64_t)t * a.Hq + h;
    for (int e = 0; e < 2; ++e)
        if (tid + e * kThreads < d) io<T>::st((T *)a.o + row * d + tid + e * kThreads, l == 0.f ? 0.f : o[e] * vs / l);
    if (tid == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t paged_prefill_workspace_bytes(const gdn_kv_cache &, int, int, int) { return 256; }

cudaError_t launch_paged_prefill(const PrefillArgs &a, cudaStream_t stream) {
    const dim3 grid((unsigned)a.n, (unsigned)a.Hq);
    if (a.c.dtype == GDN_BF16) return launch_kernel(false, prefill_simple<__nv_bfloat16, __nv_bfloat16>, grid, kThreads, 0, stream, a);
    if (a.c.dtype == GDN_E4M3) return launch_kernel(false, prefill_simple<__nv_fp8_e4m3, __nv_bfloat16>, grid, kThreads, 0, stream, a);
    return launch_kernel(false, prefill_simple<float, float>, grid, kThreads, 0, stream, a);
}

}  // namespace gdn
