// k_paged_decode.cu -- softmax attention of one new token per request over the paged cache.
//
// First form: one CTA per (request, query head), one warp per token in turn, with
// a running maximum and sum per warp, joined in shared memory.
#include "paged.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;

template <typename T> __device__ __forceinline__ float ld(const T *p) { return io<T>::ld(p); }
template <> __device__ __forceinline__ float ld(const __nv_fp8_e4m3 *p) { return (float)*p; }

template <typename Q, typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) decode_kernel(AttendArgs a) {
    constexpr int N = D / 32;
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
    const int b = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, hk = h / (a.Hq / a.c.Hkv);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t len = min((int64_t)max(a.lens[b], 0), (int64_t)a.max_pages * a.c.page);
    const int64_t start = a.window > 0 ? max((int64_t)0, len - a.window) : 0;
    const float ks = a.c.k_scale ? a.c.k_scale[hk] : 1.f, vs = a.c.v_scale ? a.c.v_scale[hk] : 1.f;
    float q[N], o[N], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        q[i] = io<Q>::ld((const Q *)a.q + b * a.q_req + h * a.q_head + lane + 32 * i) * (a.scale * ks);
        o[i] = 0.f;
    }
    for (int64_t j = start + warp; j < len; j += kWarps) {
        const int64_t page = a.table[b * a.table_stride + j / a.c.page];
        if (page < 0 || page >= a.c.pages) continue;
        const int64_t at = page * a.c.stride_page + (j % a.c.page) * a.c.stride_token + hk * a.c.stride_head + lane;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) s += q[i] * ld((const T *)a.c.k + at + 32 * i);
#pragma unroll
        for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
        const float f = expf(m - ref), p = expf(s - ref);
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = o[i] * f + p * ld((const T *)a.c.v + at + 32 * i);
        m = mn;
    }
    if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
    for (int i = 0; i < N; ++i) so[warp][lane + 32 * i] = o[i];
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
    const float ref = M == -INFINITY ? 0.f : M;
    for (int w = 0; w < kWarps; ++w) L += sl[w] * expf(sm[w] - ref);
    for (int i = threadIdx.x; i < D; i += 32 * kWarps) {
        float x = 0.f;
        for (int w = 0; w < kWarps; ++w) x += so[w][i] * expf(sm[w] - ref);
        io<Q>::st((Q *)a.o + ((int64_t)b * a.Hq + h) * D + i, L == 0.f ? 0.f : x * vs / L);
    }
    if (threadIdx.x == 0 && a.lse) a.lse[(int64_t)b * a.Hq + h] = L == 0.f ? -INFINITY : ref + logf(L);
}

template <typename Q, typename T>
void launch(const AttendArgs &a, cudaStream_t stream) {
    const unsigned grid = (unsigned)(a.B * a.Hq);
    if (a.c.d == 64) decode_kernel<Q, T, 64><<<grid, 32 * kWarps, 0, stream>>>(a);
    else if (a.c.d == 128) decode_kernel<Q, T, 128><<<grid, 32 * kWarps, 0, stream>>>(a);
    else decode_kernel<Q, T, 256><<<grid, 32 * kWarps, 0, stream>>>(a);
}

}  // namespace

size_t paged_decode_workspace_bytes(const gdn_kv_cache &, int) { return 0; }

cudaError_t launch_paged_decode(const AttendArgs &a, cudaStream_t stream) {
    if (a.c.dtype == GDN_BF16) launch<__nv_bfloat16, __nv_bfloat16>(a, stream);
    else if (a.c.dtype == GDN_E4M3) launch<__nv_bfloat16, __nv_fp8_e4m3>(a, stream);
    else launch<float, float>(a, stream);
    return cudaGetLastError();
}

}  // namespace gdn
