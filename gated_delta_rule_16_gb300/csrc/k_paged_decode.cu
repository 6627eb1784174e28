// k_paged_decode.cu -- one-token attention over the paged cache: the launch, and the join of
// rows that were cut between CTAs (paged_decode.cuh has the main kernel).
//
// A row cut into parts (m_i, l_i, o_i) is o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i, M = max m_i.  One
// CTA per (CTA edge, query head): the first edge inside a row joins all of the row's parts, in the order of
// the tokens, so the result does not depend on which part was done first.  At most 2 x 304 parts of up to 16
// heads, read back from L2: latency, hidden in part by a programmatic dependent launch.
#include "paged_decode.cuh"

namespace gdn {
namespace paged {
namespace {

constexpr int kThreads = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) join_kernel(AttendArgs a, int heads) {
    __shared__ float weight[kMaxCtas];
    __shared__ float2 red[kThreads / 32];
    __shared__ float4 acc[kThreads];
    const WsView ws = ws_view(a.ws, heads);
    const int i = blockIdx.x + 1;
    pdl_wait();
    const int4 at = ws.joins[i];
    const int parts = at.w;
    if (parts == 0) return;
    const int group = a.Hq / a.c.Hkv, passes = (group + heads - 1) / heads;
    const int h = at.y / passes, hh = at.y % passes * heads + blockIdx.y;
    if (hh >= group) return;
    // the row's last in CTA i - 1 (or its only one), then the first of each CTA up to the row's end
    auto part = [&](int k) { return k == 0 ? at.z : 2 * (i + k - 1); };

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float top = -INFINITY;
    for (int k = tid; k < parts; k += kThreads) top = fmaxf(top, ws.ml[(int64_t)part(k) * heads + blockIdx.y].x);
    for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (lane == 0) red[warp].x = top;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, red[w].x);
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int k = tid; k < parts; k += kThreads) {
        const float2 x = ws.ml[(int64_t)part(k) * heads + blockIdx.y];
        const float f = exp2_fast(x.x - ref);
        weight[k] = f;
        sum += f * x.y;
    }
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) red[warp].y = sum;
    __syncthreads();
    sum = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) sum += red[w].y;

    constexpr int kLanes = D / 4, kGroups = kThreads / kLanes;
    const int d4 = tid % kLanes * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = tid / kLanes; k < parts; k += kGroups) {
        const float4 y = *(const float4 *)(ws.o + ((int64_t)part(k) * heads + blockIdx.y) * D + d4);
        const float f = weight[k];
        x.x += f * y.x, x.y += f * y.y, x.z += f * y.z, x.w += f * y.w;
    }
    acc[tid] = x;
    __syncthreads();
    if (tid >= kLanes) return;
    for (int gr = 1; gr < kGroups; ++gr) {
        const float4 y = acc[gr * kLanes + tid];
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
    }
    float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (a.c.v_scale) inv *= a.c.v_scale[h];
    const int64_t out = (int64_t)at.x * a.Hq + h * group + hh;
    io<T>::st((T *)a.o + out * D + d4, x.x * inv);
    io<T>::st((T *)a.o + out * D + d4 + 1, x.y * inv);
    io<T>::st((T *)a.o + out * D + d4 + 2, x.z * inv);
    io<T>::st((T *)a.o + out * D + d4 + 3, x.w * inv);
    if (tid == 0 && a.lse) a.lse[out] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
}

template <typename T>
cudaError_t join(const AttendArgs &a, int grid, int heads, cudaStream_t stream) {
    const dim3 g(grid - 1, min(heads, a.Hq / a.c.Hkv));
    switch (a.c.d) {
        case 64: return launch_kernel(true, join_kernel<T, 64>, g, kThreads, 0, stream, a, heads);
        case 128: return launch_kernel(true, join_kernel<T, 128>, g, kThreads, 0, stream, a, heads);
        default: return launch_kernel(true, join_kernel<T, 256>, g, kThreads, 0, stream, a, heads);
    }
}

}  // namespace
}  // namespace paged

size_t paged_decode_workspace_bytes(const gdn_kv_cache &c, int Hq) {
    return paged::ws_bytes(paged::pass_heads(Hq / c.Hkv), c.d);
}

cudaError_t launch_paged_decode(const AttendArgs &args, cudaStream_t stream) {
    AttendArgs a = args;
    if (a.max_pages == 0) a.c.k = a.c.v = (void *)a.q;  // an address for copies of no bytes
    // slices of 16 tokens of a row as long as the table or the window (whose first slice it need not fill)
    int64_t tokens = (int64_t)a.max_pages * a.c.page;
    if (a.window > 0) tokens = min(tokens, (int64_t)a.window + 15);
    const int64_t slices = max((int64_t)1, (tokens + 15) / 16);
    int grid = 0;
    cudaError_t e;
    if (a.c.dtype == GDN_BF16) e = paged::launch_kind<GDN_BF16>(a, slices, stream, &grid);
    else if (a.c.dtype == GDN_E4M3) e = paged::launch_kind<GDN_E4M3>(a, slices, stream, &grid);
    else e = paged::launch_kind<GDN_F32>(a, slices, stream, &grid);
    if (e != cudaSuccess || grid < 2 || slices <= paged::tile_of(a.c) / 16) return e;  // a row of one tile cannot be cut
    const int heads = paged::pass_heads(a.Hq / a.c.Hkv);
    return a.c.dtype == GDN_F32 ? paged::join<float>(a, grid, heads, stream) : paged::join<__nv_bfloat16>(a, grid, heads, stream);
}

}  // namespace gdn
