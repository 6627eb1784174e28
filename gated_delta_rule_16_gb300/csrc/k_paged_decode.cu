// k_paged_decode.cu -- one-token attention over the paged cache: the launch, and the join of
// rows that were cut between CTAs (paged_decode.cuh has the main kernel).
//
// A row cut into parts (m_i, l_i, o_i) is o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i, M = max m_i.  One
// CTA per (cut row, query head), in the order of the tokens, so the result does not depend on which part was done
// first.  Latency is all there is to it: the parts lie in L2, so a thread has its first four loads of outputs in
// flight beside those of maxima and sums.  With 8 CTAs or more to a row (few long rows, up to 608 parts each) there is an
// entry per row and 512 threads to every 64 dims; else one per CTA edge, of a few parts, and 128 threads.  After 1 x 131072
// tokens (4 rows of 114 parts) it adds 4 us to the call, after 64 requests up to 8192 (455 edges) 4 us, most of them the wait for
// the kernel before and three loads that depend on one another.  The choice looks at the number of rows only: where one of many is as
// long as all others together, 128 threads join its hundreds of parts (one request of 100000 tokens among 60 of 50, one KV head:
// 13 us of 31; with 4 KV heads and 18 others 6 of 43).
#include "paged_decode.cuh"

namespace gdn {
namespace paged {
namespace {

template <typename T, int D, int THREADS>
__global__ void __launch_bounds__(THREADS) join_kernel(AttendArgs a, int heads) {
    constexpr int kDims = THREADS == 512 ? 64 : D;  // of this CTA
    constexpr int kLanes = kDims / 4, kGroups = THREADS / kLanes, kFirst = 4;
    __shared__ float2 ml[kMaxCtas];
    __shared__ float2 red[THREADS / 32];
    __shared__ float4 acc[THREADS];
    const WsView ws = ws_view(a.ws, heads);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    const int4 at = ws.joins[blockIdx.x];
    const int parts = at.w;
    if (parts == 0) return;
    const int group = a.Hq / a.c.Hkv, passes = (group + heads - 1) / heads;
    const int h = at.y / passes, hh = at.y % passes * heads + blockIdx.y;
    if (hh >= group) return;
    // the row's last in its first CTA (or that CTA's only one), then the first of each CTA up to the row's end
    auto part = [&](int k) { return (int64_t)(k == 0 ? at.z : 2 * ((at.z >> 1) + k)) * heads + blockIdx.y; };
    const int own = tid / kLanes, d4 = blockIdx.z * kDims + tid % kLanes * 4;
    float4 y[kFirst];
#pragma unroll
    for (int e = 0; e < kFirst; ++e)
        if (own + e * kGroups < parts) y[e] = *(const float4 *)(ws.o + part(own + e * kGroups) * D + d4);
    float top = -INFINITY;
    for (int k = tid; k < parts; k += THREADS) {
        ml[k] = ws.ml[part(k)];
        top = fmaxf(top, ml[k].x);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (lane == 0) red[warp].x = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) top = fmaxf(top, red[w].x);
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int k = tid; k < parts; k += THREADS) sum += exp2_fast(ml[k].x - ref) * ml[k].y;
#pragma unroll
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) red[warp].y = sum;

    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int k, const float4 &z) {
        const float f = exp2_fast(ml[k].x - ref);
        x.x += f * z.x, x.y += f * z.y, x.z += f * z.z, x.w += f * z.w;
    };
#pragma unroll
    for (int e = 0; e < kFirst; ++e)
        if (own + e * kGroups < parts) add(own + e * kGroups, y[e]);
#pragma unroll 4
    for (int k = own + kFirst * kGroups; k < parts; k += kGroups) add(k, *(const float4 *)(ws.o + part(k) * D + d4));
    acc[tid] = x;
    __syncthreads();
    if (tid >= kLanes) return;
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) sum += red[w].y;
#pragma unroll
    for (int gr = 1; gr < kGroups; ++gr) {
        const float4 z = acc[gr * kLanes + tid];
        x.x += z.x, x.y += z.y, x.z += z.z, x.w += z.w;
    }
    float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (a.c.v_scale) inv *= a.c.v_scale[h];
    const int64_t out = (int64_t)at.x * a.Hq + h * group + hh;
    if constexpr (sizeof(T) == 4)
        *(float4 *)((float *)a.o + out * D + d4) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    else
        *(uint2 *)((__nv_bfloat16 *)a.o + out * D + d4) = make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
    if (d4 == 0 && a.lse) a.lse[out] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
}

template <typename T, int D>
cudaError_t join(const AttendArgs &a, int grid, int heads, cudaStream_t stream) {
    const int group = a.Hq / a.c.Hkv;
    const int64_t rows = (int64_t)a.B * a.c.Hkv * ((group + heads - 1) / heads);
    if (join_by_row(rows, grid))
        return launch_kernel(true, join_kernel<T, D, 512>, dim3((unsigned)rows, min(heads, group), D / 64), 512, 0, stream, a, heads);
    return launch_kernel(true, join_kernel<T, D, 128>, dim3(grid - 1, min(heads, group)), 128, 0, stream, a, heads);
}
template <typename T>
cudaError_t join(const AttendArgs &a, int grid, int heads, cudaStream_t stream) {
    switch (a.c.d) {
        case 64: return join<T, 64>(a, grid, heads, stream);
        case 128: return join<T, 128>(a, grid, heads, stream);
        default: return join<T, 256>(a, grid, heads, stream);
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
