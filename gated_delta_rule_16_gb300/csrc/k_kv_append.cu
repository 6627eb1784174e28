// k_kv_append.cu -- writes new tokens' keys and values into the paged cache.
//
// A pure copy (every value read once, written once; an 8-bit cache divides by the
// head's scale on the way), bound by memory.  A thread keeps one 16-byte piece of a
// cached row, (head, piece), through the tokens it takes, so its addresses, its scale
// and the scale's reciprocal are made once; four tokens' loads are in flight together.
#include "paged.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// 8-bit storage: x / scale in fp32 (one rounding), then to nearest even in e4m3, saturated: a cached value is off by
// half an e4m3 step of its own size at most.  The quotient is corrected once from the rounded reciprocal (Markstein, IBM
// J. Res. Dev. 34, 1990: with r = RN(1/s), q = RN(x r), RN(q + r RN(x - q s)) is RN(x/s) while nothing over- or underflows),
// three operations in place of a division's ten.  A scale whose reciprocal leaves the normal range is divided by.
struct Scale {
    float s, r;  // r = 0: divide
    __device__ explicit Scale(float x) : s(x), r(fabsf(x) > 1e-30f && fabsf(x) < 1e30f ? 1.f / x : 0.f) {}
    __device__ __forceinline__ float under(float x) const {
        if (r == 0.f) return x / s;
        const float q = x * r, rest = __fmaf_rn(-q, s, x);
        return fabsf(q) < 1e30f ? __fmaf_rn(rest, r, q) : q;  // past it (infinities): saturated all the same
    }
};
__device__ __forceinline__ uint32_t e4m3x4(float x0, float x1, float x2, float x3, const Scale &s) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(s.under(x0), s.under(x1)), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(s.under(x2), s.under(x3)), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

template <typename T> struct Piece;  // 16 cached 8-bit values from 16 values of type T
template <> struct Piece<__nv_bfloat16> {
    static __device__ __forceinline__ uint4 pack(const uint4 *src, const Scale &scale) {
        uint4 out;
        uint32_t *w = &out.x;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 x = src[i];
            // a bf16 is the upper half of its fp32
            w[2 * i] = e4m3x4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u),
                              __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u), scale);
            w[2 * i + 1] = e4m3x4(__uint_as_float(x.z << 16), __uint_as_float(x.z & 0xffff0000u),
                                  __uint_as_float(x.w << 16), __uint_as_float(x.w & 0xffff0000u), scale);
        }
        return out;
    }
};
template <> struct Piece<float> {
    static __device__ __forceinline__ uint4 pack(const uint4 *src, const Scale &scale) {
        uint4 out;
        uint32_t *w = &out.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 x = src[i];
            w[i] = e4m3x4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w), scale);
        }
        return out;
    }
};

template <typename T, bool QUANT>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendArgs a, int per_token, int tokens) {
    constexpr int kElem = QUANT ? 1 : sizeof(T), kPer = 16 / kElem;  // cached values per piece
    constexpr int kLoads = QUANT ? sizeof(T) : 1, kAhead = QUANT ? 2 : 4;  // 16-byte loads per piece; tokens in flight
    // `tokens` tokens of `per_token` pieces side by side in a CTA, a token's pieces over several CTAs in y if they are more
    const int lane = threadIdx.x / per_token, piece = blockIdx.y * kThreads + threadIdx.x % per_token;
    const int pieces = a.c.d / kPer, h = piece / pieces, e = piece % pieces * kPer;
    if (lane >= tokens || h >= a.c.Hkv) return;
    const T *k = (const T *)a.k + h * a.k_head + e, *v = (const T *)a.v + h * a.v_head + e;
    char *kc = (char *)a.c.k + (h * a.c.stride_head + e) * kElem, *vc = (char *)a.c.v + (h * a.c.stride_head + e) * kElem;
    const Scale ks(QUANT ? a.c.k_scale[h] : 1.f), vs(QUANT ? a.c.v_scale[h] : 1.f);
    const int64_t cells = a.c.pages * a.c.page;
    const bool pow2 = (a.c.page & (a.c.page - 1)) == 0;
    const int shift = 31 - __clz(a.c.page);
    const int stride = gridDim.x * tokens;
    for (int64_t t0 = blockIdx.x * tokens + lane; t0 < a.n; t0 += (int64_t)kAhead * stride) {
        int64_t slot[kAhead];
        uint4 kx[kAhead][kLoads], vx[kAhead][kLoads];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t t = t0 + (int64_t)u * stride;
            slot[u] = t < a.n ? a.slots[t] : -1;
            if (slot[u] >= cells) slot[u] = -1;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t t = t0 + (int64_t)u * stride;
            if (slot[u] < 0) continue;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                kx[u][i] = ((const uint4 *)(k + t * a.k_tok))[i];
                vx[u][i] = ((const uint4 *)(v + t * a.v_tok))[i];
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (slot[u] < 0) continue;
            const int64_t page = pow2 ? slot[u] >> shift
                                 : slot[u] <= (int64_t)UINT32_MAX ? (int64_t)((uint32_t)slot[u] / (uint32_t)a.c.page) : slot[u] / a.c.page;
            const int64_t at = (page * a.c.stride_page + (slot[u] - page * a.c.page) * a.c.stride_token) * kElem;
            uint4 x, y;
            if constexpr (QUANT) {
                x = Piece<T>::pack(kx[u], ks);
                y = Piece<T>::pack(vx[u], vs);
            } else {
                x = kx[u][0];
                y = vx[u][0];
            }
            *(uint4 *)(kc + at) = x;
            *(uint4 *)(vc + at) = y;
        }
    }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs &a, cudaStream_t stream) {
    const int per = a.c.dtype == GDN_E4M3 ? 16 : (a.c.dtype == GDN_BF16 ? 8 : 4);
    const int pieces = a.c.Hkv * (a.c.d / per), per_token = min(pieces, kThreads), tokens = kThreads / per_token;
    // up to eight CTAs per SM, each taking tokens in turn; small calls one token per thread
    const int64_t want = ((int64_t)a.n + tokens - 1) / tokens;
    const dim3 grid((unsigned)min(want, (int64_t)152 * 8), (pieces + kThreads - 1) / kThreads);
    auto go = [&](auto kern) { kern<<<grid, kThreads, 0, stream>>>(a, per_token, tokens); };
    if (a.c.dtype == GDN_E4M3) {
        if (a.dtype == GDN_BF16) go(kv_append_kernel<__nv_bfloat16, true>);
        else go(kv_append_kernel<float, true>);
    } else if (a.c.dtype == GDN_BF16) {
        go(kv_append_kernel<__nv_bfloat16, false>);
    } else {
        go(kv_append_kernel<float, false>);
    }
    return cudaGetLastError();
}

}  // namespace gdn
