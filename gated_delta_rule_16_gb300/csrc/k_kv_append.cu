// k_kv_append.cu -- writes new tokens' keys and values into the paged cache.
//
// A pure copy (every value read once, written once; an 8-bit cache divides by the
// head's scale on the way), bound by memory.  A thread keeps one 16-byte piece of a
// cached row, (head, piece), through the tokens it takes, so its addresses, its scale
// and the scale's reciprocal are made once.  Copies have four tokens' loads in flight; a conversion has registers for one
// (two measured 38 us against 35, four 51, at the prompt below).  That prompt takes 31.3 us, 6.05 TB/s or 89 % of a copy; 64 tokens of
// a decode step 2.0 us, a launch.
#include "paged.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// 8-bit storage: x / scale in fp32 (one rounding), then to nearest even in e4m3, saturated: a cached value is off by
// half an e4m3 step of its own size at most.  The quotient is corrected once from the rounded reciprocal (Markstein, IBM
// J. Res. Dev. 34, 1990: with r = RN(1/s), q = RN(x r), RN(q + r RN(x - q s)) is RN(x/s) while nothing over- or underflows;
// an underflow here rounds to 0 all the same), three operations in place of a division's ten.  Where the reciprocal
// or a quotient of the piece leaves the range (infinities among them) the piece is divided.  With a division each a prompt
// of 32805 tokens, 8 heads of 128, took 39 us.
struct Scale {
    float s, r, most;  // |x| < most: corrected quotients
    __device__ explicit Scale(float x) : s(x), r(1.f / x), most(fabsf(x) > 1e-30f && fabsf(x) < 1e30f ? 1e6f * fabsf(x) : 0.f) {}
    __device__ __forceinline__ float quotient(float x) const {
        const float q = x * r;
        return __fmaf_rn(__fmaf_rn(-q, s, x), r, q);
    }
};
__device__ __forceinline__ uint32_t e4m3x4(float x0, float x1, float x2, float x3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x2, x3), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}
// 16 cached 8-bit values from 16 values of type T.
template <typename T>
__device__ __forceinline__ uint4 quantised(const uint4 *src, const Scale &s) {
    float x[16], top = 0.f;
    const uint32_t *w = &src[0].x;
    if constexpr (sizeof(T) == 2) {
        __nv_bfloat162 m = __habs2(*(const __nv_bfloat162 *)w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m = __hmax2(m, __habs2(*(const __nv_bfloat162 *)(w + i)));
            x[2 * i] = __uint_as_float(w[i] << 16);  // a bf16 is the upper half of its fp32
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
        top = fmaxf(__low2float(m), __high2float(m));
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = __uint_as_float(w[i]);
            top = fmaxf(top, fabsf(x[i]));
        }
    }
    if (top < s.most) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = s.quotient(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = x[i] / s.s;
    }
    return make_uint4(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]), e4m3x4(x[8], x[9], x[10], x[11]),
                      e4m3x4(x[12], x[13], x[14], x[15]));
}

template <typename T, bool QUANT>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendArgs a, int per_token, int tokens) {
    constexpr int kElem = QUANT ? 1 : sizeof(T), kPer = 16 / kElem;  // cached values per piece
    constexpr int kLoads = QUANT ? sizeof(T) : 1, kAhead = QUANT ? 1 : 4;  // 16-byte loads per piece; tokens in flight
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
                x = quantised<T>(kx[u], ks);
                y = quantised<T>(vx[u], vs);
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
    // one wave of CTAs that take tokens in turn, eight per SM for copies, four for conversions (31.4 us against 32.3 with
    // eight, 38.5 without turns); small calls one token per thread
    const int64_t want = ((int64_t)a.n + tokens - 1) / tokens;
    const dim3 grid((unsigned)min(want, (int64_t)152 * (a.c.dtype == GDN_E4M3 ? 4 : 8)), (pieces + kThreads - 1) / kThreads);
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
