// k_kv_append.cu -- writes new tokens' keys and values into the paged cache.
//
// A pure copy (every value read once, written once; an 8-bit cache divides by the
// head's scale on the way), bound by memory.  One thread moves one 16-byte piece of
// a cached row: the rows of a token are spread by the caches' strides, the pieces
// of a row are contiguous on both sides.
#include "paged.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// 8-bit storage: x / scale in fp32 (one rounding), then to nearest even in e4m3,
// saturated: a cached value is off by half an e4m3 step of its own size at most.
__device__ __forceinline__ uint32_t e4m3x4(float x0, float x1, float x2, float x3, float scale) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x0 / scale, x1 / scale), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x2 / scale, x3 / scale), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

template <typename T> struct Piece;  // 16 cached 8-bit values from 16 values of type T
template <> struct Piece<__nv_bfloat16> {
    static __device__ __forceinline__ uint4 pack(const uint4 *src, float scale) {
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
    static __device__ __forceinline__ uint4 pack(const uint4 *src, float scale) {
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
__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendArgs a) {
    constexpr int kElem = QUANT ? 1 : sizeof(T);
    constexpr int kPer = 16 / kElem;  // cached values per piece
    const int pieces = a.c.d / kPer;  // per row
    const int64_t total = (int64_t)a.n * a.c.Hkv * pieces;
    const int64_t cells = a.c.pages * a.c.page;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int e = (int)(i % pieces) * kPer;
        const int64_t row = i / pieces;
        const int h = (int)(row % a.c.Hkv);
        const int64_t t = row / a.c.Hkv, slot = a.slots[t];
        if (slot < 0 || slot >= cells) continue;
        const int64_t dst = (slot / a.c.page) * a.c.stride_page + (slot % a.c.page) * a.c.stride_token +
                            h * a.c.stride_head + e;
        const uint4 *ks = (const uint4 *)((const T *)a.k + t * a.k_tok + h * a.k_head + e);
        const uint4 *vs = (const uint4 *)((const T *)a.v + t * a.v_tok + h * a.v_head + e);
        uint4 kx, vx;
        if constexpr (QUANT) {
            kx = Piece<T>::pack(ks, a.c.k_scale[h]);
            vx = Piece<T>::pack(vs, a.c.v_scale[h]);
        } else {
            kx = *ks;
            vx = *vs;
        }
        *(uint4 *)((char *)a.c.k + dst * kElem) = kx;
        *(uint4 *)((char *)a.c.v + dst * kElem) = vx;
    }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs &a, cudaStream_t stream) {
    const int per = a.c.dtype == GDN_E4M3 ? 16 : (a.c.dtype == GDN_BF16 ? 8 : 4);
    const int64_t blocks = ((int64_t)a.n * a.c.Hkv * (a.c.d / per) + kThreads - 1) / kThreads;
    const unsigned grid = (unsigned)(blocks < (1 << 20) ? blocks : 1 << 20);
    if (a.c.dtype == GDN_E4M3) {
        if (a.dtype == GDN_BF16) kv_append_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, stream>>>(a);
        else kv_append_kernel<float, true><<<grid, kThreads, 0, stream>>>(a);
    } else if (a.c.dtype == GDN_BF16) {
        kv_append_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, stream>>>(a);
    } else {
        kv_append_kernel<float, false><<<grid, kThreads, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace gdn
