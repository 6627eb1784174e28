// k_qk_rope.cu -- per-head norm and rotary positions of new tokens' queries and keys, in one pass.
//
// y = x w / sqrt(mean(x^2) + eps); a pair (a, b) of y turns by the angle positions[t] * freqs[i].  A pair's factors do not
// depend on the head, so a group of lanes that holds one row in registers (16 bytes each) keeps its token's cosines and sines,
// with the weights and mscale multiplied in, through all of the token's heads: per element two products and one scale remain,
// out = r (x (w c) + x' (w' s)), r = 1 / sqrt(..), x' the pair's other element.  It comes from a lane of the same group by a
// shuffle; where `pairs` is no multiple of a lane's elements it comes from shared memory.
//
// The angle in turns is position * (freqs / 2 pi) modulo 1, and the position is a whole number: the fraction of freqs / 2 pi as a
// 64-bit whole number F makes it the low 64 bits of position * F, exact however far the position.  The conversion takes a few
// 64-bit floating operations, of which an SM does two per clock: one thread per pair and CTA makes F, not one per token.
//
// What bounds it: HBM, each value read and written once, as long as enough loads are on their way: four rows to a lane and 32 warps to an SM.
// 16411 tokens of 40 heads of 128 bf16 (336 MB) 65.5 us, 5.1 TB/s or 76 % of a copy, 10 points of which are the second, two-thirds full wave
// of CTAs; with 24 warps 74 us, two rows to a lane 73, heads dealt out to two CTAs 72 to 78 (each makes the cosines again), rows copied
// ahead to shared memory by cp.async 73, factors in shared memory for CTAs that go along a token's heads 112.  64 tokens 5 us: the launch,
// and two dependent loads.
#include "paged.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256, kUnroll = 4;

template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&p);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

// The fraction of freqs / 2 pi in units of 2^-64 of a turn.
__device__ __forceinline__ uint64_t turns(double f) {
    const double t = f * 0.15915494309189533577;  // 1 / 2 pi
    return __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
}
// (cos, sin) of a fraction of a turn: to the nearest quarter, whose rest keeps 24 bits
__device__ __forceinline__ void cos_sin(uint64_t turn, float &c, float &s) {
    const uint32_t hi = (uint32_t)(turn >> 32), quarter = (hi + 0x20000000u) >> 30;
    const float r = (float)(int32_t)(hi - (quarter << 30)) * 4.656612873077393e-10f;  // 2^-31: sincospi takes half turns
    float y, x;
    sincospif(r, &y, &x);
    c = quarter & 1 ? y : x;
    s = quarter & 1 ? x : y;
    if (quarter == 1 || quarter == 2) c = -c;
    if (quarter >= 2) s = -s;
}

// Lanes to a row: 16 bytes each, twice for rows of more than 512 bytes.  PAIRS: 0 interleaved, 1 half layout with the pair's
// other element at the same place of another 16 bytes, 2 half layout with any number of pairs.
template <typename T, int D, int PAIRS>
__global__ void __launch_bounds__(kThreads, sizeof(T) * D > 512 ? 3 : 4) qk_rope_kernel(RopeArgs a) {
    constexpr int N = Vec<T>::N, kChunks = D / N, kLanes = kChunks < 32 ? kChunks : 32, C = kChunks / kLanes, kSlots = kThreads / kLanes;
    __shared__ uint64_t freq[D / 2];
    __shared__ float rows[PAIRS == 2 ? kThreads * N * C : 1];
    const int tid = threadIdx.x, lane = tid % kLanes, slot = tid / kLanes;
    for (int i = tid; i < a.pairs; i += kThreads) freq[i] = turns(a.freqs[i]);
    __syncthreads();
    const int t = blockIdx.x * kSlots + slot;
    const bool real = (unsigned)t < (unsigned)a.n;  // the last CTA's groups may pass 2^31
    const int64_t pos = real ? a.positions[t] : 0;

    float cs[C][N], sn[C][N];
    int turned[C], other[C];  // elements of a chunk that turn; the chunk with their other halves
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e0 = (lane + c * kLanes) * N;
        turned[c] = max(0, min(N, 2 * a.pairs - e0));
        other[c] = lane + c * kLanes;
        if (PAIRS == 1 && turned[c]) other[c] += e0 < a.pairs ? a.pairs / N : -(a.pairs / N);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (PAIRS == 0 && (j & 1)) {
                cs[c][j] = cs[c][j - 1];
                sn[c][j] = -sn[c][j - 1];
                continue;
            }
            const int e = e0 + j, i = PAIRS == 0 ? e >> 1 : (e < a.pairs ? e : e - a.pairs);
            cs[c][j] = 1.f;
            sn[c][j] = 0.f;
            if (j < turned[c]) {
                cos_sin((uint64_t)pos * freq[i], cs[c][j], sn[c][j]);
                cs[c][j] *= a.mscale;
                sn[c][j] *= PAIRS == 0 || e < a.pairs ? -a.mscale : a.mscale;
            }
        }
    }

    // heads [h0, h1) of one of the two tensors
    auto heads = [&](const T *x, int64_t x_tok, int64_t x_head, T *y, int64_t y_tok, int64_t y_head, const float *w, int h0, int h1) {
        if (h0 >= h1) return;
        float wc[C][N], ws[C][N];  // factors of an element and of its pair's other element
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int e = (lane + c * kLanes) * N + j;
                const int p = j >= turned[c] ? e : (PAIRS == 0 ? e ^ 1 : (e < a.pairs ? e + a.pairs : e - a.pairs));
                wc[c][j] = w ? cs[c][j] * w[e] : cs[c][j];
                ws[c][j] = w ? sn[c][j] * w[p] : sn[c][j];
            }
        x += (real ? t : 0) * x_tok + lane * N;
        y += (real ? t : 0) * y_tok + lane * N;
#pragma unroll 1
        for (int h = h0; h < h1; h += kUnroll) {
            uint4 in[kUnroll][C];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
#pragma unroll
                for (int c = 0; c < C; ++c)
                    in[u][c] = real && h + u < h1 ? *reinterpret_cast<const uint4 *>(x + (h + u) * x_head + c * kLanes * N) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                float v[C][N], r = 1.f;
#pragma unroll
                for (int c = 0; c < C; ++c) Vec<T>::unpack(in[u][c], v[c]);
                if (w) {
                    float sum = 0.f;
#pragma unroll
                    for (int c = 0; c < C; ++c)
#pragma unroll
                        for (int j = 0; j < N; ++j) sum += v[c][j] * v[c][j];
#pragma unroll
                    for (int off = kLanes / 2; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                    r = rsqrtf(sum * (1.f / D) + a.eps);
                }
                float z[C][N];  // the pairs' other elements
                if constexpr (PAIRS == 0) {
#pragma unroll
                    for (int c = 0; c < C; ++c)
#pragma unroll
                        for (int j = 0; j < N; ++j) z[c][j] = v[c][j ^ 1];
                } else if constexpr (PAIRS == 1) {
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        uint4 got;
                        const int from = other[c] % kLanes;
                        const uint4 &s = in[u][0];
                        got.x = __shfl_sync(0xffffffffu, s.x, from, kLanes);
                        got.y = __shfl_sync(0xffffffffu, s.y, from, kLanes);
                        got.z = __shfl_sync(0xffffffffu, s.z, from, kLanes);
                        got.w = __shfl_sync(0xffffffffu, s.w, from, kLanes);
                        if constexpr (C == 2) {
                            const uint4 &s1 = in[u][1];
                            uint4 g1;
                            g1.x = __shfl_sync(0xffffffffu, s1.x, from, kLanes);
                            g1.y = __shfl_sync(0xffffffffu, s1.y, from, kLanes);
                            g1.z = __shfl_sync(0xffffffffu, s1.z, from, kLanes);
                            g1.w = __shfl_sync(0xffffffffu, s1.w, from, kLanes);
                            if (other[c] >= kLanes) got = g1;
                        }
                        Vec<T>::unpack(got, z[c]);
                    }
                } else {
                    float *row = rows + slot * D;
#pragma unroll
                    for (int c = 0; c < C; ++c)
#pragma unroll
                        for (int j = 0; j < N; ++j) row[(lane + c * kLanes) * N + j] = v[c][j];
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < C; ++c)
#pragma unroll
                        for (int j = 0; j < N; ++j) {
                            const int e = (lane + c * kLanes) * N + j;
                            z[c][j] = row[j >= turned[c] ? e : (e < a.pairs ? e + a.pairs : e - a.pairs)];
                        }
                    __syncwarp();
                }
#pragma unroll
                for (int c = 0; c < C; ++c) {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const float whole = v[c][j] * wc[c][j];
                        v[c][j] = r * (j < turned[c] ? whole + z[c][j] * ws[c][j] : whole);
                    }
                    if (real && h + u < h1) *reinterpret_cast<uint4 *>(y + (h + u) * y_head + c * kLanes * N) = Vec<T>::pack(v[c]);
                }
            }
        }
    };
    const int h0 = blockIdx.y * a.heads_per_cta, h1 = min(h0 + a.heads_per_cta, a.Hq + a.Hkv);
    heads((const T *)a.q, a.q_tok, a.q_head, (T *)a.q_out, a.qo_tok, a.qo_head, a.q_weight, h0, min(h1, a.Hq));
    heads((const T *)a.k, a.k_tok, a.k_head, (T *)a.k_out, a.ko_tok, a.ko_head, a.k_weight, max(h0, a.Hq) - a.Hq, h1 - a.Hq);
}

template <typename T, int D>
cudaError_t launch(RopeArgs a, cudaStream_t stream) {
    constexpr int kChunks = D / Vec<T>::N, kLanes = kChunks < 32 ? kChunks : 32, kSlots = kThreads / kLanes;
    const unsigned groups = (unsigned)((a.n + (int64_t)kSlots - 1) / kSlots);
    // Every CTA makes its own cosines, which pays off over a token's heads; few tokens have their heads dealt out instead, down to
    // one round of loads, until there are some CTAs for every SM.
    const int heads = a.Hq + a.Hkv, rounds = (heads + kUnroll - 1) / kUnroll;
    const int split = (int)max((int64_t)1, min((int64_t)rounds, (int64_t)4 * 152 / (int64_t)groups));
    a.heads_per_cta = (rounds + split - 1) / split * kUnroll;
    const dim3 grid(groups, (heads + a.heads_per_cta - 1) / a.heads_per_cta);
    auto fn = a.interleaved ? qk_rope_kernel<T, D, 0> : a.pairs % Vec<T>::N == 0 ? qk_rope_kernel<T, D, 1> : qk_rope_kernel<T, D, 2>;
    return launch_kernel(false, fn, grid, kThreads, 0, stream, a);
}
template <typename T>
cudaError_t launch(const RopeArgs &a, cudaStream_t stream) {
    return a.d == 64 ? launch<T, 64>(a, stream) : a.d == 128 ? launch<T, 128>(a, stream) : launch<T, 256>(a, stream);
}

}  // namespace

cudaError_t launch_qk_rope(const RopeArgs &a, cudaStream_t stream) {
    return a.dtype == GDN_BF16 ? launch<__nv_bfloat16>(a, stream) : launch<float>(a, stream);
}

}  // namespace gdn
