// k_paged_prefill_f32.cu -- softmax attention of new tokens over the paged cache in 32-bit storage.
//
// Every operand is split into two tf32 terms of 11 bits, x = hi + lo to 2^-22 of x, and a product of two takes three warp MMAs
// (lo hi, hi lo, hi hi); the tensor core's sums run over 32 terms of each only, longer ones are fp32 additions, which round where the
// tensor core cuts.  An m16n8k8 takes 8 clocks of an SM quarter's tensor core (measured, 300 TFLOP/s in all), so three make 100 TFLOP/s at most; 41 % of
// that is reached (3 requests up to 2031 tokens, d 64: 188 us), the rest waits for operands and between the tile's two barriers.  One after the other for all sums instead of three to a sum: 197 us.
// Keys and values are split once, when they come (as part of each product it took ten instructions to three MMAs: 202 us against 188 for
// 3 requests up to 2031 tokens, d 64): a thread loads its pieces of the next tile into registers while this one is worked
// on, and stores (hi, hi, lo, lo) of two neighbours - two dims of a key, two keys of a dim of the values - as the 16 bytes that one
// thread's operand is.  Contraction indices are dealt to the fragments' places so that a thread's scores are its A operand of
// the second product; rows are padded so that loads have no bank conflicts.  q is split beforehand too where it has room (d <= 128).
#include "paged_decode.cuh"
#include "paged_prefill.cuh"

namespace gdn {
namespace prefill {
namespace {

using paged::exp2_fast;
using paged::mma_tf32;
using paged::split_tf32;

constexpr int kWarps = 8, kThreads = 32 * kWarps, kRows = 16 * kWarps;

template <int D> struct Cfg {
    static constexpr int kKeys = D == 256 ? 16 : 32;
    static constexpr bool kSplitQ = D < 256;
    static constexpr int kPitchQ = kSplitQ ? 2 * D + 16 : D + 8, kPitchK = 2 * D + 16;  // floats to a row
    static constexpr int kPitchV = D + 2;                                               // 16 bytes to two keys of a dim
    static constexpr int kK = kKeys * D / 4 / kThreads, kV = kKeys / 2 * D / kThreads;  // pieces of a thread: four dims of a key; two keys of a dim
    static constexpr int kSmem = 4 * (kRows * kPitchQ + kKeys * kPitchK) + 16 * (kKeys / 2 * kPitchV);
};

__device__ __forceinline__ uint32_t range_bits(int kb, int lo, int hi) {
    const int l = lo - kb, h = hi - kb;
    if (l > 31 || h < 0) return 0;
    return (l <= 0 ? ~0u : ~0u << l) & (h >= 31 ? ~0u : (2u << h) - 1);
}

// (hi, hi, lo, lo) of two values
__device__ __forceinline__ uint4 split2(float x, float y) {
    uint4 r;
    split_tf32(__float_as_uint(x), r.x, r.z);
    split_tf32(__float_as_uint(y), r.y, r.w);
    return r;
}
__device__ __forceinline__ uint4 lds(const float *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7fffffffu) < 0x7f7ff000u; }  // and so is its high term, rounded to 11 bits

// c += a b in three products, the small ones first
__device__ __forceinline__ void mma_split(float (&c)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4], const uint4 &b) {
    mma_tf32(c, al, b.x, b.y);
    mma_tf32(c, ah, b.z, b.w);
    mma_tf32(c, ah, b.x, b.y);
}

template <int D>
__global__ void __launch_bounds__(kThreads, D == 64 ? 2 : 1) prefill_f32_kernel(PrefillArgs a) {
    using C = Cfg<D>;
    constexpr int kKeys = C::kKeys, kTiles = kKeys / 8;
    constexpr uint32_t kAll = kKeys == 32 ? ~0u : (1u << (kKeys & 31)) - 1;
    extern __shared__ __align__(16) float sm[];
    __shared__ uint32_t ok_bits[2];
    float *const qs = sm, *const ks = qs + kRows * C::kPitchQ, *const vs = ks + kKeys * C::kPitchK;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
    const int group = (int)a.group.by, room = a.max_pages * a.c.page;
    View view;
    layout(a.ws, a.B, a.n, a.Hq, a.c.Hkv, D, kRows, gridDim.x, &view);
    pdl_wait();
    pdl_trigger();
    Walk walk;
    walk.start(view, blockIdx.x);
    const float zs = a.scale * 1.4426950408889634f;

    while (walk.next()) {
        const Unit u = walk.u;
        const int lo = u.lo, all_lo = u.all_lo[0], all_hi = u.all_hi[0];
        const int32_t *table = a.table + u.b * a.table_stride;
        // this thread's two rows
        int64_t out[2];
        Reach reach[2];
        bool there[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            int head;
            const int r = 16 * warp + g + 8 * e, token = u.first + a.group.quotient(u.row + min(r, u.rows - 1), head);
            there[e] = r < u.rows;
            out[e] = (int64_t)token * a.Hq + walk.h * group + head;
            reach[e] = reach_of(token + u.shift, a.window, room);
        }
        // ---- loads of the next tile, into registers
        const int end = min(u.hi, u.key + kKeys * walk.t1 - 1);
        float4 kx[C::kK];
        float2 vx[C::kV];
        // a lane knows where the tile's key of its number is; its page is looked up a tile ahead
        int cell_next = 0, page_next = -1;
        auto look_up = [&](int t) {
            const int key = u.key + kKeys * t + lane;
            page_next = -1;
            if (lane < kKeys && key >= lo && key <= end) page_next = table[a.page.quotient(key, cell_next)];
        };
        auto load = [&](int t) {
            const bool real = page_next >= 0 && page_next < a.c.pages;
            const int64_t row = real ? page_next * a.c.stride_page + cell_next * a.c.stride_token + walk.h * a.c.stride_head : -1;
            if (t + 1 < walk.t1) look_up(t + 1);
            const uint32_t bits = __ballot_sync(0xffffffffu, real);
            if (tid == 0) ok_bits[t & 1] = bits;
#pragma unroll
            for (int i = 0; i < C::kK; ++i) {
                const int at = tid + i * kThreads;
                const int64_t from = __shfl_sync(0xffffffffu, row, at / (D / 4));
                kx[i] = from >= 0 ? *(const float4 *)((const float *)a.c.k + from + at % (D / 4) * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < C::kV; ++i) {
                const int at = tid + i * kThreads, pair = at / D, d = at % D;
                const int64_t from = __shfl_sync(0xffffffffu, row, 2 * pair), from1 = __shfl_sync(0xffffffffu, row, 2 * pair + 1);
                vx[i].x = from >= 0 ? ((const float *)a.c.v)[from + d] : 0.f;
                vx[i].y = from1 >= 0 ? ((const float *)a.c.v)[from1 + d] : 0.f;
            }
        };
        // ---- the tile that the registers hold, split, to shared memory; whether its values are numbers
        auto store = [&] {
            bool numbers = true;
#pragma unroll
            for (int i = 0; i < C::kK; ++i) {
                const int at = tid + i * kThreads;
                float *to = ks + at / (D / 4) * C::kPitchK + at % (D / 4) * 8;
                *(uint4 *)to = split2(kx[i].x, kx[i].y);
                *(uint4 *)(to + 4) = split2(kx[i].z, kx[i].w);
            }
#pragma unroll
            for (int i = 0; i < C::kV; ++i) {
                const int at = tid + i * kThreads, pair = at / D, d = at % D;
                *(uint4 *)(vs + (pair * C::kPitchV + d) * 4) = split2(vx[i].x, vx[i].y);
                numbers = numbers && finite(vx[i].x) && finite(vx[i].y);
            }
            return numbers;
        };
        __syncthreads();  // the piece before is done with shared memory
        if (walk.t0 < walk.t1) {
            look_up(walk.t0);
            load(walk.t0);
#pragma unroll 4
            for (int r = warp; r < kRows; r += kWarps) {
                int head;
                const int token = u.first + a.group.quotient(u.row + min(r, u.rows - 1), head);
                const float *src = (const float *)a.q + token * a.q_tok + (walk.h * group + head) * a.q_head;
#pragma unroll
                for (int c = lane; c < D / 4; c += 32) {
                    const float4 x = r < u.rows ? *(const float4 *)(src + 4 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
                    if constexpr (C::kSplitQ) {
                        *(uint4 *)(qs + r * C::kPitchQ + 8 * c) = split2(x.x, x.y);
                        *(uint4 *)(qs + r * C::kPitchQ + 8 * c + 4) = split2(x.z, x.w);
                    } else {
                        *(float4 *)(qs + r * C::kPitchQ + 4 * c) = x;
                    }
                }
            }
        }
        float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        for (int t = walk.t0; t < walk.t1; ++t) {
            if (t > walk.t0) __syncthreads();  // the tile before has been read
            const bool numbers = store();
            if (t + 1 < walk.t1) load(t + 1);
            // a masked weight of 0 times an infinity or NaN is none: values that only some rows attend to have to be numbers
            const bool some = __syncthreads_or(!numbers);
            float s[kTiles][4];
#pragma unroll
            for (int i = 0; i < kTiles; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
            const float *qw = qs + (16 * warp + g) * C::kPitchQ + (C::kSplitQ ? 4 : 2) * q4, *kw = ks + g * C::kPitchK + 4 * q4;
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += 32) {
                float c[kTiles][4];
#pragma unroll
                for (int i = 0; i < kTiles; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint4 x, y;
                    if constexpr (C::kSplitQ) {
                        x = lds(qw + 2 * d0 + 16 * k);
                        y = lds(qw + 8 * C::kPitchQ + 2 * d0 + 16 * k);
                    } else {
                        const float2 p = *(const float2 *)(qw + d0 + 8 * k), q = *(const float2 *)(qw + 8 * C::kPitchQ + d0 + 8 * k);
                        x = split2(p.x, p.y);
                        y = split2(q.x, q.y);
                    }
                    const uint32_t ah[4] = {x.x, y.x, x.y, y.y}, al[4] = {x.z, y.z, x.w, y.w};
#pragma unroll
                    for (int i = 0; i < kTiles; ++i) mma_split(c[i], ah, al, lds(kw + 8 * i * C::kPitchK + 2 * d0 + 16 * k));
                }
#pragma unroll
                for (int i = 0; i < kTiles; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[i][j] += c[i][j];
            }
            const int kb = u.key + kKeys * t;
            const uint32_t ok = ok_bits[t & 1];
            const bool edge = kb < all_lo || kb + kKeys - 1 > all_hi || ok != kAll;
            const uint32_t bits[2] = {ok & range_bits(kb, reach[0].lo, reach[0].hi), ok & range_bits(kb, reach[1].lo, reach[1].hi)};
            float top[2] = {m[0], m[1]};
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = !edge || (bits[j >> 1] >> (8 * i + 2 * q4 + (j & 1)) & 1) ? s[i][j] * zs : -INFINITY;
                    top[j >> 1] = fmaxf(top[j >> 1], s[i][j]);
                }
            bool moved = false;
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
                top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
                f[e] = 1.f;
                if (top[e] > m[e]) {
                    moved = true;
                    f[e] = exp2_fast(m[e] - top[e]);
                    m[e] = top[e];
                    l[e] *= f[e];
                }
            }
            if (__any_sync(0xffffffffu, moved) && t > walk.t0)
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[i][j] *= f[j >> 1];
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = exp2_fast(s[i][j] - (m[j >> 1] == -INFINITY ? 0.f : m[j >> 1]));
                    l[j >> 1] += s[i][j];
                }
            if (some && edge) {
#pragma unroll 1
                for (int k = 0; k < kKeys; ++k) {
                    float p[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = 0.f;
#pragma unroll
                        for (int i = 0; i < kTiles; ++i)
                            if (k >> 3 == i) x = k & 1 ? s[i][2 * e + 1] : s[i][2 * e];
                        p[e] = __shfl_sync(0xffffffffu, x, (lane & ~3) | (k >> 1 & 3));
                    }
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            // hi + lo: to 2^-22 of the value, or what it has of NaN and infinity
                            const float *at = vs + ((k >> 1) * C::kPitchV + 8 * i + 2 * q4 + j) * 4 + (k & 1);
                            const float v = at[2] == 0.f ? at[0] : at[0] + at[2];
                            if (bits[0] >> k & 1) o[i][j] += p[0] * v;
                            if (bits[1] >> k & 1) o[i][2 + j] += p[1] * v;
                        }
                }
            } else {
                uint32_t ph[kTiles][4], pl[kTiles][4];
#pragma unroll
                for (int k = 0; k < kTiles; ++k) {
                    split_tf32(__float_as_uint(s[k][0]), ph[k][0], pl[k][0]);
                    split_tf32(__float_as_uint(s[k][2]), ph[k][1], pl[k][1]);
                    split_tf32(__float_as_uint(s[k][1]), ph[k][2], pl[k][2]);
                    split_tf32(__float_as_uint(s[k][3]), ph[k][3], pl[k][3]);
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < kTiles; ++k) mma_split(c, ph[k], pl[k], lds(vs + ((4 * k + q4) * C::kPitchV + 8 * i + g) * 4));
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[i][j] += c[j];
                }
            }
        }
        // ---- the rows' end in this CTA
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            if (!there[e]) continue;
            if (walk.whole()) {
                const bool none = m[e] == -INFINITY && l[e] == 0.f;
                const float inv = none ? 0.f : 1.f / l[e];
                float *to = (float *)a.o + out[e] * D + 2 * q4;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) *(float2 *)(to + 8 * i) = none ? make_float2(0.f, 0.f) : make_float2(o[i][2 * e] * inv, o[i][2 * e + 1] * inv);
                if (a.lse && q4 == 0) a.lse[out[e]] = none ? -INFINITY : (m[e] + log2f(l[e])) * 0.6931471805599453f;
            } else {
                const int slot = walk.slot(), r = 16 * warp + g + 8 * e;
                float *to = view.o + ((size_t)slot * (D / 4) * kRows + r) * 4;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const int col = 8 * i + 2 * q4;
                    *(float2 *)(to + (size_t)(col / 4) * kRows * 4 + col % 4) = make_float2(o[i][2 * e], o[i][2 * e + 1]);
                }
                if (q4 == 0) view.ml[(size_t)slot * kRows + r] = make_float2(m[e], l[e]);
            }
        }
    }
}

template <int D>
cudaError_t launch(const PrefillArgs &a, int grid, cudaStream_t stream) {
    const cudaError_t e = cudaFuncSetAttribute(prefill_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
    return e != cudaSuccess ? e : launch_kernel(true, prefill_f32_kernel<D>, grid, kThreads, Cfg<D>::kSmem, stream, a);
}

}  // namespace

cudaError_t launch_f32(const PrefillArgs &a, int grid, cudaStream_t stream) {
    return a.c.d == 64 ? launch<64>(a, grid, stream) : a.c.d == 128 ? launch<128>(a, grid, stream) : launch<256>(a, grid, stream);
}

}  // namespace prefill
}  // namespace gdn
