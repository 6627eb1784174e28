// k_paged_prefill_f32.cu -- softmax attention of new tokens over the paged cache in 32-bit storage.
//
// Every operand is split into two tf32 terms of 11 bits, x = hi + lo to 2^-22 of x, and a product of two takes three warp MMAs
// (lo hi, hi lo, hi hi); the tensor core's sums run over 32 terms of each only, longer ones are fp32 additions, which round where the
// tensor core cuts.  A warp has 16 rows, a CTA eight warps, a tile 32 keys; keys and values are copied in turns, one while the
// other is worked on.  Contraction indices are dealt to the fragments' places so that a thread's scores are its A operand of
// the second product and its operands of the first are 8-byte loads; rows are padded so that neither has bank conflicts.
#include "paged_decode.cuh"
#include "paged_prefill.cuh"

namespace gdn {
namespace prefill {
namespace {

using paged::cp16;
using paged::cp_commit;
using paged::cp_wait;
using paged::exp2_fast;
using paged::mma_tf32;
using paged::split_tf32;

constexpr int kWarps = 8, kThreads = 32 * kWarps, kRows = 16 * kWarps, kKeys = 32;

template <int D> struct Cfg {
    static constexpr int kPitchK = D + 8, kPitchV = D + 4;  // floats; q's rows as the keys'
    static constexpr int kSmem = 4 * (kRows * kPitchK + kKeys * (kPitchK + kPitchV));
};

__device__ __forceinline__ uint32_t range_bits(int kb, int lo, int hi) {
    const int l = lo - kb, h = hi - kb;
    if (l > 31 || h < 0) return 0;
    return (l <= 0 ? ~0u : ~0u << l) & (h >= 31 ? ~0u : (2u << h) - 1);
}

// c += a b in three products, the small ones first
__device__ __forceinline__ void mma_split(float (&c)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4], uint32_t b0, uint32_t b1) {
    uint32_t h0, l0, h1, l1;
    split_tf32(b0, h0, l0);
    split_tf32(b1, h1, l1);
    mma_tf32(c, al, h0, h1);
    mma_tf32(c, ah, l0, l1);
    mma_tf32(c, ah, h0, h1);
}

template <int D>
__global__ void __launch_bounds__(kThreads, D < 256 ? 2 : 1) prefill_f32_kernel(PrefillArgs a) {
    using C = Cfg<D>;
    extern __shared__ __align__(16) float sm[];
    __shared__ uint32_t ok_bits[kWarps];
    float *const qs = sm, *const ks = qs + kRows * C::kPitchK, *const vs = ks + kKeys * C::kPitchK;
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
        const int lo = u.lo, hi = u.hi, all_lo = u.all_lo[0], all_hi = u.all_hi[0];
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
        // ---- copies: warp w has keys 4 w .. 4 w + 3 of a tile; lanes 0 to 3 know where they are
        int64_t row = 0;
        bool real = false;
        auto find = [&](int t) {
            const int key = u.key + kKeys * t + 4 * warp + lane;
            real = false;
            row = 0;
            if (lane < 4 && key >= lo && key <= hi) {
                int cell;
                const int page = table[a.page.quotient(key, cell)];
                real = page >= 0 && page < a.c.pages;
                if (real) row = page * a.c.stride_page + cell * a.c.stride_token + walk.h * a.c.stride_head;
            }
            const uint32_t bits = __ballot_sync(0xffffffffu, real);
            if (lane == 0) ok_bits[warp] = bits;
        };
        auto copy = [&](const void *base, float *to, int pitch) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t off = __shfl_sync(0xffffffffu, row, k);
                const bool is = __shfl_sync(0xffffffffu, (int)real, k);
                const uint32_t dst = paged::smem_addr(to + (4 * warp + k) * pitch);
                for (int c = lane; c < D / 4; c += 32) cp16(dst + 16 * c, (const float *)base + off + 4 * c, is);
            }
            cp_commit();
        };
        __syncthreads();  // the piece before is done with shared memory
        const int n = walk.t1 - walk.t0;
        if (n > 0) {
            for (int r = warp; r < kRows; r += kWarps) {
                int head;
                const int token = u.first + a.group.quotient(u.row + min(r, u.rows - 1), head);
                const float *src = (const float *)a.q + token * a.q_tok + (walk.h * group + head) * a.q_head;
                for (int c = lane; c < D / 4; c += 32) cp16(paged::smem_addr(qs + r * C::kPitchK) + 16 * c, src + 4 * c, r < u.rows);
            }
            find(walk.t0);
            copy(a.c.k, ks, C::kPitchK);
        }
        float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        for (int t = walk.t0; t < walk.t1; ++t) {
            cp_wait<0>();
            __syncthreads();  // keys are there; the values before have been read
            copy(a.c.v, vs, C::kPitchV);
            float s[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
            const float *qw = qs + (16 * warp + g) * C::kPitchK + 2 * q4, *kw = ks + g * C::kPitchK + 2 * q4;
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += 32) {
                float c[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 x = *(const float2 *)(qw + d0 + 8 * k), y = *(const float2 *)(qw + 8 * C::kPitchK + d0 + 8 * k);
                    uint32_t ah[4], al[4];
                    split_tf32(__float_as_uint(x.x), ah[0], al[0]);
                    split_tf32(__float_as_uint(y.x), ah[1], al[1]);
                    split_tf32(__float_as_uint(x.y), ah[2], al[2]);
                    split_tf32(__float_as_uint(y.y), ah[3], al[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 b = *(const float2 *)(kw + 8 * i * C::kPitchK + d0 + 8 * k);
                        mma_split(c[i], ah, al, __float_as_uint(b.x), __float_as_uint(b.y));
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[i][j] += c[i][j];
            }
            const int kb = u.key + kKeys * t;
            uint32_t ok = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) ok |= ok_bits[w] << (4 * w);
            const bool edge = kb < all_lo || kb + kKeys - 1 > all_hi || ok != ~0u;
            const uint32_t bits[2] = {ok & range_bits(kb, reach[0].lo, reach[0].hi), ok & range_bits(kb, reach[1].lo, reach[1].hi)};
            float top[2] = {m[0], m[1]};
#pragma unroll
            for (int i = 0; i < 4; ++i)
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
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = exp2_fast(s[i][j] - (m[j >> 1] == -INFINITY ? 0.f : m[j >> 1]));
                    l[j >> 1] += s[i][j];
                }
            cp_wait<0>();
            int tainted = 0;
            if (edge) {
                // a masked weight of 0 times an infinity or NaN is none: values that only some rows attend to have to be numbers
                __syncthreads();
                for (int c = tid; c < kKeys * (D / 4); c += kThreads) {
                    const float4 x = *(const float4 *)(vs + c / (D / 4) * C::kPitchV + c % (D / 4) * 4);
                    tainted |= !(fabsf(x.x) < INFINITY) | !(fabsf(x.y) < INFINITY) | !(fabsf(x.z) < INFINITY) | !(fabsf(x.w) < INFINITY);
                }
            }
            tainted = __syncthreads_or(tainted);  // values are there; the keys have been read
            if (t + 1 < walk.t1) {
                find(t + 1);
                copy(a.c.k, ks, C::kPitchK);
            }
            if (tainted) {
#pragma unroll 1
                for (int k = 0; k < kKeys; ++k) {
                    float p[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = 0.f;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (k >> 3 == i) x = k & 1 ? s[i][2 * e + 1] : s[i][2 * e];
                        p[e] = __shfl_sync(0xffffffffu, x, (lane & ~3) | (k >> 1 & 3));
                    }
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        const float2 v = *(const float2 *)(vs + k * C::kPitchV + 8 * i + 2 * q4);
                        if (bits[0] >> k & 1) o[i][0] += p[0] * v.x, o[i][1] += p[0] * v.y;
                        if (bits[1] >> k & 1) o[i][2] += p[1] * v.x, o[i][3] += p[1] * v.y;
                    }
                }
            } else {
                uint32_t ph[4][4], pl[4][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    split_tf32(__float_as_uint(s[k][0]), ph[k][0], pl[k][0]);
                    split_tf32(__float_as_uint(s[k][2]), ph[k][1], pl[k][1]);
                    split_tf32(__float_as_uint(s[k][1]), ph[k][2], pl[k][2]);
                    split_tf32(__float_as_uint(s[k][3]), ph[k][3], pl[k][3]);
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float *v = vs + (8 * k + 2 * q4) * C::kPitchV + 8 * i + g;
                        mma_split(c, ph[k], pl[k], __float_as_uint(v[0]), __float_as_uint(v[C::kPitchV]));
                    }
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
