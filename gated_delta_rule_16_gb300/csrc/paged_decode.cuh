// paged_decode.cuh -- one-token attention over the paged cache: the kernel template that
// k_paged_decode_{bf16,e4m3,f32}.cu instantiate.
//
// o = sum_j p_j v_j / sum_j p_j with p_j = 2^(z_j - max z), z_j = scale log2(e) <q, k_j>: one pass over K and V
// with a running maximum, sum and output per (request, query head).
//
// What bounds it: every cached byte is read once and used for 2 G operations (G query heads per KV head; at most
// 16 to a pass), so HBM, as long as tensor and issue slots keep up.  Measured: 64 requests of up to 8192 bf16 tokens
// (8 KV heads of 128, G = 4) 170 us, 6.2 TB/s or 92 % of a copy; one of 131072 tokens 48 us; 32 e4m3 requests of up to 32768
// (G = 8) 87 us, 6.0 TB/s; 256 dims 5.6 TB/s; fp32 5.7 TB/s; 16 heads to a pass 5.4 (bf16), 3.4 (e4m3).  The design
// follows from the bound:
//   - Work is cut by cached tokens, not by requests.  All (request, KV head) rows are laid end to end in tiles of
//     16 tokens per warp and the CTAs of one wave get equal runs of tiles.  A row inside one CTA is written out
//     directly; a row cut by a CTA's edge leaves unnormalised fp32 parts that a second, dependent launch joins in a
//     fixed order.  Lengths are only known on the GPU, so each CTA finds its run from a scan over them.
//   - Each warp streams its own 16-token slices of K and V through a ring of shared-memory slots by 16-byte
//     cp.async, whose source address is free per token: any page size, any storage order.  No CTA barrier inside a
//     row: the warps keep their own maxima and meet at the row's end.
//   - Products on warp MMAs with the cached tokens as M and 8 query heads as N: S^T = K Q^T (16 tokens x 8 heads) and
//     O^T += V^T P^T (16 dims x 8 heads), so 8 heads waste nothing (heads as M would pad them to 16), and K and V
//     are the A operands straight from shared memory.  The tensor cores' tcgen05 form wants 64 rows of M or more and
//     both operands in shared memory; at 2 G flops a byte the warp form has the rate needed, and P stays in registers.
//     P^T comes from the S^T fragment by transposing 8x8 tiles between registers (movmatrix).
//   - Rounding: scores, maxima, sums and outputs are fp32.  P enters the second product as two bf16 terms (16 bits
//     together) for a bf16 cache; for an 8-bit cache as f16 of 2^15 P (11 bits down to 2^-29 of a warp's largest weight, an
//     absolute 2^-40 of it below, so that a long tail of small weights keeps its mass; a second f16 term would bring the outputs
//     five times as near to those of fp32 weights, below bf16's own rounding, and take 5 % more time), where K and V are
//     converted exactly to f16 and q, scaled by a power of two to below 2, loses nothing unless it is 2^14 times smaller than the row's largest.  A
//     32-bit cache splits every operand into two tf32 terms, drops the product of the low ones (2^-22) and adds each
//     8-wide product to its sum outside the tensor core, whose own accumulation cuts instead of rounding: that
//     drift alone put scores of thousands past 1e-5.
//   - Tokens outside [max(0, L - window), L) or on a page outside the pool are zero-filled, never read, and their
//     scores set to -inf, so that what the cache holds there cannot reach a product.
#pragma once

#include "paged.cuh"

namespace gdn {
namespace paged {

constexpr int kSMs = 152;
constexpr int kMaxCtas = 4 * kSMs;   // one wave
constexpr int kPadded = 8;           // tiles per CTA from which on a row counts one tile more

// Workspace.  A row cut between CTAs is described by one entry {request, row in request, first part, parts}: entry r of row
// r = request * rows + row if rows are few (join_by_row; parts 0: not cut), else entry i - 1 of the
// CTA i that is the second of the row's.  Then two parts per CTA: 2 i of CTA i's first row, 2 i + 1 of its last.
struct WsView {
    int4 *joins;
    float2 *ml;   // [2 * kMaxCtas][heads] {maximum, sum}
    float *o;     // [2 * kMaxCtas][heads][d]
};
__host__ __device__ inline WsView ws_view(void *ws, int heads) {
    char *p = (char *)ws;
    WsView w;
    w.joins = (int4 *)p;
    w.ml = (float2 *)(p + kMaxCtas * sizeof(int4));
    w.o = (float *)(p + kMaxCtas * sizeof(int4) + (size_t)2 * kMaxCtas * heads * sizeof(float2));
    return w;
}
inline size_t ws_bytes(int heads, int d) {
    return kMaxCtas * sizeof(int4) + (size_t)2 * kMaxCtas * heads * (sizeof(float2) + (size_t)d * sizeof(float));
}

inline bool join_by_row(int64_t rows, int grid) { return rows * 8 <= grid; }

// Query heads per pass over a KV head's tokens: 8 or 16 (a larger group takes several passes, as rows of their own).
__host__ __device__ constexpr int pass_heads(int group) { return group <= 8 ? 8 : 16; }

// By the bytes of a cached row: warps per CTA (rows wider than 512 bytes leave room for two warps' rings), and 16-token
// parts of a warp's slice (narrow rows take two at a time: half the waits, maxima and addresses per token).
__host__ __device__ constexpr int warps_of(int row) { return row > 512 ? 2 : 4; }
__host__ __device__ constexpr int sub_slices(int row) { return row <= 128 ? 2 : 1; }

template <gdn_dtype KIND, int D, int NT>
struct Cfg {
    static constexpr int kBytes = KIND == GDN_BF16 ? 2 : (KIND == GDN_E4M3 ? 1 : 4);
    static constexpr int kRow = D * kBytes;           // bytes of a cached row
    static constexpr int kChunks = kRow / 16;
    static constexpr int kWarps = warps_of(kRow);
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kSub = sub_slices(kRow);     // 16-token parts of a slice
    static constexpr int kTok = 16 * kSub;            // tokens of a warp's slice
    static constexpr int kTile = kTok * kWarps;       // tokens of a tile
    static constexpr int kHalf = kTok * kRow;          // bytes of one warp's K (or V) slice
    // CTAs per SM and ring slots of half a slice (K or V) per warp.  Warps hide each other's waits, so as many CTAs as the
    // registers allow (16 heads, or 256 dims, of output per warp take twice the registers of 8 heads of 128) with three
    // slots or more; what shared memory is left deepens the ring.  Measured against one CTA less per SM: 32 x 8192 bf16 tokens of
    // 64 dims 56 -> 53 us, 64 x 8192 of 128 dims 175 -> 170, of 64 dims for 16 heads 66 -> 60, 16 x 8192 fp32 138 -> 99.
    static constexpr int kOcc = kHalf > 8192 && NT == 2 ? 1 : kHalf > 4096 || D == 256 ? 2
                                : NT == 2 ? (D == 64 && KIND != GDN_F32 ? 3 : 2) : kHalf > 2048 ? (KIND == GDN_BF16 && D == 64 ? 4 : 3) : 4;
    static constexpr int kSlots = kOcc == 1 ? 6 : kHalf > 4096 ? 3 : kOcc == 2 ? (kHalf > 2048 ? 6 : 8) : kOcc == 3 ? 4 : kHalf > 2048 ? 3 : kHalf > 1024 ? 5 : 8;
    static constexpr int kRing = kSlots * kHalf;      // per warp
    static constexpr float kUnit = KIND == GDN_E4M3 ? 32768.f : 1.f;  // of weights and of outputs until a row's end
    static constexpr int kMergeDims = (KIND == GDN_F32 && NT == 2) || (kOcc == 4 && kHalf > 2048) ? 32 : 64;  // output dims joined per round at a row's end
    static constexpr int kMerge = kWarps * 8 * (kMergeDims + 4) * 4;
    static constexpr int kQ = KIND == GDN_F32 ? NT * (D / 8) * 32 * 8 : 0;
    static constexpr int kSmem = kWarps * kRing + kMerge + kWarps * NT * 8 * 8 + kQ + kWarps * kSlots * 4;
    static_assert(KIND != GDN_F32 || kSub == 1, "the fp32 products take one part");
    static_assert((kSmem + 1024) * kOcc <= 228 * 1024, "shared memory of an SM");
};

inline int tile_of(const gdn_kv_cache &c) {  // Cfg::kTile
    const int row = c.d * (c.dtype == GDN_BF16 ? 2 : c.dtype == GDN_E4M3 ? 1 : 4);
    return 16 * sub_slices(row) * warps_of(row);
}

// ---- instructions -----------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
    return r;
}
__device__ __forceinline__ void lds128(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo to 2^-24 of x, each rounded to tf32's 11 bits.  In integer arithmetic at the full rate, as the conversion
// instruction has a quarter of it (16 requests up to 8192 tokens, 8 KV heads of 128: 91 us with it against 84; of 256 dims 213
// against 181).  lo cut instead of rounded takes 0 to 6 % less, but scores in the thousands then lose the bits that order their softmax.
// hi's rounding may carry a NaN's bits over into a zero's, so lo has to keep the NaN: it has 12 bits at most, for which a product
// with 1 + 2^-11 that is cut rounds the same as an addition of half a unit would, and a NaN stays one.
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t &hi, uint32_t &lo) {
    hi = (x + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint((__uint_as_float(x) - __uint_as_float(hi)) * 1.00048828125f) & 0xffffe000u;
}
// both 8-bit values of x's low (high) half as f16: exact
__device__ __forceinline__ uint32_t f16_lo(uint32_t x) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)x));
    return r;
}
__device__ __forceinline__ uint32_t f16_hi(uint32_t x) { return f16_lo(x >> 16); }
__device__ __forceinline__ float exp2_fast(float x) {  // 2^-22 relative
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ---- a place in the list of tiles -------------------------------------------------------------------
struct Cursor {
    int b, row, tile, tiles;  // request, row in request, tile in row, tiles of the row
    int start, len;           // tokens attended: [start, len)

    template <int TILE> __device__ __forceinline__ void load(const AttendArgs &a) {
        tiles = 1;
        start = len = 0;
        if (b >= a.B) return;
        const int64_t room = (int64_t)a.max_pages * a.c.page;
        len = (int)min((int64_t)max(a.lens[b], 0), room);
        start = a.window > 0 ? max(0, len - a.window) : 0;
        tiles = max(1, (len - (start & ~15) + TILE - 1) / TILE);  // an empty request keeps one, to be written
    }
    template <int TILE> __device__ __forceinline__ void next(const AttendArgs &a, int rows) {
        if (++tile < tiles) return;
        tile = 0;
        if (++row < rows) return;
        row = 0;
        ++b;
        load<TILE>(a);
    }
};

__device__ __forceinline__ int64_t split_at(int64_t total, int ctas, int i) {
    return total < (1 << 22) ? (int64_t)((uint32_t)total * (uint32_t)i / (uint32_t)ctas) : total * i / ctas;  // ctas < 2^10
}

template <int THREADS>
__device__ int64_t block_sum(int64_t x, int64_t *buf) {
#pragma unroll
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) x += buf[w];
    __syncthreads();
    return x;
}

template <gdn_dtype KIND, int D, int NT>
__global__ void __launch_bounds__(Cfg<KIND, D, NT>::kThreads, Cfg<KIND, D, NT>::kOcc) paged_decode_kernel(AttendArgs a, bool by_row) {
    using C = Cfg<KIND, D, NT>;
    constexpr int W = C::kWarps, TILE = C::kTile, SUB = C::kSub, kMergeDims = C::kMergeDims;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, q4 = lane & 3;  // fragment row, fragment column pair
    float *merge = (float *)(smem + W * C::kRing);
    float2 *ml = (float2 *)(smem + W * C::kRing + C::kMerge);
    float2 *qs = (float2 *)((uint8_t *)ml + W * NT * 8 * 8);                         // 32-bit storage: q by fragment
    uint32_t *real = (uint32_t *)((uint8_t *)qs + C::kQ) + warp * C::kSlots;         // of the slice in a slot: bit t: token t is real
    const uint32_t ring = smem_addr(smem) + warp * C::kRing;
    const int group = a.Hq / a.c.Hkv, passes = (group + NT * 8 - 1) / (NT * 8), rows = a.c.Hkv * passes;
    const WsView ws = ws_view(a.ws, NT * 8);
    pdl_trigger();

    // ---- this CTA's run of tiles [t0, t0 + n): requests lie one after the other, `rows` rows of the same tiles each.  To begin
    // and end a row takes a CTA about as long as a tile, so where runs are long enough to divide so finely a row counts one
    // tile more (pad), which nobody has to do.  Without it CTAs with many short rows are the last: 32 e4m3 requests up to 32768
    // tokens 92 us against 86, 256 bf16 requests up to 300 43 against 36, 16 fp32 up to 8192 95 against 82.  (Two or three tiles
    // more: within 2 % of one, and 36 -> 38 us for the 256.)
    __shared__ int64_t scan[W];
    __shared__ int4 found;
    Cursor cur;
    int64_t total, t0, n;
    int ctas, pad;
    const int cta = blockIdx.x;
    auto settle = [&](int64_t per_row) {  // false: no tiles for this CTA
        pad = per_row * rows >= (int64_t)kPadded * gridDim.x;
        total = (per_row + pad * a.B) * rows;
        ctas = (int)min((int64_t)gridDim.x, total);
        if (cta >= ctas) {
            if (tid == 0 && !by_row) ws.joins[cta - 1] = make_int4(0, 0, 0, 0);
            return false;
        }
        t0 = split_at(total, ctas, cta);
        n = split_at(total, ctas, cta + 1) - t0;
        return true;
    };
    if (a.B <= 32) {
        // a lane per request, every warp for itself
        cur.b = lane;
        cur.load<TILE>(a);
        const int mine = lane < a.B ? cur.tiles : 0;
        int64_t incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += x;
        }
        if (!settle(__shfl_sync(0xffffffffu, incl, 31))) return;
        const int64_t want = t0 / rows;
        const int at = __popc(__ballot_sync(0xffffffffu, lane < a.B && incl + pad * (lane + 1) <= want));  // requests that end before
        const int64_t off = t0 - (__shfl_sync(0xffffffffu, incl - mine, at) + pad * at) * rows;
        const int tiles = __shfl_sync(0xffffffffu, mine, at) + pad;
        cur.b = at;
        cur.load<TILE>(a);
        cur.row = (int)(off / tiles);
        cur.tile = (int)(off % tiles);
    } else {
        int64_t sum = 0;
        for (int b = tid; b < a.B; b += C::kThreads) {
            cur.b = b;
            cur.load<TILE>(a);
            sum += cur.tiles;
        }
        if (!settle(block_sum<C::kThreads>(sum, scan))) return;
        const int64_t want = t0 / rows;
        int64_t before = 0;
        for (int b0 = 0; b0 < a.B; b0 += C::kThreads) {
            cur.b = b0 + tid;
            cur.load<TILE>(a);
            const int64_t mine = cur.b < a.B ? cur.tiles + pad : 0;
            int64_t incl = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += x;
            }
            if (lane == 31) scan[warp] = incl;
            __syncthreads();
            int64_t base = before, step = 0;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                if (w < warp) base += scan[w];
                step += scan[w];
            }
            const int64_t excl = base + incl - mine;
            if (mine > 0 && excl <= want && want < excl + mine) {
                const int64_t at = t0 - excl * rows;
                found = make_int4(cur.b, (int)(at / mine), (int)(at % mine), (int)mine);
            }
            before += step;
            __syncthreads();
            if (before > want) break;
        }
        cur.b = found.x;
        cur.load<TILE>(a);
        cur.row = found.y;
        cur.tile = found.z;
    }

    // ---- loads, in parts of 16 tokens.  Where a page holds whole parts (page a multiple of 16, as parts are aligned to 16
    // tokens) one table entry and one address serve the warp: its lanes' pieces lie at fixed distances.  Else lane l finds
    // the row of token l & 15 and the lanes pass them on.  `off`: of the part's first token, or of the lane's; `mask`: the
    // real tokens of the slice.
    const bool whole_pages = (a.c.page & 15) == 0, pow2 = (a.c.page & (a.c.page - 1)) == 0;
    const int shift = 31 - __clz(a.c.page);
    struct Next { int64_t off[SUB]; uint32_t mask; };
    auto find = [&](const Cursor &c) -> Next {
        Next x;
        x.mask = 0u;
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
            const int t0 = (c.start & ~15) + c.tile * TILE + warp * C::kTok + 16 * u, t = whole_pages ? t0 : t0 + (lane & 15);
            const int lo = max(c.start - t0, 0), hi = min(c.len - t0, 16);
            x.off[u] = 0;
            if (hi <= lo) continue;
            uint32_t mask = (0xffffu >> (16 - hi)) & (0xffffu << lo);
            int id = -1, cell = 0;
            if (whole_pages || (mask >> (lane & 15) & 1)) {
                const int slot = pow2 ? t >> shift : t / a.c.page;
                cell = t - slot * a.c.page;
                id = a.table[c.b * a.table_stride + slot];
            }
            const bool real = id >= 0 && id < a.c.pages;
            if (whole_pages) mask = real ? mask : 0u;
            else mask &= __ballot_sync(0xffffffffu, real);
            if (real) x.off[u] = id * a.c.stride_page + cell * a.c.stride_token + (c.row / passes) * a.c.stride_head;
            x.mask |= mask << (16 * u);
        }
        return x;
    };
    auto swizzled = [](int row, int chunk) -> uint32_t {
        const int x = C::kChunks >= 8 ? row & 7 : (row >> 1) & 3;
        return (uint32_t)(row * C::kRow + ((chunk ^ x) << 4));
    };
    const int64_t token_bytes = a.c.stride_token * C::kBytes;
    const int64_t lane_bytes = (lane / C::kChunks) * token_bytes + lane % C::kChunks * 16;
    auto issue = [&](int slot, const Next &x, const void *cache) {
        if (lane == 0) real[slot] = x.mask;
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
            const uint32_t dst = ring + slot * C::kHalf + u * (16 * C::kRow), mask = x.mask >> (16 * u);
            if (whole_pages && C::kChunks <= 32) {
                constexpr int kRows = C::kChunks <= 32 ? 32 / C::kChunks : 1;  // per instruction
                const char *src = (const char *)cache + (x.off[u] * C::kBytes + lane_bytes);
#pragma unroll
                for (int i = 0; i < 16 / kRows; ++i) {
                    const int row = i * kRows + lane / C::kChunks;
                    cp16(dst + swizzled(row, lane % C::kChunks), src, mask >> row & 1);
                    src += kRows * token_bytes;
                }
            } else {
#pragma unroll 4
                for (int i = 0; i < 16 * C::kChunks / 32; ++i) {
                    const int idx = i * 32 + lane, row = idx / C::kChunks, chunk = idx % C::kChunks;
                    const int64_t at = whole_pages ? x.off[u] + row * a.c.stride_token : __shfl_sync(0xffffffffu, x.off[u], row);
                    const bool have = mask >> row & 1;
                    cp16(dst + swizzled(row, chunk), (const char *)cache + (have ? at : 0) * C::kBytes + chunk * 16, have);
                }
            }
        }
    };

    // ---- a row's state
    uint32_t qf[KIND == GDN_F32 ? 1 : D / 16][NT][2];
    float z_scale[NT][2];                       // per query head 2 q4 + j of tile nt
    float m[NT][2], l[NT][2], o[D / 16][NT][4];
    auto begin_row = [&](const Cursor &c) {
        const int h = c.row / passes, first = (c.row % passes) * NT * 8;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int hh = first + nt * 8 + g;
            const bool have = hh < group;
            const int64_t off = c.b * a.q_req + (int64_t)(h * group + (have ? hh : 0)) * a.q_head;
            float unit = 1.f;
            if constexpr (KIND == GDN_BF16) {
                const __nv_bfloat16 *q = (const __nv_bfloat16 *)a.q + off;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        qf[kk][nt][i] = have ? *(const uint32_t *)(q + 16 * kk + 8 * i + 2 * q4) : 0u;
            } else if constexpr (KIND == GDN_E4M3) {
                // K's bytes 4 q4 .. 4 q4 + 3 of a 16-byte piece are this lane's k indices 2 q4, 2 q4 + 1, 2 q4 + 8, 2 q4 + 9
                const __nv_bfloat16 *q = (const __nv_bfloat16 *)a.q + off;
                float top = 0.f;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint2 x = have ? *(const uint2 *)(q + 16 * kk + 4 * q4) : make_uint2(0u, 0u);
                    qf[kk][nt][0] = x.x;
                    qf[kk][nt][1] = x.y;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qf[kk][nt][i] << 16)),
                                               fabsf(__uint_as_float(qf[kk][nt][i] & 0xffff0000u))));
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = (int)(__float_as_uint(top) >> 23);        // top = 2^(e-127) * [1, 2); 0 or infinite: left as it is
                float down = 1.f;
                if (e > 0 && e < 255) {
                    unit = __uint_as_float((uint32_t)e << 23);
                    down = e < 254 ? __uint_as_float((uint32_t)(254 - e) << 23) : __uint_as_float(1u << 22);
                }
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        qf[kk][nt][i] = pack_f16(__uint_as_float(qf[kk][nt][i] << 16) * down,
                                                 __uint_as_float(qf[kk][nt][i] & 0xffff0000u) * down);
            } else {
                const float *q = (const float *)a.q + off;
                for (int kk = warp; kk < D / 8; kk += W)
                    qs[(nt * (D / 8) + kk) * 32 + lane] = have ? make_float2(q[8 * kk + q4], q[8 * kk + q4 + 4]) : make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float f = a.scale * 1.4426950408889634f;
                if constexpr (KIND == GDN_E4M3) f *= a.c.k_scale ? a.c.k_scale[h] : 1.f;
                z_scale[nt][j] = f * (KIND == GDN_E4M3 ? __shfl_sync(0xffffffffu, unit, (2 * q4 + j) * 4) : 1.f);
                m[nt][j] = -INFINITY;
                l[nt][j] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[mt][nt][i] = 0.f;
        }
        if constexpr (KIND == GDN_F32) __syncthreads();
    };

    // ---- one slice.  Scores and the running softmax, from the K slice at kb
    const int mrow = lane & 7, mid = lane >> 3;  // ldmatrix: row in matrix, matrix
    float p[SUB][NT][4];  // scores, then weights
    auto scores = [&](uint32_t kb, uint32_t mask) {
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) p[u][nt][i] = 0.f;
        if constexpr (KIND == GDN_BF16) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                uint32_t k[4];
                ldsm4(k, kb + u * (16 * C::kRow) + swizzled(mrow + (mid & 1) * 8, 2 * kk + (mid >> 1)));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_bf16(p[u][nt], k, qf[kk][nt][0], qf[kk][nt][1]);
            }
        } else if constexpr (KIND == GDN_E4M3) {
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                uint32_t k[4];  // rows 0-7 and 8-15 of one 16-byte piece, then of the next
                ldsm4(k, kb + u * (16 * C::kRow) + swizzled(mrow + (mid & 1) * 8, 2 * kk + (mid >> 1)));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t a0 = f16_lo(k[2 * i]), a1 = f16_lo(k[2 * i + 1]), a2 = f16_hi(k[2 * i]), a3 = f16_hi(k[2 * i + 1]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(p[u][nt], a0, a1, a2, a3, qf[2 * kk + i][nt][0], qf[2 * kk + i][nt][1]);
                }
            }
        } else {
#pragma unroll
            for (int kk = 0; kk < D / 8; ++kk)
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                uint32_t k[4], kh[4], kl[4];
                ldsm4(k, kb + u * (16 * C::kRow) + swizzled(mrow + (mid & 1) * 8, 2 * kk + (mid >> 1)));
#pragma unroll
                for (int i = 0; i < 4; ++i) split_tf32(k[i], kh[i], kl[i]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float2 x = qs[(nt * (D / 8) + kk) * 32 + lane];
                    uint32_t h0, l0, h1, l1;
                    split_tf32(__float_as_uint(x.x), h0, l0);
                    split_tf32(__float_as_uint(x.y), h1, l1);
                    float t[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_tf32(t, kl, h0, h1);
                    mma_tf32(t, kh, l0, l1);
                    mma_tf32(t, kh, h0, h1);
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[u][nt][i] += t[i];
                }
            }
        }

        // running softmax; token g of a part in p[u][.][0..1], token g + 8 in p[u][.][2..3], heads 2 q4 and 2 q4 + 1
        bool moved = false;
        float f[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float top = -INFINITY;
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float &x = p[u][nt][2 * i + j];
                        x = mask >> (16 * u + 8 * i + g) & 1 ? x * z_scale[nt][j] : -INFINITY;
                        top = fmaxf(top, x);
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                top = fmaxf(top, m[nt][j]);
                const float ref = top == -INFINITY ? 0.f : top;
                moved |= top != m[nt][j];
                f[nt][j] = exp2_fast(m[nt][j] - ref);
                m[nt][j] = top;
                float sum = 0.f;
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float &x = p[u][nt][2 * i + j];
                        x = exp2_fast(x - ref);
                        sum += x;
                    }
                l[nt][j] = l[nt][j] * f[nt][j] + sum;
            }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[mt][nt][i] *= f[nt][i & 1];
        }

    };
    // The weighted sum, from the V slice at vb
    auto values = [&](uint32_t vb) {
        if constexpr (KIND == GDN_BF16) {
            uint32_t hi[SUB][NT][2], lo[SUB][NT][2];
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float p0 = p[u][nt][2 * i], p1 = p[u][nt][2 * i + 1];
                        // cut, not rounded, so that both terms of a weight are positive: an infinite value stays infinite.  The low
                        // one is at least 2^-24 of the weight: a fixed least would let values of 1e38 in that have no weight
                        const uint32_t h = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
                        const uint32_t r = pack_bf16(fmaxf(p0 - __uint_as_float(h << 16), p0 * 5.9604645e-8f),
                                                     fmaxf(p1 - __uint_as_float(h & 0xffff0000u), p1 * 5.9604645e-8f));
                        hi[u][nt][i] = transpose8x8(h);
                        lo[u][nt][i] = transpose8x8(r);
                    }
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    uint32_t v[4];
                    ldsm4t(v, vb + u * (16 * C::kRow) + swizzled(mrow + (mid >> 1) * 8, 2 * mt + (mid & 1)));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_bf16(o[mt][nt], v, lo[u][nt][0], lo[u][nt][1]);
                        mma_bf16(o[mt][nt], v, hi[u][nt][0], hi[u][nt][1]);
                    }
                }
        } else if constexpr (KIND == GDN_E4M3) {
            uint32_t b[SUB][NT][2];
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        b[u][nt][i] = transpose8x8(pack_f16(p[u][nt][2 * i] * C::kUnit, p[u][nt][2 * i + 1] * C::kUnit));
            // a lane's 4 bytes of a token are dims 4 g .. 4 g + 3 of a block of 32; bytes of neighbouring tokens are
            // paired into the A fragments of two 16-row tiles whose rows g, g + 8 are dims 4 g, 4 g + 1 and 4 g + 2, 4 g + 3
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = lds32(vb + u * (16 * C::kRow) + swizzled(2 * q4 + (i & 1) + (i >> 1) * 8, 2 * kk + (g >> 2)) + (g & 3) * 4);
                    const uint32_t t01 = __byte_perm(w[0], w[1], 0x5140), t23 = __byte_perm(w[2], w[3], 0x5140);
                    const uint32_t u01 = __byte_perm(w[0], w[1], 0x7362), u23 = __byte_perm(w[2], w[3], 0x7362);
                    const uint32_t ta[4] = {f16_lo(t01), f16_hi(t01), f16_lo(t23), f16_hi(t23)};
                    const uint32_t ua[4] = {f16_lo(u01), f16_hi(u01), f16_lo(u23), f16_hi(u23)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_f16(o[2 * kk][nt], ta[0], ta[1], ta[2], ta[3], b[u][nt][0], b[u][nt][1]);
                        mma_f16(o[2 * kk + 1][nt], ua[0], ua[1], ua[2], ua[3], b[u][nt][0], b[u][nt][1]);
                    }
                }
        } else {
            // k index q4 of step i is token 8 i + 2 q4, k index q4 + 4 is token 8 i + 2 q4 + 1; rows as for 8 bits
            uint32_t ph[NT][2][2], pl[NT][2][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t x = __float_as_uint(p[0][nt][2 * i]), y = __float_as_uint(p[0][nt][2 * i + 1]);
                    const uint32_t top = transpose8x8(__byte_perm(x, y, 0x7632)), low = transpose8x8(__byte_perm(x, y, 0x5410));
                    split_tf32(__byte_perm(low, top, 0x5410), ph[nt][i][0], pl[nt][i][0]);
                    split_tf32(__byte_perm(low, top, 0x7632), ph[nt][i][1], pl[nt][i][1]);
                }
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t x[4], y[4];
                    lds128(x, vb + swizzled(8 * i + 2 * q4, 8 * kk + g));
                    lds128(y, vb + swizzled(8 * i + 2 * q4 + 1, 8 * kk + g));
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const uint32_t v[4] = {x[2 * t], x[2 * t + 1], y[2 * t], y[2 * t + 1]};
                        uint32_t vh[4], vl[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) split_tf32(v[e], vh[e], vl[e]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float r[4] = {0.f, 0.f, 0.f, 0.f};
                            mma_tf32(r, vl, ph[nt][i][0], ph[nt][i][1]);
                            mma_tf32(r, vh, pl[nt][i][0], pl[nt][i][1]);
                            mma_tf32(r, vh, ph[nt][i][0], ph[nt][i][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[2 * kk + t][nt][e] += r[e];
                        }
                    }
                }
        }
    };

    // ---- a row's (or part's) end: the warps' sums meet
    auto end_row = [&](const Cursor &c, bool whole, int part) {
        const int h = c.row / passes, first = (c.row % passes) * NT * 8;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float x = l[nt][j];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                if (g == 0) ml[warp * NT * 8 + nt * 8 + 2 * q4 + j] = make_float2(m[nt][j], x);
            }
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float f[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < W; ++w) top = fmaxf(top, ml[w * NT * 8 + nt * 8 + 2 * q4 + j].x);
                f[j] = exp2_fast(m[nt][j] - (top == -INFINITY ? 0.f : top)) * (1.f / C::kUnit);
            }
#pragma unroll
            for (int r = 0; r < D / kMergeDims; ++r) {
                float *mine = merge + warp * 8 * (kMergeDims + 4);
#pragma unroll
                for (int mt = 0; mt < kMergeDims / 16; ++mt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // dim of fragment row g + 8 (i / 2) of tile mt: in order for bf16, else two tiles interleave by 4
                        const int dim = KIND == GDN_BF16 ? 16 * mt + g + 8 * (i >> 1) : 32 * (mt >> 1) + 4 * g + 2 * (mt & 1) + (i >> 1);
                        mine[(2 * q4 + (i & 1)) * (kMergeDims + 4) + dim] = o[r * (kMergeDims / 16) + mt][nt][i] * f[i & 1];
                    }
                __syncthreads();
                for (int idx = tid; idx < 8 * kMergeDims / 4; idx += C::kThreads) {
                    const int head = idx / (kMergeDims / 4), d4 = idx % (kMergeDims / 4) * 4, hh = first + nt * 8 + head;
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    float top = -INFINITY, sum = 0.f;
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const float4 y = *(const float4 *)(merge + (w * 8 + head) * (kMergeDims + 4) + d4);
                        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
                        top = fmaxf(top, ml[w * NT * 8 + nt * 8 + head].x);
                    }
                    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const float2 y = ml[w * NT * 8 + nt * 8 + head];
                        sum += y.y * exp2_fast(y.x - ref);
                    }
                    if (hh >= group) continue;
                    const int d = r * kMergeDims + d4;
                    if (whole) {
                        float inv = sum == 0.f ? 0.f : 1.f / sum;
                        if constexpr (KIND == GDN_E4M3) inv *= a.c.v_scale ? a.c.v_scale[h] : 1.f;
                        const int64_t at = (int64_t)c.b * a.Hq + h * group + hh;
                        if constexpr (KIND == GDN_F32)
                            *(float4 *)((float *)a.o + at * D + d) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
                        else
                            *(uint2 *)((__nv_bfloat16 *)a.o + at * D + d) = make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
                        if (d == 0 && a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
                    } else {
                        const int64_t at = (int64_t)part * NT * 8 + nt * 8 + head;
                        *(float4 *)(ws.o + at * D + d) = x;
                        if (d == 0) ws.ml[at] = make_float2(top, sum);
                    }
                }
                __syncthreads();
            }
        }
    };

    int64_t done = 0;  // of the run, behind `cur`
    if (cur.tile >= cur.tiles) {
        done = cur.tiles + pad - cur.tile;
        cur.tile = cur.tiles - 1;
        cur.next<TILE>(a, rows);
    }
    Cursor ahead = cur;  // the tile whose loads go out next
    int64_t left = n - done;  // of the run from there on
    bool second = false;      // V's half
    Next next;
    if (left > 0) next = find(ahead);
    int feed_slot = 0;
    auto feed = [&]() {
        if (left > 0) {
            issue(feed_slot, next, second ? a.c.v : a.c.k);
            if (second) {
                left -= ahead.tile == ahead.tiles - 1 ? 1 + pad : 1;
                ahead.next<TILE>(a, rows);
                if (left > 0) next = find(ahead);
            }
            second = !second;
        }
        feed_slot = feed_slot == C::kSlots - 1 ? 0 : feed_slot + 1;
        cp_commit();
    };
#pragma unroll 1
    for (int i = 0; i < C::kSlots - 1; ++i) feed();
    // the number of CTAs that a row's tiles [t0, t1) are spread over, if its first is in CTA i
    auto spread = [&](int i, int64_t t1) {  // its last CTA: the last j with floor(total j / ctas) < t1
        const int64_t j = total < (1 << 22) ? ((uint32_t)t1 * (uint32_t)ctas + (uint32_t)total - 1) / (uint32_t)total : (t1 * ctas + total - 1) / total;
        return min(ctas, (int)j) - i;
    };
    if (tid == 32 && !by_row && cta > 0) {  // beside the first loads
        const int64_t row0 = t0 - cur.tile, before = split_at(total, ctas, cta - 1);
        const bool cut = cur.tile > 0 && before <= row0;
        ws.joins[cta - 1] = make_int4(cur.b, cur.row, 2 * (cta - 1) + (before < row0), cut ? spread(cta - 1, row0 + cur.tiles) : 0);
    }
    bool open = false, began_here = false;
    int part = 2 * cta, slot = 0;
    auto arrive = [&]() -> uint32_t {  // at the next half
        cp_wait<C::kSlots - 2>();
        __syncwarp();  // every lane's copies into this slot have landed, and the slot before is read
        feed();
        const uint32_t at = ring + slot * C::kHalf;
        slot = slot == C::kSlots - 1 ? 0 : slot + 1;
        return at;
    };
    while (done < n) {
        if (!open) {
            begin_row(cur);
            open = true;
            began_here = cur.tile == 0;
            part = 2 * cta + (done > 0);
            if (by_row && began_here && tid == 32) {
                const int parts = n - done < cur.tiles ? spread(cta, t0 + done + cur.tiles) : 0;
                ws.joins[cur.b * rows + cur.row] = make_int4(cur.b, cur.row, part, parts);
            }
        }
        const int k_slot = slot;
        const uint32_t kb = arrive(), mask = real[k_slot];
        if (mask) scores(kb, mask);
        const uint32_t vb = arrive();
        if (mask) values(vb);
        const bool row_ends = cur.tile == cur.tiles - 1;
        done += row_ends ? 1 + pad : 1;
        if (row_ends || done == n) {
            end_row(cur, began_here && row_ends, part);
            open = false;
        }
        cur.next<TILE>(a, rows);
    }
}

template <gdn_dtype KIND, int D, int NT>
cudaError_t launch_one(const AttendArgs &a, int64_t most_tiles16, cudaStream_t stream, int *grid_out) {
    using C = Cfg<KIND, D, NT>;
    auto kern = paged_decode_kernel<KIND, D, NT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t most = (most_tiles16 + C::kSub * C::kWarps - 1) / (C::kSub * C::kWarps);  // tiles of a row, were it as long as the table
    const int group = a.Hq / a.c.Hkv, rows = a.c.Hkv * ((group + NT * 8 - 1) / (NT * 8));
    const int64_t wave = (int64_t)kSMs * C::kOcc;
    int64_t ctas = (int64_t)a.B * rows;
    ctas = ctas >= wave || most >= wave ? wave : min(ctas * most, wave);
    *grid_out = (int)ctas;
    kern<<<(unsigned)ctas, C::kThreads, C::kSmem, stream>>>(a, join_by_row((int64_t)a.B * rows, (int)ctas));
    return cudaGetLastError();
}

// Launches the kernel of one storage type; defined in k_paged_decode_{bf16,e4m3,f32}.cu.
template <gdn_dtype KIND>
cudaError_t launch_kind(const AttendArgs &a, int64_t most_tiles16, cudaStream_t stream, int *grid);

template <gdn_dtype KIND>
cudaError_t dispatch(const AttendArgs &a, int64_t most_tiles16, cudaStream_t stream, int *grid) {
    const bool one = pass_heads(a.Hq / a.c.Hkv) == 8;
    switch (a.c.d) {
        case 64: return one ? launch_one<KIND, 64, 1>(a, most_tiles16, stream, grid) : launch_one<KIND, 64, 2>(a, most_tiles16, stream, grid);
        case 128: return one ? launch_one<KIND, 128, 1>(a, most_tiles16, stream, grid) : launch_one<KIND, 128, 2>(a, most_tiles16, stream, grid);
        default: return one ? launch_one<KIND, 256, 1>(a, most_tiles16, stream, grid) : launch_one<KIND, 256, 2>(a, most_tiles16, stream, grid);
    }
}

}  // namespace paged
}  // namespace gdn
