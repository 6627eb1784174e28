// paged_prefill_tc.cuh -- softmax attention of new tokens over the paged cache on tcgen05 tensor cores: the
// kernel template that k_paged_prefill_{bf16,e4m3}.cu instantiate.
//
// S = Q K^T, P = 2^(z - ref), O += P V with z = scale log2(e) S, for tiles of 128 rows and 64 keys; S and O are accumulators in
// tensor memory, P is written over S in 16 bits and read from there as the second product's A operand.  ref follows the running
// maximum of a row lazily: only when z passes it by kSlack is ref raised and O, in tensor memory, rescaled.
//
// One CTA of 16 warps per SM:
//   warps 0-3, 4-7   softmax of the unit's first and second 128 rows, a thread per row.  Each has two S tiles: the tensor core makes
//                    one while the other is worked on, so that neither waits for the other's latency (with one S tile of 128 keys a
//                    tile took 4600 clocks of 2048 in the tensor core);
//   warp 14          copies keys and values into a ring of shared memory, in the 128-byte swizzle, by TMA: one box to a slab and as many tokens
//                    as lie together whatever the page (16 for pages of 16 or 48, 64 for pages of 64).  8-bit values go to a ring of their own,
//                    from which warps 8-11 convert them to f16;
//   warps 8-11       load q.  Pages of which no 8 tokens lie together (pages of 1, say) are copied by them, 16 bytes at a time by cp.async, at
//                    a sixth of the tokens per instruction;
//   warps 12, 13     issue the scores' products of the first and second row tile, warp 15 those with the values.  Between two batches of MMAs
//                    a warp has some tens of instructions to go through, which beside the busy softmax warps take hundreds of clocks,
//                    more than the tensor core has queued: the other warps' batches fill the gap.  (One warp for all of them: a pair of tiles
//                    took 2900 clocks; a warp for each row tile 2100.)
// With 256 dims O fills the tensor memory of two row tiles, and a unit has one.
//
// What bounds it.  8192 bf16 tokens at once (32 query and 8 KV heads of 128): 476 us, 1155 TFLOP/s, 60 % of a large library product; 2048 tokens
// over 131072: 1480 us, 1470 TFLOP/s in some tens of launches, 1690 us, 1290 TFLOP/s where the power limit holds the clock at 1.54 GHz; 8-bit chunks over 16000: 279 us, 1000 TFLOP/s; 256 dims in a
// window of 4096: 331 us, 880 TFLOP/s.  A pair of S tiles takes about 1850 clocks of which the tensor core works 1280 (the scores' product, 64 keys
// wide, reads q and k from shared memory at its full rate, 48 clocks to an MMA instead of 32).  The rest is the chain from a tile's scores over its softmax (950) and
// product to the scores two tiles on, with four waits of 200 to 400 clocks in it; tensor memory holds no third S tile beside two O of 128 dims.  With
// 256 dims it is also the copies: 64 KB for every 64 keys of 128 rows, and a ring of little more than two tiles.
// Tried and not kept: S of 128 keys, one to a row tile (1900 us for the long chunk), one warp issuing both products of a row tile in turn (1880 us and
// 454 us for 256 dims: what it issues next waits behind what the tensor core has not begun), a warp for each row tile's products with the values and three instead of
// four to load q (8192 tokens 552 us), four S tiles and scores 128 keys wide for 256 dims (347 us), polling instead of suspended waits
// (549 us, as the waiting warps take issue slots), keys and values by cp.async where TMA can take them (573 us).
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "paged_prefill.cuh"
#include "tc.cuh"
#include "tmap.cuh"

namespace gdn {
namespace prefill {

using namespace tc;

constexpr int kThreads = 512;
constexpr uint32_t kSlab = 16384;  // [128 rows][128 bytes]
constexpr int kTileKeys = 64;
constexpr int kWords = 16;         // stages whose masks of real keys are kept

template <gdn_dtype KIND, int D>
struct Cfg {
    static constexpr bool kE4M3 = KIND == GDN_E4M3;
    static constexpr int kDims = D < 128 ? D : 128;    // of a ring stage, which has 128 keys: two tiles
    static constexpr int kParts = D / kDims;           // stages of a tile of keys (and of one of values)
    static constexpr int kSlabs = kDims / 64;
    static constexpr uint32_t kStage = kSlabs * kSlab;
    static constexpr int kTiles = D == 256 ? 1 : 2;    // of 128 rows
    static constexpr uint32_t kQTile = D / 64 * kSlab;
    static constexpr int kStages = kE4M3 ? (D == 64 ? 6 : D == 128 ? 3 : 4) : (D == 64 ? 10 : 5);
    static constexpr int kRaw = kE4M3 ? (D == 64 ? 8 : D == 128 ? 4 : 2) : 0;  // stages of 8-bit values on their way
    static constexpr uint32_t kRawStage = 128 * kDims;
    static constexpr uint32_t kSmem = kTiles * kQTile + kStages * kStage + kRaw * kRawStage;  // and Bars behind it
    static constexpr uint32_t kO = 256;                // tensor memory: S at 0, 64 (first row tile), 128, 192 (second), O from here on
    // ref is raised when a score passes it by 2^kSlack; weights are 2^kShift times 2^(z - ref).  bf16 has fp32's range; f16 gets
    // 11 bits for weights down to 2^-25 of the largest, and what sums to less than 2^-36 of it is lost.
    static constexpr float kSlack = kE4M3 ? 4.f : 8.f, kShift = kE4M3 ? 11.f : 0.f;
    static constexpr uint32_t kKindBits = kE4M3 ? 0u : (1u << 7) | (1u << 10);  // instruction descriptor: A and B are f16 or bf16
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void tma_load_4d_at(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void mma_commit_at(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Arrive on `bar` once this thread's copies so far are there.
__device__ __forceinline__ void cp_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void lds128(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint32_t f16_of_e4m3(uint32_t x) {  // both values of the low half: exact
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)x));
    return r;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Four K steps of D[tmem] (+)= A B, issued by the lane with `issue`: both operands K-major in shared memory, or A in tensor memory and B
// MN-major.  One block of predicated instructions with their descriptors counted up in it: with a branch and descriptors of its own for
// each, the MMAs of a tile took longer to issue, beside the other warps of the scheduler, than to run.
__device__ __forceinline__ void mma4_ss(bool issue, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n"
        ".reg .pred p, q, t;\n"
        ".reg .b64 a, b;\n"
        "setp.ne.b32 q, %5, 0;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "setp.eq.b32 t, 0, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        "add.s64 a, %1, 2;\n"
        "add.s64 b, %2, 2;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        "add.s64 a, %1, 4;\n"
        "add.s64 b, %2, 4;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        "add.s64 a, %1, 6;\n"
        "add.s64 b, %2, 6;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        "}\n" ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate), "r"((uint32_t)issue)
        : "memory");
}
__device__ __forceinline__ void mma4_ts(bool issue, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n"
        ".reg .pred p, q, t;\n"
        ".reg .b64 b;\n"
        ".reg .b32 a;\n"
        "setp.ne.b32 q, %5, 0;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "setp.eq.b32 t, 0, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
        "add.s32 a, %1, 8;\n"
        "add.s64 b, %2, 128;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
        "add.s32 a, %1, 16;\n"
        "add.s64 b, %2, 256;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
        "add.s32 a, %1, 24;\n"
        "add.s64 b, %2, 384;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
        "}\n" ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate), "r"((uint32_t)issue)
        : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "elect.sync _|p, 0xffffffff;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n" : "=r"(r));
    return r != 0;
}
template <int N> __device__ __forceinline__ void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_less() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
// Waits on mbarriers end after kWaitLimitNs, or soon after another thread's did.  A try suspends the warp for up to a millisecond, so that
// those that wait leave the issue slots to the others.
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000000;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n" : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}
struct Waiter {
    volatile int *gave_up;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity, uint64_t limit_ns = kWaitLimitNs) const {
        if (try_wait(bar, parity)) return true;
        const uint64_t since = globaltimer();
#pragma unroll 1
        while (!try_wait(bar, parity))
            if (*gave_up || globaltimer() - since > limit_ns) {
                *gave_up = 1;
                return false;
            }
        return true;
    }
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const { return (*this)(smem_addr(bar), parity); }
};

struct Bars {
    static constexpr int kMaxStages = 10;
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t raw_full[8], raw_empty[8];  // of 8-bit stages
    uint64_t q_full[2], q_empty[2];  // of a row tile
    uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // of a group's two S tiles
    uint64_t joint[2], drain[3];    // joint: a group's votes
    uint32_t words[kWords][4];      // real keys of a stage
    int8_t lift[3][256];            // e4m3: exponents that q's rows were lifted by, of three units by turns: q of one is loaded while the next one's
                                    // first scores are made and the softmax may still begin the one before
    int vote[2][3];                 // of a group, by turns
    int skip[2][2];                 // the group has added this tile's P V itself
    int gave_up;
    uint32_t tmem;
    uint64_t never;                 // self-test: nothing arrives
};

static_assert(sizeof(Bars) <= 3 * 1024, "shared memory");

// A warp's waits succeed or fail for all of its lanes.
template <typename Bar> __device__ __forceinline__ bool warp_wait(const Waiter &wait, Bar bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(bar, parity));
}
// One arrival for a warp, after what all of its lanes did: 32 of them on one address take as many turns.
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}
// Whether any thread of a group says x, in `any`; false: a wait ran out.  `turn` counts the group's votes.
__device__ __forceinline__ bool group_any(const Waiter &wait, Bars &bars, int group, int &turn, bool x, bool &any) {
    if (x) *(volatile int *)&bars.vote[group][turn % 3] = 1;
    mbar_arrive(&bars.joint[group]);
    const bool ok = warp_wait(wait, &bars.joint[group], turn & 1);
    any = *(volatile int *)&bars.vote[group][turn % 3];
    // the turn before has been read by all who came here, and nobody gets to the one after next before this thread does
    if ((threadIdx.x & 127) == 0) *(volatile int *)&bars.vote[group][(turn + 2) % 3] = 0;
    ++turn;
    return ok;
}

// Four lanes' 16-byte pieces of four rows change places: lane q of the four gets piece q of each of their rows.
__device__ __forceinline__ void transpose4(uint4 (&a)[4], int lane) {
    auto swap = [&](uint4 x, int with) {
        return make_uint4(__shfl_xor_sync(0xffffffffu, x.x, with), __shfl_xor_sync(0xffffffffu, x.y, with), __shfl_xor_sync(0xffffffffu, x.z, with),
                          __shfl_xor_sync(0xffffffffu, x.w, with));
    };
    auto pick = [](bool first, const uint4 &x, const uint4 &y) { return make_uint4(first ? x.x : y.x, first ? x.y : y.y, first ? x.z : y.z, first ? x.w : y.w); };
    const bool odd = lane & 1, high = lane & 2;
    uint4 x = swap(pick(odd, a[0], a[1]), 1), y = swap(pick(odd, a[2], a[3]), 1);
    a[0] = pick(odd, x, a[0]), a[1] = pick(odd, a[1], x), a[2] = pick(odd, y, a[2]), a[3] = pick(odd, a[3], y);
    x = swap(pick(high, a[0], a[2]), 2), y = swap(pick(high, a[1], a[3]), 2);
    a[0] = pick(high, x, a[0]), a[2] = pick(high, a[2], x), a[1] = pick(high, y, a[1]), a[3] = pick(high, a[3], y);
}

// Bits of keys kb + 32 part .. inside [lo, hi].
__device__ __forceinline__ uint32_t range_bits(int part, int kb, int lo, int hi) {
    const int l = lo - kb - 32 * part, h = hi - kb - 32 * part;
    if (l > 31 || h < 0) return 0;
    return (l <= 0 ? ~0u : ~0u << l) & (h >= 31 ? ~0u : (2u << h) - 1);
}

// Whether half of a key's values in a ring stage are finite: thread r of a group has key r % 64 of a tile's, and its first or second half.
// Values that only some rows attend to have to be; those of a key that none does (`live` false) become zeros.
template <gdn_dtype KIND, int D>
__device__ __noinline__ bool all_numbers(uint32_t stage, int key0, int r, bool live) {
    using C = Cfg<KIND, D>;
    uint32_t bad = 0;
#pragma unroll 4
    for (int e = 0; e < C::kDims / 16; ++e) {
        const int piece = (r >> 6) * (C::kDims / 16) + e;
        const uint32_t at = stage + piece / 8 * kSlab + sw128_offset(key0 + (r & 63), piece % 8 * 8);
        if (live) {
            uint32_t x[4];
            lds128(x, at);
#pragma unroll
            for (int w = 0; w < 4; ++w)
                bad |= C::kE4M3 ? ((x[w] & 0x7c007c00u) + 0x04000400u) & 0x80008000u : ((x[w] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
        } else {
            sts128(at, 0, 0, 0, 0);
        }
    }
    if (!live) fence_async_smem();
    return bad == 0;
}

// O += P V of one tile for a group's rows without the tensor core, which multiplies a masked weight of 0 with what it masks: a tile of
// values with an infinity or NaN that some of the rows do not attend to.  P is in tensor memory, a row's thread reads its own; the
// values are rows `key0` on of the stages from stage0 on.
template <gdn_dtype KIND, int D>
__device__ __noinline__ void add_masked(uint32_t t_p, uint32_t t_o, const uint8_t *ring, int stage0, int key0, uint32_t bits0, uint32_t bits1, bool first) {
    using C = Cfg<KIND, D>;
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
        float o[32];
        tmem_ld32(t_o + 32 * c, o);
        tmem_ld_wait();
        if (first)
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.f;
        const int d0 = 32 * c;
        const uint32_t stage = smem_addr(ring) + (uint32_t)((stage0 + d0 / C::kDims) % C::kStages) * C::kStage + d0 % C::kDims / 64 * kSlab;
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
            const uint32_t bits = part ? bits1 : bits0;
            float p[16];
            tmem_ld16(t_p + 16 * part, p);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                if (!(bits >> k & 1)) continue;
                const uint32_t w = __float_as_uint(p[k / 2]);
                float x;
                if constexpr (C::kE4M3) x = __half2float(__ushort_as_half((unsigned short)(k & 1 ? w >> 16 : w & 0xffff)));
                else x = __uint_as_float(k & 1 ? w & 0xffff0000u : w << 16);
                const int key = key0 + 32 * part + k;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t v[4];
                    lds128(v, stage + sw128_offset(key, d0 % 64 + 8 * e));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float lo, hi;
                        if constexpr (C::kE4M3) {
                            lo = __half2float(__ushort_as_half((unsigned short)(v[i] & 0xffff)));
                            hi = __half2float(__ushort_as_half((unsigned short)(v[i] >> 16)));
                        } else {
                            lo = __uint_as_float(v[i] << 16);
                            hi = __uint_as_float(v[i] & 0xffff0000u);
                        }
                        o[8 * e + 2 * i] += x * lo;
                        o[8 * e + 2 * i + 1] += x * hi;
                    }
                }
            }
            __syncwarp();
        }
        tmem_st32(t_o + 32 * c, o);
        tmem_st_wait();
    }
}

// TMA: keys and values come by TMA, in boxes of `box` tokens of one page.  LOST: the self-test of waits, instances of its own, as the same few
// instructions in the others take 2 % of a call.
template <gdn_dtype KIND, int D, bool TMA, bool LOST>
__global__ void __launch_bounds__(kThreads, 1) prefill_tc_kernel(PrefillArgs a, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, int box) {
    using C = Cfg<KIND, D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars &bars = *reinterpret_cast<Bars *>(smem + C::kSmem);
    uint8_t *const q_smem = smem, *const ring = smem + C::kTiles * C::kQTile;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warpgroup = warp >> 2;
    const int group = (int)a.group.by, room = a.max_pages * a.c.page;
    const Waiter wait = {&bars.gave_up};
    View view;
    layout(a.ws, a.B, a.n, a.Hq, a.c.Hkv, D, 128 * C::kTiles, gridDim.x, &view);

    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&bars.full[i], C::kE4M3 ? 4 : TMA ? 1 : 128 + 4);
            mbar_init(&bars.empty[i], C::kTiles);
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(&bars.raw_full[i], 1);
            mbar_init(&bars.raw_empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.q_full[i], 128);
            mbar_init(&bars.q_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            for (int j = 0; j < 2; ++j) {
                mbar_init(&bars.s_full[i][j], 1);
                mbar_init(&bars.p_full[i][j], 4);
                mbar_init(&bars.pv_done[i][j], 1);
                bars.skip[i][j] = 0;
            }
            mbar_init(&bars.joint[i], 128);
            for (int j = 0; j < 3; ++j) bars.vote[i][j] = 0;
        }
        for (int i = 0; i < 3; ++i) mbar_init(&bars.drain[i], 1);
        if constexpr (LOST) mbar_init(&bars.never, 1);
        bars.gave_up = 0;
        fence_mbar_init();
    }
    if (warp == 12) tmem_alloc<512>(&bars.tmem);
    pdl_wait();  // the plan
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;
    Walk walk;
    walk.start(view, blockIdx.x);
    auto never = [&] { return __all_sync(0xffffffffu, wait(smem_addr(&bars.never), 0, a.lost_ns)) != 0; };
    if (smem_addr(smem) & 1023u) walk.at.x = -1, bars.gave_up = 1;  // the swizzle needs aligned tiles, which shared memory without static parts is

    if (warpgroup == 2) {
        // ---- copies ---------------------------------------------------------------------------------------
        regs_less<80>();
        const int pt = tid - 256, pw = pt >> 5;
        constexpr int kChunks = C::kDims * (C::kE4M3 ? 1 : 2) / 16, kAtOnce = 32 / kChunks, kSteps = 32 / kAtOnce;  // 16-byte pieces of a row; rows per copy
        const int chunk = lane % kChunks, sub = lane / kChunks;
        int stage_in = 0, stage_out = 0, tiles = 0;  // stages issued, stages converted (e4m3)
        int units = 0, units1 = 0;                    // units, and those with a second row tile
        bool ok = true;
        const uint32_t ring_at = smem_addr(ring), raw_at = smem_addr(ring + C::kStages * C::kStage);
        auto free_stage = [&](int n) { return n < C::kStages || warp_wait(wait, &bars.empty[n % C::kStages], (n / C::kStages - 1) & 1); };
        // e4m3: 8-bit values of the oldest stage become f16; a thread reads what it copied itself
        auto convert = [&] {
            const int n = stage_out;
            if (TMA && !warp_wait(wait, &bars.raw_full[n % (C::kRaw ? C::kRaw : 1)], n / (C::kRaw ? C::kRaw : 1) & 1)) return false;
            if (!free_stage(n)) return false;
            const uint32_t from = raw_at + n % (C::kRaw ? C::kRaw : 1) * C::kRawStage, to = ring_at + n % C::kStages * C::kStage;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int key = 32 * pw + i * kAtOnce + sub;
                uint32_t x[4];
                lds128(x, from + key * C::kDims + 16 * chunk);
                const uint32_t at = to + chunk / 4 * kSlab;
                sts128(at + sw128_offset(key, chunk % 4 * 16), f16_of_e4m3(x[0]), f16_of_e4m3(x[0] >> 16), f16_of_e4m3(x[1]), f16_of_e4m3(x[1] >> 16));
                sts128(at + sw128_offset(key, chunk % 4 * 16 + 8), f16_of_e4m3(x[2]), f16_of_e4m3(x[2] >> 16), f16_of_e4m3(x[3]), f16_of_e4m3(x[3] >> 16));
            }
            fence_async_smem();
            warp_arrive(&bars.full[n % C::kStages], lane);
            if (TMA && lane == 0) mbar_arrive(&bars.raw_empty[n % (C::kRaw ? C::kRaw : 1)]);
            ++stage_out;
            return true;
        };
        auto copy = [&](const void *base, int part, int64_t row, bool real) {  // one stage; row: this lane's key's offset in elements
            const uint8_t *src = (const uint8_t *)base + part * C::kDims * (C::kE4M3 ? 1 : 2) + 16 * chunk;
            if (!C::kE4M3 && !free_stage(stage_in)) return false;
            const uint32_t dst = C::kE4M3 ? raw_at + stage_in % (C::kRaw ? C::kRaw : 1) * C::kRawStage : ring_at + stage_in % C::kStages * C::kStage + chunk / 8 * kSlab;
#pragma unroll 4
            for (int i = 0; i < kSteps; ++i) {
                const int from = i * kAtOnce + sub, key = 32 * pw + from;
                const int64_t off = __shfl_sync(0xffffffffu, row, from);
                const bool there = __shfl_sync(0xffffffffu, (int)real, from);
                if constexpr (C::kE4M3) cp16(dst + key * C::kDims + 16 * chunk, src + off, there);
                else cp16(dst + sw128_offset(key, chunk % 8 * 8), src + off * 2, there);
            }
            if constexpr (C::kE4M3) {
                cp_commit();
                if (++stage_in - stage_out < C::kRaw) return true;
                cp_wait<(C::kRaw > 0 ? C::kRaw - 1 : 0)>();
                return convert();
            } else {
                uint64_t *bar = &bars.full[stage_in++ % C::kStages];
                cp_arrive(bar);
                if (lane == 0) mbar_arrive(bar);  // and the mask of real keys
                return true;
            }
        };
        auto settle = [&] {  // e4m3: everything issued has been converted
            if constexpr (C::kE4M3 && !TMA) {
                cp_wait<0>();
                while (stage_out < stage_in)
                    if (!convert()) return false;
            }
            return true;
        };
        // the unit's rows of q, a tile of 128 after the other; rows behind the last are zeros.  A row is (token, head of the group): a lane
        // counts its own up instead of dividing for each, which made a unit's beginning 6 us longer
        constexpr int kLanes = D / 8, kRowStep = 4 * (32 / kLanes);  // 16 bytes to a lane; rows that the warps have at a time
        const int piece = lane % kLanes, step_token = a.group.quotient(kRowStep), step_head = kRowStep - step_token * group;
        const int64_t step = step_token * a.q_tok + step_head * a.q_head, carry = a.q_tok - group * a.q_head;
        auto load_q = [&](const Unit &u, int h) {
            if (!settle()) return false;
            int r = pw * (32 / kLanes) + lane / kLanes, head;
            const int token = u.first + a.group.quotient(u.row + r, head);
            const uint16_t *src = (const uint16_t *)a.q + token * a.q_tok + (h * group + head) * a.q_head + 8 * piece;
#pragma unroll 1
            for (int m = 0; m < C::kTiles && 128 * m < u.rows; ++m) {
                const int uses = m ? units1 : units;
                if (uses > 0 && !warp_wait(wait, &bars.q_empty[m], (uses - 1) & 1)) return false;
                const uint32_t dst = smem_addr(q_smem) + m * C::kQTile + piece / 8 * kSlab;
                constexpr int kBatch = C::kE4M3 ? 8 : 4;  // rows of a lane whose loads are on their way together
#pragma unroll 1
                for (int i = 0; i < 128 / kRowStep; i += kBatch) {
                    uint4 x[C::kE4M3 ? kBatch : 1];
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        const int row = r + j * kRowStep;
                        const bool there = row < u.rows;
                        if constexpr (C::kE4M3) x[j] = there ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0, 0, 0, 0);
                        else cp16(dst + sw128_offset(row & 127, piece % 8 * 8), there ? src : (const uint16_t *)a.q, there);
                        src += step;
                        if ((head += step_head) >= group) head -= group, src += carry;
                    }
                    if constexpr (C::kE4M3) {
                        // f16 of q times a power of two that takes the row's largest to 2^14 or so: 8 bits of any value down to 2^-30 of it,
                        // and what it loses below is lost in the fp32 sum too
#pragma unroll
                        for (int j = 0; j < kBatch; ++j) {
                            const int row = r + j * kRowStep;
                            const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
                            uint32_t most = 0;
#pragma unroll
                            for (int k = 0; k < 4; ++k) most = max(most, max(w[k] & 0x7fffu, w[k] >> 16 & 0x7fffu));
#pragma unroll
                            for (int off = kLanes / 2; off; off >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
                            const int e = min((int)(most >> 7), 254), lift = min(141 - e, 126);
                            const float f = __uint_as_float((uint32_t)(127 + lift) << 23);
                            uint32_t y[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) y[k] = pack_f16x2(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xffff0000u) * f);
                            sts128(dst + sw128_offset(row & 127, piece % 8 * 8), y[0], y[1], y[2], y[3]);
                            if (piece == 0) bars.lift[uses % 3][row] = (int8_t)lift;
                        }
                    }
                    r += kBatch * kRowStep;
                }
                if constexpr (C::kE4M3) {
                    fence_async_smem();
                    mbar_arrive(&bars.q_full[m]);
                } else {
                    cp_arrive(&bars.q_full[m]);
                }
            }
            ++units;
            units1 += u.rows > 128;
            return true;
        };
        while (ok && walk.next()) {
            const Unit u = walk.u;
            if (walk.t0 == walk.t1) continue;
            const int n = (walk.t1 - walk.t0 + 1) / 2;
            if constexpr (TMA) {
                // bf16: q is all there is to do; e4m3: the unit's stages too, q after the first keys
                for (int i = 0; ok && i < (C::kE4M3 ? 2 * C::kParts * n : 1); ++i) {
                    if (i == (C::kE4M3 ? C::kParts : 0) && !(ok = load_q(u, walk.h))) break;
                    if constexpr (C::kE4M3) ok = convert();
                }
                continue;
            }
            const int32_t *table = a.table + u.b * a.table_stride;
            const int lo = u.lo, begin = u.key + kTileKeys * walk.t0, end = min(u.hi, u.key + kTileKeys * walk.t1 - 1);
            auto entry = [&](int key, int &cell) {  // the key's page, -1 where it has none
                const int page = a.page.quotient(key, cell);
                return key >= lo && key <= end ? table[page] : -1;
            };
            int cell_next, page_next = entry(begin + pt, cell_next);
            for (int t = 0; ok && t < n; ++t) {
                if (LOST && tiles == 1 && !(ok = never())) break;
                const int page = page_next, cell = cell_next;
                if (t + 1 < n) page_next = entry(begin + 128 * (t + 1) + pt, cell_next);
                const bool real = page >= 0 && page < a.c.pages;
                const int64_t row = real ? page * a.c.stride_page + cell * a.c.stride_token + walk.h * a.c.stride_head : 0;
                const uint32_t word = __ballot_sync(0xffffffffu, real);
                if (lane == 0) bars.words[tiles % kWords][pw] = word;
                ++tiles;
#pragma unroll 1
                for (int part = 0; ok && part < 2 * C::kParts; ++part) {
                    if (t == 0 && part == C::kParts && !(ok = load_q(u, walk.h))) break;
                    ok = copy(part < C::kParts ? a.c.k : a.c.v, part % C::kParts, row, real);
                }
            }
        }
        if (ok) settle();
        cp_commit();
        cp_wait<0>();
    } else if (warpgroup == 3) {
        // ---- products -------------------------------------------------------------------------------------
        regs_less<48>();
        if (warp < 12 + C::kTiles || warp == 15) {
            // the whole warp goes along, so that descriptors are uniform values, and one lane issues: with one lane in a branch of
            // its own an MMA took four times as long to issue as to run
            const bool leader = elect_one();
            constexpr uint32_t kBase = (1u << 4) | C::kKindBits | (128u >> 4 << 24);
            constexpr uint32_t id_qk = kBase | ((uint32_t)kTileKeys >> 3 << 17), id_pv = kBase | (1u << 16) | ((uint32_t)C::kDims >> 3 << 17);
            const uint64_t q_desc = kmajor_desc(smem_addr(q_smem), 0, kSlab), k_desc = kmajor_desc(smem_addr(ring), 0, kSlab), v_desc = mnmajor_desc(smem_addr(ring), 0, kSlab);
            const uint32_t full_at = smem_addr(&bars.full), empty_at = smem_addr(&bars.empty), s_at = smem_addr(&bars.s_full), p_at = smem_addr(&bars.p_full),
                           pv_at = smem_addr(&bars.pv_done);
            int units = 0, done[2] = {0, 0};  // units, and tiles of a row tile, before this piece; tiles take a row tile's two places by turns
            bool ok = true;
            // copies by cp.async and the tensor core see shared memory through different proxies
            auto ready = [&](uint32_t bar, uint32_t parity) {
                if (!warp_wait(wait, bar, parity)) return false;
                if constexpr (!C::kE4M3 && !TMA) fence_async_smem();
                return true;
            };
            auto commit = [&](uint32_t bar) {
                if (leader) mma_commit_at(bar);
            };
            // a place in the ring: the first stage of a tile pair's keys or values
            struct Place {
                int slot;
                uint32_t parity;
                __device__ __forceinline__ void step(int by) {
                    slot += by;
                    if (slot >= C::kStages) slot -= C::kStages, parity ^= 1;
                }
            };
            auto stages_ready = [&](Place at) {
                bool there = ready(full_at + 8 * at.slot, at.parity);
                if constexpr (C::kParts == 2) {
                    at.step(1);
                    there = there && ready(full_at + 8 * at.slot, at.parity);
                }
                return there;
            };
            auto release_stages = [&](Place at, int times) {
#pragma unroll
                for (int part = 0; part < C::kParts; ++part) {
                    for (int i = 0; i < times; ++i) commit(empty_at + 8 * at.slot);
                    at.step(1);
                }
            };
            if (warp < 15) {
                const int m = warp - 12;
                Place at = {0, 0};
                while (ok && walk.next()) {
                    const int n = walk.t1 - walk.t0;
                    if (n == 0) continue;
                    if (m == 1 && walk.u.rows <= 128) {
                        // Nothing to do but to say so, stage by stage.  A wait tells a phase from the one before it only, copies arrive in any
                        // order, and a stage has keys and values by turns: so the values of the units before have to have come, and
                        // those of this one are waited for like the keys.
                        if (done[0] > 0 && !(ok = warp_wait(wait, pv_at + 16 + 8 * ((done[0] - 1) & 1), (done[0] - 1) >> 1 & 1))) break;
                        for (int i = 0; i < (n + 1) / 2 * 2; ++i) {
                            if (!(ok = warp_wait(wait, full_at + 8 * at.slot, at.parity))) break;
                            if (leader) mbar_arrive(&bars.empty[at.slot]);
                            at.step(1);
                        }
                        continue;
                    }
#pragma unroll 1
                    for (int i = 0; i < n; ++i) {
                        const int tile = done[0] + i, place = tile & 1, half = i & 1;
                        // the weights that lie over the scores of two tiles before have been used; before the wait for keys, whose stage may have
                        // held the values of two pairs before: of those it is known now that they had come
                        if (tile >= 2 && !(ok = warp_wait(wait, pv_at + 16 * m + 8 * place, ((tile >> 1) - 1) & 1))) break;
                        if (!half && !(ok = stages_ready(at))) break;
                        if (i == 0) {
                            if (!(ok = warp_wait(wait, smem_addr(&bars.q_full[m]), units & 1))) break;
                            if constexpr (!C::kE4M3) fence_async_smem();  // q is copied by cp.async
                        }
                        tc_fence_after();
                        Place from = at;
#pragma unroll
                        for (int part = 0; part < C::kParts; ++part) {
                            const uint64_t k = k_desc + (uint32_t)(from.slot * (int)(C::kStage >> 4) + half * (int)(kSlab >> 5));
#pragma unroll
                            for (int slab = 0; slab < C::kSlabs; ++slab)
                                mma4_ss(leader, tmem + 128 * m + 64 * place, q_desc + ((m * C::kQTile + (part * C::kSlabs + slab) * kSlab) >> 4), k + (slab * kSlab >> 4), id_qk, part + slab > 0);
                            from.step(1);
                        }
                        commit(s_at + 16 * m + 8 * place);
                        if (half || i == n - 1) {
                            release_stages(at, 1);
                            at.step(2 * C::kParts);
                        }
                    }
                    commit(smem_addr(&bars.q_empty[m]));
                    done[0] += n;
                    ++units;
                }
            } else {
                Place at = {C::kParts, 0};
                while (ok && walk.next()) {
                    const int n = walk.t1 - walk.t0, row_tiles = walk.u.rows > 128 ? 2 : 1;
                    if (n == 0) continue;
#pragma unroll 1
                    for (int i = 0; ok && i < n; ++i) {
                        const int half = i & 1;
                        if (!half && !(ok = stages_ready(at))) break;
#pragma unroll
                        for (int m = 0; m < C::kTiles; ++m) {
                            if (m >= row_tiles) break;
                            const int tile = done[m] + i, place = tile & 1;
                            if (!(ok = warp_wait(wait, p_at + 16 * m + 8 * place, tile >> 1 & 1))) break;
                            tc_fence_after();
                            if (!*(volatile int *)&bars.skip[m][place]) {
                                Place from = at;
#pragma unroll
                                for (int part = 0; part < C::kParts; ++part) {
                                    mma4_ts(leader, tmem + C::kO + m * D + part * C::kDims, tmem + 128 * m + 64 * place, v_desc + (uint32_t)(from.slot * (int)(C::kStage >> 4) + half * (int)(kSlab >> 5)), id_pv, i > 0);
                                    from.step(1);
                                }
                            }
                            commit(pv_at + 16 * m + 8 * place);
                        }
                        if (half || i == n - 1) {
                            release_stages(at, row_tiles);  // the other row tile's warp says the rest
                            at.step(2 * C::kParts);
                        }
                    }
                    done[0] += n;
                    if (row_tiles == 2) done[1] += n;
                }
            }
            commit(smem_addr(&bars.drain[warp == 15 ? 2 : warp - 12]));
            mbar_wait(&bars.drain[warp == 15 ? 2 : warp - 12], 0);
        }
        if (TMA && warp == 14) {
            // ---- copies by TMA ----------------------------------------------------------------------------
            constexpr int kRing = C::kE4M3 ? C::kRaw : C::kStages;
            constexpr uint32_t kBytes = C::kE4M3 ? C::kRawStage : C::kStage;
            const int boxes = 128 / box, shift = 31 - __clz(box);
            const uint32_t ring_at = smem_addr(ring) + (C::kE4M3 ? C::kStages * C::kStage : 0);
            int slot = 0, tiles = 0;
            uint32_t turn = 0;
            bool ok = true;
            while (ok && walk.next()) {
                const Unit u = walk.u;
                if (walk.t0 == walk.t1) continue;
                const int32_t *table = a.table + u.b * a.table_stride;
                const int lo = u.lo, begin = u.key + kTileKeys * walk.t0, end = min(u.hi, u.key + kTileKeys * walk.t1 - 1), n = (walk.t1 - walk.t0 + 1) / 2;
                // lane l has the l-th box of 128 keys
                auto entry = [&](int key, int &cell) {
                    const int page = a.page.quotient(key, cell);
                    return lane < boxes && key + box > lo && key <= end ? table[page] : -1;
                };
                int cell_next, page_next = entry(begin + lane * box, cell_next);
                for (int t = 0; ok && t < n; ++t) {
                    if (LOST && tiles == 1 && !(ok = never())) break;
                    const int cell = cell_next, page = page_next >= 0 && page_next < a.c.pages ? page_next : -1;  // outside the pool TMA fills with zeros
                    if (t + 1 < n) page_next = entry(begin + 128 * (t + 1) + lane * box, cell_next);
                    const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t word = __ballot_sync(0xffffffffu, there >> ((32 * c + lane) >> shift) & 1) & range_bits(c, begin + 128 * t, lo, end);
                        if (lane == 0) bars.words[tiles % kWords][c] = word;
                    }
                    ++tiles;
#pragma unroll 1
                    for (int part = 0; part < 2 * C::kParts; ++part) {
                        uint64_t *bar = C::kE4M3 ? &bars.raw_full[slot] : &bars.full[slot];
                        if (turn > 0 && !(ok = warp_wait(wait, C::kE4M3 ? &bars.raw_empty[slot] : &bars.empty[slot], (turn - 1) & 1))) break;
                        if (lane == 0) mbar_arrive_expect_tx(bar, kBytes);
                        __syncwarp();
                        if (lane < boxes) {
                            const CUtensorMap *map = part < C::kParts ? &k_map : &v_map;
                            const int x = part % C::kParts * C::kDims;
                            const uint32_t dst = ring_at + slot * kBytes + lane * box * (C::kE4M3 ? C::kDims : 128);
#pragma unroll
                            for (int slab = 0; slab < (C::kE4M3 ? 1 : C::kSlabs); ++slab) tma_load_4d_at(dst + slab * kSlab, map, x + 64 * slab, cell, walk.h, page, smem_addr(bar));
                        }
                        if (++slot == kRing) slot = 0, ++turn;
                    }
                }
            }
            // what was asked for has to arrive before the memory may go, whether or not a wait has run out
            for (int i = 0; i < kRing; ++i) {
                const int s = (slot + i) % kRing;
                const uint32_t last = turn - (s >= slot);  // of the slot's turns
                if (turn > 0 || s < slot) mbar_wait(C::kE4M3 ? &bars.raw_full[s] : &bars.full[s], last & 1);
            }
        }
        __syncwarp();
    } else {
        // ---- softmax --------------------------------------------------------------------------------------
        regs_more<192>();
        const int m = warpgroup, r = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // tensor memory lanes of this warp
        const float log2e = 1.4426950408889634f;
        int stage = 0, units = 0, loads = 0, done = 0, votes = 0;  // before this piece: ring stages, units, masks of keys, tiles
        bool ok = true;
        while (ok && walk.next()) {
            const Unit u = walk.u;
            const int n = walk.t1 - walk.t0;
            const bool two = u.rows > 128;
            if (m == 1 && !two) {  // the first group has all of it
                stage += 2 * C::kParts * ((n + 1) / 2);
                loads += (n + 1) / 2;
                continue;
            }
            const int rows = min(128, u.rows - 128 * m);
            int head;
            const int token = u.first + a.group.quotient(u.row + 128 * m + min(r, rows - 1), head);
            const Reach mine = reach_of(token + u.shift, a.window, room);
            // keys that all rows attend to
            const int all_lo = m ? u.all_lo[1] : u.all_lo[0], all_hi = m ? u.all_hi[1] : u.all_hi[0];
            const uint32_t t_o = tmem + lanes + C::kO + m * D;
            float ref = -INFINITY, sum = 0.f, zs = a.scale * log2e;
            if (a.c.k_scale) zs *= a.c.k_scale[walk.h];
            for (int i = 0; ok && i < n; ++i) {
                const int place = (done + i) & 1;
                const uint32_t t_s = tmem + lanes + 128 * m + 64 * place;
                // the product of tile j has ended; tile i's scores say so for j <= i - 2
                auto ended = [&](int j) { return warp_wait(wait, &bars.pv_done[m][(done + j) & 1], (done + j) >> 1 & 1); };
                if (!(ok = warp_wait(wait, &bars.s_full[m][place], (done + i) >> 1 & 1))) break;
                tc_fence_after();
                if (C::kE4M3 && i == 0) zs *= __uint_as_float((uint32_t)(127 - bars.lift[units % 3][128 * m + r]) << 23);
                float s[2][32];
                tmem_ld32(t_s, s[0]);
                tmem_ld32(t_s + 32, s[1]);
                const int kb = u.key + kTileKeys * (walk.t0 + i);
                uint32_t bits[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) bits[c] = bars.words[(loads + (i >> 1)) % kWords][2 * (i & 1) + c];
                const bool edge = kb < all_lo || kb + kTileKeys - 1 > all_hi || (bits[0] & bits[1]) != ~0u;
                tmem_ld_wait();
                float f = zs;
                if (__builtin_expect(!(zs > 0.f), 0)) {  // the maximum below is that of s
                    f = 1.f;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int j = 0; j < 32; ++j) s[c][j] *= zs;
                }
                if (__builtin_expect(edge, 0)) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        bits[c] &= range_bits(c, kb, mine.lo, mine.hi);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(bits[c] >> j & 1)) s[c][j] = -INFINITY;
                    }
                }
                float mx[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) mx[j] = fmaxf(s[j / 2][j % 2 * 16], s[j / 2][j % 2 * 16 + 1]);
#pragma unroll
                for (int k = 2; k < 16; k += 2)
#pragma unroll
                    for (int j = 0; j < 4; ++j) mx[j] = fmaxf(fmaxf(mx[j], s[j / 2][j % 2 * 16 + k]), s[j / 2][j % 2 * 16 + k + 1]);
                const float most = f * fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                const bool raise = most > ref + C::kSlack || (ref == -INFINITY && most > -INFINITY);
                if (__any_sync(0xffffffffu, raise)) {
                    float lower = 1.f;
                    if (raise) {
                        lower = ex2(ref - most);
                        ref = most;
                        sum *= lower;
                    }
                    if (i > 0) {
                        if (!(ok = ended(i - 1))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            float o[16];
                            tmem_ld16(t_o + 16 * c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] *= lower;
                            tmem_st16(t_o + 16 * c, o);
                        }
                        tmem_st_wait();
                    }
                }
                const float base = ref == -INFINITY ? 0.f : ref - C::kShift;
                // two at once: a product and a sum to each instruction
                const uint64_t f2 = pair(f, f), base2 = pair(-base, -base);
                uint64_t part[2] = {0, 0};
                float p[32];
#pragma unroll
                for (int j = 0; j < 64; j += 2) {
                    float x, y;
                    unpair(fma2(pair(s[j / 32][j % 32], s[j / 32][j % 32 + 1]), f2, base2), x, y);
                    x = ex2(x), y = ex2(y);
                    part[j / 2 % 2] = add2(part[j / 2 % 2], pair(x, y));
                    p[j / 2] = __uint_as_float(C::kE4M3 ? pack_f16x2(x, y) : pack_bf16x2(x, y));
                }
                tmem_st32(t_s, p);
                float even, odd;
                unpair(add2(part[0], part[1]), even, odd);
                sum += even + odd;
                tmem_st_wait();
                if (__builtin_expect(edge, 0)) {
                    const int at = stage + 2 * C::kParts * (i >> 1) + C::kParts;
                    bool numbers = true;
                    const bool live = bars.words[(loads + (i >> 1)) % kWords][2 * (i & 1) + (r >> 5 & 1)] >> (r & 31) & 1;
                    for (int k = 0; ok && k < C::kParts; ++k) {
                        ok = warp_wait(wait, &bars.full[(at + k) % C::kStages], (at + k) / C::kStages & 1);
                        numbers = numbers && all_numbers<KIND, D>(smem_addr(ring) + (uint32_t)((at + k) % C::kStages) * C::kStage, (i & 1) * kTileKeys, r, live);
                    }
                    bool tainted = false;
                    if (!(ok = ok && group_any(wait, bars, m, votes, !numbers, tainted))) break;
                    if (tainted) {
                        if (!(ok = i == 0 || ended(i - 1))) break;
                        tc_fence_after();
                        add_masked<KIND, D>(t_s, t_o, ring, at, (i & 1) * kTileKeys, bits[0], bits[1], i == 0);
                    }
                    if (r == 0) bars.skip[m][place] = tainted;
                } else if (r == 0) {
                    bars.skip[m][place] = 0;
                }
                tc_fence_before();
                warp_arrive(&bars.p_full[m][place], lane);
            }
            if (!ok) break;
            if (n > 0) {
                if (!(ok = warp_wait(wait, &bars.pv_done[m][(done + n - 1) & 1], (done + n - 1) >> 1 & 1))) break;
                tc_fence_after();
            }
            stage += 2 * C::kParts * ((n + 1) / 2);
            loads += (n + 1) / 2;
            units += n > 0;
            done += n;
            // ---- the row's end in this CTA
            const bool there = r < rows;
            if (32 * (warp & 3) >= rows) {
                // none of this warp's
            } else if (walk.whole()) {
                const bool none = n == 0 || (ref == -INFINITY && sum == 0.f);  // NaN is not nothing
                float inv = none ? 0.f : 1.f / sum;
                if (a.c.v_scale) inv *= a.c.v_scale[walk.h];
                const int64_t out = (int64_t)token * a.Hq + walk.h * group + head;
                // a thread has a row, whose pieces alone would be 32 places to a store: four lanes write 64 bytes of a row together
                __nv_bfloat16 *to[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int64_t row = __shfl_sync(0xffffffffu, out, (lane & ~3) + k);
                    to[k] = (lane & ~3) + k + 32 * (warp & 3) < rows ? (__nv_bfloat16 *)a.o + row * D + 8 * (lane & 3) : nullptr;
                }
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    tmem_ld32(t_o + 32 * c, o);
                    tmem_ld_wait();
                    uint4 w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w[j] = none ? make_uint4(0, 0, 0, 0)
                                    : make_uint4(pack_bf16x2(o[8 * j] * inv, o[8 * j + 1] * inv), pack_bf16x2(o[8 * j + 2] * inv, o[8 * j + 3] * inv),
                                                 pack_bf16x2(o[8 * j + 4] * inv, o[8 * j + 5] * inv), pack_bf16x2(o[8 * j + 6] * inv, o[8 * j + 7] * inv));
                    transpose4(w, lane);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (to[k]) *(uint4 *)(to[k] + 32 * c) = w[k];
                }
                if (there && a.lse) a.lse[out] = none ? -INFINITY : (ref - C::kShift + log2f(sum)) * 0.6931471805599453f;
            } else {
                const int slot = walk.slot(), tile = 128 * C::kTiles, row = 128 * m + r;
                float4 *o_at = (float4 *)view.o + (size_t)slot * (D / 4) * tile + row;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    tmem_ld32(t_o + 32 * c, o);
                    tmem_ld_wait();
                    if (there)
#pragma unroll
                        for (int j = 0; j < 8; ++j) o_at[(size_t)(8 * c + j) * tile] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                }
                if (there) view.ml[(size_t)slot * tile + row] = make_float2(ref == -INFINITY ? -INFINITY : ref - C::kShift, sum);
            }
            tc_fence_before();
        }
    }
    __syncthreads();
    if (bars.gave_up && tid == 0) atomicOr(view.status, 1);
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc<512>(tmem);
    }
}

// A cache tensor as a map of (dim, cell, head, page), boxes of `box` cells and the dims of a swizzled row, or of an 8-bit stage.
inline bool make_tmap_cache(CUtensorMap *map, const gdn_kv_cache &c, const void *base, int box) {
    auto enc = tmap_encoder();
    if (!enc) return false;
    const int bytes = c.dtype == GDN_E4M3 ? 1 : 2;
    const cuuint64_t dims[4] = {(cuuint64_t)c.d, (cuuint64_t)c.page, (cuuint64_t)c.Hkv, (cuuint64_t)c.pages};
    const int64_t step[3] = {c.stride_token, c.stride_head, c.stride_page};
    cuuint64_t strides[3];
    for (int i = 0; i < 3; ++i) {
        strides[i] = (cuuint64_t)(dims[i + 1] == 1 ? c.d : step[i]) * bytes;  // of one element any will do
        if (strides[i] == 0 || strides[i] >> 40) return false;
    }
    const cuuint32_t boxes[4] = {(cuuint32_t)(bytes == 1 ? (c.d < 128 ? c.d : 128) : 64), (cuuint32_t)box, 1, 1}, each[4] = {1, 1, 1, 1};
    return enc(map, bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, boxes, each,
               CU_TENSOR_MAP_INTERLEAVE_NONE, bytes == 1 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <gdn_dtype KIND, int D, bool TMA, bool LOST>
cudaError_t launch_tc(const PrefillArgs &a, int grid, int box, const CUtensorMap (&maps)[2], cudaStream_t stream) {
    using C = Cfg<KIND, D>;
    constexpr int kSmem = (int)(C::kSmem + sizeof(Bars));
    // the warp groups' shares of registers are what a block of 128 to a thread has: with fewer they would wait for ever
    static std::atomic<int> regs{0};
    if (regs.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes attr;
        const cudaError_t e = cudaFuncGetAttributes(&attr, prefill_tc_kernel<KIND, D, TMA, LOST>);
        if (e != cudaSuccess) return e;
        regs.store(attr.numRegs, std::memory_order_relaxed);
    }
    if (regs.load(std::memory_order_relaxed) != 128) return cudaErrorInvalidConfiguration;
    const cudaError_t e = cudaFuncSetAttribute(prefill_tc_kernel<KIND, D, TMA, LOST>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    return e != cudaSuccess ? e : launch_kernel(true, prefill_tc_kernel<KIND, D, TMA, LOST>, grid, kThreads, kSmem, stream, a, maps[0], maps[1], box);
}
template <gdn_dtype KIND, bool TMA, bool LOST = false>
cudaError_t launch_tc(const PrefillArgs &a, int grid, int box, const CUtensorMap (&maps)[2], cudaStream_t stream) {
    switch (a.c.d) {
        case 64: return launch_tc<KIND, 64, TMA, LOST>(a, grid, box, maps, stream);
        case 128: return launch_tc<KIND, 128, TMA, LOST>(a, grid, box, maps, stream);
        default: return launch_tc<KIND, 256, TMA, LOST>(a, grid, box, maps, stream);
    }
}

}  // namespace prefill
}  // namespace gdn
