// k_paged_prefill.cu -- softmax attention of new tokens over the paged cache: the plan before the attention
// kernels, and the join of rows that were cut between CTAs after them (paged_prefill.cuh has the scheme).
//
// Both are latency.  The plan is one CTA's scans and searches, 6 to 8 us by itself with cold caches (every instruction of it comes from
// afar once); the attention kernel's CTAs start beside it and set up their barriers and tensor memory meanwhile.  The join reads at most 40 MB of
// parts: 4 us where there are few, 16 us (cold) for 151 cut units of 256 rows of 128 dims, 3 % of a call that has so many.
#include "paged_prefill_tc.cuh"

namespace gdn {
namespace prefill {
namespace {

constexpr int kPlanThreads = 1024, kHeldUnits = 2048;

// Running sum over the CTA, inclusive; `all` gets the total.
__device__ int64_t scan(int64_t x, int64_t *buf, int64_t &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) buf[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int64_t y = buf[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t z = __shfl_up_sync(0xffffffffu, y, off);
            if (lane >= off) y += z;
        }
        buf[lane] = y;
    }
    __syncthreads();
    if (warp) x += buf[warp - 1];
    all = buf[31];
    __syncthreads();
    return x;
}

// One CTA: a thread per request counts its units, a thread per unit finds its request, rows and keys, a thread per CTA its run.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PrefillArgs a, int tile, int keys, int grid, int pad, Weights weights) {
    __shared__ int64_t buf[32];
    __shared__ int64_t held[kHeldUnits];
    View v;
    layout(a.ws, a.B, a.n, a.Hq, a.c.Hkv, a.c.d, tile, grid, &v);
    const int tid = threadIdx.x, group = a.Hq / a.c.Hkv, room = a.max_pages * a.c.page;
    pdl_trigger();
    auto rows_of = [&](int b, int &first) {
        first = min(max(a.cu[b], 0), a.n);
        return max(min(a.cu[b + 1], a.n) - first, 0) * group;
    };
    int64_t units = 0;
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        int first;
        const int b = b0 + tid, mine = b < a.B ? (rows_of(b, first) + tile - 1) / tile : 0;
        int64_t all;
        const int64_t incl = scan(mine, buf, all);
        if (b < a.B) v.first[b] = (int)min(units + incl - mine, (int64_t)INT32_MAX);
        units += all;
    }
    // cu_new that goes back and forth names rows more often than there is room for: the last units are left out
    units = min(units, unit_capacity(a.B, (int64_t)a.n * group, tile));
    __syncthreads();
    int64_t cost = 0;
    for (int64_t i0 = 0; i0 < units; i0 += kPlanThreads) {
        const int64_t i = i0 + tid;
        int mine = 0;
        if (i < units) {
            int lo = 0, hi = a.B;  // the last request whose first unit is at or before i: requests without units are skipped
            while (lo + 1 < hi) {
                const int mid = (lo + hi) >> 1;
                if (v.first[mid] <= i) lo = mid;
                else hi = mid;
            }
            Unit u;
            u.b = lo;
            const int rows = rows_of(lo, u.first);
            u.row = (int)(i - v.first[lo]) * tile;
            u.rows = min(tile, rows - u.row);
            u.shift = max(a.lens[lo], 0) - a.cu[lo + 1];  // with a row at all cu is positive, and its positions are below its length
            auto reach = [&](int row) { return reach_of(u.first + a.group.quotient(u.row + row) + u.shift, a.window, room); };
            const Reach r0 = reach(0), r1 = reach(u.rows - 1);
            u.lo = r0.lo;
            u.hi = r1.hi;
            u.key = r0.lo / keys * keys;
            u.tiles = r1.hi >= r0.lo ? (r1.hi - u.key) / keys + 1 : 0;
            u.all_hi[0] = r0.hi;
            u.all_lo[0] = reach(min(u.rows, 128) - 1).lo;
            u.all_hi[1] = reach(min(u.rows - 1, 128)).hi;
            u.all_lo[1] = r1.lo;
            u.pad[0] = u.pad[1] = u.pad[2] = 0;
            v.unit[i] = u;
            mine = (u.rows > 128 ? weights.two : weights.one) * (u.tiles + pad);
        }
        int64_t all;
        const int64_t incl = cost + scan(mine, buf, all);
        if (i < units) {
            v.ends[i] = incl;
            if (i < kHeldUnits) held[i] = incl;
        }
        cost += all;
    }
    __syncthreads();
    const int64_t *ends = units <= kHeldUnits ? held : v.ends;
    const int64_t total = cost * a.c.Hkv;
    const int ctas = (int)max((int64_t)1, min((int64_t)grid, total / (weights.one * (pad + 1))));  // no two edges at the same tile
    for (int i = tid; i <= grid; i += kPlanThreads) {
        int4 run = make_int4(-1, 0, 0, 0);
        if (i == ctas || total == 0) run = i <= ctas ? make_int4(a.c.Hkv, 0, 0, 0) : run;
        else if (i < ctas) {
            const int64_t x = split_at(total, ctas, i), head = x / cost, rest = x % cost;
            int lo = 0, hi = (int)units - 1;  // the first unit that ends behind it
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (ends[mid] > rest) hi = mid;
                else lo = mid + 1;
            }
            const int64_t begin = lo ? ends[lo - 1] : 0;
            const Unit &u = v.unit[lo];
            run = make_int4((int)head, lo, (int)(rest - begin) / (u.rows > 128 ? weights.two : weights.one), u.tiles);
        }
        v.runs[i] = run;
    }
    if (tid == 0) {
        *v.status = 0;
        *v.units = (int)units;
    }
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A unit cut into parts (m_i, l_i, o_i): o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i, M = max m_i, in the keys' order.
// Grid: an entry per edge between two CTAs, which is idle unless it is the first inside its unit; times the tile's blocks of rows; times
// blocks of dims.  A thread has 8 dims of a row.
constexpr int kJoinRows = 32, kJoinThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(PrefillArgs a, int tile, int grid) {
    View v;
    layout(a.ws, a.B, a.n, a.Hq, a.c.Hkv, a.c.d, tile, grid, &v);
    pdl_wait();
    const int edge = blockIdx.x + 1;
    auto inside = [&](const int4 &r) { return r.x >= 0 && r.z > 0 && r.z < r.w; };
    const int4 r = v.runs[edge];
    if (!inside(r)) return;
    const int4 before = v.runs[edge - 1];
    if (inside(before) && before.x == r.x && before.y == r.y) return;
    int parts = 2;
    for (; edge + parts - 1 <= grid; ++parts) {
        const int4 next = v.runs[edge + parts - 1];
        if (!inside(next) || next.x != r.x || next.y != r.y) break;
    }
    const Unit u = v.unit[r.y];
    const int row = blockIdx.y * kJoinRows + threadIdx.x % kJoinRows;
    const int d0 = (blockIdx.z * (kJoinThreads / kJoinRows) + threadIdx.x / kJoinRows) * 8;
    if (row >= u.rows || d0 >= a.c.d) return;
    // the unit's beginning is the last piece of the CTA before the edge, the rest are first pieces
    auto slot = [&](int k) { return k == 0 ? 2 * (edge - 1) + 1 : 2 * (edge - 1 + k); };
    float top = -INFINITY;
    for (int k = 0; k < parts; ++k) top = fmaxf(top, v.ml[(size_t)slot(k) * tile + row].x);
    const float ref = top == -INFINITY ? 0.f : top;
    float x[8] = {}, sum = 0.f;
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
        const float2 ml = v.ml[(size_t)slot(k) * tile + row];
        const float4 *o = (const float4 *)v.o + ((size_t)slot(k) * (a.c.d / 4) + d0 / 4) * tile + row;
        const float4 lo = o[0], hi = o[tile];
        const float f = exp2_fast(ml.x - ref);
        sum += f * ml.y;
        x[0] += f * lo.x, x[1] += f * lo.y, x[2] += f * lo.z, x[3] += f * lo.w;
        x[4] += f * hi.x, x[5] += f * hi.y, x[6] += f * hi.z, x[7] += f * hi.w;
    }
    int head;
    const int token = u.first + a.group.quotient(u.row + row, head);
    float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (a.c.v_scale) inv *= a.c.v_scale[r.x];
    const int64_t out = (int64_t)token * a.Hq + r.x * (int)a.group.by + head;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = sum == 0.f ? 0.f : x[i] * inv;
    if constexpr (sizeof(T) == 4) {
        float4 *o = (float4 *)((float *)a.o + out * a.c.d + d0);
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        __nv_bfloat162 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        *(uint4 *)((__nv_bfloat16 *)a.o + out * a.c.d + d0) = *(const uint4 *)p;
    }
    if (d0 == 0 && a.lse) a.lse[out] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace
}  // namespace prefill

size_t paged_prefill_workspace_bytes(const gdn_kv_cache &c, int B, int n, int Hq) {
    return prefill::layout(nullptr, B, n, Hq, c.Hkv, c.d, prefill::row_tile(c.dtype, c.d), prefill::wave(c.dtype, c.d), nullptr);
}

cudaError_t launch_paged_prefill(const PrefillArgs &args, cudaStream_t stream) {
    using namespace prefill;
    PrefillArgs a = args;
    if (a.max_pages == 0) a.c.k = a.c.v = (void *)a.q;  // an address for copies of no bytes
    a.group = divisor(a.Hq / a.c.Hkv);
    a.page = divisor(a.c.page);
    const int tile = row_tile(a.c.dtype, a.c.d), grid = wave(a.c.dtype, a.c.d);
    cudaError_t e = launch_kernel(false, plan_kernel, 1, kPlanThreads, 0, stream, a, tile, key_tile(a.c.dtype, a.c.d), grid, unit_pad(a.c.dtype),
                                  unit_weights(a.c.dtype, a.c.d));
    if (e != cudaSuccess) return e;
    if (a.c.dtype == GDN_F32) {
        e = launch_f32(a, grid, stream);
    } else {
        // tokens of a page that lie together in every tile of 64 keys: a TMA box from 8 on, the rows of a swizzle pattern
        int box = 64;
        while (a.c.page % box) box /= 2;
        CUtensorMap maps[2];
        const bool tma = box >= 8 && a.max_pages > 0 && make_tmap_cache(&maps[0], a.c, a.c.k, box) && make_tmap_cache(&maps[1], a.c, a.c.v, box);
        if (a.lost_ns) e = (a.c.dtype == GDN_BF16 ? launch_lost_bf16 : launch_lost_e4m3)(a, tma, grid, box, maps, stream);
        else e = a.c.dtype == GDN_BF16 ? (tma ? launch_bf16_tma : launch_bf16)(a, grid, box, maps, stream) : (tma ? launch_e4m3_tma : launch_e4m3)(a, grid, box, maps, stream);
    }
    if (e != cudaSuccess) return e;
    const int dims = kJoinThreads / kJoinRows * 8;
    const int64_t rows = (int64_t)a.n * (a.Hq / a.c.Hkv);
    const dim3 blocks(grid - 1, (unsigned)((min((int64_t)tile, rows) + kJoinRows - 1) / kJoinRows), a.c.d / dims);
    return a.c.dtype == GDN_F32 ? launch_kernel(true, join_kernel<float>, blocks, kJoinThreads, 0, stream, a, tile, grid)
                                : launch_kernel(true, join_kernel<__nv_bfloat16>, blocks, kJoinThreads, 0, stream, a, tile, grid);
}

}  // namespace gdn
