// paged_prefill.cuh -- softmax attention of new tokens over the paged cache: how the work is cut and where the
// parts of cut rows lie, shared by the kernels that k_paged_prefill*.cu instantiate.
//
// A unit is a tile of rows (new token t, query head of one KV head's group, in this order) of one request with all the keys
// they attend to, in tiles of 64 keys (32-bit storage: 32 or 16).  The units of all requests are laid end to end, once for each KV head, and the CTAs of one
// wave get equal runs of key tiles (weighed where units of one row tile take less); a unit cut by a CTA's edge leaves unnormalised fp32 parts that a last launch joins in
// the keys' order.  Lengths are only known on the GPU, so a first launch of one CTA lists the units and finds the runs.  Causal rows
// make units of 1 to hundreds of tiles, and equal runs need no luck with their order: of 8192 tokens at once every CTA
// has the same number of tiles, and one row over 131072 is shared by all of them.
#pragma once

#include <cuda.h>

#include "paged.cuh"

namespace gdn {
namespace prefill {

constexpr int kMaxCtas = 304;  // of a wave, at most two per SM

// What the kernels need of a unit is worked out once, in the plan: instructions that a CTA goes through once come from afar, some 250
// clocks to every eight of them, and with the arithmetic repeated by each kind of warp the first product was asked for 9 us after the start.
struct alignas(16) Unit {
    int b, first;             // request; its first row of q
    int row, rows;            // of the request's (token, head of the group) rows: the first, and how many
    int shift;                // position of a token: its row of q + shift
    int key, tiles;           // first key, a multiple of the tile; tiles of keys
    int lo, hi;               // keys that any row attends to: [lo, hi]
    int all_lo[2], all_hi[2]; // of the two tiles of 128 rows: keys that all of its rows attend to
    int pad[3];
};

struct View {
    int32_t *status;  // bits, 0: nothing ran out
    int4 *runs;       // [kMaxCtas + 1] {KV head, unit, place in the unit, its tiles}; x < 0: no such CTA
    int32_t *units;   // how many
    Unit *unit;
    int64_t *ends;    // running sum of the units' costs
    int32_t *first;   // of each request: its first unit
    float2 *ml;       // [2 CTAs][rows of a unit] reference and sum of a part
    float *o;         // [2 CTAs][d / 4][rows of a unit][4]
};

inline __host__ __device__ int64_t unit_capacity(int B, int64_t rows, int tile) { return rows / tile + 1 + B; }

// Byte offsets of View's parts; returns the size.
inline __host__ __device__ size_t layout(void *ws, int B, int n, int Hq, int Hkv, int d, int tile, int ctas, View *v) {
    const int64_t units = unit_capacity(B, (int64_t)n * (Hq / Hkv), tile);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) & ~(size_t)255;
        return (uint8_t *)ws + here;
    };
    View x;
    x.status = (int32_t *)take(256);
    x.units = x.status + 1;
    x.runs = (int4 *)take((kMaxCtas + 1) * sizeof(int4));
    x.unit = (Unit *)take(units * sizeof(Unit));
    x.ends = (int64_t *)take(units * sizeof(int64_t));
    x.first = (int32_t *)take(((size_t)B + 1) * sizeof(int32_t));
    x.ml = (float2 *)take((size_t)2 * ctas * tile * sizeof(float2));
    x.o = (float *)take((size_t)2 * ctas * tile * d * sizeof(float));
    if (v) *v = x;
    return at;
}

// Rows and keys of a tile: what the kernels are built for.
inline __host__ __device__ int row_tile(gdn_dtype kind, int d) { return kind == GDN_F32 || d == 256 ? 128 : 256; }
inline __host__ __device__ int key_tile(gdn_dtype kind, int d) { return kind != GDN_F32 ? 64 : d == 256 ? 16 : 32; }
// A unit costs its tiles and this many more, for its beginning and end (8-bit caches: most of all for q's conversion, in turn with the keys'),
// and a CTA takes one more than that at least.  8192 bf16 tokens at once: 484 us with 2, 476 with 3, 479 with 4; 8-bit chunks of up to 512
// tokens over 16000: 329 with 3, 314 with 5, 299 with 8, 290 with 10, 294 with 12 (279 with 10 since units of one row tile are weighed and a tile's product is waited for ahead of its keys).
inline __host__ __device__ int unit_pad(gdn_dtype kind) { return kind == GDN_E4M3 ? 10 : 3; }
// What a tile costs in a unit of one row tile of 128, and of two.  With 256 bytes to a bf16 row the copies take as long for one as for two:
// 32 requests of mostly one new token, up to 4096 behind them, 85.9 us with 1:1, 87.5 with 3:4, 92.2 with 2:3.  Rows of 128 bytes or less: bf16 of 64
// dims 76.9, 71.2 and 74.2 us, 8-bit of 128 104, 96 and 101, of 64 89.8, 84.7 and 84.3.
struct Weights { int one, two; };
inline __host__ __device__ Weights unit_weights(gdn_dtype kind, int d) {
    return row_tile(kind, d) == 128 || (kind == GDN_BF16 && d == 128) ? Weights{1, 1} : Weights{3, 4};
}
// CTAs of a wave: one per SM, two where the registers of the warp-MMA kernel allow.
inline __host__ __device__ int wave(gdn_dtype kind, int d) { return kind == GDN_F32 && d == 64 ? kMaxCtas : kMaxCtas / 2; }

inline __host__ __device__ int64_t split_at(int64_t total, int ctas, int i) { return total / ctas * i + total % ctas * i / ctas; }

// Keys [lo, hi] that a token attends to.
struct Reach { int lo, hi; };
__device__ __forceinline__ Reach reach_of(int pos, int window, int room) {
    const int lo = window > 0 && pos >= window ? pos - window + 1 : 0;
    return {min(lo, room), max(min(pos, room - 1), -1)};
}

// What a CTA does, one piece of a unit after the other.  Every thread that walks it sees the same pieces.
struct Walk {
    View v;
    int4 at, end;
    int units;
    Unit u;           // the piece's unit
    int h;            // its KV head
    int t0, t1;       // its tiles [t0, t1)
    int cta;

    __device__ __forceinline__ void start(const View &view, int which) {
        v = view;
        cta = which;
        at = v.runs[which];
        end = v.runs[which + 1];
        units = *v.units;
    }
    // The next piece that has something to do; false: there is none.
    __device__ __forceinline__ bool next() {
        for (;;) {
            if (at.x < 0 || end.x < 0) return false;
            const bool last = at.x == end.x && at.y == end.y;
            if (at.x > end.x || (at.x == end.x && at.y > end.y) || (last && at.z >= end.z)) return false;
            u = v.unit[at.y];
            h = at.x;
            const bool begin = at.z == 0;
            t0 = min(at.z, u.tiles);
            t1 = last ? min(end.z, u.tiles) : u.tiles;
            at.z = 0;
            if (++at.y == units) at.y = 0, ++at.x;
            if (t0 < t1 || (u.tiles == 0 && begin)) return true;
        }
    }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == u.tiles; }
    // Where a part lies: a CTA's first piece if its unit began in another CTA, else its last.
    __device__ __forceinline__ int slot() const { return 2 * cta + (t0 > 0 ? 0 : 1); }
};

// prefill kernels: a.ws holds the View; launched as programmatic dependents of the plan
cudaError_t launch_bf16(const PrefillArgs &a, int grid, int box, const CUtensorMap (&maps)[2], cudaStream_t stream);
cudaError_t launch_bf16_tma(const PrefillArgs &a, int grid, int box, const CUtensorMap (&maps)[2], cudaStream_t stream);
cudaError_t launch_e4m3(const PrefillArgs &a, int grid, int box, const CUtensorMap (&maps)[2], cudaStream_t stream);
cudaError_t launch_e4m3_tma(const PrefillArgs &a, int grid, int box, const CUtensorMap (&maps)[2], cudaStream_t stream);
cudaError_t launch_lost_bf16(const PrefillArgs &a, bool tma, int grid, int box, const CUtensorMap (&maps)[2], cudaStream_t stream);  // self-test of waits
cudaError_t launch_lost_e4m3(const PrefillArgs &a, bool tma, int grid, int box, const CUtensorMap (&maps)[2], cudaStream_t stream);
cudaError_t launch_f32(const PrefillArgs &a, int grid, cudaStream_t stream);

}  // namespace prefill
}  // namespace gdn
