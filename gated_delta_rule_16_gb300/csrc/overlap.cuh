// overlap.cuh -- whether strided tensors of one call share memory (host only): an output over an input, or over itself, would be
// written by one CTA while another reads or writes it, which is refused before anything is launched.
#pragma once

#include <stdint.h>

namespace gdn {

// Pieces of `len` contiguous bytes along up to three axes of non-negative strides, in bytes.  Bounds are those of a tensor in memory, below 2^62.
struct Pieces {
    uintptr_t at;
    int64_t len;
    struct Axis { int64_t n, step; } axis[3];
};

inline Pieces pieces(const void *p, int64_t len) { return {(uintptr_t)p, len, {{1, 0}, {1, 0}, {1, 0}}}; }
inline Pieces pieces(const void *p, int64_t len, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2 = 1, int64_t s2 = 0) {
    return {(uintptr_t)p, len, {{n0, s0}, {n1, s1}, {n2, s2}}};
}

namespace overlap_detail {

inline bool empty(const Pieces &p) { return p.len <= 0 || p.axis[0].n <= 0 || p.axis[1].n <= 0 || p.axis[2].n <= 0; }
inline int64_t floor_div(int64_t x, int64_t by) { return x / by - (x % by < 0); }  // by > 0

// Axes that lie densely become part of the piece, those of one element or no stride go; the longest that is left comes first.
inline Pieces merged(Pieces p) {
    for (bool again = true; again;) {
        again = false;
        for (Pieces::Axis &x : p.axis) {
            if (x.n > 1 && x.step > 0 && x.step <= p.len) p.len += (x.n - 1) * x.step, x.n = 1, again = true;
            if (x.n <= 1 || x.step == 0) x = {1, 0};
        }
    }
    for (int i = 1; i < 3; ++i)
        if (p.axis[i].n > p.axis[0].n) {
            const Pieces::Axis x = p.axis[i];
            p.axis[i] = p.axis[0];
            p.axis[0] = x;
        }
    return p;
}

inline uintptr_t end_of(const Pieces &p) {
    uintptr_t end = p.at + p.len;
    for (const Pieces::Axis &x : p.axis) end += (x.n - 1) * x.step;
    return end;
}

// Whether low <= at + k step <= high for a k of [first, last].
inline bool meets(int64_t at, int64_t step, int64_t first, int64_t last, int64_t low, int64_t high) {
    if (step == 0) return at >= low && at <= high;
    int64_t k = -floor_div(at - low, step);  // the first that is not below
    if (k < first) k = first;
    return k <= last && at + k * step <= high;
}

}  // namespace overlap_detail

inline bool overlap(const Pieces &x, const Pieces &y) {
    using namespace overlap_detail;
    if (empty(x) || empty(y)) return false;
    if (x.at >= end_of(y) || y.at >= end_of(x)) return false;
    const Pieces a = merged(x), b = merged(y);
    const Pieces::Axis &u = a.axis[0], &v = b.axis[0];
    for (int64_t i = 0; i < a.axis[1].n * a.axis[2].n; ++i)
        for (int64_t j = 0; j < b.axis[1].n * b.axis[2].n; ++j) {
            // b's piece behind a's; they share bytes where it is in (-b.len, a.len)
            const int64_t off = (int64_t)(b.at - a.at) + j % b.axis[1].n * b.axis[1].step + j / b.axis[1].n * b.axis[2].step -
                                i % a.axis[1].n * a.axis[1].step - i / a.axis[1].n * a.axis[2].step;
            if (u.step == v.step || u.n == 1 || v.n == 1) {
                const int64_t step = v.n == 1 ? u.step : v.step;
                if (meets(off, step, 1 - u.n, v.n - 1, 1 - b.len, a.len - 1)) return true;
            } else {
                for (int64_t k = 0; k < u.n; ++k)
                    if (meets(off - k * u.step, v.step, 0, v.n - 1, 1 - b.len, a.len - 1)) return true;
            }
        }
    return false;
}

// Whether pieces of one tensor share bytes.
inline bool overlaps_itself(const Pieces &p) {
    using namespace overlap_detail;
    if (empty(p)) return false;
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)  // by stride
        for (int j = 0; j < 2 - i; ++j)
            if (p.axis[order[j]].step > p.axis[order[j + 1]].step) {
                const int t = order[j];
                order[j] = order[j + 1];
                order[j + 1] = t;
            }
    int64_t span = p.len;  // of what lies inside an axis: apart if every stride passes it
    bool apart = true;
    for (int i : order) {
        const Pieces::Axis &x = p.axis[i];
        if (x.n == 1) continue;
        if (x.step < p.len) return true;
        apart = apart && x.step >= span;
        span += (x.n - 1) * x.step;
    }
    if (apart) return false;
    // two pieces at distances (i, j, k) of the axes, not all 0; the largest first, so that the other two take fewer turns
    Pieces::Axis x = p.axis[0], y = p.axis[1], z = p.axis[2];
    if (y.n > x.n) { const Pieces::Axis t = x; x = y; y = t; }
    if (z.n > x.n) { const Pieces::Axis t = x; x = z; z = t; }
    for (int64_t j = 1 - y.n; j < y.n; ++j)
        for (int64_t k = 1 - z.n; k < z.n; ++k) {
            const int64_t off = j * y.step + k * z.step;
            if (j == 0 && k == 0) continue;  // along one axis alone every stride is a piece long
            if (meets(off, x.step, 1 - x.n, x.n - 1, 1 - p.len, p.len - 1)) return true;
        }
    return false;
}

}  // namespace gdn
