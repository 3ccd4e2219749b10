// Whether what a call writes lies on other arrays of it.  Host code alone.
#pragma once
#include <stdint.h>

#include <algorithm>
#include <numeric>

namespace fp4 {

typedef __int128 wide_t;  // counts times strides pass 64 bits where the arguments make no sense

// The bytes p + i * stride[0] + j * stride[1] + [0, width), i < count[0], j < count[1],
// all of them below `end`.
struct Span {
    uintptr_t p, end;
    int64_t width, count[2], stride[2];
};

inline Span span_of(const void* p, int64_t width, int64_t n0 = 1, int64_t s0 = 0, int64_t n1 = 1, int64_t s1 = 0) {
    Span s{reinterpret_cast<uintptr_t>(p), 0, width, {n0, n1}, {s0, s1}};
    const wide_t end = (wide_t)s.p + (wide_t)(n0 - 1) * s0 + (wide_t)(n1 - 1) * s1 + width;
    s.end = end > (wide_t)UINTPTR_MAX ? UINTPTR_MAX : (uintptr_t)end;
    return s;
}

// 16-bit rows: strides in elements.
inline Span span_of_rows(const void* p, int64_t width, int64_t rows, int64_t stride, int64_t heads = 1, int64_t hs = 0) {
    return span_of(p, width * 2, rows, stride * 2, heads, hs * 2);
}

// The same elements under the same indices.
inline bool same_span(const Span& a, const Span& b) {
    for (int d = 0; d < 2; ++d)
        if (a.count[d] != b.count[d] || (a.count[d] > 1 && a.stride[d] != b.stride[d])) return false;
    return a.p == b.p && a.width == b.width;
}

// Steps of c bytes, lo to hi of them.
struct SpanSteps {
    int64_t c;
    wide_t lo, hi;
};

// Whether some sum of the steps (largest c first) lies in [from, to].  Only those counts
// of a step are tried that the smaller ones can still make up for, and none where no
// multiple of the steps' common divisor lies there (views of one array side by side).
inline bool steps_reach(const SpanSteps* s, int n, wide_t from, wide_t to, int& budget) {
    if (from > to) return false;
    if (n == 0) return from <= 0 && to >= 0;
    auto below = [](wide_t a, wide_t b) { return a / b - (a % b < 0); };  // floor(a / b), b > 0
    wide_t least = 0, most = 0;
    for (int i = 1; i < n; ++i) least += s[i].c * s[i].lo, most += s[i].c * s[i].hi;
    if (to < least + s[0].c * s[0].lo || from > most + s[0].c * s[0].hi) return false;  // all of it elsewhere
    int64_t g = s[0].c;
    for (int i = 1; i < n; ++i) g = std::gcd(g, s[i].c);
    if (below(to, g) * g < from) return false;
    const wide_t lo = std::max(s[0].lo, -below(most - from, s[0].c)), hi = std::min(s[0].hi, below(to - least, s[0].c));
    for (wide_t k = lo; k <= hi; ++k) {
        if (n == 1) return true;
        if (--budget < 0) return false;
        if (steps_reach(s + 1, n - 1, from - k * s[0].c, to - k * s[0].c, budget)) return true;
    }
    return false;
}

// Whether two spans share a byte.  A search of more than 2^16 counts (arrays of unlike
// strides and many rows inside one another) ends as if they shared none.
inline bool spans_meet(const Span& a, const Span& b) {
    if (!a.p || !b.p || a.end <= b.p || b.end <= a.p) return false;
    SpanSteps s[4];
    int n = 0;
    wide_t width[2] = {a.width, b.width};
    for (int side = 0; side < 2; ++side) {
        const Span& x = side ? b : a;
        int order[2] = {0, 1};
        if (x.stride[0] < x.stride[1]) std::swap(order[0], order[1]);  // the larger stride first
        for (int i = 1; i >= 0; --i) {
            const int64_t count = x.count[order[i]], c = x.stride[order[i]];
            if (count < 1) return false;
            if (count == 1 || c == 0) continue;
            if (c <= width[side]) {  // rows without a gap are one row
                width[side] += (count - 1) * c;
                continue;
            }
            int k = 0;
            while (k < n && s[k].c != c) ++k;
            if (k == n) s[n++] = {c, 0, 0};
            (side ? s[k].hi : s[k].lo) += side ? count - 1 : 1 - count;
        }
    }
    for (int i = 1; i < n; ++i)
        for (int k = i; k > 0 && s[k].c > s[k - 1].c; --k) std::swap(s[k], s[k - 1]);
    const wide_t apart = (wide_t)b.p - (wide_t)a.p;  // b's first byte from a's
    int budget = 1 << 16;
    return width[0] > 0 && width[1] > 0 && steps_reach(s, n, 1 - width[1] - apart, width[0] - 1 - apart, budget);
}

// An output that may be this input, element by element, or else has to lie apart from it.
inline bool span_may_be(const Span& to, const Span& from) { return same_span(to, from) || !spans_meet(to, from); }

}  // namespace fp4
