// overlap.h -- host: whether tensors of strided rows share memory.
//
// A tensor [n0, n1, n2] of contiguous rows: row (i0, i1, i2) begins at p +
// i0 step0 + i1 step1 + i2 step2.  Two tensors share a byte iff some
// difference of two such beginnings is smaller than a row: a bounded linear
// equation in six whole numbers, solved by trying the values of the largest
// step first.  The other steps reach only a few values of it, because rows of
// real layouts nest; a query projection and a key projection side by side in
// one buffer are told apart in a handful of tries.
#pragma once

#include <stdint.h>

namespace fa {

struct Rows {
    const void *p;
    int64_t width;  // bytes of a row
    int64_t n[3], step[3];  // bytes; n >= 1
};

namespace overlap_detail {

typedef __int128 wide;

struct Equation {  // sum of x_k step_k + offset within [low, high], lo_k <= x_k <= hi_k
    struct Term {
        wide step, lo, hi;
    } t[6];
    int n = 0;
    wide low, high;
    wide least[7], most[7];  // of the terms from k on
    int tries = 0;

    void add(wide step, wide lo, wide hi) {
        if (step == 0 || (lo == 0 && hi == 0)) return;
        if (step < 0) {
            const wide l = -hi;
            step = -step, hi = -lo, lo = l;
        }
        int k = 0;
        while (k < n && t[k].step > step) ++k;
        if (k < n && t[k].step == step) {
            t[k].lo += lo, t[k].hi += hi;
            return;
        }
        for (int j = n++; j > k; --j) t[j] = t[j - 1];
        t[k] = Term{step, lo, hi};
    }
    static wide floor_div(wide a, wide b) { return a >= 0 ? a / b : -((-a + b - 1) / b); }

    bool from(int k, wide offset) {
        if (offset + most[k] < low || offset + least[k] > high) return false;
        if (k == n) return true;
        const Term &x = t[k];
        wide a = -floor_div(-(low - offset - most[k + 1]), x.step), b = floor_div(high - offset - least[k + 1], x.step);
        if (a < x.lo) a = x.lo;
        if (b > x.hi) b = x.hi;
        for (; a <= b; ++a) {
            if (++tries > 20000) return true;  // not shown to be apart
            if (from(k + 1, offset + a * x.step)) return true;
        }
        return false;
    }
    bool solvable(wide offset) {
        least[n] = most[n] = 0;
        for (int k = n - 1; k >= 0; --k) {
            least[k] = least[k + 1] + t[k].lo * t[k].step;
            most[k] = most[k + 1] + t[k].hi * t[k].step;
        }
        return from(0, offset);
    }
};

}  // namespace overlap_detail

// First byte and the one behind the last.
inline void rows_span(const Rows &a, overlap_detail::wide *first, overlap_detail::wide *end) {
    *first = *end = (overlap_detail::wide)(uintptr_t)a.p;
    for (int k = 0; k < 3; ++k) *(a.step[k] < 0 ? first : end) += (overlap_detail::wide)(a.n[k] - 1) * a.step[k];
    *end += a.width;
}

// Some byte belongs to both (or 20000 tries did not settle it).
inline bool rows_meet(const Rows &a, const Rows &b) {
    overlap_detail::wide a0, a1, b0, b1;
    rows_span(a, &a0, &a1);
    rows_span(b, &b0, &b1);
    if (a1 <= b0 || b1 <= a0) return false;  // nearly always
    overlap_detail::Equation e;
    e.low = 1 - b.width, e.high = a.width - 1;
    for (int k = 0; k < 3; ++k) {
        e.add(b.step[k], 0, b.n[k] - 1);
        e.add(a.step[k], 1 - a.n[k], 0);
    }
    return e.solvable((overlap_detail::wide)(uintptr_t)b.p - (overlap_detail::wide)(uintptr_t)a.p);
}

// Two different rows of `a` share a byte (or 20000 tries did not settle it).
inline bool rows_meet_themselves(const Rows &a) {
    // Of the differences of two rows one sign is enough: the first index that
    // differs is larger, the ones after it are anything.
    for (int first = 0; first < 3; ++first) {
        if (a.n[first] == 1) continue;
        if (a.step[first] == 0) return true;
        overlap_detail::Equation e;
        e.low = 1 - a.width, e.high = a.width - 1;
        e.add(a.step[first], 1, a.n[first] - 1);
        for (int k = first + 1; k < 3; ++k) e.add(a.step[k], 1 - a.n[k], a.n[k] - 1);
        if (e.solvable(0)) return true;
    }
    return false;
}

}  // namespace fa
