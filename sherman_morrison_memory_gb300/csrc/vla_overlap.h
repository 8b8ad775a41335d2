// vla_overlap.h -- whether the arrays of a call share memory (host code).
//
// A kernel's blocks read inputs while others write outputs, so an output on top
// of an input gives results that depend on which came first: such calls are
// refused. Outputs that lie between the rows of an input, or of each other (dq,
// dk and dv as slices of one projection's gradient), share none and are taken.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <initializer_list>

namespace vla_layer {

// Device memory that a call reads or writes: rows of `row` bytes at strides st[i]
// (bytes) apart in each of three dimensions.
struct Region {
    uintptr_t p;
    long long row, st[3];
    int n[3];
};
template <typename S>
inline Region region(const S* s, int B, int H, int T, int d, int es) {
    auto bytes = [&](int n, long long st) { return n > 1 ? st * es : 0; };
    return Region{reinterpret_cast<uintptr_t>(s->data), (long long)d * es,
                  {bytes(B, s->stride_b), bytes(H, s->stride_h), bytes(T, s->stride_t)}, {B, H, T}};
}
// n values of `bits` bits, one after another (more than the address space holds counts as that)
inline Region region(const void* p, __int128 n, int bits) {
    const __int128 bytes = std::min<__int128>(n * bits / 8, (__int128)1 << 60);
    return Region{reinterpret_cast<uintptr_t>(p), p ? (long long)bytes : 0, {0, 0, 0}, {1, 1, 1}};
}
inline bool same(const Region& a, const Region& b) {
    bool s = a.p == b.p && a.row == b.row;
    for (int i = 0; i < 3; ++i) s = s && a.n[i] == b.n[i] && (a.st[i] == b.st[i]);
    return s;
}

// Whether whole numbers k_i in [lo_i, hi_i] with sum k_i st_i in [from, to] exist
// (`other`: besides all k_i = 0). Strides in falling order; a search over the few k
// that the strides behind leave open. Where it takes long, the answer is yes.
struct Term {
    long long st, lo, hi;
};
inline bool reaches(const Term* t, int n, __int128 from, __int128 to, bool other, int& steps) {
    if (n == 0) return !other && from <= 0 && to >= 0;
    __int128 lo = 0, hi = 0;  // what the terms behind can add
    for (int i = 1; i < n; ++i) lo += (__int128)t[i].lo * t[i].st, hi += (__int128)t[i].hi * t[i].st;
    auto floor_div = [](__int128 a, long long b) { return a >= 0 ? a / b : -((b - 1 - a) / b); };
    const __int128 first = std::max<__int128>(t->lo, -floor_div(hi - from, t->st)),
                   last = std::min<__int128>(t->hi, floor_div(to - lo, t->st));
    for (__int128 k = first; k <= last; ++k) {
        if (--steps < 0) return true;
        if (reaches(t + 1, n - 1, from - k * t->st, to - k * t->st, other && k == 0, steps)) return true;
    }
    return false;
}
inline void in_order(Term* t, int n) {
    std::sort(t, t + n, [](const Term& a, const Term& b) { return a.st > b.st; });
}
// a and b have a byte in common
inline bool overlap(const Region& a, const Region& b) {
    if (!a.p || !b.p || a.row <= 0 || b.row <= 0) return false;
    __int128 ea = a.row, eb = b.row;
    for (int i = 0; i < 3; ++i) {
        if (a.n[i] <= 0 || b.n[i] <= 0) return false;
        if (a.n[i] > 1) ea += (__int128)(a.n[i] - 1) * a.st[i];
        if (b.n[i] > 1) eb += (__int128)(b.n[i] - 1) * b.st[i];
    }
    const __int128 off = (__int128)b.p - (__int128)a.p;
    if (off >= ea || -off >= eb) return false;
    Term t[6];
    int n = 0;
    auto add = [&](long long st, long long lo, long long hi) {
        for (int i = 0; i < n; ++i)
            if (t[i].st == st) {
                t[i].lo += lo, t[i].hi += hi;
                return;
            }
        t[n++] = Term{st, lo, hi};
    };
    for (int i = 0; i < 3; ++i) {
        if (a.n[i] > 1) add(a.st[i], 0, a.n[i] - 1);
        if (b.n[i] > 1) add(b.st[i], -(b.n[i] - 1), 0);
    }
    in_order(t, n);
    int steps = 4096;
    return reaches(t, n, off - (a.row - 1), off + (b.row - 1), false, steps);
}
// two rows of a have a byte in common
inline bool overlaps_itself(const Region& a) {
    if (!a.p || a.row <= 0) return false;
    Term t[3];
    int n = 0;
    for (int i = 0; i < 3; ++i)
        if (a.n[i] > 1) t[n++] = Term{a.st[i], -(a.n[i] - 1), a.n[i] - 1};
    in_order(t, n);
    int steps = 4096;
    return reaches(t, n, -(a.row - 1), a.row - 1, true, steps);
}
// No output overlaps itself, another or an input. The first output may be the very
// rows of one of the first `in_place` inputs.
inline bool apart(std::initializer_list<Region> outs, std::initializer_list<Region> ins, int in_place = 0) {
    for (const Region* o = outs.begin(); o != outs.end(); ++o) {
        if (overlaps_itself(*o)) return false;
        for (const Region* x = o + 1; x != outs.end(); ++x)
            if (overlap(*o, *x)) return false;
        for (const Region* x = ins.begin(); x != ins.end(); ++x)
            if (!(x - ins.begin() < in_place && o == outs.begin() && same(*o, *x)) && overlap(*o, *x)) return false;
    }
    return true;
}

}  // namespace vla_layer
