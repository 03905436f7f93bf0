// overlap.h -- do two tensors of a call share memory?
//
// A tensor here is a set of rows of bytes: n[0] x n[1] of them, s[0] and s[1] apart.  Two
// column slices of one buffer interleave without sharing anything, so extents alone do not
// tell.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace m2 {

struct Rows {
    int64_t at, row;        // address of the first row, bytes of each
    int64_t n[2], s[2];     // rows and bytes between them

    // Rows that follow one another are one; a dimension of one row has no step.
    void tidy() {
        for (int k = 0; k < 2; ++k)
            if (n[k] <= 1 || s[k] == 0) n[k] = 1, s[k] = 0;
        for (int pass = 0; pass < 2; ++pass)
            for (int k = 0; k < 2; ++k)
                if (n[k] > 1 && s[k] == row) row *= n[k], n[k] = 1, s[k] = 0;
    }
    int64_t end() const { return at + (n[0] - 1) * s[0] + (n[1] - 1) * s[1] + row; }
    bool one() const { return n[0] == 1 && n[1] == 1; }
};

// Some row of r meets the bytes [lo, hi): the shorter dimension is walked, the other solved.
inline bool meets(int64_t lo, int64_t hi, const Rows& r) {
    const int walk = r.n[0] <= r.n[1] ? 0 : 1;
    const int64_t n = r.n[1 - walk], s = r.s[1 - walk];
    for (int64_t i = 0; i < r.n[walk]; ++i) {
        const int64_t first = r.at + i * r.s[walk], behind = lo - r.row - first;   // first + j s > lo - row
        const int64_t j = n == 1 || behind < 0 ? 0 : behind / s + 1;
        if (j < n && first + j * s < hi && first + j * s + r.row > lo) return true;
    }
    return false;
}

// True when a and b share a byte.  Views of two different pitches with very many rows are
// not walked: false.
inline bool overlap(Rows a, Rows b) {
    if (a.row <= 0 || b.row <= 0 || a.n[0] <= 0 || a.n[1] <= 0 || b.n[0] <= 0 || b.n[1] <= 0) return false;
    if (a.end() <= b.at || b.end() <= a.at) return false;
    a.tidy();
    b.tidy();
    if (a.one()) return meets(a.at, a.at + a.row, b);
    if (b.one()) return meets(b.at, b.at + b.row, a);
    // The same steps in both (a missing one is free): a row of a meets one of b where a's first
    // row meets b moved back by every step a takes.
    int64_t step[2] = {0, 0}, na[2] = {1, 1}, nb[2] = {1, 1};
    int steps = 0;
    const auto put = [&](const Rows& r, int64_t* n) {
        for (int k = 0; k < 2; ++k) {
            if (r.n[k] == 1) continue;
            int at = 0;
            while (at < steps && (step[at] != r.s[k] || n[at] != 1)) ++at;
            if (at == 2) return false;
            if (at == steps) step[steps++] = r.s[k];
            n[at] = r.n[k];
        }
        return true;
    };
    if (put(a, na) && put(b, nb)) {
        Rows d{b.at, b.row, {na[0] + nb[0] - 1, na[1] + nb[1] - 1}, {step[0], step[1]}};
        for (int k = 0; k < 2; ++k) d.at -= (na[k] - 1) * step[k];
        return meets(a.at, a.at + a.row, d);
    }
    if (a.n[0] * a.n[1] * std::min(b.n[0], b.n[1]) > (int64_t(1) << 16)) std::swap(a, b);
    if (a.n[0] * a.n[1] * std::min(b.n[0], b.n[1]) > (int64_t(1) << 16)) return false;
    for (int64_t i = 0; i < a.n[0]; ++i)
        for (int64_t j = 0; j < a.n[1]; ++j) {
            const int64_t lo = a.at + i * a.s[0] + j * a.s[1];
            if (meets(lo, lo + a.row, b)) return true;
        }
    return false;
}

}  // namespace m2
