// rows.h -- whether the rows of two strided tensors overlap in memory (host only).
#pragma once
#include <stdint.h>

namespace fa {

// Rows of `row` bytes at first + sum_i k_i stride_i for 0 <= k_i < count_i.
struct Rows {
    int64_t first, row;
    int n = 0;  // dimensions, by falling stride; none with a single entry or a stride of 0
    int64_t stride[3], count[3];

    Rows(const void *at, int64_t bytes) : first((int64_t)(uintptr_t)at), row(bytes) {}
    // False for a stride out of all proportion.
    bool add(int64_t s, int64_t entries) {
        if (entries <= 1 || s == 0) return true;
        const int64_t far = (int64_t)1 << 50, size = s < 0 ? -s : s;
        if (size > far / entries || s == INT64_MIN) return false;
        if (s < 0) first += (entries - 1) * s;
        int i = n++;
        for (; i > 0 && stride[i - 1] < size; --i) stride[i] = stride[i - 1], count[i] = count[i - 1];
        stride[i] = size, count[i] = entries;
        return true;
    }
    // From the first row's start to the last one's end, without the first `from` dimensions.
    int64_t reach(int from) const {
        int64_t r = row;
        for (int i = from; i < n; ++i) r += (count[i] - 1) * stride[i];
        return r;
    }
};

inline int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0 ? 1 : 0); }  // b > 0

// Whether any row of a meets one of b, whose first row lies `off` behind a's, from dimensions ia and ib on. The dimension of the
// greatest stride is gone through, one that both have in one: only places whose reaches overlap are looked at, one or two
// for rows that nest. After `budget` of them the answer is yes.
inline bool rows_meet(const Rows &a, const Rows &b, int64_t off, int ia, int ib, int &budget) {
    if (off >= a.reach(ia) || off <= -b.reach(ib)) return false;
    if (--budget < 0 || (ia == a.n && ib == b.n)) return true;
    const int64_t sa = ia < a.n ? a.stride[ia] : 0, sb = ib < b.n ? b.stride[ib] : 0, s = sa > sb ? sa : sb;
    const int ja = ia + (sa == s), jb = ib + (sb == s);
    // off + k s for k = (entry of b) - (entry of a), within (-reach of b, reach of a)
    int64_t lo = sa == s ? 1 - a.count[ia] : 0, hi = sb == s ? b.count[ib] - 1 : 0;
    const int64_t least = floor_div(-b.reach(jb) - off, s) + 1, most = floor_div(a.reach(ja) - off - 1, s);
    if (lo < least) lo = least;
    if (hi > most) hi = most;
    for (int64_t k = lo; k <= hi; ++k)
        if (rows_meet(a, b, off + k * s, ja, jb, budget)) return true;
    return false;
}
inline bool rows_meet(const Rows &a, const Rows &b) {
    int budget = 4096;
    return rows_meet(a, b, b.first - a.first, 0, 0, budget);
}

}  // namespace fa
