"""The search for the least weight that an eviction keeps, restated on the CPU step by step (fa_kvq8_evict.cu): integers of
the weights' order, 2048 bins between the least and the greatest of them, then within the bin that the count is reached in.
`end` gives a bin's last integer, so that a wrong one can be planted."""
import numpy as np

TOP = 2 ** 32 - 1


def orders(w):
    """Integers of the weights' order; NaN above all, -0 with 0."""
    u = (np.asarray(w, np.float32) + np.float32(0)).view(np.uint32)
    v = np.where(u >> 31 == 1, ~u, u | np.uint32(1 << 31))
    return np.where(np.isnan(w), np.uint32(TOP), v).astype(np.int64)


def bin_end(lo, hi, shift):
    return lo + min(hi - lo, (1 << shift) - 1)


def bin_end_wrapped(lo, hi, shift):
    """In 32 bits, where the end of the top bin may pass the greatest integer."""
    return min(hi, (lo + (1 << shift) - 1) & TOP)


def select(w, need, end=bin_end):
    """Positions taken of the weights w, by the rule that the kernel writes by: all above T and, of those equal to it, as
    many as are missing."""
    v = orders(w)
    lo, hi, above = int(v.min()), int(v.max()), 0
    T, steps = lo, 0
    while lo < hi:
        steps += 1
        assert steps <= 3
        shift = max(0, (hi - lo).bit_length() - 11)
        top = (hi - lo) >> shift
        assert top < 2048
        in_range = (v >= lo) & (v <= hi)
        count = np.bincount(top - ((v[in_range] - lo) >> shift), minlength=2048)
        reached = above + np.cumsum(count)
        k = int(np.argmax(reached >= need))
        above += int(count[:k].sum())
        lo += (top - k) << shift
        hi = end(lo, hi, shift)
        T = lo
        if above + int(count[k]) == need:
            above, T = need, lo - 1
            break
    taken, equal = [], need - above
    for i, x in enumerate(v):
        if x > T or (x == T and equal > 0):
            taken.append(i)
            equal -= x == T
    return taken
