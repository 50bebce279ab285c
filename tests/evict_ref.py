"""Weights and eviction of the 8-bit cache, and rotary positions, from their definitions in 64 bits on the CPU (numpy;
shares no code with the kernels). Caches are arrays of the numbers that the codes stand for, [pages, Hkv, page, d]."""
import numpy as np

import kvq8_ref as ref


def keep_positions(w, keep, recent):
    """Old positions of the tokens kept of one head with weights w, in order."""
    n = len(w)
    if n <= keep:
        return list(range(n))
    old = n - recent
    rank = [(-np.inf if np.isnan(x) else -float(x), not np.isnan(x), i) for i, x in enumerate(w[:old])]
    rank = [(0 if not number else 1, a, i) for a, number, i in rank]  # NaN before all numbers
    return sorted(i for _, _, i in sorted(rank)[: keep - recent]) + list(range(old, n))


def evict(codes, scales, fmt, table, lens, kept):
    """In place: the kept tokens of each (sequence, head) to the front of the sequence's pages."""
    page, d = codes.shape[2], codes.shape[3]
    for s, n in enumerate(lens):
        for h in range(codes.shape[1]):
            at = kept[s][h]
            if not at:
                continue
            x = ref.gather(codes, scales, table[s], n)[h][at]  # a copy
            for j in range(0, len(at), page):
                if at[j : j + page] == list(range(j, min(j + page, len(at)))):
                    continue
                p, v = table[s][j // page], x[j : j + page]
                now = ref.scale_for(np.abs(v).max(), fmt)
                scales[p, h] = now
                codes[p, h, : len(v)] = ref.round_code(v / now, fmt) if now > 0 else 0.0


def weights(q, k, lse, scale, causal):
    """One sequence: q [H, Nq, d], k [Hkv, n, d], lse [H, Nq]. Returns the weight that each key receives [Hkv, n] and a
    bound of what 32-bit arithmetic may make of it: a score is a sum of d products (each addition off by 2^-23 of the
    sum of magnitudes at most), the exponent takes three roundings of its terms and the exponential two units."""
    H, Nq, d = q.shape
    n, group = k.shape[1], H // k.shape[0]
    out, bound = np.zeros(k.shape[:2]), np.zeros(k.shape[:2])
    for h in range(H):
        s = scale * (q[h] @ k[h // group].T)  # [Nq, n]
        mag = scale * (np.abs(q[h]) @ np.abs(k[h // group]).T)
        seen = np.ones((Nq, n), bool)
        if causal:
            seen = np.arange(n)[None, :] <= np.arange(Nq)[:, None] + n - Nq
        l = lse[h][:, None]
        with np.errstate(invalid="ignore", over="ignore"):
            p = np.where(seen & np.isfinite(l), np.exp(s - l), 0.0)
        rel = d * 2.0 ** -23 * mag + 2.0 ** -21 * (1 + np.abs(s) + np.where(np.isfinite(l), np.abs(l), 0.0))
        out[h // group] += p.sum(0)
        bound[h // group] += (p * rel).sum(0) * 1.1
    return out, bound + 2.0 ** -22 * H * Nq * out + 1e-37


def rotary(x, positions, inv_freq, axis, inverse):
    """x [..., d] with positions [axes, ...] without the heads; x's axis -2 is the heads. Angles in extended precision."""
    r = len(inv_freq)
    two_pi = np.longdouble(2) * np.arctan2(np.longdouble(0), np.longdouble(-1))
    y = x.astype(np.float64).copy()
    for i in range(r):
        turns = positions[axis[i]].astype(np.longdouble) * np.longdouble(inv_freq[i]) / two_pi
        a = ((turns - np.rint(turns)) * two_pi).astype(np.float64)[..., None]
        if inverse:
            a = -a
        y[..., i] = x[..., i] * np.cos(a) - x[..., i + r] * np.sin(a)
        y[..., i + r] = x[..., i] * np.sin(a) + x[..., i + r] * np.cos(a)
    return y
