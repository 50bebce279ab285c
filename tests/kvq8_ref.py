"""The 8-bit cache and attention over it from their definitions, in 64 bits on the CPU (numpy; shares no code with
the kernels). A cache is a dict of codes as the numbers they stand for, [pages, Hkv, page, d], and scales."""
import numpy as np

QMAX = {"int8": 127.0, "e4m3": 448.0}


def round_code(x, fmt):
    """Nearest code, ties to even, saturated; x already divided by the scale."""
    if fmt == "int8":
        return np.clip(np.rint(x), -127, 127)
    a = np.abs(x)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    step = 2.0 ** (np.maximum(e, -6) - 3)  # 3 mantissa bits; subnormals share the step of 2^-6
    return np.clip(np.rint(x / step) * step, -448, 448)


def scale_for(most, fmt):
    if most == 0:
        return 0.0
    e = -110
    while most > QMAX[fmt] * 2.0 ** e and e < 120:
        e += 1
    return 2.0 ** e


def append(codes, scales, fmt, x, table, cu, lens):
    """In place: tokens x [total, Hkv, d] of each sequence behind its lens[s] held ones. Non-finite values count as 0."""
    page = codes.shape[2]
    x = np.where(np.isfinite(x), x, 0.0)
    for s in range(len(lens)):
        new = x[cu[s] : cu[s + 1]]
        for t in range(lens[s] // page, (lens[s] + len(new) + page - 1) // page if len(new) else 0):
            lo, hi = max(lens[s] - t * page, 0), min(lens[s] + len(new) - t * page, page)
            at = new[t * page + lo - lens[s] : t * page + hi - lens[s]]  # [hi - lo, Hkv, d]
            for h in range(codes.shape[1]):
                p = table[s][t]
                now = scale_for(np.abs(at[:, h]).max(), fmt)
                if lo > 0:
                    old = float(scales[p, h])
                    now = max(now, old)
                    if now > 0:
                        codes[p, h, :lo] = round_code(codes[p, h, :lo] * (old / now), fmt)
                scales[p, h] = now
                codes[p, h, lo:hi] = round_code(at[:, h] / now, fmt) if now > 0 else 0.0


def gather(codes, scales, table_row, n):
    """Values of a sequence's first n positions: [Hkv, n, d]."""
    page = codes.shape[2]
    pages = np.asarray(table_row[: (n + page - 1) // page], dtype=np.int64)
    v = codes[pages].astype(np.float64) * scales[pages].astype(np.float64)[:, :, None, None]
    return v.transpose(1, 0, 2, 3).reshape(codes.shape[1], -1, codes.shape[3])[:, :n]


def attend(q, k, v, scale, causal):
    """One sequence: q [H, Nq, d], k, v [Hkv, n, d]. Returns out, lse, and for tolerances sum_j p_ij |v_j| (per output
    element), the largest |score| of each row, and the sum of exp(score - max)."""
    H, Nq, d = q.shape
    n = k.shape[1]
    out, mag = np.zeros((H, Nq, d)), np.zeros((H, Nq, d))
    lse, top, tot = np.full((H, Nq), -np.inf), np.zeros((H, Nq)), np.ones((H, Nq))
    for h in range(H):
        kk, vv = k[h // (H // k.shape[0])], v[h // (H // k.shape[0])]
        for i in range(Nq):
            last = n if not causal else min(n, i + n - Nq + 1)
            if last <= 0:
                continue
            s = scale * (kk[:last] @ q[h, i])
            m = s.max()
            p = np.exp(s - m)
            tot[h, i] = p.sum()
            lse[h, i] = m + np.log(tot[h, i])
            top[h, i] = np.abs(s).max()
            out[h, i] = (p / tot[h, i]) @ vv[:last]
            mag[h, i] = (p / tot[h, i]) @ np.abs(vv[:last])
    return out, lse, mag, top, tot
