"""CPU model of the barrier protocol of the d = 64 backward over keys of another length, in which a CTA goes through
several key blocks (fa_bwd_cross_kernel_h64). It steps the roles in random orders, with each issuing warp's products
in order in a queue of its own and copies landing in any order, and keeps track of what every buffer holds."""
import random

from pipeline_model import Bar, Deadlock


def simulate_bwd_cross(counts, stages, seed, acc_free=True, kv_free_count=2, acc_waits=True, readout_first=True):
    """counts: iterations of each of the CTA's key blocks. Iterations are numbered through (g); block n uses K/V buffer
    n & 1. Hazards that fail here: a K/V buffer or a Q/dO stage refilled while a product still reads it; S/dP, packed
    P^T, dS rows or dQ columns overwritten before their reader; dV/dK restarted before the gradient warps have taken the
    last block's; a block's dV/dK taken before its last product. Mutations that must be caught: acc_free=False (the
    first dV/dK product of a block does not wait for the last block's read-out), kv_free_count=1, acc_waits=False,
    readout_first=False (dV/dK taken without waiting for the block's last dQ)."""
    rnd = random.Random(seed)
    block = [n for n, c in enumerate(counts) for _ in range(c)]           # block of iteration g
    first = [g == 0 or block[g] != block[g - 1] for g in range(len(block))]
    last = [g + 1 == len(block) or block[g] != block[g + 1] for g in range(len(block))]
    G = len(block)
    B = {}
    for name, c in (("dq_full", 1), ("dq_free", 256), ("drain", 2), ("acc_free", 256)):
        B[name] = Bar(name, c)
    for h in range(2):
        for name, c in (("sp_full", 1), ("p_full", 128), ("stats", 128), ("acc_done", 1), ("kv_full", 1),
                        ("kv_free", kv_free_count)):
            B[f"{name}{h}"] = Bar(f"{name}{h}", c)
    for s in range(stages):
        B[f"qd_full{s}"] = Bar(f"qd_full{s}", 1)
        B[f"qd_empty{s}"] = Bar(f"qd_empty{s}", 2)
    stage, kv = [None] * stages, [None, None]
    sdp, dq, acc = [None, None], [None], [set()]      # acc: iterations and halves summed in dV/dK
    taken = [[None] * 4, [None] * 4]                  # block whose dV (half 0) or dK (half 1) a warp has taken
    pt = [[None] * 4 for _ in range(2)]
    ds = [[[None] * 4 for _ in range(2)] for _ in range(2)]
    q1, q2, tma = [], [], []

    def s_mma(g, h):
        def run():
            assert stage[g % stages] == g, f"S({g},{h}) reads stage holding {stage[g % stages]}"
            assert kv[block[g] & 1] == block[g], f"S({g},{h}) reads K of block {kv[block[g] & 1]}"
            sdp[h] = g
        return ("mma", run)

    def acc_mma(g, h):
        def run():
            assert stage[g % stages] == g
            assert all(x == g for x in pt[h]), f"dV({g},{h}) reads P^T {pt[h]}"
            assert all(x == ("dS", g) for x in ds[g & 1][h]), f"dK({g},{h}) reads dS rows {ds[g & 1][h]}"
            if first[g] and h == 0:
                if block[g] > 0:
                    assert all(x == block[g] - 1 for t in taken for x in t), f"block {block[g]} restarts dV/dK: {taken}"
                acc[0] = set()
            acc[0].add((g, h))
        return ("mma", run)

    def dq_mma(g):
        def run():
            assert kv[block[g] & 1] == block[g], f"dQ({g}) reads K of block {kv[block[g] & 1]}"
            for h in range(2):
                assert all(x == ("dS", g) for x in ds[g & 1][h]), f"dQ({g}) reads dS rows {ds[g & 1][h]}"
            dq[0] = g
        return ("mma", run)

    def producer():
        g = 0
        for n, c in enumerate(counts):
            yield ("wait", f"kv_free{n & 1}", (n >> 1) - 1)
            tma.append((f"kv_full{n & 1}", kv, n & 1, n))
            for _ in range(c):
                s = g % stages
                yield ("wait", f"qd_empty{s}", g // stages - 1)
                tma.append((f"qd_full{s}", stage, s, g))
                g += 1

    def warp1():
        if G:
            yield ("wait", "kv_full0", 0)
            yield ("wait", "qd_full0", 0)
            q1.extend([s_mma(0, 0), ("commit", "sp_full0"), s_mma(0, 1), ("commit", "sp_full1"), ("commit", "qd_empty0")])
            if last[0]:
                q1.append(("commit", "kv_free0"))
        for g in range(G):
            more = g + 1 < G
            yield ("wait", "p_full0", g)
            if more:
                n = block[g + 1]
                if first[g + 1]:
                    yield ("wait", f"kv_full{n & 1}", n >> 1)
                yield ("wait", f"qd_full{(g + 1) % stages}", (g + 1) // stages)
                q1.extend([s_mma(g + 1, 0), ("commit", "sp_full0")])
            yield ("wait", "p_full1", g)
            if more:
                q1.extend([s_mma(g + 1, 1), ("commit", "sp_full1"), ("commit", f"qd_empty{(g + 1) % stages}")])
                if last[g + 1]:
                    q1.append(("commit", f"kv_free{n & 1}"))
        q1.append(("commit", "drain"))
        yield ("wait", "drain", 0)

    def warp2():
        for g in range(G):
            n, s = block[g], g % stages
            if first[g]:
                yield ("wait", f"kv_full{n & 1}", n >> 1)
            yield ("wait", "p_full0", g)
            yield ("wait", f"qd_full{s}", g // stages)
            if first[g] and n > 0 and acc_free:
                yield ("wait", "acc_free", n - 1)
            q2.extend([acc_mma(g, 0), ("commit", "acc_done0")])
            yield ("wait", "p_full1", g)
            q2.extend([acc_mma(g, 1), ("commit", "acc_done1"), ("commit", f"qd_empty{s}")])
            if g > 0:
                yield ("wait", "dq_free", g - 1)
            q2.extend([dq_mma(g), ("commit", "dq_full")])
            if last[g]:
                q2.append(("commit", f"kv_free{n & 1}"))
        q2.append(("commit", "drain"))

    def grads(h, w):
        def readout(g):
            yield ("wait", "dq_full", g)
            assert dq[0] == g, f"readout({g}) finds dQ of {dq[0]}"
            yield ("arrive", "dq_free", 32)
            assert ds[g & 1][h][w] == ("dS", g)
            ds[g & 1][h][w] = ("stage", g)

        def take(n):  # dV (half 0) or dK (half 1) of block n, after the first pass of the next block
            want = {(g, k) for g in range(G) if block[g] == n for k in range(2)}
            assert acc[0] == want, f"block {n}: dV/dK taken with {acc[0]}"
            taken[h][w] = n

        for g in range(G):
            yield ("arrive", f"stats{h}", 32)
            yield ("wait", f"stats{h}", g)
            yield ("wait", f"sp_full{h}", g)
            assert sdp[h] == g, f"pass({g},{h}) reads S/dP of {sdp[h]}"
            if g > 0 and acc_waits:
                yield ("wait", f"acc_done{h}", g - 1)
            pt[h][w] = g
            ds[g & 1][h][w] = ("dS", g)
            yield ("arrive", f"p_full{h}", 32)
            if g > 0:
                if first[g] and not readout_first:
                    take(block[g - 1])
                yield from readout(g - 1)
                if first[g]:
                    if readout_first:
                        take(block[g - 1])
                    yield ("arrive", "acc_free", 32)
        if G:
            yield from readout(G - 1)
            take(block[G - 1])
            yield ("arrive", "acc_free", 32)

    agents = {"producer": producer(), "warp1": warp1(), "warp2": warp2()}
    for h in range(2):
        for w in range(4):
            agents[f"g{h}.{w}"] = grads(h, w)
    waiting = {k: None for k in agents}
    # kv_full0/1, sp_full0/1 and the like are told apart by name; index -1 is a phase before the first
    while agents or q1 or q2 or tma:
        ready = [k for k in agents if waiting[k] is None or B[waiting[k][1]].done(waiting[k][2])]
        ready += ["#q1"] * bool(q1) + ["#q2"] * bool(q2) + ["#tma"] * bool(tma)
        if not ready:
            raise Deadlock(f"deadlock: {[(k, waiting[k]) for k in agents]}")
        c = rnd.choice(ready)
        if c in ("#q1", "#q2"):
            kind, x = (q1 if c == "#q1" else q2).pop(0)
            if kind == "mma":
                x()
            else:
                B[x].arrive(1)
        elif c == "#tma":
            name, where, slot, what = tma.pop(rnd.randrange(len(tma)))
            where[slot] = what
            B[name].arrive(1)
        else:
            try:
                while True:
                    ev = next(agents[c])
                    if ev[0] == "arrive":
                        B[ev[1]].arrive(ev[2])
                        continue
                    waiting[c] = ev
                    break
            except StopIteration:
                del agents[c]
                waiting[c] = None
    return True


def plan(valid, n_it, num_sms):
    """bwd_cross_plan: (full, parts, items) of `valid` key blocks of n_it iterations each."""
    tail = valid % num_sms
    parts, best = 1, n_it + 1
    for m in (1, 2):
        if tail:
            k = min(m * num_sms // tail, n_it)
            cost = -(-tail * k // num_sms) * (-(-n_it // k) + 2)
            if k > 1 and cost < best:
                best, parts = cost, k
    return valid - tail, parts, valid - tail + tail * parts


def slots(blocks, n_it, num_sms):
    """bwd_cross_slots: workspace slots for any number of blocks up to `blocks`."""
    return 0 if n_it < 2 else min(min(blocks, num_sms) * n_it, 2 * num_sms)


def item(full, parts, a, n_it):
    """cross_item: (rank of the block, first iteration, iterations, slot) of item a."""
    if a < full or parts == 1:
        return a, 0, n_it, -1
    part = (a - full) % parts
    each, more = divmod(n_it, parts)
    return full + (a - full) // parts, part * each + min(part, more), each + (part < more), a - full
