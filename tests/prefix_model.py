"""CPU model of the barrier protocol of the kernel that attends to a shared prefix for the rows of all sequences
(fa_kvq8_prefix_tc.cu). It steps the roles in random orders, with each issuing warp's products in order in a queue of
its own and copies landing in any order, and keeps track of what every buffer holds."""
import random

from pipeline_model import Bar, Deadlock

WARPS = 8  # converters


def simulate_prefix(blocks, tiles, raw, seed, dead=(), s_free=True, k_empty=True, v_empty=True, raw_empty=True,
                    v_empty_count=None, dead_wait=True, pv_wait=True):
    """One CTA's run of `blocks` 128-key blocks for `tiles` tiles of query rows, with `raw` tiles of raw codes in flight.
    `dead`: (tile, warp) pairs without rows, which only keep the barriers. Hazards that fail here: a raw slot refilled
    before every converter has read it, a K or V tile rewritten while a product still reads it, the S buffer overwritten
    before it is copied out, P overwritten before its product has read it, an O that misses a block. Mutations that must be
    caught: each of the flags off, v_empty_count=1 with two tiles."""
    rnd = random.Random(seed)
    B = {}
    for name, count in (("s_free", 128), ("drain", tiles + 1), ("scan", WARPS * 32)):
        B[name] = Bar(name, count)
    for s in range(raw):
        B[f"raw_full{s}"] = Bar(f"raw_full{s}", 1)
        B[f"raw_empty{s}"] = Bar(f"raw_empty{s}", WARPS * 32)
    for s in range(2):
        B[f"k_full{s}"] = Bar(f"k_full{s}", WARPS * 32)
        B[f"v_full{s}"] = Bar(f"v_full{s}", WARPS * 32)
        B[f"k_empty{s}"] = Bar(f"k_empty{s}", 1)
        B[f"v_empty{s}"] = Bar(f"v_empty{s}", tiles if v_empty_count is None else v_empty_count)
    for t in range(tiles):
        B[f"q_full{t}"] = Bar(f"q_full{t}", 128)
        B[f"s_full{t}"] = Bar(f"s_full{t}", 1)
        B[f"p_full{t}"] = Bar(f"p_full{t}", 128)
        for b in range(2):
            B[f"pv_done{t}{b}"] = Bar(f"pv_done{t}{b}", 1)
            B[f"s_issued{t}{b}"] = Bar(f"s_issued{t}{b}", 1)
    raw_holds = [None] * raw
    kv = {"k": [[None] * WARPS for _ in range(2)], "v": [[None] * WARPS for _ in range(2)]}
    s_buf, s_read = [None], [None]                        # (tile, block) in S; warps that have copied it out
    p_buf = [[None] * 4 for _ in range(tiles)]            # block in each warp's rows of P
    o_sum = [[] for _ in range(tiles)]
    queues = {"S": [], **{f"PV{t}": [] for t in range(tiles)}}
    copies = []
    order = []                                            # of the tiles of codes
    for j in range(-1, blocks):
        if j + 1 < blocks:
            order.append(("k", j + 1))
        if j >= 0:
            order.append(("v", j))

    def s_mma(t, j):
        def run():
            assert kv["k"][j % 2] == [j] * WARPS, f"S({t},{j}) reads K of {kv['k'][j % 2]}"
            if s_buf[0] is not None:
                assert s_read[0] == set(range(4)), f"S({t},{j}) overwrites S{s_buf[0]}, read by {s_read[0]}"
            s_buf[0], s_read[0] = (t, j), set()
        return ("mma", run)

    def pv_mma(t, j):
        def run():
            assert kv["v"][j % 2] == [j] * WARPS, f"PV({t},{j}) reads V of {kv['v'][j % 2]}"
            for w in range(4):
                assert (t, w) in dead or p_buf[t][w] == j, f"PV({t},{j}) reads P of {p_buf[t]}"
                p_buf[t][w] = ("read", j)
            o_sum[t].append(j)
        return ("mma", run)

    def loader():
        for pos, (what, j) in enumerate(order):
            s = pos % raw
            if raw_empty:
                yield ("wait", f"raw_empty{s}", pos // raw - 1)
            copies.append((s, (what, j)))
            yield ("step",)

    def converter(w):
        yield ("arrive", "scan", 32)
        for pos, (what, j) in enumerate(order):
            s, slot = pos % raw, j % 2
            yield ("wait", f"raw_full{s}", pos // raw)
            if k_empty if what == "k" else v_empty:
                yield ("wait", f"{what}_empty{slot}", j // 2 - 1)
            yield ("step",)
            assert raw_holds[s] == (what, j), f"{what}{j} converted from a slot that holds {raw_holds[s]}"
            kv[what][slot][w] = j
            yield ("arrive", f"raw_empty{s}", 32)
            yield ("arrive", f"{what}_full{slot}", 32)

    def s_issuer():
        for t in range(tiles):
            yield ("wait", f"q_full{t}", 0)
        issued = 0
        yield ("wait", "k_full0", 0)
        for j in range(blocks):
            for t in range(tiles):
                if t == tiles - 1 and j + 1 < blocks:
                    yield ("wait", f"k_full{(j + 1) % 2}", (j + 1) // 2)
                if issued and s_free:
                    yield ("wait", "s_free", issued - 1)
                issued += 1
                queues["S"] += [s_mma(t, j), ("commit", f"s_full{t}")]
                yield ("arrive", f"s_issued{t}{j & 1}", 1)
            queues["S"].append(("commit", f"k_empty{j % 2}"))
        queues["S"].append(("commit", "drain"))

    def pv_issuer(t):
        for j in range(blocks):
            yield ("wait", f"v_full{j % 2}", j // 2)
            yield ("wait", f"p_full{t}", j)
            if j + 1 < blocks:
                yield ("wait", f"s_issued{t}{(j + 1) & 1}", (j + 1) >> 1)
            queues[f"PV{t}"] += [pv_mma(t, j), ("commit", f"pv_done{t}{j & 1}"), ("commit", f"v_empty{j % 2}")]
        queues[f"PV{t}"].append(("commit", "drain"))

    def softmax(t, w):
        yield ("arrive", f"q_full{t}", 32)
        yield ("wait", "scan", 0)
        for j in range(blocks):
            yield ("wait", f"s_full{t}", j)
            if (t, w) not in dead:
                assert s_buf[0] == (t, j), f"softmax({t},{j}) finds S{s_buf[0]}"
            s_read[0].add(w)
            yield ("arrive", "s_free", 32)
            if j > 0 and (pv_wait if (t, w) not in dead else dead_wait):
                yield ("wait", f"pv_done{t}{(j - 1) & 1}", (j - 1) >> 1)
            if (t, w) not in dead:
                if j > 0:
                    assert p_buf[t][w] == ("read", j - 1), f"P({t},{j}) overwrites P of {p_buf[t][w]}"
                p_buf[t][w] = j
            yield ("arrive", f"p_full{t}", 32)
        yield ("wait", f"pv_done{t}{(blocks - 1) & 1}", (blocks - 1) >> 1)
        if (t, w) not in dead:
            assert o_sum[t] == list(range(blocks)), f"O of tile {t} sums {o_sum[t]}"

    agents = {"loader": loader(), "S": s_issuer()}
    for w in range(WARPS):
        agents[f"c{w}"] = converter(w)
    for t in range(tiles):
        agents[f"PV{t}"] = pv_issuer(t)
        for w in range(4):
            agents[f"m{t}.{w}"] = softmax(t, w)
    waiting = {k: None for k in agents}
    while agents or copies or any(queues.values()):
        ready = [k for k in agents if waiting[k] is None or waiting[k][0] == "step" or B[waiting[k][1]].done(waiting[k][2])]
        ready += ["#" + q for q in queues if queues[q]] + ["#copy"] * bool(copies)
        if not ready:
            raise Deadlock(f"deadlock: {[(k, waiting[k]) for k in agents]}")
        c = rnd.choice(ready)
        if c == "#copy":
            s, what = copies.pop(rnd.randrange(len(copies)))
            raw_holds[s] = what
            B[f"raw_full{s}"].arrive(1)
        elif c[0] == "#":
            kind, x = queues[c[1:]].pop(0)
            if kind == "mma":
                x()
            else:
                B[x].arrive(1)
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
    assert B["drain"].phase == 1
    return True
