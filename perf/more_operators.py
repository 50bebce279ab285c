"""What is measured of serving from the 8-bit key/value cache with a shared prefix and under a memory budget, and of
rotary positions with several axes.

Four operators, each a case's "op":

  prefix   attention of 1 to 16 query rows per sequence over a prefix that all sequences share and the sequence's own
           cached tokens behind it
  weights  the softmax weight that each cached key receives, summed over the query rows that share its head and added
           to what it has received so far
  evict    the cache cut down to the keys of the greatest weight and the latest ones, each head's kept tokens moved to
           the front of its pages
  rotary   queries and keys rotated by angles of several axes (time, height, width), and the gradient of that

`run` computes them in elementary torch operations in 32 bits (angles in 64), or, where `own` is set, through the
package's entry points. `exact` computes them from the definitions in 64 bits.

The cache: codes [pages, Hkv, page, d] (int8, or float8_e4m3fn), one fp32 scale for each page and head, K and V
apart; a value is code * scale. Eviction leaves a page alone whose kept tokens all stay where they are; any other
page gets the smallest power of two that holds its tokens (2^-110 to 2^120; 0 when all are 0) and its codes rounded
to it.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
QMAX = {"int8": 127.0, "e4m3": 448.0}
DEV = "cuda"


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a small batch behind a short instruction: latency
        dict(name="prefix_small", op="prefix", fmt="int8", dtype="bf16", B=3, H=8, Hkv=8, Nq=1, d=64, page=16, prefix=1000,
             length=100, causal=False, ragged=True),
        # an ordinary decoding step behind a system prompt, grouped heads
        dict(name="prefix_step", op="prefix", fmt="int8", dtype="bf16", B=16, H=32, Hkv=8, Nq=1, d=128, page=16,
             prefix=8192, length=1024, causal=False, ragged=True),
        # checking drafted tokens: five causal rows per sequence
        dict(name="prefix_draft", op="prefix", fmt="e4m3", dtype="fp16", B=12, H=16, Hkv=4, Nq=5, d=64, page=64,
             prefix=6001, length=700, causal=True, ragged=True),
        # a large serving batch that asks about one long document
        dict(name="prefix_large", op="prefix", fmt="e4m3", dtype="bf16", B=64, H=64, Hkv=8, Nq=1, d=128, page=64,
             prefix=32768, length=2048, causal=False, ragged=True),
        # one user's weights after a step: latency
        dict(name="weights_one", op="weights", fmt="int8", dtype="bf16", B=1, H=8, Hkv=8, Nq=1, d=64, page=16, length=509,
             causal=False, ragged=False),
        # weights after drafted tokens, many rows to a key
        dict(name="weights_draft", op="weights", fmt="e4m3", dtype="fp16", B=12, H=16, Hkv=4, Nq=5, d=64, page=64,
             length=6001, causal=True, ragged=True),
        # weights after a step of a large batch
        dict(name="weights_step", op="weights", fmt="int8", dtype="bf16", B=64, H=32, Hkv=8, Nq=1, d=128, page=16,
             length=8192, causal=False, ragged=True),
        # one conversation cut down
        dict(name="evict_one", op="evict", fmt="e4m3", B=1, Hkv=4, d=64, page=32, length=1500, keep=1100, recent=100,
             ragged=False),
        # a batch over its budget
        dict(name="evict_batch", op="evict", fmt="int8", B=24, Hkv=8, d=128, page=16, length=12000, keep=5000, recent=500,
             ragged=True),
        # a decoding step's queries and keys
        dict(name="rotary_step", op="rotary", dtype="bf16", layout="packed", B=1, N=16, H=32, Hkv=8, d=128, pairs=64, far=40000,
             inverse=False),
        # prompts with images and video, packed
        dict(name="rotary_prompt", op="rotary", dtype="bf16", layout="packed", B=1, N=30011, H=32, Hkv=8, d=128, pairs=64,
             far=100000, inverse=False),
        # gradients of a training batch, rotated back
        dict(name="rotary_grad", op="rotary", dtype="fp16", layout="heads", B=4, N=4099, H=16, Hkv=16, d=64, pairs=24, far=0,
             inverse=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "weights", "evict", "rotary"])
    c = dict(op=op, d=rng.choice([64, 128]), Hkv=rng.choice([1, 2, 5, 8]))
    if op != "evict":
        c["dtype"] = rng.choice(["bf16", "fp16"])
        c["H"] = c["Hkv"] * rng.choice([1, 2, 4, 5, 8])
    if op == "rotary":
        c.update(layout=rng.choice(["packed", "heads"]), inverse=rng.random() < 0.4, far=_log(rng, 1, 200000),
                 pairs=rng.choice([c["d"] // 2, c["d"] // 2, 24, 16]))
        c["B"] = 1 if c["layout"] == "packed" else _log(rng, 1, 16)
        c["N"] = _log(rng, 1, max(1, min(40000, 30011 * 40 * 128 // (c["B"] * (c["H"] + c["Hkv"]) * c["d"]))))
        return c
    c.update(fmt=rng.choice(["int8", "e4m3"]), page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.7)
    if op == "evict":
        c["B"] = _log(rng, 1, 40)
        c["length"] = _log(rng, 2, max(2, min(16000, 24 * 8 * 4000 * 128 // (c["B"] * c["Hkv"] * c["d"]))))
        c["keep"] = rng.randint(1, c["length"])
        c["recent"] = rng.randint(0, c["keep"])
        return c
    c.update(Nq=rng.choice([1, 1, 1, 2, 3, 7, 16]), B=_log(rng, 1, 64), causal=rng.random() < 0.5)
    rows = c["B"] * c["H"] * c["Nq"]
    if op == "weights":
        most = 64 * 8 * 5000 * 128 // (c["B"] * c["Hkv"] * c["d"])
        c["length"] = _log(rng, 1, max(1, min(20000, most, 64 * 32 * 5000 * 128 // (rows * c["d"]))))
    else:
        c["length"] = _log(rng, 1, max(1, min(4096, 64 * 8 * 2048 * 128 // (c["B"] * c["Hkv"] * c["d"]),
                                              64 * 64 * 32768 // (2 * rows))))
        c["prefix"] = _log(rng, 1, max(1, min(32768, 64 * 64 * 32768 // (2 * rows))))
    return c


def _lengths(case):
    """Whole lengths of a ragged batch, from the case alone: a quarter of the longest to the longest, the first one that."""
    most, count = case["length"], case["B"]
    if not case["ragged"]:
        return [most] * count
    r = np.random.RandomState(count * 7919 + most)
    got = [int(x) for x in r.randint(max(1, most // 4), most + 1, count)]
    got[0] = most
    return got


def _pages(case, n):
    return (n + case["page"] - 1) // case["page"]


def work(case):
    """Each input read once, each output written once; products counted for the visible pairs. Of an eviction's cache the
    kept tokens of the sequences that are over the budget are read and written."""
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    if op == "rotary":
        values = case["B"] * case["N"] * (case["H"] + Hkv) * d
        return {"bytes": values * 4 + 12 * case["B"] * case["N"],
                "flops": 3 * case["B"] * case["N"] * (case["H"] + Hkv) * 2 * case["pairs"]}
    lens = _lengths(case)
    if op == "evict":
        over = sum(n > case["keep"] for n in lens)
        moved = over * Hkv * case["keep"] * d * 2
        scales = over * Hkv * _pages(case, case["keep"]) * 8
        return {"bytes": 2 * (moved + scales) + sum(lens) * Hkv * 4 + case["B"] * Hkv * (_capacity(case) + case["keep"]) * 4,
                "flops": 0}
    rows = case["B"] * case["H"] * case["Nq"]
    own_bytes = sum(lens) * Hkv * d + sum(_pages(case, n) for n in lens) * Hkv * 4
    pairs = sum(lens) * case["H"] * case["Nq"]
    if op == "weights":
        return {"bytes": own_bytes + sum(lens) * Hkv * 8 + rows * (d * 2 + 4), "flops": 2 * pairs * d}
    shared = case["prefix"] * Hkv * d + _pages(case, case["prefix"]) * Hkv * 4
    return {"bytes": 2 * (own_bytes + shared) + rows * (d * 4 + 4), "flops": 4 * (pairs + rows * case["prefix"]) * d}


# ---------------------------------------------------------------- inputs
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _power(e):
    """2^e as fp32, by its bits (a pow is not exact everywhere)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _capacity(case):
    """Positions that a row of the page table reaches."""
    return _pages(case, case["length"]) * case["page"]


def _cache(case, g, extra):
    """A cache with room for every sequence's tokens and for `extra` tokens of a prefix, its pages in a random order, every
    page holding codes of normal values under scales of the size that an append gives them."""
    page, heads, d = case["page"], case["Hkv"], case["d"]
    need = [_pages(case, n) for n in _lengths(case)]
    shared = _pages(case, extra)
    total = sum(need) + shared + 3
    order = torch.randperm(total, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    width = max(need)
    first = torch.tensor([0] + [int(x) for x in np.cumsum(need)][:-1], device=DEV).unsqueeze(1)
    at = first + torch.arange(width, device=DEV).unsqueeze(0)
    table = order[at.clamp(max=total - 1)].contiguous()
    table[torch.arange(width, device=DEV).unsqueeze(0) >= torch.tensor(need, device=DEV).unsqueeze(1)] = 0
    shape = (total, heads, page, d)
    state = {"table": table, "prefix_table": order[sum(need) : sum(need) + max(shared, 1)].contiguous()}
    for n in ("k", "v"):
        x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float16)
        if case["fmt"] == "int8":
            state[n + "_codes"] = (x * 27).round_().clamp_(-127, 127).to(torch.int8)
            e = -5
        else:
            state[n + "_codes"] = (x * 90).clamp_(-448, 448).to(torch.float8_e4m3fn)
            e = -7
        more = torch.randint(-1, 2, (total, heads), generator=g, device=DEV)
        state[n + "_scale"] = _power(more + e)
    return state


def _positions(case, g):
    """Positions [3, B, N] of text with pictures in between: along text all axes count on together; within a picture
    time stands still and height and width go over its grid."""
    B, N = case["B"], case["N"]
    token = torch.arange(N, device=DEV).expand(B, N)
    start = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device=DEV)
    side, period = 24, 24 * 24 + 200
    inside, block = token % period, token // period
    base = start + block * (200 + side)
    text, patch = inside < 200, inside - 200
    t = torch.where(text, base + inside, base + 200)
    h = torch.where(text, base + inside, base + 200 + patch // side)
    w = torch.where(text, base + inside, base + 200 + patch % side)
    return torch.stack([t, h, w]).int().contiguous()


def _frequencies(case):
    """10000^(-i / pairs) for the pair i, and the axis that its angle goes by: the first quarter of the pairs time, the
    rest halved between height and width."""
    n = case["pairs"]
    inv = torch.tensor([10000.0 ** (-i / n) for i in range(n)], dtype=torch.float64)
    a, b = n // 4, n // 4 + (n - n // 4) // 2
    axis = torch.tensor([0 if i < a else 1 if i < b else 2 for i in range(n)], dtype=torch.int32)
    return inv, axis


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2 + 1)
    op, d = case["op"], case["d"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(DTYPES[case["dtype"]])

    if op == "rotary":
        B, N, H, Hkv = case["B"], case["N"], case["H"], case["Hkv"]
        inv, axis = _frequencies(case)
        s = {"inv_freq": inv, "axis": axis, "positions": _positions(case, g)}
        if case["layout"] == "packed":  # parts of one projection's output
            qkv = normal(N, H + 2 * Hkv, d)
            s.update(q=qkv[:, :H], k=qkv[:, H : H + Hkv])
            s["positions"] = s["positions"][:, 0].contiguous()
        else:
            s.update(q=normal(B, H, N, d), k=normal(B, Hkv, N, d))
    else:
        lens = _lengths(case)
        s = _cache(case, g, case.get("prefix", 0))
        s["lens"] = _ints(lens)
        if op == "evict":  # weights as steps leave them: a few keys have most, many have next to none, some nothing
            w = torch.exp(3.0 * torch.randn((case["B"], case["Hkv"], _capacity(case)), generator=g, device=DEV) - 4.0)
            w = torch.where(torch.rand(w.shape, generator=g, device=DEV) < 0.1, torch.zeros_like(w), w)
            held = torch.arange(_capacity(case), device=DEV) < s["lens"][:, None]
            s["weight"] = torch.where(held[:, None], w, torch.zeros_like(w))
        else:
            s.update(q=normal(case["B"], case["H"], case["Nq"], d), max_len=max(lens))
            if op == "prefix":
                s["prefix_len"] = _ints([case["prefix"]])
            else:
                s["lse"] = _attend(s, case, False)[1]  # what the attention left behind
                s["weight"] = torch.rand((case["B"], case["Hkv"], _capacity(case)), generator=g, device=DEV)
    s["case"] = dict(case)
    return s


# ---------------------------------------------------------------- plain forms
def _values(s, n, table):
    """Codes of a table's pages times their scales, [..., Hkv, tokens, d] in 32 bits."""
    codes, t = s[n + "_codes"], table.long()
    x = codes.view(torch.uint8)[t].view(codes.dtype).float() * s[n + "_scale"][t][..., None, None]
    return x.transpose(-4, -3).flatten(-3, -2)


def _own_scores(s, case):
    """Scores over each sequence's own keys, [B, Hkv, group, Nq, keys], excluded ones -inf."""
    B, H, Nq, d, Hkv = case["B"], case["H"], case["Nq"], case["d"], case["Hkv"]
    q = s["q"].float().view(B, Hkv, H // Hkv * Nq, d)
    scores = (q @ _values(s, "k", s["table"]).transpose(-1, -2)) * (1.0 / math.sqrt(d))
    scores = scores.view(B, Hkv, H // Hkv, Nq, -1)
    key = torch.arange(scores.shape[-1], device=DEV)
    last = s["lens"].long()[:, None] - 1
    if case["causal"]:
        last = last + torch.arange(Nq, device=DEV)[None, :] - (Nq - 1)
    seen = key[None, None, :] <= last[:, :, None]  # [B, Nq or 1, keys]
    return scores.masked_fill(~seen[:, None, None], float("-inf"))


def _attend(s, case, shared):
    B, H, Nq, d, Hkv = case["B"], case["H"], case["Nq"], case["d"], case["Hkv"]
    group = H // Hkv
    own_s = _own_scores(s, case)
    parts = [own_s]
    if shared:  # one product for all sequences' rows
        q = s["q"].float().view(B, Hkv, group * Nq, d).transpose(0, 1).reshape(Hkv, B * group * Nq, d)
        k = _values(s, "k", s["prefix_table"])[:, : case["prefix"]]
        a = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
        a = a.view(Hkv, B, group, Nq, -1).transpose(0, 1)
        if case["causal"]:  # a sequence with fewer tokens of its own than rows: the first rows end inside the prefix
            last = case["prefix"] + s["lens"].long()[:, None] - Nq + torch.arange(Nq, device=DEV)[None, :]
            seen = torch.arange(case["prefix"], device=DEV)[None, None, :] <= last[:, :, None]
            a = a.masked_fill(~seen[:, None, None], float("-inf"))
        parts.append(a)
    m = torch.stack([x.amax(-1) for x in parts]).amax(0)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)[..., None]
    e = [torch.exp(x - m) for x in parts]
    total = sum(x.sum(-1, keepdim=True) for x in e)
    out = e[0].view(B, Hkv, group * Nq, -1) @ _values(s, "v", s["table"])
    if shared:
        v = _values(s, "v", s["prefix_table"])[:, : case["prefix"]]
        p = e[1].transpose(0, 1).reshape(Hkv, B * group * Nq, -1) @ v
        out = out + p.view(Hkv, B, group * Nq, d).transpose(0, 1)
    out = out.view(B, Hkv, group, Nq, d) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (m + torch.log(total)).squeeze(-1)
    return out.reshape(B, H, Nq, d).to(s["q"].dtype), lse.reshape(B, H, Nq)


def _weights(s, case):
    B, H, Nq, Hkv = case["B"], case["H"], case["Nq"], case["Hkv"]
    lse = s["lse"].view(B, Hkv, H // Hkv, Nq, 1)
    p = torch.exp(_own_scores(s, case) - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse))
    s["weight"] += p.sum((2, 3))
    return {"weight": s["weight"]}


def _code(x, fmt):
    if fmt == "int8":
        return x.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _evict(s, case):
    B, Hkv, d, page, fmt, keep = case["B"], case["Hkv"], case["d"], case["page"], case["fmt"], case["keep"]
    n, weight, capacity = s["lens"].long(), s["weight"], s["weight"].shape[-1]
    pos = torch.arange(capacity, device=DEV)
    late = pos >= (n - case["recent"])[:, None]
    rank = torch.where(late[:, None], torch.full_like(weight, float("inf")), weight)
    rank = torch.where((pos < n[:, None])[:, None], rank, torch.full_like(weight, float("-inf")))
    most = min(keep, capacity)
    kept = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :most].sort(-1).values
    slot = torch.arange(most, device=DEV)
    lens = torch.minimum(n, torch.full_like(n, keep))
    held = (slot < lens[:, None])[:, None].expand(B, Hkv, most)
    kept = torch.where((n <= keep)[:, None, None], slot.expand(B, Hkv, most), kept)
    new_weight = torch.zeros_like(weight)
    new_weight[..., :most] = torch.where(held, weight.gather(-1, kept), torch.zeros_like(weight[..., :most]))
    # the kept tokens, page by page of their new places
    pages = (most + page - 1) // page
    pad = pages * page - most
    src, valid = torch.nn.functional.pad(kept, (0, pad)), torch.nn.functional.pad(held, (0, pad))
    to = torch.arange(pages * page, device=DEV)
    moves = (valid & (src != to)).view(B, Hkv, pages, page).any(-1)
    head = torch.arange(Hkv, device=DEV)[None, :, None]
    seq = torch.arange(B, device=DEV)[:, None, None]
    at = s["table"].long()[seq, src // page]
    put = s["table"].long()[:, :pages]  # [B, pages]
    write = valid.view(B, Hkv, pages, page) & moves[..., None]
    top, bits = (0.9921875, 7) if fmt == "int8" else (0.875, 9)  # QMAX = top * 2^bits
    result = {"lens": lens.int(), "kept": torch.where(held, kept, torch.full_like(kept, -1)).int(), "weight": new_weight}
    if most < keep:  # a budget beyond every sequence
        result["kept"] = torch.nn.functional.pad(result["kept"], (0, keep - most), value=-1)
    for name in ("k", "v"):
        codes, scale = s[name + "_codes"], s[name + "_scale"]
        raw = codes.view(torch.uint8)
        x = raw[at, head, src % page].view(codes.dtype).float() * scale[at, head][..., None]
        x = torch.where(valid[..., None], x, torch.zeros_like(x)).view(B, Hkv, pages, page, d)
        amax = x.abs().amax((-1, -2))
        frac, e = torch.frexp(amax)
        e = (e - bits + (frac > top).int()).clamp(-110, 120)
        now = torch.where(amax > 0, _power(e), torch.zeros_like(amax))
        inv = torch.where(now > 0, 1.0 / now.clamp(min=2.0 ** -120), torch.zeros_like(now))
        fresh = _code(x * inv[..., None, None], fmt)
        b, h, g = (i.expand(B, Hkv, pages) for i in (seq, head, torch.arange(pages, device=DEV)[None, None]))
        b, h, g = b[moves], h[moves], g[moves]
        where = put[b, g]
        raw[where, h] = torch.where(write[b, h, g][..., None], fresh[b, h, g], raw[where, h])
        scale[where, h] = now[b, h, g]
        result.update({name + "_codes": codes, name + "_scale": scale})
    return result


def _rotary(s, case):
    r = case["pairs"]
    angle = s["positions"].double()[s["axis"].long().to(DEV)] * s["inv_freq"].to(DEV).view(-1, *[1] * (s["positions"].dim() - 1))
    angle = angle.movedim(0, -1)  # [..., pairs]
    if case["inverse"]:
        angle = -angle
    head = 1 if case["layout"] == "heads" else -2
    cos, sin = torch.cos(angle).float().unsqueeze(head), torch.sin(angle).float().unsqueeze(head)

    def one(x):
        f = x.float()
        a, b = f[..., :r], f[..., r : 2 * r]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, f[..., 2 * r :]], -1).to(x.dtype)

    return {"q": one(s["q"]), "k": one(s["k"])}


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return _own(s, case, op)
    if op == "prefix":
        out, lse = _attend(s, case, True)
        return {"out": out, "lse": lse}
    if op == "weights":
        return _weights(s, case)
    return _evict(s, case) if op == "evict" else _rotary(s, case)


def _own(s, case, op):
    from io_aware_exact_13_gb300 import fa

    if op == "rotary":
        turn = fa.rotary_backward if case["inverse"] else fa.rotary
        q, k = turn(s["q"], s["k"], s["positions"], s["inv_freq"], s["axis"])
        return {"q": q, "k": k}
    cache = fa.KVCacheQ8(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    if op == "prefix":
        out, lse = fa.attention_kvq8_prefix(s["q"], cache, s["prefix_table"], s["prefix_len"], s["table"], s["lens"],
                                            causal=case["causal"], max_prefix=case["prefix"], max_len=s["max_len"])
        return {"out": out, "lse": lse}
    if op == "weights":
        fa.kvq8_weights(s["q"], cache, s["table"], s["lens"], s["lse"], s["weight"], causal=case["causal"],
                        max_len=s["max_len"])
        return {"weight": s["weight"]}
    lens, kept, weight = fa.kvq8_evict(cache, s["table"], s["lens"], s["weight"], case["keep"], case["recent"])
    return {"lens": lens, "kept": kept, "weight": weight, "k_codes": s["k_codes"], "k_scale": s["k_scale"],
            "v_codes": s["v_codes"], "v_scale": s["v_scale"]}


# ---------------------------------------------------------------- the definitions in 64 bits
def _power64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(x):
    """Nearest 8-bit float (4 exponent bits, 3 mantissa bits, bias 7), ties to the even mantissa."""
    _, e = torch.frexp(x)
    step = _power64((e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _tokens64(s, case, name, h, table, n):
    """The first n tokens of a row of pages, one head: [n, d]."""
    pages = table[: _pages(case, n)].long()
    codes = s[name + "_codes"][:, h].view(torch.uint8)[pages].view(s[name + "_codes"].dtype).double()
    return (codes * s[name + "_scale"][pages, h].double()[:, None, None]).reshape(-1, case["d"])[:n]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        return _exact_rotary(s, case)
    if op == "evict":
        return _exact_evict(s, case)
    lens, d, Nq = _lengths(case), case["d"], case["Nq"]
    group = case["H"] // case["Hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=DEV)
    weight = s["weight"].double().clone() if op == "weights" else None
    before = case.get("prefix", 0)
    for h in range(case["Hkv"]):
        heads = slice(h * group, (h + 1) * group)
        kp, vp = (_tokens64(s, case, n, h, s["prefix_table"], before) for n in ("k", "v"))
        for b, n in enumerate(lens):
            k, v = (torch.cat([p, _tokens64(s, case, m, h, s["table"][b], n)]) for m, p in (("k", kp), ("v", vp)))
            a = torch.einsum("gid,jd->gij", s["q"][b, heads].double(), k) / math.sqrt(d)
            if case["causal"]:
                a = a.masked_fill(torch.ones(a.shape[1:], dtype=torch.bool, device=DEV).triu(before + n - Nq + 1), -math.inf)
            if op == "weights":
                given = s["lse"][b, heads].double()[..., None]
                p = torch.exp(a - given).nan_to_num(0.0)  # a row that sees no key has -inf - -inf
                weight[b, h, :n] += p.sum((0, 1))
                continue
            l = torch.logsumexp(a, -1)
            lse[b, heads] = l
            out[b, heads] = torch.einsum("gij,jd->gid", torch.exp(a - l[..., None]).nan_to_num(0.0), v)
    return {"weight": weight} if op == "weights" else {"out": out, "lse": lse}


def _exact_rotary(s, case):
    r = case["pairs"]
    got = {}
    for name in ("q", "k"):
        x = s[name].double()
        y = x.clone()
        for i in range(r):  # the plane of dims i and r + i turned by one angle
            angle = s["positions"][int(s["axis"][i])].double() * float(s["inv_freq"][i]) * (-1.0 if case["inverse"] else 1.0)
            angle = angle.unsqueeze(1)  # over the heads, in either layout
            turn = torch.polar(torch.ones_like(angle), angle) * torch.complex(x[..., i], x[..., i + r])
            y[..., i], y[..., i + r] = turn.real, turn.imag
        got[name] = y
    return got


def _exact_evict(s, case):
    page, fmt, keep, d = case["page"], case["fmt"], case["keep"], case["d"]
    lens = _lengths(case)
    got = {"lens": _ints([min(n, keep) for n in lens]), "weight": torch.zeros_like(s["weight"], dtype=torch.float64),
           "kept": torch.full((case["B"], case["Hkv"], keep), -1, dtype=torch.int32, device=DEV)}
    for m in ("k", "v"):
        raw = s[m + "_codes"]
        got[m + "_codes"] = raw.clone() if fmt == "int8" else raw.double()
        got[m + "_scale"] = s[m + "_scale"].double()
    weights = s["weight"].cpu().double().numpy()
    for b, n in enumerate(lens):
        for h in range(case["Hkv"]):
            w = weights[b, h, :n]
            if n <= keep:
                stay = np.arange(n)
            else:
                old = n - case["recent"]
                order = np.lexsort((np.arange(old), -w[:old]))  # greatest first, then lowest place
                stay = np.sort(np.concatenate([order[: keep - case["recent"]], np.arange(old, n)]))
            got["weight"][b, h, : len(stay)] = torch.from_numpy(w[stay]).to(DEV)
            got["kept"][b, h, : len(stay)] = torch.from_numpy(stay).int().to(DEV)
            changed = [j for j in range(_pages(case, len(stay)))
                       if np.any(stay[j * page : (j + 1) * page] != np.arange(len(stay))[j * page : (j + 1) * page])]
            if not changed:
                continue
            first = changed[0] * page  # everything behind the first token that moves has moved
            index = torch.from_numpy(stay[first:]).to(DEV)
            pages = s["table"][b, changed[0] : _pages(case, len(stay))].long()
            for m in ("k", "v"):
                x = _tokens64(s, case, m, h, s["table"][b], n)[index]
                x = torch.nn.functional.pad(x, (0, 0, 0, len(pages) * page - len(x))).view(len(pages), page, d)
                most = x.abs().amax((-1, -2))
                frac, e = torch.frexp(most / QMAX[fmt])  # frac in [0.5, 1): the next power of two is 2^e, or itself
                now = _power64((e - (frac == 0.5).int()).clamp(-110, 120))
                now = torch.where(most > 0, now, torch.zeros_like(now))
                value = x / now.clamp(min=2.0 ** -200)[:, None, None]
                value = torch.round(value).clamp(-127, 127) if fmt == "int8" else _round_e4m3(value)
                codes = got[m + "_codes"]
                at = torch.arange(len(pages) * page, device=DEV).view(-1, page, 1)
                codes[pages, h] = torch.where(at < len(stay) - first, value.to(codes.dtype), codes[pages, h])
                got[m + "_scale"][pages, h] = now
    return got
