"""What is measured of the 8-bit key/value cache and of attention over keys of another length.

Five operators, each a case's "op":

  append     new tokens' K and V quantised into a paged 8-bit cache
  read       cached tokens given back as 16-bit K and V, packed
  attend     attention of 1 to 16 query rows per sequence over the 8-bit cache
  cross      attention of Nq queries over Nk keys of another sequence, each batch entry with its own key count
  cross_bwd  its gradients

`run` computes them in elementary torch operations in 32 bits, or, where `own` is set, through the package's
entry points. `exact` computes them from the definitions in 64 bits.

The cache: codes [pages, Hkv, page, d] (int8, or float8_e4m3fn), one fp32 scale for each page and head, K and V
apart; a value is code * scale. A page written by `append` has the smallest power of two that holds the largest
magnitude of its tokens (2^-110 to 2^120; 0 when all are 0); a page that held tokens before keeps its scale, or
takes the larger one and has its codes rounded to it.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
QMAX = {"int8": 127.0, "e4m3": 448.0}
DEV = "cuda"


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of a small batch: every sequence appends its token's K and V
        dict(name="append_step", op="append", fmt="int8", dtype="bf16", nseq=8, Hkv=8, d=128, page=16, new=1, old=2000,
             ragged=False),
        # prompts of a batch written into the cache after their prefill
        dict(name="append_prompts", op="append", fmt="e4m3", dtype="bf16", nseq=24, Hkv=8, d=128, page=64, new=4100,
             old=300, ragged=True),
        # a short conversation read back
        dict(name="read_short", op="read", fmt="e4m3", dtype="fp16", nseq=1, Hkv=4, d=64, page=32, length=700,
             ragged=False),
        # a batch's prefixes read back for the packed forward
        dict(name="read_batch", op="read", fmt="int8", dtype="bf16", nseq=24, Hkv=8, d=128, page=16, length=5000,
             ragged=True),
        # one user, short context, one token: latency
        dict(name="attend_one", op="attend", fmt="int8", dtype="bf16", B=1, H=8, Hkv=8, Nq=1, d=64, page=16, length=509,
             causal=False, ragged=False),
        # an ordinary decoding step with grouped heads and ragged contexts
        dict(name="attend_step", op="attend", fmt="int8", dtype="bf16", B=16, H=32, Hkv=8, Nq=1, d=128, page=16,
             length=8192, causal=False, ragged=True),
        # checking drafted tokens: five causal rows per sequence
        dict(name="attend_draft", op="attend", fmt="e4m3", dtype="fp16", B=12, H=16, Hkv=4, Nq=5, d=64, page=64,
             length=6001, causal=True, ragged=True),
        # a large serving batch with long contexts
        dict(name="attend_large", op="attend", fmt="e4m3", dtype="bf16", B=64, H=64, Hkv=8, Nq=1, d=128, page=64,
             length=16384, causal=False, ragged=True),
        # a decoder's short prompt over an encoder's states
        dict(name="cross_prompt", op="cross", dtype="fp16", B=2, H=8, Hkv=8, d=64, Nq=35, Nk=1500, ragged=False),
        # training: a padded batch, decoder over encoder
        dict(name="cross_train", op="cross", dtype="bf16", B=4, H=32, Hkv=8, d=128, Nq=4096, Nk=6000, ragged=True),
        # its gradients, at a small and a large size
        dict(name="cross_bwd_small", op="cross_bwd", dtype="fp16", B=8, H=16, Hkv=16, d=64, Nq=448, Nk=1500, ragged=True),
        dict(name="cross_bwd_train", op="cross_bwd", dtype="bf16", B=4, H=32, Hkv=8, d=128, Nq=2500, Nk=4096,
             ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "cross", "cross_bwd"])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), d=rng.choice([64, 128]))
    group = rng.choice([1, 2, 4, 5, 8])
    if op in ("append", "read"):
        c.update(fmt=rng.choice(["int8", "e4m3"]), nseq=_log(rng, 1, 40), Hkv=rng.choice([1, 2, 5, 8]),
                 page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.7)
        most = max(1, min(8000, 24 * 4100 * 8 * 128 // (2 * c["nseq"] * c["Hkv"] * c["d"])))
        if op == "append":
            c.update(new=_log(rng, 1, most), old=_log(rng, 1, 3000))
        else:
            c.update(length=_log(rng, 1, most))
    elif op == "attend":
        c.update(fmt=rng.choice(["int8", "e4m3"]), Hkv=rng.choice([1, 2, 5, 8]), page=rng.choice([16, 32, 64, 128]),
                 Nq=rng.choice([1, 1, 1, 2, 3, 7, 16]), B=_log(rng, 1, 48), causal=rng.random() < 0.5,
                 ragged=rng.random() < 0.7)
        c["H"] = c["Hkv"] * group
        most = 64 * 8 * 16384 * 64 // (4 * c["B"] * c["Hkv"] * group * c["Nq"])
        c["length"] = _log(rng, 1, max(1, min(20000, most)))
    else:
        c.update(Hkv=rng.choice([1, 2, 4, 7]), B=_log(rng, 1, 12), ragged=rng.random() < 0.7)
        c["H"] = c["Hkv"] * group
        heads = c["B"] * c["H"]
        c["Nq"] = _log(rng, 1, 4000)
        c["Nk"] = _log(rng, 1, max(1, min(6000, 4 * 32 * 2500 * 4096 // (2 * heads * c["Nq"]))))
    return c


def _lengths(case, count, most):
    """Whole lengths of a ragged batch, from the case alone: a quarter of `most` to `most`, the first one `most`."""
    if not case["ragged"]:
        return [most] * count
    r = np.random.RandomState(count * 7919 + most)
    got = [int(x) for x in r.randint(max(1, most // 4), most + 1, count)]
    got[0] = most
    return got


def _new_lengths(case):
    return _lengths(case, case["nseq"], case["new"])


def work(case):
    """Each input read once, each output written once; products counted for the visible pairs."""
    op, d = case["op"], case["d"]
    if op == "append":  # 16-bit K and V in, 8-bit codes and the touched pages' scales out
        t = sum(_new_lengths(case))
        pages = sum((n + case["page"] - 1) // case["page"] for n in _new_lengths(case))
        return {"bytes": t * case["Hkv"] * d * 2 * 3 + pages * case["Hkv"] * 8, "flops": 0}
    if op == "read":
        lens = _lengths(case, case["nseq"], case["length"])
        pages = sum((n + case["page"] - 1) // case["page"] for n in lens)
        return {"bytes": sum(lens) * case["Hkv"] * d * 2 * 3 + pages * case["Hkv"] * 8, "flops": 0}
    if op == "attend":
        lens = _lengths(case, case["B"], case["length"])
        pages = sum((n + case["page"] - 1) // case["page"] for n in lens)
        rows = case["B"] * case["H"] * case["Nq"]
        return {"bytes": sum(lens) * case["Hkv"] * d * 2 + pages * case["Hkv"] * 8 + rows * (d * 4 + 4),
                "flops": 4 * sum(lens) * case["H"] * case["Nq"] * d}
    lens = _lengths(case, case["B"], case["Nk"])
    q, kv = case["B"] * case["H"] * case["Nq"] * d * 2, case["B"] * case["Hkv"] * case["Nk"] * d * 2
    pairs = sum(lens) * case["H"] * case["Nq"]
    if op == "cross":
        return {"bytes": 2 * q + 2 * kv + case["B"] * case["H"] * case["Nq"] * 4, "flops": 4 * pairs * d}
    return {"bytes": 4 * q + 4 * kv + case["B"] * case["H"] * case["Nq"] * 4, "flops": 10 * pairs * d}


# ---------------------------------------------------------------- inputs
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cumulative(lens):
    return _ints([0] + [int(x) for x in np.cumsum(lens)])


def _power(e):
    """2^e as fp32, by its bits (a pow is not exact everywhere)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _cache(case, g, capacity):
    """A cache with room for `capacity` tokens of each sequence, its pages in a random order, every page holding
    codes of normal values under scales of the size that `append` gives them."""
    page, heads, d = case["page"], case["Hkv"], case["d"]
    need = [(n + page - 1) // page for n in capacity]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    width = max(need)
    first = torch.tensor([0] + [int(x) for x in np.cumsum(need)][:-1], device=DEV).unsqueeze(1)
    at = first + torch.arange(width, device=DEV).unsqueeze(0)
    table = order[at.clamp(max=total - 1)].contiguous()
    table[torch.arange(width, device=DEV).unsqueeze(0) >= torch.tensor(need, device=DEV).unsqueeze(1)] = 0
    shape = (total, heads, page, d)
    state = {"table": table}
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


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2 + 1)
    op, d, dtype = case["op"], case["d"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)

    if op == "append":
        new = _new_lengths(case)
        old = _lengths(case, case["nseq"], case["old"])
        s = _cache(case, g, [a + b for a, b in zip(old, new)])
        t = sum(new)
        # K and V are two parts of one projection's output: rows of a wider buffer
        qkv = normal(t, 2 * case["Hkv"] + 2, d)
        s.update(k=qkv[:, 2 : 2 + case["Hkv"]], v=qkv[:, 2 + case["Hkv"] :], cu=_cumulative(new), old=_ints(old),
                 max_new=max(new))
    elif op == "read":
        lens = _lengths(case, case["nseq"], case["length"])
        s = _cache(case, g, lens)
        s.update(cu=_cumulative(lens), max_len=max(lens), total=sum(lens))
    elif op == "attend":
        lens = _lengths(case, case["B"], case["length"])
        s = _cache(case, g, lens)
        s.update(q=normal(case["B"], case["H"], case["Nq"], d), lens=_ints(lens), max_len=max(lens))
    else:
        lens = _lengths(case, case["B"], case["Nk"])
        q = normal(case["B"], case["H"], case["Nq"], d)
        k, v = (normal(case["B"], case["Hkv"], case["Nk"], d) for _ in range(2))
        s = dict(q=q, k=k, v=v, lens=_ints(lens))
        if op == "cross_bwd":  # what the forward pass left behind
            out, lse = _cross(s, case)
            s.update(out=out, lse=lse, dout=normal(case["B"], case["H"], case["Nq"], d))
    s["case"] = dict(case)
    return s


# ---------------------------------------------------------------- plain forms
def _append(s, case):
    page, heads, d, fmt = case["page"], case["Hkv"], case["d"], case["fmt"]
    top, bits = (0.9921875, 7) if fmt == "int8" else (0.875, 9)  # QMAX = top * 2^bits
    token = torch.arange(s["k"].shape[0], device=DEV)
    seq = torch.searchsorted(s["cu"].long(), token, right=True) - 1
    pos = s["old"].long()[seq] + token - s["cu"].long()[seq]
    to, slot = s["table"].long()[seq, pos // page], pos % page
    # the pages that hold tokens already, one for each sequence (as many as sequences; some hold none)
    old = s["old"].long()
    held = torch.minimum(old // page, torch.tensor(s["table"].shape[1] - 1, device=DEV))
    part = s["table"].long()[torch.arange(old.numel(), device=DEV), held]
    kept = torch.arange(page, device=DEV).unsqueeze(0) < (old % page).unsqueeze(1)  # [nseq, page]
    grows = ((old % page) > 0) & (s["cu"][1:] > s["cu"][:-1])
    result = {}

    def one(n):
        x, codes, scale = s[n].float(), s[n + "_codes"], s[n + "_scale"]
        most = torch.full((scale.shape[0], heads), -1.0, device=DEV)
        most.scatter_reduce_(0, to[:, None].expand(-1, heads), x.abs().amax(-1), "amax")
        touched = most >= 0
        frac, e = torch.frexp(most.clamp(min=0))
        e = (e - bits + (frac > top).int()).clamp(-110, 120)
        fresh = torch.where(most > 0, _power(e), torch.zeros_like(most))
        before = torch.zeros_like(most)
        before[part] = torch.where(grows.unsqueeze(1), scale[part], before[part])
        now = torch.maximum(fresh, before)
        raw = codes.view(torch.uint8)
        # the earlier tokens' codes under the page's new scale
        ratio = torch.where(now[part] > 0, before[part] / now[part].clamp(min=2.0 ** -120), torch.ones_like(now[part]))
        was = codes[part].float() if fmt == "int8" else raw[part].view(torch.float8_e4m3fn).float()
        again = _code(was * ratio[:, :, None, None], fmt)
        keep = (kept & grows.unsqueeze(1))[:, None, :, None].expand(-1, heads, -1, d)
        raw[part] = torch.where(keep, again, raw[part])
        by = now[to]
        inv = torch.where(by > 0, 1.0 / by.clamp(min=2.0 ** -120), torch.zeros_like(by))
        raw[to[:, None], torch.arange(heads, device=DEV)[None, :], slot[:, None]] = _code(x * inv[:, :, None], fmt)
        scale.copy_(torch.where(touched, now, scale))
        result.update({n + "_codes": codes, n + "_scale": scale})

    one("k")
    one("v")
    return result


def _code(x, fmt):
    if fmt == "int8":
        return x.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(s, n):
    """[pages, Hkv, page, d] codes of the table's pages times their scales: [B, Hkv, tokens, d] in 32 bits."""
    codes, table = s[n + "_codes"], s["table"].long()
    x = codes.view(torch.uint8)[table].view(codes.dtype).float() * s[n + "_scale"][table][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _read(s, case):
    token = torch.arange(s["total"], device=DEV)
    seq = torch.searchsorted(s["cu"].long(), token, right=True) - 1
    pos = token - s["cu"].long()[seq]
    to, slot = s["table"].long()[seq, pos // case["page"]], pos % case["page"]
    head = torch.arange(case["Hkv"], device=DEV)[None, :]

    def one(n):
        codes = s[n + "_codes"]
        x = codes.view(torch.uint8)[to[:, None], head, slot[:, None]].view(codes.dtype).float()
        return (x * s[n + "_scale"][to][..., None]).to(DTYPES[case["dtype"]])

    return {"k": one("k"), "v": one("v")}


def _softmax(scores):
    """Probabilities and log-sum-exp of rows in which excluded scores are -inf; a row with none left has zeros."""
    m = scores.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(scores - m)
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    return p / torch.where(total > 0, total, torch.ones_like(total)), lse


def _attend(s, case):
    B, H, Nq, d, Hkv = case["B"], case["H"], case["Nq"], case["d"], case["Hkv"]
    q = s["q"].float().view(B, Hkv, H // Hkv * Nq, d)
    k, v = _values(s, "k"), _values(s, "v")
    scores = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    scores = scores.view(B, Hkv, H // Hkv, Nq, -1)
    key = torch.arange(k.shape[2], device=DEV)
    last = s["lens"].long()[:, None] - 1
    if case["causal"]:
        last = last + torch.arange(Nq, device=DEV)[None, :] - (Nq - 1)
    seen = key[None, None, :] <= last[:, :, None]  # [B, Nq or 1, keys]
    scores = scores.masked_fill(~seen[:, None, None], float("-inf"))
    p, lse = _softmax(scores)
    out = p.view(B, Hkv, H // Hkv * Nq, -1) @ v
    return {"out": out.view(B, H, Nq, d).to(s["q"].dtype), "lse": lse.reshape(B, H, Nq)}


def _cross_scores(s, case):
    B, H, Nq, d, Hkv = case["B"], case["H"], case["Nq"], case["d"], case["Hkv"]
    q = s["q"].float().view(B, Hkv, H // Hkv * Nq, d)
    scores = (q @ s["k"].float().transpose(-1, -2)) * (1.0 / math.sqrt(d))
    seen = torch.arange(case["Nk"], device=DEV)[None, :] < s["lens"][:, None]
    return q, scores.masked_fill_(~seen[:, None, None], float("-inf"))


def _cross(s, case):
    B, H, Nq, d = case["B"], case["H"], case["Nq"], case["d"]
    _, scores = _cross_scores(s, case)
    p, lse = _softmax(scores)
    out = p @ s["v"].float()
    return out.view(B, H, Nq, d).to(s["q"].dtype), lse.reshape(B, H, Nq)


def _cross_bwd(s, case):
    B, H, Nq, d, Hkv = case["B"], case["H"], case["Nq"], case["d"], case["Hkv"]
    q, scores = _cross_scores(s, case)
    p, _ = _softmax(scores)
    g = s["dout"].float().view(B, Hkv, H // Hkv * Nq, d)
    dv = p.transpose(-1, -2) @ g
    dp = g @ s["v"].float().transpose(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * (1.0 / math.sqrt(d))
    dq = (ds @ s["k"].float()).view(B, H, Nq, d)
    dk = ds.transpose(-1, -2) @ q
    t = s["q"].dtype
    return {"dq": dq.to(t), "dk": dk.to(t), "dv": dv.to(t)}


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return _own(s, case, op)
    if op == "append":
        return _append(s, case)
    if op == "read":
        return _read(s, case)
    if op == "attend":
        return _attend(s, case)
    if op == "cross":
        out, lse = _cross(s, case)
        return {"out": out, "lse": lse}
    return _cross_bwd(s, case)


def _own(s, case, op):
    from io_aware_exact_13_gb300 import fa

    if op == "cross":
        out, lse = fa.attention_cross(s["q"], s["k"], s["v"], kv_lens=s["lens"])
        return {"out": out, "lse": lse}
    if op == "cross_bwd":
        dq, dk, dv = fa.attention_cross_backward(s["q"], s["k"], s["v"], s["out"], s["dout"], s["lse"], kv_lens=s["lens"])
        return {"dq": dq, "dk": dk, "dv": dv}
    cache = fa.KVCacheQ8(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    if op == "append":
        fa.kvq8_append(cache, s["k"], s["v"], s["table"], s["cu"], s["old"], s["max_new"])
        return {n: s[n] for n in ("k_codes", "k_scale", "v_codes", "v_scale")}
    if op == "read":
        k, v = fa.kvq8_read(cache, s["table"], s["cu"], s["total"], s["max_len"], dtype=DTYPES[case["dtype"]])
        return {"k": k, "v": v}
    out, lse = fa.attention_kvq8(s["q"], cache, s["table"], s["lens"], max_len=s["max_len"], causal=case["causal"])
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------- the definitions in 64 bits
def _power64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(x):
    """Nearest 8-bit float (4 exponent bits, 3 mantissa bits, bias 7), ties to the even mantissa."""
    _, e = torch.frexp(x)
    step = _power64((e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op == "append":
        return _exact_append(s, case)
    if op == "read":
        lens, out = _lengths(case, case["nseq"], case["length"]), {}
        for n in ("k", "v"):
            rows = []
            for b, length in enumerate(lens):
                pages = s["table"][b, : (length + case["page"] - 1) // case["page"]].long()
                x = s[n + "_codes"].view(torch.uint8)[pages].view(s[n + "_codes"].dtype).double()
                x = x * s[n + "_scale"][pages].double()[:, :, None, None]
                rows.append(x.permute(0, 2, 1, 3).reshape(-1, case["Hkv"], d)[:length])
            out[n] = torch.cat(rows)
        return out
    group = case["H"] // case["Hkv"]
    lens = _lengths(case, case["B"], case["length"] if op == "attend" else case["Nk"])
    if 4 * sum(lens) * case["H"] * case["Nq"] * d > 1e13:  # minutes in 64 bits
        return None
    q = s["q"].double()
    got = {n: torch.zeros_like(q) for n in ("out", "dq")}
    got["lse"] = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=DEV)
    if op != "attend":
        got["dk"], got["dv"] = (torch.zeros_like(s[n], dtype=torch.float64) for n in ("k", "v"))
    for b, length in enumerate(lens):
        for h in range(case["Hkv"]):
            if op == "attend":
                pages = s["table"][b, : (length + case["page"] - 1) // case["page"]].long()
                k, v = ((s[n + "_codes"][:, h].view(torch.uint8)[pages].view(s[n + "_codes"].dtype).double()
                         * s[n + "_scale"][pages, h].double()[:, None, None]).reshape(-1, d)[:length] for n in ("k", "v"))
            else:
                k, v = s["k"][b, h, :length].double(), s["v"][b, h, :length].double()
            for i in range(h * group, (h + 1) * group):
                a = torch.einsum("id,jd->ij", q[b, i], k) / math.sqrt(d)
                if op == "attend" and case["causal"]:
                    shift = length - case["Nq"]
                    a = a.masked_fill(torch.ones_like(a, dtype=torch.bool).triu(shift + 1), -math.inf)
                l = torch.logsumexp(a, -1)
                p = torch.exp(a - l[:, None]).nan_to_num(0.0)
                if op != "cross_bwd":
                    got["lse"][b, i] = l
                    got["out"][b, i] = torch.einsum("ij,jd->id", p, v)
                    continue
                g = s["dout"][b, i].double()
                got["dv"][b, h, :length] += torch.einsum("ij,id->jd", p, g)
                t = torch.einsum("id,jd->ij", g, v)
                t = p * (t - (p * t).sum(-1, keepdim=True)) / math.sqrt(d)
                got["dq"][b, i] = torch.einsum("ij,jd->id", t, k)
                got["dk"][b, h, :length] += torch.einsum("ij,id->jd", t, q[b, i])
    return {n: got[n] for n in (("dq", "dk", "dv") if op == "cross_bwd" else ("out", "lse"))}


def _exact_append(s, case):
    page, fmt = case["page"], case["fmt"]
    new, old = _new_lengths(case), _lengths(case, case["nseq"], case["old"])
    got, start = {}, 0
    for n in ("k", "v"):
        raw = s[n + "_codes"]
        got[n + "_codes"] = raw.clone() if fmt == "int8" else raw.double()
        got[n + "_scale"] = s[n + "_scale"].double()
    for b, (a, t) in enumerate(zip(old, new)):
        first, last = a // page, (a + t - 1) // page
        pages = s["table"][b, first : last + 1].long()
        for n in ("k", "v"):
            x = s[n][start : start + t].double()
            x = torch.nn.functional.pad(x, (0, 0, 0, 0, a % page, -(a + t) % page))
            x = x.view(-1, page, *x.shape[1:]).transpose(1, 2)  # pages, heads, tokens, d
            most = x.abs().amax((-1, -2))
            frac, e = torch.frexp(most / QMAX[fmt])  # frac in [0.5, 1): the next power of two is 2^e, or itself
            need = _power64((e - (frac == 0.5).int()).clamp(-110, 120))
            need = torch.where(most > 0, need, torch.zeros_like(need))
            codes, scale = got[n + "_codes"], got[n + "_scale"]
            now = need.clone()
            if a % page:
                now[0] = torch.maximum(need[0], scale[pages[0]])
            by = now.clamp(min=2.0 ** -200)[:, :, None, None]
            value = x / by
            if a % page:
                was = codes[pages[0], :, : a % page].double() * scale[pages[0]][:, None, None]
                value[0, :, : a % page] = was / by[0]
            value = torch.round(value).clamp(-127, 127) if fmt == "int8" else _round_e4m3(value)
            held = codes[pages].clone()
            at = torch.arange(page * len(pages), device=DEV).view(-1, 1, page, 1)
            codes[pages] = torch.where(at < a % page + t, value.to(codes.dtype), held)
            scale[pages] = now
        start += t
    return got
