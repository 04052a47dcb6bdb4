"""A paged key-value cache in 8 bits and the attention that reads it, measured: keys and values
quantised as they are written, read back as 16-bit rows, attended to by prompts, chunks and single
tokens (causal, with a sliding window and a few first keys that stay visible) and by the drafted
tokens of a tree.

Each case has a plain form (elementary torch operations in 32 bits) and the framework's call.
"""
import math
import random

import torch

own = False

DEV = "cuda"
F16, BF16 = "fp16", "bf16"
DT = {F16: torch.float16, BF16: torch.bfloat16}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
# symmetric int8: 127 steps to a row's largest magnitude; E4M3: its largest value
TOP = {"int8": 127.0, "e4m3": 448.0}


def _case(name, op, B, L, n, Hq, Hkv, D, dtype, cache, page, window=0, sinks=0, mix=0):
    """B sequences of up to L positions, up to n of them new; `mix` spreads the lengths (-1: all
    alike)."""
    return {"name": name, "op": op, "B": B, "L": L, "n": n, "Hq": Hq, "Hkv": Hkv, "D": D,
            "dtype": dtype, "cache": cache, "page": page, "window": window, "sinks": sinks,
            "mix": mix}


def listed():
    return [
        # one decoded token's keys and values, heads of Llama-3-8B
        _case("write int8 T=1", "write", 1, 1500, 1, 32, 8, 128, BF16, "int8", 64, mix=-1),
        # a batch of prompts, written in one call
        _case("write e4m3 prompts", "write", 7, 6001, 6001, 64, 8, 128, F16, "e4m3", 64, mix=1),
        # short sequences read back, small heads
        _case("read int8 short", "read", 3, 333, 333, 9, 3, 64, F16, "int8", 16, mix=2),
        # a long context read back whole
        _case("read e4m3 long", "read", 1, 131072, 131072, 32, 8, 128, BF16, "e4m3", 64, mix=-1),
        # one decoded token, one sequence, heads of Llama-3-8B
        _case("decode B=1", "attend", 1, 1500, 1, 32, 8, 128, BF16, "int8", 64, mix=-1),
        # a decode batch of ragged lengths, heads of Llama-3-70B
        _case("decode B=64", "attend", 64, 8192, 1, 64, 8, 128, F16, "e4m3", 64, mix=3),
        # two long contexts
        _case("decode long", "attend", 2, 131072, 1, 32, 8, 128, BF16, "int8", 128, mix=4),
        # a decode batch with a window and sinks, small heads, three rows a key head
        _case("decode window", "attend", 48, 32768, 1, 24, 8, 64, BF16, "e4m3", 16, 4096, 4, mix=5),
        # a prompt, causal
        _case("prompt 8192", "attend", 1, 8192, 8192, 32, 8, 128, BF16, "int8", 64, mix=-1),
        # ragged chunks of prompts on what the cache holds, with a window and sinks
        _case("chunks window", "attend", 6, 9001, 1511, 40, 8, 64, F16, "e4m3", 32, 2048, 16, mix=6),
        # one sequence's tree of 64 drafted tokens
        _case("tree B=1", "tree", 1, 2112, 64, 32, 8, 128, BF16, "int8", 64, mix=-1),
        # trees of a batch, with a window and sinks
        _case("tree B=32", "tree", 32, 8192, 48, 64, 8, 128, F16, "e4m3", 64, 4096, 4, mix=7),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("write", "read", "attend", "attend", "attend", "tree"))
    D = rng.choice((64, 128, 128))
    Hkv = rng.choice((1, 2, 3, 4, 8, 8))
    group = rng.choice((1, 2, 3, 4, 4, 5, 7, 8, 8, 16))
    page = rng.choice((16, 32, 64, 64, 128, 256))
    B = _log(rng, 1, 64)
    # what the plain form holds at once is bounded: keys and values, and the scores
    L = _log(rng, 16, min(131072, 131072 * 8 * 128 // (B * Hkv * D)))
    window = sinks = 0
    if op in ("write", "read"):
        n = L if rng.random() < 0.6 else _log(rng, 1, L)
    else:
        most = max(1, min(L, (1 << 30) // (B * Hkv * group * L)))
        kind = rng.random()
        if op == "tree":
            n = _log(rng, 2, max(2, min(L, 128, most)))
        elif kind < 0.5:
            n = 1
        else:
            n = _log(rng, 1, most)
        if rng.random() < 0.4:
            window, sinks = _log(rng, 16, 8192), rng.choice((0, 1, 4, 16, 100))
    c = _case("", op, B, L, n, Hkv * group, Hkv, D, rng.choice((F16, BF16)),
              rng.choice(("int8", "e4m3")), page, window, sinks, mix=rng.randrange(1 << 20))
    del c["name"]
    return c


def _batch(case):
    """(rows, lengths) of the sequences."""
    B, L, n = case["B"], case["L"], case["n"]
    if case["mix"] < 0:
        return [n] * B, [L] * B
    r = random.Random(case["mix"])
    lens = [L] + [r.randint(max(1, L // 16), L) for _ in range(B - 1)]
    rows = [min(k, n if n < 2 or b == 0 else r.randint(max(1, n // 8), n))
            for b, k in enumerate(lens)]
    return rows, lens


def _tree(case):
    """[T, n] truth values: the drafted tokens that each one sees, itself and its ancestors."""
    r = random.Random(case["mix"] + 1)
    rows, _ = _batch(case)
    mask = torch.zeros(sum(rows), max(rows), dtype=torch.bool)
    at = 0
    for n in rows:
        for t in range(n):
            parent = r.randint(max(-1, t - 8), t - 1)  # -1: the tree's root, held by the cache
            if parent >= 0:
                mask[at + t] = mask[at + parent]
            mask[at + t, t] = True
        at += n
    return mask


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    rows, lens = _batch(case)
    B, Hq, Hkv, D, page = (case[k] for k in ("B", "Hq", "Hkv", "D", "page"))
    dt, T = DT[case["dtype"]], sum(rows)
    s["T"], s["rows"], s["most"] = T, max(rows), max(lens)
    starts = [0]
    for n in rows:
        starts.append(starts[-1] + n)
    # pages in no order; entries past a sequence's last page are no page's
    used = [-(-k // page) for k in lens]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    table = torch.full((B, max(used)), -1, device=DEV, dtype=torch.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    s["table"] = table
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    # keys have a few large channels, as a transformer's have
    wide = 1 + 6 * (torch.rand(Hkv, 1, D, generator=g, device=DEV) < 0.03)
    if case["op"] == "write":
        # rows of the product that makes queries, keys and values in one
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device=DEV).to(dt)
        k = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        k *= wide.squeeze(1).to(dt)
        s["k_new"], s["v_new"] = k, qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        filled = [torch.zeros(pages, Hkv, page, D, device=DEV).to(CODES[case["cache"]])
                  for _ in range(2)]
        scales = [torch.zeros(pages, Hkv, page, device=DEV) for _ in range(2)]
    else:
        filled, scales = [], []
        for spread in (wide, 1.0):
            x = torch.randn(pages, Hkv, page, D, generator=g, device=DEV) * spread
            codes, scale = _quantised(x, case["cache"])
            filled.append(codes)
            scales.append(scale)
            del x
    s["k"], s["v"], s["k_scales"], s["v_scales"] = *filled, *scales
    if case["op"] in ("attend", "tree"):
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device=DEV).to(dt)
        s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
    if case["op"] == "tree":
        s["mask"] = _tree(case).to(DEV)
    if own:  # the cache's arrays as a program holds them
        import int4_weight_mixed_gb300 as w4
        s["held"] = w4.KVCache(s["k"], s["v"], s["k_scales"], s["v_scales"])
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import int4_weight_mixed_gb300 as w4
    held, plan = s["held"], (s["table"], s["starts"], s["lens"])
    if s["op"] == "write":
        w4.cache_write(held, s["k_new"], s["v_new"], *plan)
        return {"k": held.k, "v": held.v, "k_scales": held.k_scales, "v_scales": held.v_scales}
    if s["op"] == "read":
        k, v = w4.cache_read(held, *plan, s["T"], DT[s["dtype"]])
        return {"k": k, "v": v}
    if s["op"] == "tree":
        return {"out": w4.tree_attention(held, s["q"], s["mask"], *plan, window=s["window"],
                                         sinks=s["sinks"])}
    return {"out": w4.cache_attention(held, s["q"], *plan, window=s["window"], sinks=s["sinks"])}


def _quantised(x, cache):
    """Codes and scales of rows x: scale = largest magnitude / top, code = x / scale rounded once;
    a row of zeros has scale 0 and codes 0."""
    scale = x.abs().amax(-1) / TOP[cache]
    q = x / torch.where(scale > 0, scale, 1.0)[..., None]
    return (torch.round(q) if cache == "int8" else q).to(CODES[cache]), scale


def _places(s):
    """Page and slot of every row's position."""
    row = torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(s["starts"][1:].long(), row, right=True)
    pos = row + (s["lens"].long() - s["starts"][1:].long())[b]
    return s["table"].long()[b, pos // s["page"]], pos % s["page"]


def _plain(s):
    if s["op"] == "write":
        page, slot = _places(s)
        for new, codes, scales in (("k_new", "k", "k_scales"), ("v_new", "v", "v_scales")):
            q, scale = _quantised(s[new].float(), s["cache"])
            s[codes].view(torch.uint8)[page, :, slot] = q.view(torch.uint8)
            s[scales][page, :, slot] = scale
        return {n: s[n] for n in ("k", "v", "k_scales", "v_scales")}
    if s["op"] == "read":
        page, slot = _places(s)
        return {n: (s[n].view(torch.uint8)[page, :, slot].view(s[n].dtype).float()
                    * s[n + "_scales"][page, :, slot][..., None]).to(DT[s["dtype"]])
                for n in ("k", "v")}
    # every sequence padded to the longest one: [B, rows, ...] queries, [B, keys, ...] keys
    B, Hq, Hkv, D, n, L = s["B"], s["Hq"], s["Hkv"], s["D"], s["rows"], s["most"]
    starts, lens = s["starts"].long(), s["lens"].long()[:, None, None]
    count = (starts[1:] - starts[:-1])[:, None, None]
    i = torch.arange(n, device=DEV)[None, :, None]
    j = torch.arange(L, device=DEV)[None, None, :]
    row = (starts[:-1, None, None] + i).clamp(max=s["T"] - 1).squeeze(2)  # [B, n]
    first = lens - count
    if s["op"] == "tree":
        m = s["mask"][row]  # [B, n, drafts]
        at = first + (m.sum(-1, keepdim=True) - 1).clamp(min=0)
        draft = (j - first).clamp(0, m.shape[2] - 1).expand(B, n, L)
        seen = torch.where(j < first, torch.ones_like(draft, dtype=torch.bool),
                           m.gather(2, draft) & (j - first < m.shape[2])) & (j < lens)
        prefix = j < first
    else:
        at = first + i
        seen = j <= at
        prefix = torch.ones_like(seen)
    if s["window"] > 0:
        seen = seen & (~prefix | (j > at - s["window"]) | (j < s["sinks"]))
    pages = s["table"].long().clamp(min=0)

    def held(name):
        x = s[name].view(torch.uint8)[pages].view(s[name].dtype).float()
        x = x * s[name + "_scales"][pages][..., None]
        return x.transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :L]

    q = s["q"].float()[row].view(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    q = q.reshape(B, Hkv, -1, D)
    t = (q @ held("k").transpose(2, 3)).view(B, Hkv, Hq // Hkv, n, L)
    t.mul_(1 / math.sqrt(D)).masked_fill_(~seen[:, None, None], float("-inf"))
    top = t.amax(-1, keepdim=True)
    t.sub_(torch.where(torch.isinf(top), 0.0, top)).exp_()
    total = t.sum(-1)[..., None]
    o = (t.view(B, Hkv, -1, L) @ held("v")).view(B, Hkv, Hq // Hkv, n, D)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(B * n, Hq, D).to(DT[s["dtype"]])
    # the padded rows leave
    r = torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(starts[1:], r, right=True)
    return {"out": o[b * n + r - starts[b]]}


def _seen(case):
    """For every sequence: keys that any of its rows sees, and the sum over its rows of the keys
    that each sees."""
    rows, lens = _batch(case)
    window, sinks = case["window"], case["sinks"]
    drafts = _tree(case).sum(1).tolist() if case["op"] == "tree" else None
    found, at = [], 0
    for n, k in zip(rows, lens):
        first = k - n

        def prefix(p):  # keys before `first` that a row at position p sees
            if window <= 0:
                return first
            low = min(first, max(0, p - window + 1))
            return first - low + min(low, sinks)

        if drafts is not None:
            each = sum(prefix(first + d - 1) + d for d in drafts[at:at + n])
            some = prefix(first) + n
        elif window <= 0:
            each, some = n * first + n * (n + 1) // 2, k
        else:
            each = 0
            for p in range(first, k):
                low = max(0, p - window + 1)
                each += p + 1 - low + min(low, sinks)
            low = max(0, first - window + 1)
            some = k - low + min(low, sinks)
        found.append((some, each))
        at += n
    return found


def work(case):
    rows, _ = _batch(case)
    T, Hq, Hkv, D = sum(rows), case["Hq"], case["Hkv"], case["D"]
    if case["op"] in ("write", "read"):
        return {"bytes": 2 * T * Hkv * (2 * D + D + 4), "flops": 2 * T * Hkv * D}
    seen = _seen(case)
    keys = sum(k for k, _ in seen)
    return {"bytes": keys * Hkv * 2 * (D + 4) + 2 * T * Hq * D * 2,
            "flops": 4 * D * Hq * sum(e for _, e in seen)}


def exact(case, seed):
    s = prepare(case, seed)
    rows, lens = _batch(case)
    B, Hkv, D, P = case["B"], case["Hkv"], case["D"], case["page"]
    table = s["table"].cpu()

    def line(name, b, lo, hi):
        """Positions lo..hi-1 of sequence b as one [Hkv, hi - lo, ...] array."""
        p = torch.arange(lo, hi)
        pg, sl = table[b, p // P].long().to(DEV), (p % P).to(DEV)
        x = s[name]
        if x.element_size() == 1:
            x = x.view(torch.uint8)[pg, :, sl].view(x.dtype)
        else:
            x = x[pg, :, sl]
        return x.to(torch.float64).movedim(1, 0)

    if case["op"] == "write":
        out, at = {}, 0
        for n in ("k", "v"):
            out[n] = None if case["cache"] == "int8" else s[n].to(torch.float64)
            out[n + "_scales"] = s[n + "_scales"].double()
        for b in range(B):
            p = torch.arange(lens[b] - rows[b], lens[b])
            pg, sl = table[b, p // P].long().to(DEV), (p % P).to(DEV)
            for n in ("k", "v"):
                x = s[n + "_new"][at:at + rows[b]].double()
                scale = x.abs().max(-1).values / TOP[case["cache"]]
                out[n + "_scales"][pg, :, sl] = scale
                if out[n] is not None:  # the E4M3 value nearest to x / scale: 2^-3 of its binade
                    t = x / scale[..., None]
                    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0**-6))) - 3)
                    out[n][pg, :, sl] = torch.round(t / step) * step
            at += rows[b]
        return out
    if case["op"] == "read":
        got = {"k": [], "v": []}
        for b in range(B):
            for n in got:
                span = (n, b, lens[b] - rows[b], lens[b])
                x = line(*span) * line(n + "_scales", *span[1:])[..., None]
                got[n].append(x.movedim(0, 1))
        return {n: torch.cat(x) for n, x in got.items()}
    seen = _seen(case)
    if 4 * D * case["Hq"] * sum(e for _, e in seen) > 4e12:
        return None
    out, at = torch.empty(s["T"], case["Hq"], D, dtype=torch.float64, device=DEV), 0
    group = case["Hq"] // Hkv
    for b in range(B):
        n, k = rows[b], lens[b]
        keys = line("k", b, 0, k) * line("k_scales", b, 0, k)[..., None]
        values = line("v", b, 0, k) * line("v_scales", b, 0, k)[..., None]
        pos = torch.arange(k - n, k, device=DEV)
        hide = torch.arange(k, device=DEV)[None] > pos[:, None]
        if case["op"] == "tree":
            m = s["mask"][at:at + n, :n]
            hide[:, k - n:] = ~m
            pos = k - n + m.sum(1) - 1
        if case["window"] > 0:
            far = torch.arange(k, device=DEV)[None] + case["window"] <= pos[:, None]
            far[:, :case["sinks"]] = False
            if case["op"] == "tree":
                far[:, k - n:] = False
            hide |= far
        for h in range(Hkv):
            for c in range(group):
                q = s["q"][at:at + n, h * group + c].double()
                score = torch.mm(q, keys[h].T) / D**0.5
                score[hide] = float("-inf")
                out[at:at + n, h * group + c] = torch.mm(torch.softmax(score, 1), values[h])
        at += n
    return {"out": out}
