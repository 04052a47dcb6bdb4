"""Batches over a paged key-value cache, and the definitions of its calls in 64
bits (shared by the tests of the cache and of the attention over it)."""
import math
import random

import numpy as np
import torch

import int4_weight_mixed_gb300 as w4

TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


def quantised(x, codes):
    """Codes (as a tensor of that type) and scales of rows x by the definition,
    every step in fp32 (numpy)."""
    x = x.float().numpy()
    with np.errstate(all="ignore"):
        top = np.abs(x).max(-1)
        s = top * (np.float32(1) / np.float32(TOP[codes]))
        assert s.dtype == np.float32
        s = np.where(np.isfinite(top), np.where(s < np.float32(2.0**-100), np.float32(0), s),
                     np.float32(np.nan))
        q = np.where((s > 0)[..., None], x / s[..., None], np.float32(0)).astype(np.float32)
    if codes == torch.int8:
        return torch.from_numpy(np.rint(q).astype(np.int8)), torch.from_numpy(s)
    return torch.from_numpy(q).to(codes), torch.from_numpy(s)


class Batch:
    """rows[b] rows and lens[b] positions of each sequence, pages in no order,
    the unused entries of the table no page's.  wide: a table with room for far
    longer sequences, for which calls of more than 16 rows a key head go to the
    tensor cores' kernel."""

    def __init__(self, rows, lens, page, seed=0, spare=3, behind=0, wide=False):
        self.rows, self.lens, self.page = list(rows), list(lens), page
        used = [-(-k // page) for k in lens]
        self.pages = sum(used) + spare
        order = list(range(self.pages))
        random.Random(seed).shuffle(order)
        self.width = max([1 << 16 if wide else 1, *used])
        self.table = torch.full((len(rows), self.width), -1, dtype=torch.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = torch.tensor(order[at:at + u], dtype=torch.int32)
            at += u
        self.starts = torch.tensor([0, *np.cumsum(rows)], dtype=torch.int32)
        self.T = int(sum(rows)) + behind  # rows, those of no sequence among them

    def plan(self, dev):
        return (self.table.to(dev), self.starts.to(dev),
                torch.tensor(self.lens, dtype=torch.int32, device=dev))

    def slots(self, b, lo, hi):
        """(page, slot) of positions lo..hi-1 of sequence b."""
        p = torch.arange(lo, hi)
        return self.table[b, p // self.page].long(), p % self.page


def random_cache(batch, heads, dim, codes, seed=0, spread=3.0, garbage=True):
    """A cache whose every slot holds a quantised row; slots that no sequence
    owns hold NaN scales (and E4M3 NaN codes) where `garbage`."""
    g = torch.Generator().manual_seed(seed)
    out = []
    own = torch.zeros(batch.pages, batch.page, dtype=torch.bool)
    for b, k in enumerate(batch.lens):
        pg, sl = batch.slots(b, 0, k)
        own[pg, sl] = True
    for kv in range(2):
        x = torch.randn(batch.pages, heads, batch.page, dim, generator=g)
        x *= torch.exp(torch.randn(batch.pages, heads, batch.page, 1, generator=g) * 0.5)
        if kv == 0:
            x[..., ::17] *= spread
        c, s = quantised(x, codes)
        if garbage:
            free = ~own[:, None].expand(-1, heads, -1)
            s[free] = float("nan")
            c.view(torch.uint8)[free] = 0x7F
        out.append((c, s))
    (k, ks), (v, vs) = out
    return w4.KVCache(k, v, ks, vs)


def dequantised(cache, batch, b):
    """Keys and values of sequence b in 64 bits: [heads, len, dim]."""
    pg, sl = batch.slots(b, 0, batch.lens[b])
    out = []
    for c, s in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
        x = c.view(torch.uint8)[pg, :, sl].view(c.dtype).double() * s[pg, :, sl].double()[..., None]
        out.append(x.movedim(1, 0))
    return out


def seen(n, k, window, sinks, mask=None):
    """[n, k] truth: which keys each of the last n positions of k sees; mask
    [n, drafts]: a tree's."""
    first = k - n
    j = torch.arange(k)[None]
    i = torch.arange(n)[:, None]
    if mask is None:
        p = first + i
        see = j <= p
        near = torch.ones(n, k, dtype=torch.bool)
    else:
        w = min(n, mask.shape[1])
        m = torch.zeros(n, n, dtype=torch.bool)
        m[:, :w] = mask[:, :w]
        p = first + (m.sum(1, keepdim=True) - 1).clamp(min=0)
        see = torch.ones(n, k, dtype=torch.bool)
        lo = max(first, 0)
        see[:, lo:] = m[:, lo - first:]
        near = (j < first).expand(n, k)
    if window > 0:
        see = see & ((j > p - window) | (j < sinks) | ~near if mask is not None
                     else (j > p - window) | (j < sinks))
    return see


def attention(q, cache, batch, window=0, sinks=0, mask=None, scale=None):
    """(out, bound) of the definition in 64 bits, [T, heads, dim]; rows of no
    sequence are NaN.

    The bound, per output.  With t a score and T = sum_d |q k| * scale:
      a score is off by at most (D + 8) 2^-23 T (fp32 sums of D exact products,
        each addition off by a unit in the last place, whichever way it rounds;
        q as fp16 times a power of two loses at most 2^-25 of the row's largest
        value, which T's share covers only where the keys are alike, so it is
        added: 2^-25 max|q| sum|k| scale) and by |t| 2^-21 (its scaling, and the
        logarithm of the value's scale, in fp32);
      a probability is then off by twice the largest of these (numerator and
        denominator), by 2^-17 (exponential, reciprocals, sums; the logarithm
        of a value's scale by 2^-22 of itself, so 2^-22 of its magnitude where
        that is above 2^5; a scale of 0 counts as 2^-60) and by half a
        step of fp16, 2^-11, or by 2^-25 of the row's largest probability times
        scale where fp16 has no more bits;
      the output is rounded by half a step of its type."""
    T, Hq, D = q.shape
    Hkv = cache.k.shape[1]
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.float64)
    bound = torch.zeros_like(out)
    at = 0
    for b, (n, k) in enumerate(zip(batch.rows, batch.lens)):
        if n == 0:
            continue
        if k == 0:  # no keys: zeros
            out[at:at + n], bound[at:at + n] = 0.0, 0.0
            at += n
            continue
        m = mask[at:at + n] if mask is not None else None
        see = seen(n, k, window, sinks, m)
        K, V = dequantised(cache, batch, b)
        g = Hq // Hkv
        x = q[at:at + n].double().view(n, Hkv, g, D).permute(1, 2, 0, 3)  # [Hkv, g, n, D]
        t = torch.einsum("hgnd,hkd->hgnk", x, K) * scale
        size = torch.einsum("hgnd,hkd->hgnk", x.abs(), K.abs()) * abs(scale)
        lost = x.abs().amax(-1)[..., None] * K.abs().sum(-1)[:, None, None] * abs(scale)
        off = (D + 8) * 2.0**-23 * size + 2.0**-25 * lost + t.abs() * 2.0**-21
        t = t.masked_fill(~see, float("-inf"))
        off = off.masked_fill(~see, 0.0)
        any_ = see.any(-1)
        top = torch.where(any_, t.amax(-1), 0.0)[..., None]
        e = torch.exp(t - top)
        total = e.sum(-1, keepdim=True)
        p = torch.where(total > 0, e / total, 0.0)
        o = torch.einsum("hgnk,hkd->hgnd", p, V)
        mag = torch.einsum("hgnk,hkd->hgnd", p, V.abs())
        worst = off.amax(-1, keepdim=True)
        # p' below fp16's normal range: 2^-25 of the largest p' = p * scale
        pg, sl = batch.slots(b, 0, k)
        vs = cache.v_scales[pg, :, sl].double().movedim(1, 0)[:, None, None]  # [Hkv,1,1,k]
        log = torch.where(vs > 0, vs, 2.0**-60).log2().abs().amax()
        rel = 2 * worst + 2.0**-22 * log.clamp(min=32.0) + 2.0**-11
        big = torch.where(see, p * vs, 0.0).amax(-1, keepdim=True)
        codes = (V.abs() / torch.where(vs[:, 0, 0] > 0, vs[:, 0, 0], 1.0)[..., None])
        tiny = 2.0**-25 * big * torch.einsum("nk,hkd->hnd", see.double(), codes)[:, None]
        eps = torch.finfo(q.dtype).eps / 2
        step = torch.finfo(q.dtype).smallest_normal * eps
        bd = mag * rel + tiny
        bd = bd + (o.abs() + bd) * eps + step
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, Hq, D)
        bound[at:at + n] = bd.permute(2, 0, 1, 3).reshape(n, Hq, D)
        at += n
    return out, bound


def on(cache, dev):
    return w4.KVCache(*(t.to(dev) for t in cache))
