"""Attention over the key-value cache for batches of more sequences than a CTA
has threads (the plan then takes them in blocks), with runs of sequences that
have no rows, and batches that mix single tokens with chunks: each kernel,
against the definition in 64 bits."""
import ctypes
import math
import random

import pytest
import torch

import int4_weight_mixed_gb300 as w4
import kv
from fake_cuda import build
from test_attention import DEV, _check, _tree
from test_kv_cache import _cache, _of

S8, F8 = torch.int8, torch.float8_e4m3fn
DEC, UNPACKED, OWN = "attn_dec_kernel", "attn_unpack_kernel", "attn_tc_kernel"


def _ragged(B, most, longest, seed):
    """Rows and lengths of B sequences: runs of sequences without rows (at the
    start, the end and across multiples of 128), then up to `most` rows each."""
    r = random.Random(seed)
    rows, lens = [], []
    while len(rows) < B:
        run = r.randint(1, 40)
        none = r.random() < 0.4 or not rows
        for _ in range(run):
            n = 0 if none else r.randint(1, most)
            rows.append(n)
            lens.append(r.randint(max(n, 1), longest) if n or r.random() < 0.5 else 0)
    rows, lens = rows[:B], lens[:B]
    for b in range(126, min(B, 131)):  # ... and around the first block's end
        rows[b], lens[b] = (0, 7) if b % 2 else (1, 300)
    if not any(rows):
        rows[0] = lens[0] = 1
    return rows, lens


# sequences, most rows, longest, query heads, key heads, dimension, table width
# (0: as wide as the longest sequence), kernel
CASES = [
    (127, 1, 500, 8, 2, 128, 0, DEC), (128, 1, 500, 8, 2, 128, 0, DEC),
    (129, 1, 500, 8, 2, 128, 0, DEC), (129, 1, 400, 6, 2, 64, 0, DEC),
    (300, 1, 300, 4, 1, 64, 0, DEC), (700, 1, 200, 4, 1, 128, 0, DEC),
    (700, 2, 200, 16, 2, 64, 0, DEC),
    (321, 9, 200, 16, 1, 64, 4096, OWN), (330, 9, 300, 16, 1, 128, 1024, OWN),
    (645, 9, 150, 16, 1, 128, 1024, OWN), (700, 9, 150, 8, 1, 64, 4096, OWN),
    (330, 260, 280, 12, 1, 128, 0, UNPACKED), (330, 260, 280, 12, 1, 64, 0, UNPACKED),
]


def _batch(B, most, longest, width, page=32, behind=2):
    rows, lens = _ragged(B, most, longest, 7 * B + most)
    batch = kv.Batch(rows, lens, page, seed=B, behind=behind)
    if width > batch.width:
        batch.table = torch.nn.functional.pad(batch.table, (0, width - batch.width), value=-1)
        batch.width = width
    return batch


def _kernels(rec, heads, kv_heads, dim, rows, sequences, width, page=32, **kw):
    rec.reset()
    cache = _cache(heads=kv_heads, head_dim=dim, page_size=page)
    st = rec.lib.w4_cache_attention(
        ctypes.byref(cache), ctypes.byref(_of(table_width=width, sequences=sequences)),
        0x80000000, w4.F16, rows, heads, heads * dim, 0.1, 0, 0, 1 << 40, 1 << 41,
        kw.get("nws", 1 << 32), None)
    assert st == w4.OK, rec.lib.w4_last_error()
    return " ".join(k for _, k in rec.launches())


@pytest.fixture(scope="module")
def rec(tmp_path_factory):
    return build(tmp_path_factory.mktemp("recorded"))


@pytest.mark.parametrize("case", CASES)
def test_kernel_of_the_case(rec, case):
    """The cases below run on the kernels that they are meant for."""
    B, most, longest, Hq, Hkv, D, width, kernel = case
    batch = _batch(B, most, longest, width)
    got = _kernels(rec, Hq, Hkv, D, batch.T, B, batch.width)
    assert kernel in got
    assert (UNPACKED in got) == (kernel == UNPACKED) and (DEC in got) == (kernel == DEC)


@pytest.mark.gpu
@pytest.mark.parametrize("codes,dt", [(S8, torch.bfloat16), (F8, torch.float16)])
@pytest.mark.parametrize("case", CASES)
def test_many_sequences(gpu_lib, case, codes, dt):
    B, most, longest, Hq, Hkv, D, width, _ = case
    batch = _batch(B, most, longest, width)
    _check(batch.rows, batch.lens, Hq, Hkv, D, 32, codes, dt, batch=batch)


@pytest.mark.gpu
@pytest.mark.parametrize("D,width", [(128, 0), (64, 0), (128, 1024), (64, 4096)])
def test_many_trees(gpu_lib, D, width):
    batch = _batch(330, 9, 200, width)
    _check(batch.rows, batch.lens, 16, 1, D, 32, S8, torch.bfloat16, 50, 3,
           _tree(batch.rows, 9), batch=batch)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("codes,dt", [(S8, torch.bfloat16), (F8, torch.float16)])
def test_tokens_beside_chunks(gpu_lib, D, codes, dt, wide):
    """Single tokens of many sequences and a few chunks, of every position among
    them, in one call."""
    r = random.Random(D)
    rows = [1] * 90
    for b, n in ((0, 300), (40, 65), (41, 129), (89, 520)):
        rows[b] = n
    lens = [max(n, r.randint(1, 900)) for n in rows]
    _check(rows, lens, 8, 2, D, 64, codes, dt, wide=wide)
    _check(rows, lens, 8, 2, D, 64, codes, dt, 100, 4, wide=wide)


# dimension, sequences, rows of each, keys above the others (one for every running
# maximum of the kernel: a warp's of the decode kernel, a half's of units of up to
# 128 rows), kernel
PEAKS = [(128, 456, 1, [70, 100, 10, 50], DEC), (64, 456, 1, [70, 100, 10, 50], DEC),
         (128, 152, 20, [70, 200], OWN), (64, 152, 20, [70, 200], OWN),
         (128, 152, 40, [70], OWN), (64, 152, 40, [70], OWN),
         (128, 3, 3201, [70], UNPACKED), (64, 3, 3201, [70], UNPACKED)]


@pytest.mark.parametrize("case", PEAKS)
def test_kernel_of_the_peaks(rec, case):
    D, B, n, peaks, kernel = case
    got = _kernels(rec, 4, 1, D, B * n, B, 2048 * len(peaks), 64)
    assert kernel in got
    assert (UNPACKED in got) == (kernel == UNPACKED) and (DEC in got) == (kernel == DEC)


def _far_apart(D, B, n, peaks, below, codes, dt):
    """131072 alike keys for each of a few (at the positions `peaks`) that weigh
    2^below of one; values of 1, or of -1, that the few share in their second half of
    the dimensions alone, with zeros in the first.  Sequences share their pages: there
    are enough of them that one CTA takes all keys of its rows.

    The results and 64 bits' of either half, for both signs: [rows, heads, D / 2], [rows]."""
    L = 131072 * len(peaks)
    one = kv.Batch([n], [L], 64, seed=3, spare=0, behind=0)
    cache = w4.kv_cache(one.pages, 1, 64, D, codes, DEV)
    high, low = (torch.tensor(s * kv.TOP[codes]).to(codes).view(torch.uint8).item() for s in (1, -1))
    pg, sl = one.table[0, torch.tensor(peaks) // 64].long().to(DEV), torch.tensor(peaks, device=DEV) % 64
    # q of ones: such a key's score is below * log 2, the others' (keys of zeros) 0
    ks = torch.tensor(below * math.log(2.0) / (kv.TOP[codes] * D**0.5))
    cache.k.view(torch.uint8)[pg, :, sl] = high
    cache.k_scales[pg, :, sl] = ks.to(DEV)
    cache.v_scales.fill_(1 / kv.TOP[codes])
    table = one.table.expand(B, one.width).contiguous().to(DEV)
    starts = torch.arange(B + 1, dtype=torch.int32, device=DEV) * n
    lens = torch.full((B,), L, dtype=torch.int32, device=DEV)
    q = torch.ones(B * n, 4, D, dtype=dt, device=DEV)
    w = len(peaks) * math.exp(float(ks.double()) * kv.TOP[codes] * D**0.5)
    keys = L - n + 1 + torch.arange(n).double().repeat(B) - len(peaks)  # alike ones that a row sees
    v = float(cache.v_scales[0, 0, 0].double()) * kv.TOP[codes]
    for sign in (1, -1):
        cache.v.view(torch.uint8).fill_(high if sign > 0 else low)
        cache.v.view(torch.uint8)[pg, :, sl, :D // 2] = 0
        cache.v.view(torch.uint8)[pg, :, sl, D // 2:] = high
        out = w4.cache_attention(cache, q, table, starts, lens).cpu().double()
        yield out[..., :D // 2], v * sign * keys / (w + keys)
        yield out[..., D // 2:], v * (w + sign * keys) / (w + keys)


@pytest.mark.gpu
@pytest.mark.parametrize("codes,dt", [(S8, torch.float16), (F8, torch.float16), (S8, torch.bfloat16)])
@pytest.mark.parametrize("below", [18, 25.01, 26, 28])
@pytest.mark.parametrize("case", PEAKS)
def test_many_small_weights(gpu_lib, case, below, codes, dt):
    """Weights of 2^-below of the largest are not lost on their way into 16 bits.

    The bound, relative to the largest weight, in the half of the dimensions where it
    has no value.  With it at 2^6 at least, a weight in fp16 is off by 2^-11 of itself
    or by 2^-25, 2^-31 of the largest, 131072 by 2^-14.  The tensor cores drop up to
    2^-24 of a sum from each product that they add to it: 2^-7 of the result.  The sum
    of the weights is off by 2^-9 (2^14 additions a lane, half a unit in the last
    place each; small ones lost beside a large one, 2^-9 of it all together), the
    scores and their exponentials by 2^-17, the result by half a step.  In the other
    half the dropped parts are of the largest weight's value: 2^-7 of it."""
    for i, (out, ref) in enumerate(_far_apart(*case[:4], below, codes, dt)):
        ref = ref[:, None, None]
        half = torch.finfo(dt).eps / 2
        rel = 2.0**-11 + 2.0**-7 + 2.0**-9 + 2.0**-17
        bound = (rel * (ref.abs() if i % 2 == 0 else 1.0) + 2.0**-14) * (1 + half) + half * ref.abs()
        off = (out - ref).abs()
        assert bool((off <= bound).all()), (i, float((off / bound).max()), float(off.max()), float(ref[0]))


@pytest.mark.gpu
@pytest.mark.parametrize("codes,dt", [(S8, torch.float16), (F8, torch.float16), (S8, torch.bfloat16)])
@pytest.mark.parametrize("below", [18, 25.01, 26, 28])
def test_many_small_weights_on_the_cuda_cores(gpu_lib, below, codes, dt):
    """The same of the kernel for other head dimensions, all in fp32: keys are added 32
    at a time, so 2^12 additions in a row to each sum, each off by half a unit in the
    last place; scores and exponentials by 2^-17, the result by half a step."""
    for i, (out, ref) in enumerate(_far_apart(96, 1, 1, [70], below, codes, dt)):
        ref = ref[:, None, None]
        half = torch.finfo(dt).eps / 2
        rel = 2 * 2.0**-12 + 2.0**-17
        bound = rel * (ref.abs() if i % 2 == 0 else 1.0) * (1 + half) + half * ref.abs()
        off = (out - ref).abs()
        assert bool((off <= bound).all()), (i, float((off / bound).max()), float(off.max()), float(ref[0]))


# ------------------------------------------------------------------ workspaces
def _size(rec, heads, kv_heads, dim, rows, sequences, width, page=32):
    return rec.lib.w4_attention_workspace_size(
        ctypes.byref(_cache(heads=kv_heads, head_dim=dim, page_size=page)),
        ctypes.byref(_of(table_width=width, sequences=sequences)), rows, heads)


def test_workspace_of_a_larger_batch(rec):
    """A workspace sized for 64 sequences, whose copies of keys and values are over the
    limit, does for one, whose are not: without them."""
    shape = dict(heads=32, kv_heads=8, dim=128, rows=16384, width=256)
    large, small = (_size(rec, sequences=n, **shape) for n in (64, 1))
    assert large < small
    assert UNPACKED in _kernels(rec, sequences=1, nws=small, **shape)
    for nws in (large, small - 1):
        got = _kernels(rec, sequences=1, nws=nws, **shape)
        assert OWN in got and UNPACKED not in got


@pytest.mark.parametrize("dim", [64, 128, 96])
def test_workspace_for_one_row_does(rec, dim):
    least = _size(rec, 32, 8, dim, 1, 1, 1)
    for rows, sequences, width in ((1, 1, 1), (300, 300, 4), (1000, 7, 64), (8192, 1, 256),
                                   (8192, 1, 1 << 20), (100000, 40, 512)):
        assert _size(rec, 32, 8, dim, rows, sequences, width) >= least
        _kernels(rec, 32, 8, dim, rows, sequences, width, nws=least)
        cache, of = _cache(heads=8, head_dim=dim, page_size=32), _of(table_width=width,
                                                                     sequences=sequences)
        st = rec.lib.w4_cache_attention(ctypes.byref(cache), ctypes.byref(of), 0x80000000, w4.F16,
                                        rows, 32, 32 * dim, 0.1, 0, 0, 1 << 40, 1 << 41, least - 1,
                                        None)
        assert st == w4.ERR_WORKSPACE


@pytest.mark.gpu
@pytest.mark.parametrize("D,codes,dt", [(128, S8, torch.bfloat16), (64, F8, torch.float16)])
def test_with_and_without_copies(gpu_lib, D, codes, dt):
    """Rows enough for copies of keys and values, in a workspace with room for them
    and in one without; and the binding's own, which has room."""
    batch = kv.Batch([300, 1, 250], [700, 90, 250], 32, seed=1, behind=0)
    cache = kv.random_cache(batch, 2, D, codes)
    held, plan = kv.on(cache, DEV), batch.plan(DEV)
    q = torch.randn(batch.T, 16, D, generator=torch.Generator().manual_seed(2)).to(dt)
    ref, bound = kv.attention(q, cache, batch, 130, 5)
    full = w4.attention_workspace_size(held, batch.T, 16, plan[0])
    least = w4.attention_workspace_size(held, 1, 16, plan[0])
    assert least < full
    out = {}
    side = torch.cuda.Stream()  # (with no workspace yet)
    with torch.cuda.stream(side):
        out[0] = w4.cache_attention(held, q.to(DEV), *plan, window=130, sinks=5)
        assert w4.workspace(held.k.device, 0).numel() >= full
    side.synchronize()
    for n in (full, least):
        ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
        out[n] = w4.cache_attention(held, q.to(DEV), *plan, window=130, sinks=5, ws=ws)
        assert w4.check_status(ws) == w4.OK
    for x in out.values():
        assert bool(((x.cpu().double() - ref).abs() <= bound).all())
    with pytest.raises(w4.W4Error):
        w4.cache_attention(held, q.to(DEV), *plan,
                           ws=torch.zeros(least - 1, dtype=torch.uint8, device=DEV))


# -------------------------------------------------------------------- queries
def _heads(rows):
    return 96 if rows == 300 else 6


@pytest.mark.parametrize("D,rows,wide,kernel", [(128, 1, False, DEC), (64, 1, False, DEC),
                                                (128, 20, True, OWN), (64, 20, True, OWN),
                                                (128, 90, True, OWN), (64, 90, True, OWN),
                                                (128, 300, False, UNPACKED), (64, 300, False, UNPACKED)])
def test_kernel_of_large_queries(rec, D, rows, wide, kernel):
    got = _kernels(rec, _heads(rows), 2, D, 3 * rows, 3, (1 << 16) if wide else 13, 32)
    assert kernel in got
    assert (UNPACKED in got) == (kernel == UNPACKED) and (DEC in got) == (kernel == DEC)


@pytest.mark.gpu
@pytest.mark.parametrize("D,rows,wide", [(128, 1, False), (64, 1, False), (128, 20, True),
                                         (64, 20, True), (128, 90, True), (64, 90, True),
                                         (128, 300, False), (64, 300, False), (96, 3, False),
                                         (256, 1, False)])
@pytest.mark.parametrize("codes", [S8, F8])
@pytest.mark.parametrize("sizes,scale,log", [((1e35, 1.0, 1e34), 1e-35, 0),
                                             ((5e34, 1e20, 1e30), -2e-35, 0),
                                             ((1e35, 1e-3, 1e35), None, -90)])
def test_large_queries(gpu_lib, D, rows, wide, codes, sizes, scale, log):
    """bf16 queries whose products with the codes pass fp32's largest number (some
    rows have the signs of a key's codes), with scores of some tens or more, beside
    rows of other sizes."""
    batch = kv.Batch([rows] * 3, [400] * 3, 32, behind=0, wide=wide)
    cache = kv.random_cache(batch, 2, D, codes)
    cache.k_scales.mul_(2.0**log)
    g = torch.Generator().manual_seed(4)
    q = torch.randn(batch.T, _heads(rows), D, generator=g).clamp(-3, 3)
    K, _ = kv.dequantised(cache, batch, 0)
    q[:rows, 0] = 2.5 * K[0, 11].sign().float()
    q[:rows, -1] = -2.5 * K[1, 11].sign().float()
    for i, size in enumerate(sizes):
        q[i * rows:(i + 1) * rows] *= size
    q[::5, 2] *= 1e-7  # (heads of other sizes beside them)
    code = cache.k.float().abs().sum(-1).nan_to_num(0).max()
    assert 2.0**128 < float(q.abs().max().double() * code) < 2.0**135
    _check(None, None, _heads(rows), 2, D, 32, codes, torch.bfloat16, q=q.to(torch.bfloat16),
           cache=cache, batch=batch, scale=scale, behind=0)


# ----------------------------------------------------------------- large caches
@pytest.mark.gpu
@pytest.mark.parametrize("D,codes", [(128, S8), (64, F8), (96, S8)])
def test_cache_beyond_32_bits(gpu_lib, D, codes):
    """Codes beyond 2^31 and 2^32 bytes into their array: rows are written, read and
    attended to as in a small cache, bit for bit."""
    H, page, dt = 2, 64, torch.bfloat16
    rows, lens = [300, 1, 40, 0], [300, 700, 90, 20]
    batch = kv.Batch(rows, lens, page, seed=5, behind=0)
    pages = (1 << 32) // (H * page * D) + batch.pages
    table, starts, n = batch.plan(DEV)
    far = torch.where(table < 0, table, pages - 1 - table)  # the last ones ...
    half = (1 << 31) // (H * page * D)
    far[1] = torch.where(table[1] < 0, table[1], half - 3 + table[1] % 6 + 6 * (table[1] // 6))
    whole = torch.tensor([0, *torch.tensor(lens).cumsum(0)], dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn(sum(lens), H, D, generator=g).to(dt).to(DEV) for _ in range(2))
    q = torch.randn(batch.T, 8, D, generator=g).to(dt).to(DEV)
    got = []
    for count, t in ((batch.pages, table), (pages, far)):
        cache = w4.kv_cache(count, H, page, D, codes, DEV)
        w4.cache_write(cache, k, v, t, whole, n)
        out = [*w4.cache_read(cache, t, whole, n, sum(lens), dt),
               w4.cache_attention(cache, q, t, starts, n),
               w4.cache_attention(cache, q[:4], t, torch.arange(5, dtype=torch.int32, device=DEV), n)]
        # the tensor cores' kernel, and with its copies of keys and values
        for heads, w in ((8, 1 << 12), (192, t.shape[1])):
            wide = torch.nn.functional.pad(t, (0, w - t.shape[1]), value=-1)
            many = q[:, :1].expand(-1, heads, -1).contiguous()
            out.append(w4.cache_attention(cache, many, wide, starts, n))
        got.append(out)
        written = cache.k.view(torch.uint8).flatten(1).any(1).sum()
        assert int(written) == len(set(t[t >= 0].tolist()))
        del cache
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("D,rows,wide", [(128, 1, False), (128, 20, True), (64, 20, True),
                                         (128, 90, True), (64, 90, True), (128, 300, False),
                                         (64, 300, False), (96, 3, False)])
@pytest.mark.parametrize("codes", [S8, F8])
@pytest.mark.parametrize("sizes,log", [((1e-30, 1e-31, 1e-29), 98), ((3e-34, 1e-35, 1e-33), 110),
                                       ((3e-37, 1e-36, 1e-37), 120)])
def test_small_queries(gpu_lib, D, rows, wide, codes, sizes, log):
    """bf16 queries near the smallest normal number, keys so large that scores are some
    ones to tens."""
    batch = kv.Batch([rows] * 3, [400] * 3, 32, behind=0, wide=wide)
    cache = kv.random_cache(batch, 2, D, codes)
    cache.k_scales.mul_(2.0**log)
    g = torch.Generator().manual_seed(4)
    q = torch.randn(batch.T, _heads(rows), D, generator=g)
    for i, size in enumerate(sizes):
        q[i * rows:(i + 1) * rows] *= size
    _check(None, None, _heads(rows), 2, D, 32, codes, torch.bfloat16, q=q.to(torch.bfloat16),
           cache=cache, batch=batch, behind=0)
