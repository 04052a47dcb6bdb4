"""Attention over the paged key-value cache (causal, window and sinks, trees of
drafts): within a derived bound (kv.attention) of the definition in 64 bits,
and the refusals (CPU)."""
import ctypes

import pytest
import torch

import int4_weight_mixed_gb300 as w4
import kv
from test_kv_cache import P, _cache, _of

DEV = "cuda:0"
S8, F8 = torch.int8, torch.float8_e4m3fn


def _tree(rows, width, seed=0, kind="tree"):
    """[T, width] truth values; rows behind the last sequence see nothing."""
    g = torch.Generator().manual_seed(seed)
    mask = torch.zeros(sum(rows), width, dtype=torch.bool)
    at = 0
    for n in rows:
        for t in range(n):
            if kind == "tree":
                p = int(torch.randint(-1, t, (1,), generator=g)) if t else -1
                if p >= 0:
                    mask[at + t] = mask[at + p]
                if t < width:
                    mask[at + t, t] = True
            elif kind == "any":  # not a tree: any drafts, some rows none
                mask[at + t] = torch.rand(width, generator=g) < (0.0 if t % 5 == 2 else 0.5)
        at += n
    return mask


def _check(rows, lens, Hq, Hkv, D, page, codes, dt, window=0, sinks=0, mask=None, scale=None,
           seed=0, q=None, cache=None, batch=None, behind=2, wide=False):
    batch = batch or kv.Batch(rows, lens, page, seed, behind=behind, wide=wide)
    cache = cache or kv.random_cache(batch, Hkv, D, codes, seed)
    g = torch.Generator().manual_seed(seed + 1)
    if q is None:  # queries as a slice of wider rows
        q = (torch.randn(batch.T, (Hq + 2) * D, generator=g) * 1.5).to(dt)[:, D:(Hq + 1) * D]
        q = q.reshape(batch.T, Hq, D)
    wide = torch.zeros(batch.T, Hq + 2, D, dtype=dt)
    wide[:, 1:Hq + 1] = q
    qd = wide.to(DEV)[:, 1:Hq + 1]
    out = torch.full((batch.T, Hq, D), 7.0, dtype=dt, device=DEV)
    held, plan = kv.on(cache, DEV), batch.plan(DEV)
    kw = dict(scale=scale, window=window, sinks=sinks, out=out)
    if mask is None:
        r = w4.cache_attention(held, qd, *plan, **kw)
    else:
        full = torch.zeros(batch.T, mask.shape[1], dtype=torch.bool)
        full[:mask.shape[0]] = mask
        r = w4.tree_attention(held, qd, full.to(DEV), *plan, **kw)
    assert r is out
    torch.cuda.synchronize()
    n = sum(batch.rows)
    got = out.cpu().double()
    assert bool((got[n:] == 7.0).all()), "rows of no sequence"
    ref, bound = kv.attention(q[:n], cache, batch, window, sinks, mask, scale)
    off = (got[:n] - ref).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (int(bad.sum()), bad.numel(), float((off / bound).nan_to_num(9e9).max()),
                           bad.any(2).nonzero()[:8].tolist())
    return out


DECODE = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 700]
HEADS = [(8, 2, 128), (4, 4, 64), (8, 1, 64), (5, 1, 128), (16, 1, 128), (24, 1, 64), (6, 2, 96),
         (4, 2, 256), (2, 1, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [S8, F8])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_decode(gpu_lib, Hq, Hkv, D, dt, codes):
    _check([1] * len(DECODE), DECODE, Hq, Hkv, D, 16 if D == 64 else 64, codes, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("codes,dt", [(S8, torch.bfloat16), (F8, torch.float16)])
@pytest.mark.parametrize("page", [16, 32, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_pages(gpu_lib, page, D, codes, dt, wide):
    _check([1, 1, 3, 40], [page - 1, page + 1, 5 * page, 3 * page + 7], 4, 2, D, page, codes, dt,
           wide=wide)


MIXED = {
    "prompt": ([200], [200]), "long prompts": ([700, 900], [1300, 900]), "prompts": ([1, 129, 64, 300], [1, 129, 64, 300]),
    "chunk": ([70], [333]), "mixed": ([1, 90, 0, 1, 17, 5], [400, 131, 40, 1, 17, 260]),
    "more rows than positions": ([6, 3, 2], [4, 0, 2]), "nothing": ([0, 0], [5, 0]),
    "long": ([2, 1], [3000, 2111]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("codes,dt", [(S8, torch.bfloat16), (F8, torch.float16), (F8, torch.bfloat16),
                                      (S8, torch.float16)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (6, 2, 64), (3, 3, 128), (16, 1, 64), (2, 1, 48)])
@pytest.mark.parametrize("kind", list(MIXED))
def test_mixed(gpu_lib, kind, Hq, Hkv, D, codes, dt, wide):
    _check(*MIXED[kind], Hq, Hkv, D, 32, codes, dt, wide=wide)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("codes,dt", [(S8, torch.bfloat16), (F8, torch.float16)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 0), (129, 33), (64, 300),
                                          (1000, 4), (5000, 1)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (3, 1, 64), (2, 1, 80)])
def test_window_and_sinks(gpu_lib, Hq, Hkv, D, window, sinks, codes, dt, wide):
    _check([1, 1, 1, 150, 40, 20], [1, 130, 900, 150, 777, 1200], Hq, Hkv, D, 16, codes, dt, window,
           sinks, wide=wide)


@pytest.mark.gpu
@pytest.mark.parametrize("codes,dt", [(S8, torch.bfloat16), (F8, torch.float16), (F8, torch.bfloat16),
                                      (S8, torch.float16)])
@pytest.mark.parametrize("window,sinks", [(1, 1), (300, 4), (1000, 200)])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 1, 128), (32, 2, 64)])
def test_window_and_sinks_of_chunks(gpu_lib, Hq, Hkv, D, window, sinks, codes, dt):
    """Rows enough for the keys and values to be unpacked first; some sequences
    have few, or none."""
    _check([1, 300, 0, 128, 63], [900, 1000, 70, 128, 1999], Hq, Hkv, D, 64, codes, dt, window, sinks)

@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("codes,dt", [(S8, torch.bfloat16), (F8, torch.float16)])
@pytest.mark.parametrize("kind", ["tree", "any", "none"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4), (3, 0)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (3, 1, 64), (2, 1, 112)])
def test_tree(gpu_lib, Hq, Hkv, D, window, sinks, kind, codes, dt, wide):
    rows = [1, 7, 64, 0, 33, 130, 4]
    lens = [1, 300, 600, 10, 33, 500, 2]
    _check(rows, lens, Hq, Hkv, D, 16, codes, dt, window, sinks, _tree(rows, 130, kind=kind),
           wide=wide)


@pytest.mark.gpu
@pytest.mark.parametrize("codes,dt", [(S8, torch.bfloat16), (F8, torch.float16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 4)])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 1, 128), (64, 2, 64)])
def test_large_trees(gpu_lib, Hq, Hkv, D, window, sinks, codes, dt):
    rows = [130, 70, 1]
    _check(rows, [900, 300, 40], Hq, Hkv, D, 16, codes, dt, window, sinks, _tree(rows, 130))


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("width", [0, 1, 20, 200])
def test_tree_masks_of_other_widths(gpu_lib, width, wide):
    rows, lens = [5, 40], [77, 140]
    _check(rows, lens, 4, 1, 64, 32, S8, torch.bfloat16, mask=_tree(rows, width), wide=wide)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
def test_chain_is_causal(gpu_lib, wide):
    """A tree that is one chain sees what the causal rows see: both within the
    bound of the causal definition."""
    rows, lens = [9, 30], [300, 64]
    mask = torch.cat([torch.ones(n, 30, dtype=torch.bool).tril() for n in rows])
    for codes, D in ((S8, 128), (F8, 64)):
        a = _check(rows, lens, 8, 2, D, 16, codes, torch.bfloat16, wide=wide)
        b = _check(rows, lens, 8, 2, D, 16, codes, torch.bfloat16, mask=mask, wide=wide)
        batch = kv.Batch(rows, lens, 16, behind=2)
        q = torch.randn(batch.T, 10 * D, generator=torch.Generator().manual_seed(1)) * 1.5
        q = q.bfloat16()[:, D:9 * D].reshape(batch.T, 8, D)
        ref, bound = kv.attention(q[:39], kv.random_cache(batch, 2, D, codes), batch)
        for x in (a, b):
            assert bool(((x[:39].cpu().double() - ref).abs() <= bound).all())


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D,rows", [(128, 1), (64, 1), (128, 90), (64, 40), (96, 3)])
@pytest.mark.parametrize("codes", [S8, F8])
def test_scales_far_apart(gpu_lib, D, rows, codes, wide):
    """Values whose scales span twenty binary orders, values of zeros, keys of
    zeros, large scores: the probabilities are rounded relative to what they
    weigh."""
    for dt in (torch.float16, torch.bfloat16):
        batch = kv.Batch([rows], [500], 32, behind=2, wide=wide)
        cache = kv.random_cache(batch, 1, D, codes)
        g = torch.Generator().manual_seed(3)
        up = torch.exp2(torch.randint(-14, 7, cache.v_scales.shape, generator=g).float())
        cache.v_scales.mul_(up)
        cache.v_scales[:, :, 3::7] = 0.0
        cache.v.view(torch.uint8)[:, :, 3::7] = 0
        cache.k_scales[:, :, 5::11] = 0.0
        cache.k.view(torch.uint8)[:, :, 5::11] = 0
        q = (torch.randn(batch.T, 4, D, generator=g) * 4).to(dt)
        _check(None, None, 4, 1, D, 32, codes, dt, q=q, cache=cache, batch=batch)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D,rows", [(128, 1), (64, 1), (128, 90), (64, 40), (96, 3)])
@pytest.mark.parametrize("log", [-40, 0, 35])
def test_values_of_zeros_weigh(gpu_lib, D, rows, log, wide):
    """Three keys of four with values of zeros beside large, ordinary and small
    values: they weigh in the sum whatever the others' scales are."""
    batch = kv.Batch([rows], [500], 32, behind=2, wide=wide)
    cache = kv.random_cache(batch, 1, D, S8)
    cache.v_scales.mul_(2.0**log)
    for i in range(3):
        cache.v_scales[:, :, i::4] = 0.0
        cache.v.view(torch.uint8)[:, :, i::4] = 0
    _check(None, None, 4, 1, D, 32, S8, torch.bfloat16, cache=cache, batch=batch)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D,rows", [(128, 1), (128, 70), (64, 70), (32, 2)])
def test_sizes_of_queries(gpu_lib, D, rows, wide):
    """Queries near the types' ends: large, small, zero rows, one channel far
    above the others."""
    for dt, sizes in ((torch.bfloat16, (1e-30, 1e-4, 1.0, 1e4)), (torch.float16, (1e-6, 1.0, 300.0))):
        batch = kv.Batch([rows] * len(sizes), [130] * len(sizes), 32, behind=0, wide=wide)
        cache = kv.random_cache(batch, 2, D, S8)
        g = torch.Generator().manual_seed(3)
        q = torch.randn(batch.T, 4, D, generator=g)
        for i, size in enumerate(sizes):
            q[i * rows:(i + 1) * rows] *= size
        q[:, 0, 7] *= 50
        q[::3, 1] = 0
        scale = 1 / D**0.5
        _check(None, None, 4, 2, D, 32, S8, dt, q=q.to(dt), cache=cache, batch=batch, scale=scale,
               behind=0)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("scale", [0.0, 1.0, -0.25])
def test_scale(gpu_lib, scale, wide):
    for D in (64, 32):
        _check([1, 40], [90, 100], 4, 2, D, 16, S8, torch.float16, scale=scale, wide=wide)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D,Hq", [(128, 4), (64, 16), (96, 2)])
@pytest.mark.parametrize("codes", [S8, F8])
def test_what_holds_nan_is_seen_by_its_rows_alone(gpu_lib, D, Hq, codes, wide):
    """A key or value written from an infinity or NaN makes the rows that see it
    NaN and no others."""
    n = 90
    batch = kv.Batch([n, 1], [n, 50], 16, behind=0, wide=wide)
    dt = torch.bfloat16
    for which in ("k_scales", "v_scales"):
        cache = kv.random_cache(batch, 1, D, codes)
        pg, sl = batch.slots(0, 60, 61)
        getattr(cache, which)[pg, :, sl] = float("nan")
        (cache.k if which[0] == "k" else cache.v).view(torch.uint8)[pg, :, sl] = 0
        q = torch.randn(batch.T, Hq, D).to(dt)
        for window in (0, 10):
            out = w4.cache_attention(kv.on(cache, DEV), q.to(DEV), *batch.plan(DEV),
                                     window=window).cpu()
            row = torch.arange(n + 1)
            sees = (row >= 60) & (row < n) & ((window == 0) | (row < 60 + 10))
            assert bool(out.isnan().all(2).all(1)[sees].all())
            assert not bool(out[~sees].isnan().any())


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D", [64, 128, 48])
def test_queries_of_nan(gpu_lib, D, wide):
    """A row of queries that holds one is NaN, the others are as without it."""
    batch = kv.Batch([20, 1], [60, 90], 16, behind=0, wide=wide)
    cache = kv.on(kv.random_cache(batch, 2, D, S8), DEV)
    q = torch.randn(batch.T, 4, D).bfloat16()
    clean = w4.cache_attention(cache, q.to(DEV), *batch.plan(DEV)).cpu()
    q[3, 1, 5] = float("nan")
    q[20, 2, 0] = float("inf")
    got = w4.cache_attention(cache, q.to(DEV), *batch.plan(DEV)).cpu()
    assert bool(got[3, 1].isnan().all()) and bool(got[20, 2].isnan().any())
    keep = torch.ones(batch.T, 4, dtype=torch.bool)
    keep[3, 1] = keep[20, 2] = False
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D", [64, 128, 160])
def test_same_bits_again(gpu_lib, D, wide):
    """Runs of a call give the same bits (no sum's order is left to chance), on
    one workspace with calls of other shapes between them."""
    batch = kv.Batch([1, 60, 3, 1], [5000, 900, 2000, 17], 32, behind=0, wide=wide)
    cache = kv.on(kv.random_cache(batch, 2, D, F8), DEV)
    q = torch.randn(batch.T, 16, D).half().to(DEV)
    small = kv.Batch([1], [100], 32, behind=0)
    first = w4.cache_attention(cache, q, *batch.plan(DEV))
    for _ in range(20):
        w4.cache_attention(cache, q[:1], small.table[:, :1].to(DEV) * 0, *small.plan(DEV)[1:])
        assert torch.equal(w4.cache_attention(cache, q, *batch.plan(DEV)), first)


@pytest.mark.gpu
@pytest.mark.parametrize("D,n", [(64, 40), (128, 40), (80, 40), (128, 1), (64, 1), (128, 1300),
                                 (64, 1300)])
@pytest.mark.parametrize("wide", [False, True])
def test_pages_that_are_none(gpu_lib, D, n, wide):
    """Keys of pages outside the cache are not seen; a row with no other is
    zeros; lengths beyond the table count as its end."""
    batch = kv.Batch([1, 1, n], [64, 64, max(64, n)], 16, behind=0, wide=wide)
    cache = kv.random_cache(batch, 1, D, S8)
    q = torch.randn(batch.T, 2, D).half()
    held = kv.on(cache, DEV)
    table, starts, lens = batch.plan(DEV)
    bad = table.clone()
    bad[0, :] = -1
    bad[1, 1] = batch.pages
    bad[2, 2] = 1 << 30
    lens[1] = 2**31 - 1  # (the entries behind its four pages are none)
    got = w4.cache_attention(held, q.to(DEV), bad, starts, lens).cpu()
    assert bool((got[0] == 0).all())
    # the same with these pages' keys cut out
    K, V = kv.dequantised(cache, batch, 1)
    see = torch.ones(64, dtype=torch.bool)
    see[16:32] = False
    t = torch.einsum("gd,kd->gk", q[1].double(), K[0]) / D**0.5
    p = torch.softmax(t.masked_fill(~see, float("-inf")), -1)
    assert torch.allclose(got[1].double(), p @ V[0], atol=4e-3, rtol=4e-3)
    assert torch.isfinite(got).all()


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D,n", [(128, 1), (64, 1), (128, 64), (96, 2), (128, 390), (64, 200)])
def test_captured_and_replayed(gpu_lib, D, n, wide):
    """A captured call follows what its arrays hold when it is replayed."""
    batch = kv.Batch([n, n], [n + 400, n + 300], 16, behind=0, wide=wide)
    cache = kv.random_cache(batch, 2, D, S8)
    held, (table, starts, lens) = kv.on(cache, DEV), batch.plan(DEV)
    q = torch.randn(batch.T, 4, D).half().to(DEV)
    out = torch.empty_like(q)
    ws = torch.zeros(w4.attention_workspace_size(held, batch.T, 4, table), dtype=torch.uint8, device=DEV)
    w4.cache_attention(held, q, table, starts, lens, out=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.cache_attention(held, q, table, starts, lens, out=out, ws=ws)
    with pytest.raises(RuntimeError, match="ws="):
        bad = torch.cuda.CUDAGraph()
        with torch.cuda.graph(bad):
            w4.cache_attention(held, q, table, starts, lens, out=out)
    for k in ([n + 400, n + 300], [n, 77], [200, n + 1]):
        lens.copy_(torch.tensor(k))
        q.copy_(torch.randn(batch.T, 4, D))
        graph.replay()
        batch.lens = k
        ref, bound = kv.attention(q.cpu(), cache, batch)
        assert bool(((out.cpu().double() - ref).abs() <= bound).all())
    assert w4.check_status(ws) == w4.OK


@pytest.mark.gpu
@pytest.mark.parametrize("n,wide", [(1, False), (40, False), (40, True), (900, False)])
def test_rows_before_the_first_sequence(gpu_lib, n, wide):
    """starts[0] rows belong to no sequence: left as they were."""
    batch = kv.Batch([n, 3], [n + 50, 90], 16, behind=0, wide=wide)
    cache = kv.random_cache(batch, 2, 128, S8)
    q = torch.randn(batch.T + 5, 8, 128).half()
    table, starts, lens = batch.plan(DEV)
    out = torch.full((batch.T + 5, 8, 128), 7.0, dtype=torch.float16, device=DEV)
    held = kv.on(cache, DEV)
    w4.cache_attention(held, q.to(DEV), table, starts + 5, lens, out=out)
    assert bool((out[:5] == 7.0).all())
    ref, bound = kv.attention(q[5:], cache, batch)
    assert bool(((out[5:].cpu().double() - ref).abs() <= bound).all())
    k, v = w4.cache_read(held, table, starts + 5, lens, batch.T + 5, torch.float16)
    k0, v0 = w4.cache_read(held, table, starts, lens, batch.T, torch.float16)
    assert torch.equal(k[5:], k0) and torch.equal(v[5:], v0)


@pytest.mark.gpu
def test_two_host_threads(gpu_lib):
    """Calls of two host threads on one stream with its cached workspace give what
    each gives alone."""
    import threading
    jobs = []
    for n, k, D in ((1, 700, 128), (300, 900, 128), (60, 2000, 64), (1, 3000, 64)):
        batch = kv.Batch([n, n], [k, k - 200], 16, behind=0)
        held = kv.on(kv.random_cache(batch, 2, D, S8), DEV)
        args = (held, torch.randn(batch.T, 16, D).half().to(DEV), *batch.plan(DEV))
        jobs.append((args, w4.cache_attention(*args)))
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(2), []

    def work(mine):
        start.wait()
        outs = [(w4.cache_attention(*args), ref) for _ in range(30) for args, ref in mine]
        wrong.extend(i for i, (out, ref) in enumerate(outs) if not torch.equal(out, ref))

    threads = [threading.Thread(target=work, args=(jobs[i::2],)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.gpu
def test_layer_step(gpu_lib):
    """The calls together as a serving step makes them: prompts, then tokens one
    by one, then a tree whose accepted path is written again; against attention
    over the same rows quantised by the definition."""
    H, Hq, D, page, dt = 2, 8, 128, 16, torch.bfloat16
    g = torch.Generator().manual_seed(0)
    B, pages = 3, 40
    cache = w4.kv_cache(pages, H, page, D, F8, DEV)
    mine = kv.Batch([1] * B, [160] * B, page, seed=1, spare=0)
    table = mine.table.to(DEV)
    past = [torch.zeros(0, 2, H, D, dtype=dt) for _ in range(B)]

    def step(rows, mask=None, keep=None):
        qkv = (torch.randn(sum(rows), (Hq + 2 * H) * D, generator=g)).to(dt)
        k, v = (qkv[:, (Hq + i * H) * D:(Hq + (i + 1) * H) * D].view(-1, H, D) for i in range(2))
        for b, n in enumerate(rows):
            at = sum(rows[:b])
            past[b] = torch.cat([past[b], torch.stack([k[at:at + n], v[at:at + n]], 1)])
        starts = torch.tensor([0, *torch.tensor(rows).cumsum(0)], dtype=torch.int32, device=DEV)
        lens = torch.tensor([len(p) for p in past], dtype=torch.int32, device=DEV)
        x = qkv.to(DEV)
        qd, kd, vd = x[:, :Hq * D].view(-1, Hq, D), x[:, Hq * D:(Hq + H) * D].view(-1, H, D), \
            x[:, (Hq + H) * D:].view(-1, H, D)
        w4.cache_write(cache, kd, vd, table, starts, lens)
        if mask is None:
            out = w4.cache_attention(cache, qd, table, starts, lens)
        else:
            out = w4.tree_attention(cache, qd, mask.to(DEV), table, starts, lens)
        # the definition over rows quantised on the host
        batch = kv.Batch(rows, [len(p) for p in past], page)
        ref = kv.random_cache(batch, H, D, F8)
        for b, p in enumerate(past):
            pg, sl = batch.slots(b, 0, len(p))
            for i, (c, s) in enumerate(((ref.k, ref.k_scales), (ref.v, ref.v_scales))):
                code, scale = kv.quantised(p[:, i], F8)
                c.view(torch.uint8)[pg, :, sl] = code.view(torch.uint8)
                s[pg, :, sl] = scale
        want, bound = kv.attention(qkv[:, :Hq * D].view(-1, Hq, D), ref, batch, mask=mask)
        assert bool(((out.cpu().double() - want).abs() <= bound).all())

    step([70, 33, 5])
    step([1, 1, 1])
    rows = [9, 9, 9]
    mask = _tree(rows, 9, seed=4)
    step(rows, mask)
    # sequence 0 keeps the path to its last draft, the others their first draft
    path = mask[8].nonzero().flatten().tolist()
    for b, keep in enumerate([path, [0], [0]]):
        drafts = past[b][-9:]
        past[b] = torch.cat([past[b][:-9], drafts[keep]])
    again = torch.cat([past[0][-len(path):], past[1][-1:], past[2][-1:]]).to(DEV)
    starts = torch.tensor([0, len(path), len(path) + 1, len(path) + 2], dtype=torch.int32, device=DEV)
    lens = torch.tensor([len(p) for p in past], dtype=torch.int32, device=DEV)
    w4.cache_write(cache, again[:, 0].contiguous(), again[:, 1].contiguous(), table, starts, lens)
    step([1, 1, 1])


# ------------------------------------------------------------------- refusals
def _attend(cache=None, batch=None, q=8 * P, type=w4.F16, rows=3, heads=4, stride=256, scale=0.1,
            window=0, sinks=0, out=9 * P, ws=0x40000000, nws=1 << 32, mask=0, width=4, tree=False):
    lib, c, b = w4.load(), ctypes.byref(cache or _cache()), ctypes.byref(batch or _of())
    rest = (type, rows, heads, stride, scale, window, sinks, out, ws, nws, None)
    return lib.w4_tree_attention(c, b, q, mask, width, *rest) if tree else lib.w4_cache_attention(
        c, b, q, *rest)


INVALID, UNSUPPORTED = w4.ERR_INVALID_ARGUMENT, w4.ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(cache=_cache(type=w4.BF16)), INVALID), (dict(type=w4.E4M3), INVALID),
    (dict(rows=-1), INVALID), (dict(heads=0), INVALID), (dict(heads=3), INVALID),
    (dict(heads=-2), INVALID), (dict(stride=255), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(sinks=-1), INVALID), (dict(q=None), INVALID),
    (dict(out=None), INVALID), (dict(q=8 * P + 1), INVALID), (dict(out=9 * P + 1), INVALID),
    (dict(out=8 * P), INVALID), (dict(out=8 * P + 1024), INVALID), (dict(ws=None), w4.ERR_WORKSPACE),
    (dict(ws=0x40000008), w4.ERR_WORKSPACE), (dict(nws=256), w4.ERR_WORKSPACE),
    (dict(out=P + 256), INVALID), (dict(out=3 * P), INVALID), (dict(heads=65536, stride=1 << 23), UNSUPPORTED),
    (dict(rows=1 << 29), UNSUPPORTED), (dict(cache=_cache(page_size=24)), UNSUPPORTED),
    (dict(cache=_cache(head_dim=40)), UNSUPPORTED), (dict(batch=_of(starts=None)), INVALID)])
@pytest.mark.parametrize("tree", [False, True])
def test_refused(kw, status, tree):
    assert _attend(tree=tree, mask=7 * P, **kw) == status, w4.load().w4_last_error()


def test_refused_masks():
    assert _attend(tree=True, mask=None) == INVALID
    assert _attend(tree=True, mask=7 * P, width=-1) == INVALID


def test_another_gpu(monkeypatch):
    """The extension module leaves calls on another GPU's tensors to be made again
    with that GPU current."""
    w4.build()
    w4._load_host()
    asked = []

    class Elsewhere:
        def __getattr__(self, name):
            return lambda *args: NotImplemented

    monkeypatch.setattr(w4, "_host", Elsewhere())
    monkeypatch.setattr(w4, "_there", lambda dev, call, args: asked.append(dev) or "done")
    cache = w4.kv_cache(2, 1, 16, 64, device="cpu")
    x = torch.zeros(1, 1, 64, dtype=torch.float16)
    plan = [torch.zeros(*z, dtype=torch.int32) for z in ((1, 1), (2,), (1,))]
    w4.cache_write(cache, x, x, *plan)
    assert w4.cache_read(cache, *plan, 1) == "done"
    assert w4.cache_attention(cache, x, *plan) == "done"
    assert w4.tree_attention(cache, x, torch.ones(1, 1, dtype=torch.bool), *plan) == "done"
    assert asked == [x.device] * 4


def test_nothing_to_do():
    for tree in (False, True):
        assert _attend(rows=0, q=None, out=None, ws=None, tree=tree, mask=7 * P) == w4.OK
        assert _attend(batch=_of(sequences=0), q=None, out=None, tree=tree, mask=7 * P) == w4.OK


@pytest.mark.gpu
def test_binding_checks_shapes(gpu_lib):
    batch = kv.Batch([3], [3], 16)
    plan = batch.plan(DEV)
    cache = w4.kv_cache(batch.pages, 2, 16, 64, S8, DEV)
    q = torch.zeros(3, 4, 64, dtype=torch.float16, device=DEV)
    mask = torch.ones(3, 3, dtype=torch.bool, device=DEV)
    for bad in (q.float(), q[..., :32], q.view(3, -1), q[:, :, ::2], q[:1].expand(3, 4, 64), q.cpu()):
        with pytest.raises(ValueError):
            w4.cache_attention(cache, bad, *plan)
    for kw in (dict(window=-1), dict(sinks=-1), dict(out=q[:2]), dict(out=q.bfloat16()),
               dict(out=torch.empty(3, 4, 128, dtype=torch.float16, device=DEV)[..., ::2])):
        with pytest.raises(ValueError):
            w4.cache_attention(cache, q, *plan, **kw)
    with pytest.raises(w4.W4Error):
        w4.cache_attention(cache, q[:, :3].contiguous(), *plan)
    with pytest.raises(w4.W4Error):
        w4.cache_attention(cache, q, *plan, out=q)
    with pytest.raises(w4.W4Error):
        w4.cache_attention(cache, q, *plan, ws=torch.zeros(256, dtype=torch.uint8, device=DEV))
    for m in (mask[:2], mask.float(), mask[0], mask.cpu(), mask.t()[:, ::1].expand(3, 3).t()[::1, ::2]):
        with pytest.raises(ValueError):
            w4.tree_attention(cache, q, m, *plan)
    with pytest.raises(TypeError):
        w4.tree_attention(cache, q, None, *plan)
    w4.cache_attention(cache, q, *plan, window=1 << 40, sinks=1 << 40)
