"""The paged key-value cache: rows written (codes and scales bit for bit those
of the definition), read back (bit for bit), and the refusals (CPU)."""
import ctypes

import pytest
import torch

import int4_weight_mixed_gb300 as w4
import kv

DEV = "cuda:0"
S8, F8 = torch.int8, torch.float8_e4m3fn


def _bits(t):
    return t.contiguous().view(torch.uint8) if t.element_size() == 1 else t


def _same(a, b):
    """Bit for bit, NaN as NaN."""
    a, b = _bits(a.cpu()), _bits(b.cpu())
    return a.shape == b.shape and bool(((a == b) | ((a != a) & (b != b))).all())


def _rows(T, H, D, dt, seed=0, extra=5):
    """Keys and values as slices of one array of rows."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, (extra + 2 * H) * D, generator=g)
    x *= torch.exp(2 * torch.randn(T, 1, generator=g))
    x = x.to(dt)
    return (x[:, extra * D:(extra + H) * D].view(T, H, D), x[:, (extra + H) * D:].view(T, H, D))


def _written(cache, batch, k, v):
    """The cache after the write, by the definition."""
    out = [t.clone() for t in cache]
    at = 0
    for b, (n, length) in enumerate(zip(batch.rows, batch.lens)):
        first = length - n
        lo = max(first, 0)
        pg, sl = batch.slots(b, lo, length)
        for i, x in enumerate((k, v)):
            c, s = kv.quantised(x[at + lo - first:at + n], out[i].dtype)
            out[i].view(torch.uint8)[pg, :, sl] = c.view(torch.uint8)
            out[2 + i][pg, :, sl] = s
        at += n
    return out


BATCHES = {
    "one": ([1], [1]), "decode": ([1] * 5, [1, 16, 17, 64, 300]),
    "prompts": ([33, 1, 200, 16], [33, 1, 200, 16]), "chunks": ([7, 0, 40, 1], [90, 5, 40, 129]),
    "more rows than positions": ([4, 3], [2, 0]), "many": ([1, 0, 2] * 30, [3, 1, 50] * 30),
    "long": ([3001, 1500], [3001, 2000]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [S8, F8])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kind,H,D,page", [
    ("one", 8, 128, 64), ("decode", 3, 64, 16), ("prompts", 2, 128, 32), ("chunks", 1, 96, 128),
    ("more rows than positions", 2, 16, 16), ("many", 4, 256, 16), ("long", 2, 128, 64),
    ("chunks", 5, 208, 256)])
def test_write_and_read(gpu_lib, kind, H, D, page, dt, codes):
    rows, lens = BATCHES[kind]
    batch = kv.Batch(rows, lens, page, behind=2)
    k, v = _rows(batch.T, H, D, dt)
    before = kv.random_cache(batch, H, D, codes, garbage=True)
    plan, cache = batch.plan(DEV), kv.on(before, DEV)
    w4.cache_write(cache, k.to(DEV).contiguous(), v.to(DEV), *plan)
    want = _written(before, batch, k, v)
    for name, got, ref in zip(cache._fields, cache, want):
        assert _same(got, ref), (name, int((_bits(got.cpu()) != _bits(ref)).sum()))
    # read back: the rows that were written, and rows of no sequence as they were
    out = [torch.full((batch.T, H, D), 7.0, dtype=dt, device=DEV) for _ in range(2)]
    got = w4.cache_read(cache, *plan, batch.T, dt, *out)
    assert got[0] is out[0] and got[1] is out[1]
    for i in range(2):
        ref, at = torch.full((batch.T, H, D), 7.0, dtype=dt), 0
        for b, (n, length) in enumerate(zip(rows, lens)):
            first, lo = length - n, max(length - n, 0)
            ref[at:at + n] = 0
            pg, sl = batch.slots(b, lo, length)
            c = want[i].view(torch.uint8)[pg, :, sl].view(codes)
            ref[at + lo - first:at + n] = (c.float() * want[2 + i][pg, :, sl][..., None]).to(dt)
            at += n
        assert _same(got[i], ref)


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [S8, F8])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_values_at_the_edges(gpu_lib, dt, codes):
    """Zeros, infinities, NaN, subnormal and largest values, ties of the codes."""
    D, H = 64, 1
    big, tiny = torch.finfo(dt).max, torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    x = torch.zeros(12, H, D)
    x[1, 0, 5] = float("inf")
    x[2, 0, 9] = float("nan")
    x[3] = big
    x[3, 0, ::2] = -big
    x[4] = tiny
    x[5, 0, 0] = tiny
    x[6, 0, :] = torch.arange(D).float() - 32  # ties against a largest value of 127 / 448
    x[6, 0, 0] = kv.TOP[codes]
    x[7, 0, :] = (torch.arange(D).float() - 32) / 2
    x[7, 0, 0] = kv.TOP[codes]
    x[8, 0, 3] = -float("inf")
    x[8, 0, 4] = float("nan")
    x[9] = 2.0**-120 if dt == torch.bfloat16 else 2.0**-24
    x[10, 0, 1], x[10, 0, 2] = big, tiny
    x[11] = torch.randn(D, generator=torch.Generator().manual_seed(1))
    x = x.to(dt)
    batch = kv.Batch([12], [12], 16)
    cache = w4.kv_cache(batch.pages, H, 16, D, codes, DEV)
    before = [t.cpu() for t in cache]
    w4.cache_write(cache, x.to(DEV), x.flip(0).contiguous().to(DEV), *batch.plan(DEV))
    want = _written(w4.KVCache(*before), batch, x, x.flip(0))
    for name, got, ref in zip(cache._fields, cache, want):
        assert _same(got, ref), name


@pytest.mark.gpu
def test_rows_anywhere_in_memory(gpu_lib):
    """Rows two bytes off a 16-byte boundary, odd strides, one row with any."""
    D, H, T = 64, 2, 5
    batch = kv.Batch([T], [T], 16)
    for stride, off in ((H * D, 1), (H * D + 3, 0), (H * D + 8, 0), (3 * H * D + 1, 5)):
        flat = torch.randn(T * stride + 16).half()
        k, v = (torch.as_strided(flat, (T, H, D), (stride, D, 1), off + e) for e in (0, 8))
        cache = w4.kv_cache(batch.pages, H, 16, D, S8, DEV)
        want = _written(w4.KVCache(*(t.cpu() for t in cache)), batch, k, v)
        held = flat.to(DEV)
        kd, vd = (torch.as_strided(held, (T, H, D), (stride, D, 1), off + e) for e in (0, 8))
        w4.cache_write(cache, kd, vd, *batch.plan(DEV))
        assert all(_same(a, b) for a, b in zip(cache, want)), (stride, off)
        line = torch.zeros(2 * T * H * D + 2, dtype=torch.float16, device=DEV)
        out = [line[1:1 + T * H * D].view(T, H, D), line[1 + T * H * D:1 + 2 * T * H * D].view(T, H, D)]
        w4.cache_read(cache, *batch.plan(DEV), T, torch.float16, *out)
        for o, c, s in zip(out, want, want[2:]):
            pg, sl = batch.slots(0, 0, T)
            assert _same(o, (c[pg, :, sl].float() * s[pg, :, sl][..., None]).half())


@pytest.mark.gpu
def test_pages_that_are_none(gpu_lib):
    """Pages below 0 and beyond the cache's, lengths beyond the table, starts
    beyond the rows: not written, read as zeros, nothing else touched."""
    D, H, page = 64, 2, 16
    table = torch.tensor([[0, -1, 1 << 30, 3], [2, 4, -7, 1]], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, 64, 1000], dtype=torch.int32, device=DEV)
    lens = torch.tensor([64, 1000], dtype=torch.int32, device=DEV)  # the second's count as 64
    k, v = (torch.randn(96, H, D).half().to(DEV) for _ in range(2))
    cache = w4.kv_cache(4, H, page, D, S8, DEV)
    w4.cache_write(cache, k, v, table, starts, lens)
    got = w4.cache_read(cache, table, starts, lens, 96, torch.float16)
    c, s = kv.quantised(k.cpu(), S8)
    ref = (c.float() * s[..., None]).half()
    ref[16:48] = 0  # no page
    # rows 64..95 are positions 32..63: pages -7 (none) and 1
    ref[64:80] = 0
    assert _same(got[0], ref)
    assert float(cache.k_scales[2].abs().sum()) == 0  # a page whose positions have no row


@pytest.mark.gpu
def test_replayed_with_other_lengths(gpu_lib):
    """A captured write and read follow what the batch's arrays hold."""
    D, H = 128, 2
    batch = kv.Batch([2, 1], [40, 90], 32)
    table, starts, lens = batch.plan(DEV)
    k, v = (torch.randn(3, H, D).bfloat16().to(DEV) for _ in range(2))
    cache = w4.kv_cache(batch.pages, H, 32, D, F8, DEV)
    out = [torch.zeros(3, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w4.cache_write(cache, k, v, table, starts, lens)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for t in cache:
        t.view(torch.uint8).zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.cache_write(cache, k, v, table, starts, lens)
        w4.cache_read(cache, table, starts, lens, 3, torch.bfloat16, *out)
    for step in range(3):
        lens.copy_(torch.tensor([10 + step, 80 - step]))
        k.copy_(torch.randn(3, H, D))
        graph.replay()
        batch.lens = [10 + step, 80 - step]
        want = _written(w4.KVCache(*(t.cpu() for t in cache)), batch, k.cpu(), v.cpu())
        assert all(_same(a, b) for a, b in zip(cache, want))
        c, s = kv.quantised(k.cpu(), F8)
        assert _same(out[0], (c.float() * s[..., None]).bfloat16())


# ------------------------------------------------------------------- refusals
P = 0x10000000


class Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("pages", ctypes.c_int64), ("heads", ctypes.c_int),
                ("page_size", ctypes.c_int), ("head_dim", ctypes.c_int), ("type", ctypes.c_int)]


class Of(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("table_width", ctypes.c_int64),
                ("starts", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("sequences", ctypes.c_int64)]


def _cache(**kw):
    d = dict(k=P, v=2 * P, k_scales=3 * P, v_scales=4 * P, pages=8, heads=2, page_size=16,
             head_dim=64, type=w4.S8)
    d.update(kw)
    return Cache(**d)


def _of(**kw):
    d = dict(table=5 * P, table_width=4, starts=6 * P, lens=7 * P, sequences=2)
    d.update(kw)
    return Of(**d)


def _write(cache=None, batch=None, k=8 * P, v=9 * P, type=w4.F16, rows=3, ks=128, vs=128):
    return w4.load().w4_cache_write(ctypes.byref(cache or _cache()), ctypes.byref(batch or _of()),
                                    k, v, type, rows, ks, vs, None)


def _read(cache=None, batch=None, k=8 * P, v=9 * P, type=w4.F16, rows=3):
    return w4.load().w4_cache_read(ctypes.byref(cache or _cache()), ctypes.byref(batch or _of()),
                                   k, v, type, rows, None)


INVALID, UNSUPPORTED = w4.ERR_INVALID_ARGUMENT, w4.ERR_UNSUPPORTED
SHARED = [
    (dict(cache=_cache(type=w4.F16)), INVALID), (dict(cache=_cache(type=7)), INVALID),
    (dict(type=w4.S8), INVALID), (dict(rows=-1), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(k=8 * P + 1), INVALID), (dict(v=9 * P + 1), INVALID),
    (dict(batch=_of(sequences=-1)), INVALID), (dict(batch=_of(table_width=-1)), INVALID),
    (dict(batch=_of(table=None)), INVALID), (dict(batch=_of(starts=None)), INVALID),
    (dict(batch=_of(lens=None)), INVALID), (dict(batch=_of(lens=7 * P + 2)), INVALID),
    (dict(cache=_cache(k=None)), INVALID), (dict(cache=_cache(v_scales=None)), INVALID),
    (dict(cache=_cache(k=P + 8)), INVALID), (dict(cache=_cache(k_scales=P + 4)), INVALID),
    (dict(cache=_cache(pages=-1)), INVALID), (dict(cache=_cache(heads=0)), INVALID),
    (dict(cache=_cache(page_size=0)), INVALID), (dict(cache=_cache(head_dim=-16)), INVALID),
    (dict(cache=_cache(page_size=8)), UNSUPPORTED), (dict(cache=_cache(page_size=48)), UNSUPPORTED),
    (dict(cache=_cache(head_dim=72)), UNSUPPORTED), (dict(cache=_cache(head_dim=272)), UNSUPPORTED),
    (dict(cache=_cache(heads=65536)), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(batch=_of(table_width=(1 << 26) + 1)), UNSUPPORTED),
]


@pytest.mark.parametrize("call", [_write, _read])
@pytest.mark.parametrize("kw,status", SHARED)
def test_refused(call, kw, status):
    kw = dict(kw)
    if call is _write and kw.get("rows", 0) > 1 << 30:
        kw.update(ks=1 << 40, vs=1 << 40)
    assert call(**kw) == status, w4.load().w4_last_error()
    assert w4.load().w4_last_error()


def test_refused_strides_and_overlap():
    assert _write(ks=127) == INVALID and _write(vs=0) == INVALID
    assert _read(v=8 * P + 256) == INVALID
    assert _read(k=P + 512) == INVALID and _read(v=4 * P + 64) == INVALID
    lib = w4.load()
    assert lib.w4_cache_write(None, ctypes.byref(_of()), P, P, w4.F16, 1, 128, 128, None) == INVALID
    assert lib.w4_cache_read(ctypes.byref(_cache()), None, P, P, w4.F16, 1, None) == INVALID


def test_nothing_to_do():
    """No rows or no sequences: nothing is looked at or launched."""
    for kw in (dict(rows=0), dict(batch=_of(sequences=0))):
        assert _write(k=None, v=None, **kw) == w4.OK
        assert _read(k=None, v=None, **kw) == w4.OK


def test_binding_refuses(monkeypatch):
    """What the binding sees of the tensors, before the library (CPU tensors stand
    for wrong ones)."""
    cache = w4.kv_cache(2, 1, 16, 64, device="cpu")
    x = torch.zeros(1, 1, 64, dtype=torch.float16)
    t, s, n = (torch.zeros(*z, dtype=torch.int32) for z in ((1, 1), (2,), (1,)))
    with pytest.raises(ValueError, match="CUDA tensor"):
        w4.cache_write(cache, x, x, t, s, n)
    with pytest.raises(ValueError, match="CUDA tensor"):
        w4.cache_read(cache, t, s, n, 1)
    with pytest.raises(ValueError, match="dtype"):
        w4.cache_read(cache, t, s, n, 1, torch.float32)
    with pytest.raises(ValueError, match="dtype"):
        w4.kv_cache(2, 1, 16, 64, torch.float16, "cpu")
    with pytest.raises(TypeError):
        w4.cache_write(cache, None, x, t, s, n)


@pytest.mark.gpu
def test_binding_checks_shapes(gpu_lib):
    D, H = 64, 2
    batch = kv.Batch([3], [3], 16)
    table, starts, lens = batch.plan(DEV)
    cache = w4.kv_cache(batch.pages, H, 16, D, S8, DEV)
    k = torch.zeros(3, H, D, dtype=torch.float16, device=DEV)
    bad = [
        (cache, k.float(), k, table, starts, lens), (cache, k, k.bfloat16(), table, starts, lens),
        (cache, k[:2], k, table, starts, lens), (cache, k[:, :1], k, table, starts, lens),
        (cache, k[..., :32], k, table, starts, lens), (cache, k.view(3, -1), k, table, starts, lens),
        (cache, k.transpose(0, 1).contiguous().transpose(0, 1), k, table, starts, lens),
        (cache, k[:1].expand(3, H, D), k, table, starts, lens),
        (cache, k, k, table.long(), starts, lens), (cache, k, k, table, starts[:1], lens),
        (cache, k, k, table, starts, torch.cat([lens, lens])), (cache, k, k, table[0], starts, lens),
        (cache, k, k, table.cpu(), starts, lens),
        (cache._replace(v=cache.v[:1]), k, k, table, starts, lens),
        (cache._replace(k=cache.k.float()), k, k, table, starts, lens),
        (cache._replace(k_scales=cache.k_scales.half()), k, k, table, starts, lens),
        (cache._replace(v_scales=cache.v_scales[..., :8]), k, k, table, starts, lens),
    ]
    for args in bad:
        with pytest.raises((ValueError, KeyError)):
            w4.cache_write(*args)
    with pytest.raises(ValueError):
        w4.cache_read(cache, table, starts, lens, 3, torch.float16, k_out=k[:2])
    with pytest.raises(ValueError):
        w4.cache_read(cache, table, starts, lens, 3, torch.bfloat16, v_out=k)
    with pytest.raises(w4.W4Error):
        w4.cache_read(cache, table, starts, lens, 3, torch.float16, k_out=k, v_out=k)


@pytest.mark.gpu
def test_another_stream(gpu_lib):
    """Calls go to the current stream."""
    batch = kv.Batch([50], [50], 16)
    k, v = _rows(50, 2, 64, torch.float16)
    cache = w4.kv_cache(batch.pages, 2, 16, 64, S8, DEV)
    want = _written(w4.KVCache(*(t.cpu() for t in cache)), batch, k, v)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        kd, vd, plan = k.to(DEV), v.to(DEV), batch.plan(DEV)
        torch.cuda._sleep(2000000)
        w4.cache_write(cache, kd, vd, *plan)
    side.synchronize()
    assert all(_same(a, b) for a, b in zip(cache, want))


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [S8, F8])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_what_the_cache_holds(gpu_lib, dt, codes):
    """Of every 16-bit value, alone and beside others: codes that are numbers, scales
    that are 0 (codes 0), 2^-100 at least, or NaN (codes 0)."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dt)
    g = torch.Generator().manual_seed(0)
    alone = torch.zeros(65536, 1, 16, dtype=dt)
    alone[:, 0, 5] = x
    mixed = x[torch.randperm(65536, generator=g)].view(-1, 1, 16)
    near = x.view(-1, 1, 16)  # values of one size
    rows = torch.cat([alone, mixed, near])
    T = rows.shape[0]
    cache = w4.kv_cache(-(-T // 64), 1, 64, 16, codes, DEV)
    table = torch.arange(cache.k.shape[0], dtype=torch.int32, device=DEV)[None].contiguous()
    starts, lens = (torch.tensor(n, dtype=torch.int32, device=DEV) for n in ([0, T], [T]))
    w4.cache_write(cache, rows.to(DEV), rows.flip(0).contiguous().to(DEV), table, starts, lens)
    for c, s in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
        c, s = c.float().view(-1, 16)[:T], s.view(-1)[:T]
        assert bool(torch.isfinite(c).all())
        assert bool((s.isnan() | (s == 0) | (s >= 2.0**-100)).all())
        assert float(c[s.isnan() | (s == 0)].abs().sum()) == 0
        assert float(c.abs().max()) == kv.TOP[codes] and not bool(torch.isinf(s).any())
