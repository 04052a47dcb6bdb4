"""The root-mean-square norm (w4_rmsnorm): 16-bit outputs within a derived
bound of the definition in 64 bits, 8-bit codes bit for bit, scales within a
derived bound, and the refusals (CPU).

Bounds.  u = 2^-24.  h is one fp32 rounding of x + r.  The sum of squares is
a sum of K positive terms in chains of at most ceil(K / 32) additions (a row
is summed by at least one warp) and ten more to join them, so its relative
error is at most (K / 32 + 14) u, of which the square root halves; the
division by K, eps, the reciprocal root (2 ulp) and the two products add less
than 8 u.  y is then off by at most eps_y |y| with
eps_y = (K / 64 + 16) u, plus half a unit of its output type.  The scale has
the same relative error.  Codes are single roundings of fp32 operations, so
they are compared bit for bit with numpy's.
"""
import ctypes

import numpy as np
import pytest
import torch

import int4_weight_mixed_gb300 as w4
from parity import ulp

DEV = "cuda:0"
TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
FMT = {torch.float16: "f16", torch.bfloat16: "bf16"}


def _inputs(M, K, dt, residual=True, weight=True, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed * 7919 + M * 131 + K)
    x = (torch.randn(M, K, generator=g) * std).to(dt)
    r = (torch.randn(M, K, generator=g) * 2 * std).to(dt) if residual else None
    w = (torch.rand(K, generator=g) * 1.6 + 0.2).to(dt) if weight else None
    return x, r, w


def _np(t):
    return None if t is None else t.float().numpy()


def _ref(x, r, w, eps):
    """(h, y) of the definition in 64 bits."""
    h = _np(x).astype(np.float64) + (0.0 if r is None else _np(r).astype(np.float64))
    rstd = 1.0 / np.sqrt((h * h).sum(1, keepdims=True) / h.shape[1] + eps)
    return h, h * rstd * (1.0 if w is None else _np(w).astype(np.float64))


def _codes(x, r, w, act):
    """Codes and A of the definition, every step in fp32 (numpy)."""
    h = _np(x) if r is None else _np(x) + _np(r)
    hw = h if w is None else h * _np(w)
    A = np.abs(hw).max(1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        up = np.where(A < np.float32(2.0**-100), np.float32(2.0**100), np.float32(1))
        q = np.where(A > 0, (hw * up) * (np.float32(TOP[act]) * (np.float32(1) / (A * up))), np.float32(0))
    if act == torch.int8:
        return np.rint(q).astype(np.int8), A
    return torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), A


def _eps_y(K):
    return (K / 64 + 16) * 2.0**-24


def _check16(got, ref, dt, K, what=""):
    got = got.float().cpu().numpy().astype(np.float64)
    bound = 0.5 * ulp(np.abs(ref) * (1 + _eps_y(K)), FMT[dt]) + _eps_y(K) * np.abs(ref)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], ref[bad][:4])


def _check8(codes, scales, x, r, w, act, eps, what=""):
    ref, _ = _codes(x, r, w, act)
    got = codes.cpu().view(torch.uint8).numpy().view(ref.dtype)
    assert np.array_equal(got, ref), (what, int((got != ref).sum()))
    _, y = _ref(x, r, w, eps)
    s = np.abs(y).max(1) / TOP[act]
    err = np.abs(scales.cpu().numpy().astype(np.float64) - s)
    assert (err <= _eps_y(x.shape[1]) * s + 2.0**-149).all(), (what, (err / s).max())


def _all(x, r, w, eps=1e-5, what=""):
    """Every output type of one input, against the definition."""
    K = x.shape[1]
    d = [None if t is None else t.to(DEV) for t in (x, w, r)]
    h = None
    y = w4.rmsnorm(d[0], d[1], eps, residual=d[2])
    if r is not None:
        y, h = y
        assert torch.equal(h.cpu(), (x.float() + r.float()).to(x.dtype)), what
    _check16(y, _ref(x, r, w, eps)[1], x.dtype, K, what)
    for act in TOP:
        out = w4.rmsnorm_quant(d[0], d[1], eps, residual=d[2], act_dtype=act)
        assert out[0].dtype == act
        _check8(out[0], out[1], x, r, w, act, eps, what)
        if r is not None:
            assert torch.equal(out[2], h), what


SHAPES = [(1, 1), (1, 8), (3, 13), (9, 64), (5, 72), (70, 128), (33, 256), (7, 1000), (6, 1024),
          (5, 1111), (3, 2048), (4, 2056), (1, 4096), (17, 8192), (2, 8200), (2, 16384),
          (3, 21760), (2, 32768), (2, 40000), (1, 65544), (1, 131071)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M,K", SHAPES)
def test_norm_matches_the_definition(gpu_lib, M, K, dt):
    x, r, w = _inputs(M, K, dt)
    _all(x, r, w, what=(M, K))
    _all(x, None, w, what=(M, K, "no residual"))
    _all(x, r, None, eps=1e-6, what=(M, K, "no weight"))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("K", [9, 10, 15, 17, 23, 255, 257, 1111, 2049, 4100, 8191, 16385, 20001])
def test_norm_rows_start_and_end_anywhere(gpu_lib, K, dt):
    """Rows whose first and last values lie anywhere between two 16-byte
    boundaries, several blocks of them a CTA: as the definition, and the same
    bits wherever in the array a row stands."""
    x, r, w = _inputs(min(700, 3_000_000 // K), K, dt, seed=5)
    _all(x, r, w, what=K)
    x, r, w = (t.to(DEV) for t in (x, r, w))
    x[8:16] = x[:8]
    r[8:16] = r[:8]
    x[19:27] = x[:8]
    r[19:27] = r[:8]
    for residual in (None, r):
        for out in (w4.rmsnorm(x, w, residual=residual),
                    w4.rmsnorm_quant(x, w, residual=residual),
                    w4.rmsnorm_quant(x, w, residual=residual, act_dtype=torch.float8_e4m3fn)):
            for t in out if isinstance(out, tuple) else (out,):
                t = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
                assert torch.equal(t[:8], t[8:16]) and torch.equal(t[:8], t[19:27])


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [(2000, 128), (3000, 520), (1500, 4096), (700, 8192)])
def test_norm_many_rows(gpu_lib, M, K):
    x, r, w = _inputs(M, K, torch.float16, seed=3)
    _all(x, r, w)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("K", [1024, 8192, 40000])
def test_norm_unaligned_arrays_give_the_same_values(gpu_lib, K, dt):
    """Arrays one element off a 16-byte boundary: the same outputs."""
    M = 3
    x, r, w = _inputs(M, K, dt, seed=1)

    def off(t):
        flat = torch.empty(t.numel() + 8, dtype=t.dtype, device=DEV)
        v = flat[1:1 + t.numel()].view(t.shape)
        v.copy_(t)
        return v

    for cx, cr, cw in ((off, off, off), (torch.Tensor.cuda, torch.Tensor.cuda, off),
                       (torch.Tensor.cuda, off, torch.Tensor.cuda)):
        q, s, h = w4.rmsnorm_quant(cx(x), cw(w), 1e-5, residual=cr(r))
        _check8(q, s, x, r, w, torch.int8, 1e-5)
        assert torch.equal(h.cpu(), (x.float() + r.float()).to(dt))
    y, _ = w4.rmsnorm(x.cuda(), w.cuda(), 1e-5, residual=r.cuda(), out=off(x))
    _check16(y, _ref(x, r, w, 1e-5)[1], dt, K)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [64, 1111, 4096, 21760, 40000])
def test_norm_in_place(gpu_lib, K):
    """residual_out may be the residual and a 16-bit output x, or the other
    way round: the same values as with arrays of their own."""
    x, r, w = (t.to(DEV) for t in _inputs(37, K, torch.float16, seed=2))
    y0, h0 = w4.rmsnorm(x, w, 1e-5, residual=r)
    a, b = x.clone(), r.clone()
    y, h = w4.rmsnorm(a, w, 1e-5, residual=b, out=a, residual_out=b)
    assert torch.equal(y, y0) and torch.equal(h, h0) and y is a and h is b
    a, b = x.clone(), r.clone()
    y, h = w4.rmsnorm(a, w, 1e-5, residual=b, out=b, residual_out=a)
    assert torch.equal(y, y0) and torch.equal(h, h0)
    q0, s0, _ = w4.rmsnorm_quant(x, w, 1e-5, residual=r)
    b = r.clone()
    q, s, h = w4.rmsnorm_quant(x, w, 1e-5, residual=b, residual_out=b)
    assert torch.equal(q, q0) and torch.equal(s, s0) and torch.equal(b, h0)
    y1, h1 = w4.rmsnorm(x, w, 1e-5, residual=x)  # x + x
    assert torch.equal(h1, (2 * x.float()).half())
    assert torch.equal(y1, w4.rmsnorm((2 * x).contiguous(), w, 1e-5))


@pytest.mark.gpu
@pytest.mark.parametrize("K", [96, 1111, 8192, 40000])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_norm_special_rows(gpu_lib, K, dt):
    """Rows of zeros, of tiny values, with one infinity or NaN: their own
    results as documented, and no effect on the rows beside them."""
    M = 9
    x, _, w = _inputs(M, K, dt, seed=4)
    x[1] = 0
    x[3] = 0
    x[3, K // 2] = 2.0**-20          # one subnormal (fp16) or small value
    x[5, K - 1] = float("inf")
    x[6, 0] = float("nan")
    x[7] = torch.finfo(dt).tiny if dt == torch.bfloat16 else 2.0**-24
    good = [0, 1, 2, 3, 4, 7, 8]
    xd, wd = x.to(DEV), w.to(DEV)
    y = w4.rmsnorm(xd, wd, 1e-5)
    _check16(y[good], _ref(x[good], None, w, 1e-5)[1], dt, K)
    # the formula in fp32: an infinity makes rstd 0, so 0 beside inf * 0
    assert torch.isnan(y[5, K - 1]) and bool((y[5, :K - 1] == 0).all())
    assert bool(torch.isnan(y[6]).all())
    for act in TOP:
        q, s = w4.rmsnorm_quant(xd, wd, 1e-5, act_dtype=act)
        _check8(q[good], s[good], x[good], None, w, act, 1e-5)
        assert bool(torch.isnan(s[5:7]).all())
        assert not q.view(torch.uint8)[[1, 5, 6]].any() and float(s[1]) == 0.0


@pytest.mark.gpu
def test_norm_sum_beyond_the_fp32_range(gpu_lib):
    """bf16 values whose squares pass the fp32 range: 16-bit outputs are
    those of an infinite sum (0), 8-bit rows are marked by a NaN scale."""
    x = torch.full((2, 512), 1.0, dtype=torch.bfloat16)
    x[1] = 2.0**80
    y = w4.rmsnorm(x.to(DEV), None, 1e-5)
    assert bool((y[1] == 0).all()) and bool((y[0] == 1).all())
    q, s = w4.rmsnorm_quant(x.to(DEV), None, 1e-5)
    assert bool(torch.isnan(s[1])) and not q[1].any() and bool((q[0] == 127).all())


@pytest.mark.gpu
def test_norm_empty_and_shapes(gpu_lib):
    for shape in ((0, 64), (3, 0), (0, 0)):
        x = torch.empty(shape, dtype=torch.float16, device=DEV)
        assert w4.rmsnorm(x).shape == shape
        q, s = w4.rmsnorm_quant(x)
        assert q.shape == shape and s.shape == shape[:1] and not s.any()
    x = torch.randn(2, 3, 4, 64, device=DEV).half()  # heads: the last dimension is normed
    w = torch.rand(64, device=DEV).half()
    y = w4.rmsnorm(x, w)
    assert y.shape == x.shape and torch.equal(y.view(-1, 64), w4.rmsnorm(x.view(-1, 64), w))
    q, s = w4.rmsnorm_quant(x, w)
    assert s.shape == (2, 3, 4)


@pytest.mark.gpu
def test_norm_is_deterministic_and_rows_stand_alone(gpu_lib):
    """The same row gives the same bits whatever M, and from call to call."""
    for K in (200, 1111, 8192, 21760):
        x, r, w = (t.to(DEV) for t in _inputs(300, K, torch.bfloat16, seed=5))
        y, h = w4.rmsnorm(x, w, 1e-5, residual=r)
        y2, _ = w4.rmsnorm(x, w, 1e-5, residual=r)
        assert torch.equal(y, y2)
        q, s, _ = w4.rmsnorm_quant(x, w, 1e-5, residual=r)
        for m in (0, 7, 299):
            ym, hm = w4.rmsnorm(x[m:m + 1], w, 1e-5, residual=r[m:m + 1])
            qm, sm, _ = w4.rmsnorm_quant(x[m:m + 1], w, 1e-5, residual=r[m:m + 1])
            assert torch.equal(ym[0], y[m]) and torch.equal(hm[0], h[m])
            assert torch.equal(qm[0], q[m]) and torch.equal(sm[0], s[m])


@pytest.mark.gpu
def test_norm_on_another_stream_and_in_a_graph(gpu_lib):
    x, r, w = (t.to(DEV) for t in _inputs(64, 4096, torch.float16, seed=6))
    y0, h0 = w4.rmsnorm(x, w, 1e-5, residual=r)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        # the input of the second norm is made on this stream by the first
        a, h1 = w4.rmsnorm(x, w, 1e-5, residual=r)
        b = w4.rmsnorm(a, w, 1e-5)
    st.synchronize()
    assert torch.equal(a, y0) and torch.equal(h1, h0)
    assert torch.equal(b, w4.rmsnorm(y0, w, 1e-5))
    out, ro = torch.empty_like(x), torch.empty_like(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.rmsnorm(x, w, 1e-5, residual=r, out=out, residual_out=ro)
        w4.rmsnorm(out, w, 1e-5, residual=ro, out=out, residual_out=ro)
    g.replay()
    torch.cuda.synchronize()
    y1, h1 = w4.rmsnorm(y0, w, 1e-5, residual=h0)
    assert torch.equal(out, y1) and torch.equal(ro, h1)


# ------------------------------------------------------------- refusals (CPU)
P = 0x10000  # pointers that are checked and never read


@pytest.fixture(scope="module")
def lib():
    w4.build()
    return w4.load()


def _call(lib, x=P, xt=0, M=4, K=64, r=0, w=0, eps=1e-5, h=0, y=0x20000, yt=0, s=0):
    return lib.w4_rmsnorm(x, xt, M, K, r, w, ctypes.c_float(eps), h, y, yt, s, None)


BAD = w4.ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), BAD), (dict(K=-1), BAD), (dict(xt=2), BAD), (dict(xt=9), BAD),
    (dict(yt=1), BAD), (dict(yt=3), BAD),                       # bf16 / int32 from fp16
    (dict(eps=-1e-6), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
    (dict(h=0x40000), BAD),                                     # no residual to add
    (dict(s=0x50000), BAD),                                     # 16 bits take no scales
    (dict(yt=2), BAD), (dict(yt=4), BAD),                       # 8 bits need them
    (dict(x=0), BAD), (dict(y=0), BAD),
    (dict(x=P + 1), BAD), (dict(w=P + 0x8001), BAD), (dict(y=0x20001), BAD),
    (dict(r=0x30001), BAD), (dict(r=0x30000, h=0x40001), BAD),
    (dict(yt=2, s=0x50002), BAD),
    # overlaps: shifted by less than the arrays are long, outputs on one another
    (dict(y=P + 64), BAD), (dict(r=0x30000, h=P + 64), BAD), (dict(r=0x30000, h=0x30040), BAD),
    (dict(r=0x30000, h=0x20000), BAD), (dict(yt=2, s=0x50000, y=P), BAD),
    (dict(w=0x20010), BAD), (dict(yt=2, s=0x20010), BAD), (dict(yt=2, s=P), BAD),
    (dict(r=0x30000, h=0x40000, yt=2, s=0x40000), BAD),
    (dict(M=2**31, K=1, y=2**40), w4.ERR_UNSUPPORTED),
    (dict(M=1, K=2**31, y=2**40), w4.ERR_UNSUPPORTED),
    (dict(M=0), w4.OK), (dict(M=0, x=0, y=0), w4.OK),
])
def test_norm_refusals(lib, kw, status):
    assert _call(lib, **kw) == status
    if status != w4.OK:
        assert w4.load().w4_last_error()


def test_norm_binding_refusals():
    x = torch.zeros(2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        w4.rmsnorm(x)
    with pytest.raises(ValueError, match="act_dtype"):
        w4.rmsnorm_quant(x, act_dtype=torch.uint8)
    with pytest.raises(ValueError, match="out must"):
        w4.rmsnorm(x, out=torch.zeros(2, 63, dtype=torch.float16))
    with pytest.raises(ValueError, match="scales must"):
        w4.rmsnorm_quant(x, scales=torch.zeros(3))


@pytest.mark.gpu
def test_norm_binding_refusals_on_the_device(gpu_lib):
    x = torch.zeros(4, 64, dtype=torch.float16, device=DEV)
    for kw in (dict(weight=torch.zeros(63, dtype=torch.float16, device=DEV)),
               dict(weight=torch.zeros(64, device=DEV)),
               dict(residual=torch.zeros(4, 63, dtype=torch.float16, device=DEV)),
               dict(residual=torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)),
               dict(residual=torch.zeros(4, 128, dtype=torch.float16, device=DEV)[:, ::2])):
        with pytest.raises(ValueError):
            w4.rmsnorm(x, **kw)
    with pytest.raises(ValueError, match="contiguous"):
        w4.rmsnorm(x.t())
    with pytest.raises(ValueError, match="fp16 or bf16"):
        w4.rmsnorm(x.float())
