"""The product's epilogue (w4_gemm_epilogue, w4_gemm_dynamic_epilogue):
activation, gate and residual on every schedule, against 64 bits.

Inputs are chosen so that the product itself is exact in fp32 whatever the
order of its sums (integer activations, power-of-two scales, sums below
2^24; W4A8 is exact by construction), so the bounds below are those of the
epilogue alone.  u = 2^-24; v has at most four roundings, of values no larger
than |product| + |bias|:

  dv       <= 4 u (|product| + |bias|)
  relu     <= dv
  silu     <= 1.1 dv + ((3 + 1.2 |v|) 2^-23 + 4 u) |silu(v)|   (e^-v: 2 + 1.173 |v| ulp)
  gelu     <= 1.13 dv + (2 v^2 + 12) u |gelu(v)| + 2^-126      (erfc: 4 ulp; its argument's
              rounding moves erfc by at most 2 z^2 + 1 of it, z^2 = v^2 / 2)
  gelu_tanh<= 1.13 dv + ((3 + 1.2 |t|) 2^-23 + 6 u |t| + 4 u) |.| , t the logistic's argument

(1.1 and 1.13 bound the slopes).  A gated product multiplies two such values,
a residual adds one more rounding, and the output rounds once more.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import int4_weight_mixed_gb300 as w4
import oracle
import w4synth
from parity import ulp

DEV = "cuda:0"
U = 2.0**-24
ACTS = {"none": w4.ACT_NONE, "relu": w4.ACT_RELU, "silu": w4.ACT_SILU, "gelu": w4.ACT_GELU,
        "gelu_tanh": w4.ACT_GELU_TANH}
SCHEDULES = ["simt", "tc16_sk", "tc32_sk", "tc64_sk", "tc128_sk", "tc128_dp", "tc256_sk",
             "tc256_dp", "tc128x2_sk", "tc128x2_dp", "tc128x2_kp", "tc256_kp", "tc256p_sk",
             "tc256p_dp", "tc128p_sk", "dk8_sk", "dk16_sk", "ds8_sk", "ds16_sk", "ds32_sk",
             "gv8_cl", "gv16_cl", "gv32_cl"]
F8_SCHEDULES = ["simt", "tc16_sk", "tc64_sk", "tc128_sk", "tc256_sk", "tc256_dp", "tc256p_sk",
                "tc256p_dp", "tc128p_sk", "gv8_cl", "gv16_cl", "gv32_cl"]
ROWS = {"dk8_sk": 8, "dk16_sk": 16, "ds8_sk": 8, "ds16_sk": 16, "ds32_sk": 32, "gv8_cl": 8,
        "gv16_cl": 16, "gv32_cl": 32}


def sched(name):
    return -1 if name is None else w4.schedule_names().index(name)


def _erfc(x):
    return np.vectorize(math.erfc, otypes=[np.float64])(x)


def _act(v, dv, act):
    """(act(v), bound on the kernel's error) in 64 bits."""
    if act == "relu":
        return np.maximum(v, 0), dv
    if act == "silu":
        r = v / (1 + np.exp(-v))
        return r, 1.1 * dv + ((3 + 1.2 * np.abs(v)) * 2 * U + 4 * U) * np.abs(r)
    if act == "gelu":
        r = 0.5 * v * _erfc(-v / math.sqrt(2))
        return r, 1.13 * dv + (2 * v * v + 12) * U * np.abs(r) + 2.0**-126
    if act == "gelu_tanh":
        t = math.sqrt(8 / math.pi) * (v + 0.044715 * v**3)
        r = v / (1 + np.exp(-t))
        return r, 1.13 * dv + ((3 + 1.2 * np.abs(t)) * 2 * U + (6 * np.abs(t) + 4) * U) * np.abs(r)
    return v, dv


def reference(prod, bias, act, gated, residual):
    """(out, bound before the output's rounding) of the definition."""
    b = 0.0 if bias is None else bias.double().numpy()
    v = prod + b
    dv = 4 * U * (np.abs(prod) + np.abs(b))
    with np.errstate(over="ignore"):
        if gated:
            (r, e), up, dup = _act(v[:, 0::2], dv[:, 0::2], act), v[:, 1::2], dv[:, 1::2]
            r, e = r * up, e * np.abs(up) + (np.abs(r) + e) * dup + U * np.abs(r * up)
        else:
            r, e = _act(v, dv, act)
    if residual is not None:
        d = residual.double().numpy()
        r, e = r + d, e + U * (np.abs(r) + np.abs(d))
    return r, e


def check(got, ref, err, fmt, what):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= 0.5 * ulp(np.abs(ref) + err, fmt) + err)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], ref[bad][:4], err[bad][:4])


def gen(t, *shape, lo=-1.0, hi=1.0, dt=torch.float16):
    return (torch.rand(*shape, generator=t) * (hi - lo) + lo).to(dt)


class Case:
    """A product that is exact in fp32, its operands and its 64-bit value."""

    def __init__(self, mode, M, N, K, gs=-1, zeros=False, seed=0):
        g = torch.Generator().manual_seed(seed + 1000 * M + N + K)
        self.M, self.N, self.K, self.g = M, N, K, g
        words = torch.randint(-2**31, 2**31 - 1, (K // 8, N), generator=g, dtype=torch.int32)
        nib = ((words[:, None, :] >> torch.arange(0, 32, 4, dtype=torch.int32)[None, :, None]) & 15)
        q = nib.reshape(K, N).double().numpy()
        self.kw = dict(group_size=gs)
        G = 1 if gs == -1 else K // gs
        rep = K // G
        self.dt = torch.float16
        if mode in ("fp16", "bf16"):
            self.dt = torch.float16 if mode == "fp16" else torch.bfloat16
            a = torch.randint(-3, 4, (M, K), generator=g).to(self.dt)
            s = torch.exp2(torch.randint(-9, -6, (G, N), generator=g).float()).to(self.dt)
            sv = np.repeat(s.double().numpy(), rep, 0)
            self.kw["scales"] = s
            if zeros:
                z = torch.randint(7, 10, (G, N), generator=g)
                zs = (z.float() * s.float()).to(self.dt)  # exact
                self.kw["zeros"], self.wtype = zs, w4.UINT4
                w = q * sv - np.repeat(zs.double().numpy(), rep, 0)
            else:
                self.wtype, w = w4.UINT4B8, (q - 8) * sv
            self.prod = a.double().numpy() @ w
        else:
            self.wtype = w4.INT4
            v = np.where(q >= 8, q - 16, q)
            if mode == "int8":
                a = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8)
                if G > 1:
                    sg = torch.randint(1, 17, (G, N), generator=g, dtype=torch.int8)
                    self.kw["scales"] = sg
                    v = v * np.repeat(sg.double().numpy(), rep, 0)
                av, size = a.double().numpy(), 73 * 4.6 * math.sqrt(K) * (9.5 if G > 1 else 1)
            else:
                a = torch.randint(-8, 9, (M, K), generator=g).float().to(torch.float8_e4m3fn)
                av, size = a.float().double().numpy(), 5 * 4.6 * math.sqrt(K)
            st = torch.rand(M, generator=g) + 0.5
            sc = (torch.rand(N, generator=g) + 0.5) * (2 / size)
            self.kw.update(token_scales=st, channel_scales=sc)
            self.prod = (av @ v) * st.double().numpy()[:, None] * sc.double().numpy()
        self.a, self.words = a, words

    def fmt(self):
        return "bf16" if self.dt == torch.bfloat16 else "f16"

    def device(self):
        b = w4.prepack_B(self.words.to(DEV), self.wtype, w4.KN_SEQ, self.K, self.N)
        kw = {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in self.kw.items()}
        return self.a.to(DEV), b, kw

    def run(self, name, act, gated, bias=True, residual=True, what=""):
        n = self.N // 2 if gated else self.N
        bt = gen(self.g, self.N, dt=self.dt) if bias else None
        rt = gen(self.g, self.M, n, lo=-2, hi=2, dt=self.dt) if residual else None
        a, b, kw = self.device()
        out = w4.gemm(a, b, self.wtype, self.N, schedule=sched(name), act=ACTS[act], gated=gated,
                      bias=None if bt is None else bt.to(DEV),
                      residual=None if rt is None else rt.to(DEV), **kw)
        ref, err = reference(self.prod, bt, act, gated, rt)
        check(out, ref, err, self.fmt(), (what, name, act, gated))


FORMS = [("silu", True), ("gelu", False), ("gelu_tanh", True), ("none", False)]


@pytest.mark.gpu
@pytest.mark.parametrize("act,gated", FORMS)
@pytest.mark.parametrize("mode", ["fp16", "bf16"])
@pytest.mark.parametrize("name", SCHEDULES)
def test_w4a16_every_schedule(gpu_lib, name, mode, act, gated):
    M = min(ROWS.get(name, 41), 41) - 1
    Case(mode, M, 384, 1280, gs=128, zeros=act == "silu").run(name, act, gated)


@pytest.mark.gpu
@pytest.mark.parametrize("act,gated", FORMS)
@pytest.mark.parametrize("gs", [-1, 128])
@pytest.mark.parametrize("name", SCHEDULES)
def test_w4a8_every_schedule(gpu_lib, name, gs, act, gated):
    M = min(ROWS.get(name, 41), 41) - 1
    Case("int8", M, 384, 2048, gs=gs).run(name, act, gated)


@pytest.mark.gpu
@pytest.mark.parametrize("act,gated", FORMS)
@pytest.mark.parametrize("name", F8_SCHEDULES)
def test_fp8_every_schedule(gpu_lib, name, act, gated):
    M = min(ROWS.get(name, 41), 41) - 1
    Case("e4m3", M, 384, 2048).run(name, act, gated)


@pytest.mark.gpu
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
def test_every_combination(gpu_lib, act, gated, bias, residual):
    for mode, M in (("bf16", 3), ("int8", 40), ("e4m3", 300)):
        Case(mode, M, 256, 1024).run(None, act, gated, bias, residual)


# lengths from one token up, ragged rows and columns, tiles that end inside a
# pair of columns' neighbours, columns that only the CUDA-core schedule takes
RAGGED = [("bf16", 1, 8, 64, -1), ("fp16", 1, 2, 64, -1), ("bf16", 2, 42, 192, 64),
          ("fp16", 17, 42, 192, 64), ("int8", 5, 10, 128, -1), ("int8", 33, 200, 640, 128),
          ("e4m3", 7, 136, 384, -1), ("e4m3", 20, 14, 128, -1), ("bf16", 129, 1032, 576, 64),
          ("int8", 257, 1048, 1152, -1), ("fp16", 65, 392, 4096, 128), ("bf16", 31, 4096, 512, -1),
          ("int8", 700, 528, 2176, 128), ("e4m3", 513, 776, 1024, -1)]


@pytest.mark.gpu
@pytest.mark.parametrize("mode,M,N,K,gs", RAGGED)
def test_ragged_sizes(gpu_lib, mode, M, N, K, gs):
    c = Case(mode, M, N, K, gs=gs, seed=1)
    for act, gated in (("silu", True), ("gelu_tanh", False)):
        c.run(None, act, gated, what=(mode, M, N, K))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [5, 40])
def test_odd_columns_without_a_gate(gpu_lib, M):
    Case("fp16", M, 43, 256, gs=64).run(None, "gelu", False)
    Case("int8", M, 131, 256).run(None, "silu", False)


@pytest.mark.gpu
@pytest.mark.parametrize("name,mode,M,N,K", [
    ("gv8_cl", "bf16", 7, 136, 640), ("gv16_cl", "int8", 16, 1032, 1664), ("gv32_cl", "e4m3", 31, 256, 1408),
    ("ds8_sk", "fp16", 8, 136, 16384), ("ds32_sk", "int8", 32, 264, 21760),
    ("dk8_sk", "bf16", 8, 43 * 2, 1152), ("tc16_sk", "int8", 16, 128, 16384),
    ("tc256p_sk", "bf16", 300, 264, 4096), ("tc128p_sk", "int8", 130, 520, 8192),
    ("tc128x2_kp", "fp16", 130, 264, 4096), ("tc256_kp", "int8", 70, 136, 21760)])
@pytest.mark.parametrize("act,gated", [("silu", True), ("relu", False)])
def test_split_sums_and_clusters(gpu_lib, name, mode, M, N, K, act, gated):
    """Tiles whose K range is split over many CTAs, clusters of every size
    the shapes give (whose column ranges fall between a gate and its pair)."""
    Case(mode, M, N, K, seed=2).run(name, act, gated)


@pytest.mark.gpu
@pytest.mark.parametrize("name", SCHEDULES)
def test_zero_residual_keeps_the_product(gpu_lib, name):
    """The kernels with an epilogue of their own compute the same sums in
    the same order: adding zeros gives the plain product bit for bit."""
    M = min(ROWS.get(name, 300), 300)
    for e, mode in ((w4synth.gen_w4a16(M, 392, 1280, act_dtype=torch.bfloat16, wtype=w4.UINT4,
                                       layout=w4.KN_SEQ, group_size=128, zeros=True, seed=3), 16),
                    (w4synth.gen_w4a8(M, 384, 2048, group_size=-1, seed=4), 8)):
        b = w4.prepack_B(e["w"].to(DEV), e["wtype"], e["layout"], e["K"], e["N"])
        kw = dict(group_size=e["group_size"], schedule=sched(name))
        if mode == 16:
            kw.update(scales=e["s"].to(DEV), zeros=e["z"].to(DEV))
        else:
            kw.update(token_scales=e["s_tok"].to(DEV), channel_scales=e["s_ch"].to(DEV))
        plain = w4.gemm(e["a"].to(DEV), b, e["wtype"], e["N"], **kw)
        zeros = torch.zeros_like(plain)
        assert torch.equal(plain, w4.gemm(e["a"].to(DEV), b, e["wtype"], e["N"], residual=zeros,
                                          **kw))
        relu = w4.gemm(e["a"].to(DEV), b, e["wtype"], e["N"], act=w4.ACT_RELU, **kw)
        assert torch.equal(relu, plain.relu())


@pytest.mark.gpu
@pytest.mark.parametrize("name,mode,M,N,K,gs", [
    # every tile split: 2, 9, 33 and more contributors; the last tile ragged
    ("tc16_sk", "bf16", 16, 392, 4096, 128), ("tc64_sk", "bf16", 64, 136, 28672, 128),
    ("tc32_sk", "int8", 20, 256, 21760, -1), ("tc128_sk", "fp16", 77, 2056, 4096, 64),
    ("tc64_sk", "e4m3", 100, 1000, 8192, -1), ("tc256_sk", "int8", 300, 272, 8192, 128),
    # some tiles split, some whole; none split
    ("tc64_sk", "bf16", 64, 20000, 2048, 128), ("tc128_sk", "int8", 513, 5000, 1024, -1),
    ("tc16_sk", "bf16", 16, 19456, 1024, 128),
    # two weight tiles a CTA, K splits
    ("tc128x2_sk", "fp16", 130, 520, 4096, 128), ("tc256_kp", "e4m3", 260, 1032, 8192, -1),
    ("tc128x2_kp", "int8", 130, 520, 8192, -1),
    # CTA pairs: two contributors a tile and more, fewer; exact chunks in a unit
    ("tc256p_sk", "bf16", 512, 4096, 2048, 128), ("tc256p_sk", "int8", 300, 1000, 8192, -1),
    ("tc128p_sk", "int8", 100, 1040, 8192, 128), ("tc256p_sk", "e4m3", 200, 2056, 4096, -1),
    ("tc256p_sk", "int8", 1000, 8192, 1024, -1), ("tc128p_sk", "fp16", 300, 6000, 1024, 128),
    ("tc256p_sk", "int8", 300, 4864, 40960, -1)])
def test_split_tiles_keep_the_product(gpu_lib, name, mode, M, N, K, gs):
    """Tiles that several CTAs share are added in the order of the plain
    product's kernels, however many share one: the same bits."""
    g = torch.Generator(device=DEV).manual_seed(11)
    b = w4.prepack_B(torch.randint(-2**31, 2**31 - 1, (K // 8, N), generator=g, device=DEV,
                                   dtype=torch.int32), w4.INT4, w4.KN_SEQ, K, N)
    G = 1 if gs == -1 else K // gs
    kw = dict(group_size=gs, schedule=sched(name))
    a = torch.randn(M, K, generator=g, device=DEV)
    if mode in ("bf16", "fp16"):
        a = a.to(torch.bfloat16 if mode == "bf16" else torch.float16)
        kw["scales"] = ((torch.rand(G, N, generator=g, device=DEV) + 0.5) / 256).to(a.dtype)
    else:
        a = (a * 30).to(torch.float8_e4m3fn) if mode == "e4m3" else (a * 30).clamp(-127, 127).to(
            torch.int8)
        if G > 1:
            kw["scales"] = torch.randint(1, 17, (G, N), generator=g, device=DEV, dtype=torch.int8)
        kw["token_scales"] = (torch.rand(M, generator=g, device=DEV) + 0.5) / 4096
        kw["channel_scales"] = (torch.rand(N, generator=g, device=DEV) + 0.5) / 64
    plain = w4.gemm(a, b, w4.INT4, N, **kw)
    assert plain.isfinite().all()
    out = w4.gemm(a, b, w4.INT4, N, residual=torch.zeros_like(plain), **kw)
    assert torch.equal(plain, out)
    for _ in range(3):  # and call after call
        assert torch.equal(out, w4.gemm(a, b, w4.INT4, N, residual=torch.zeros_like(plain), **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("name", SCHEDULES)
@pytest.mark.parametrize("gated", [False, True])
def test_residual_in_place(gpu_lib, name, gated):
    M = min(ROWS.get(name, 290), 290)
    c = Case("bf16", M, 520, 1024, seed=5)
    a, b, kw = c.device()
    r = torch.randn(M, 260 if gated else 520, device=DEV).bfloat16()
    kw.update(act=w4.ACT_SILU, gated=gated, schedule=sched(name))
    ref = w4.gemm(a, b, c.wtype, c.N, residual=r, **kw)
    out = w4.gemm(a, b, c.wtype, c.N, residual=r, out=r, **kw)
    assert out is r and torch.equal(out, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 24, 300])
def test_interleaved_columns_are_gate_and_up(gpu_lib, M):
    """interleave_columns makes the gated product of two weights: act(gate)
    * up from the two weights' own raw sums."""
    N, K = 264, 1024
    g, u = (w4synth.gen_w4a8(M, N, K, group_size=128, seed=s) for s in (6, 7))
    a, st = g["a"].to(DEV), torch.full((M,), 2.0**-10, device=DEV)
    sc = [torch.full((N,), s, device=DEV) for s in (2.0**-6, 2.0**-7)]
    accs = [w4.gemm(a, w4.prepack_B(x["w"].to(DEV), w4.INT4, x["layout"], K, N), w4.INT4, N,
                    scales=x["sg"].to(DEV), group_size=128, out_dtype=torch.int32)
            for x in (g, u)]
    for layout, dim in ((w4.KN_SEQ, 1), (w4.NK_SEQ, 0), (w4.NK_EXLLAMA, 0)):
        words = [w4.unprepack_B(w4.prepack_B(x["w"].to(DEV), w4.INT4, x["layout"], K, N), w4.INT4,
                                layout, K, N) for x in (g, u)]
        w = w4.interleave_columns(*words, dim=dim)
        b = w4.prepack_B(w, w4.INT4, layout, K, 2 * N)
        sg = w4.interleave_columns(g["sg"].to(DEV), u["sg"].to(DEV))
        out = w4.gemm(a, b, w4.INT4, 2 * N, scales=sg, group_size=128, token_scales=st,
                      channel_scales=w4.interleave_columns(*sc), act=w4.ACT_SILU, gated=True)
        v = [acc.double().cpu().numpy() * 2.0**-10 * float(s[0]) for acc, s in zip(accs, sc)]
        prod = np.stack(v, 2).reshape(M, 2 * N)
        ref, err = reference(prod, None, "silu", True, None)
        check(out, ref, err, "f16", layout)


@pytest.mark.gpu
def test_activations_far_out(gpu_lib):
    """Values far beyond the bends, up to the edge of fp32: no NaN from an
    infinite exponential or cube, the limits of the formulas."""
    N, K = 128, 128
    a = torch.ones(4, K, dtype=torch.int8, device=DEV)
    words = torch.full((K // 8, N), 0x11111111, dtype=torch.int32, device=DEV)  # acc = 128
    b = w4.prepack_B(words, w4.INT4, w4.KN_SEQ, K, N)
    st = torch.tensor([2.0**-7, -2.0**-7, 2.0**-7, -2.0**-7], device=DEV)
    mags = torch.logspace(-30, 38, N, dtype=torch.float64).float().to(DEV)
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        out = w4.gemm(a, b, w4.INT4, N, token_scales=st, channel_scales=mags, act=ACTS[act])
        v = st.sign()[:, None].double().cpu().numpy() * mags.double().cpu().numpy()
        with np.errstate(over="ignore", invalid="ignore"):
            ref = np.where(v > 60, v, np.where(v < -60, 0.0, _act(np.clip(v, -60, 60), 0 * v, act)[0]))
        got = out.double().cpu().numpy()
        assert not np.isnan(got).any(), act
        big = ref > 65520
        assert np.isinf(got[big]).all()
        assert (np.abs(got - ref)[~big] <= 2.0**-10 * np.abs(ref[~big]) + 2.0**-24).all(), act


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 24, 40, 300])
@pytest.mark.parametrize("gated", [False, True])
def test_arrays_off_a_16_byte_boundary(gpu_lib, M, gated):
    """out, residual, bias and channel scales aligned to their elements only:
    the same values by the default rule, a refusal by a tensor-core schedule."""
    N, K = 256, 512
    n = N // 2 if gated else N

    def off(shape, dt, by=1):
        flat = torch.empty(math.prod(shape) + 8, dtype=dt, device=DEV)
        return flat[by:by + math.prod(shape)].view(shape)

    for mode in ("bf16", "int8", "e4m3"):
        c = Case(mode, M, N, K, seed=13)
        a, b, kw = c.device()
        bias, r = gen(c.g, N, dt=c.dt), gen(c.g, M, n, dt=c.dt)
        ref, err = reference(c.prod, bias, "silu", gated, r)
        names = ["out", "residual", "bias"] + (["channel_scales"] if mode != "bf16" else [])
        for name in names:
            k2 = dict(kw, bias=bias.to(DEV), residual=r.to(DEV), out=torch.empty(M, n, dtype=c.dt,
                                                                                   device=DEV))
            t = off(tuple(k2[name].shape), k2[name].dtype)
            t.copy_(k2[name])
            k2[name] = t
            out = w4.gemm(a, b, c.wtype, N, act=w4.ACT_SILU, gated=gated, **k2)
            check(out, ref, err, c.fmt(), (mode, name))
            with pytest.raises(w4.W4Error) as e:
                w4.gemm(a, b, c.wtype, N, act=w4.ACT_SILU, gated=gated, schedule=sched("tc64_sk"),
                        **k2)
            assert e.value.status == w4.ERR_UNSUPPORTED
            if mode == "int8":
                x = torch.randn(M, K, device=DEV).half()
                k3 = {k: v for k, v in k2.items() if k not in ("token_scales", "group_size")}
                k4 = dict(k3)
                k4[name] = k4[name].clone() if name != "out" else torch.empty_like(t)
                two = w4.gemm_dynamic(x, b, c.wtype, N, act=w4.ACT_SILU, gated=gated, **k4)
                one = w4.gemm_dynamic(x, b, c.wtype, N, act=w4.ACT_SILU, gated=gated, **k3)
                assert torch.equal(one, two)


@pytest.mark.gpu
def test_nan_and_infinite_activations_stay_in_their_rows(gpu_lib):
    c = Case("bf16", 20, 256, 1024, seed=8)
    a, b, kw = c.device()
    r = torch.randn(20, 256, device=DEV).bfloat16()
    for act in ACTS.values():
        ref = w4.gemm(a, b, c.wtype, c.N, act=act, residual=r, **kw)
        bad = a.clone()
        bad[3, 5], bad[7, 9] = float("nan"), float("inf")
        out = w4.gemm(bad, b, c.wtype, c.N, act=act, residual=r, **kw)
        assert bool(torch.isnan(out[3]).all())
        keep = [i for i in range(20) if i not in (3, 7)]
        assert torch.equal(out[keep], ref[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 24, 300])
@pytest.mark.parametrize("act_dtype", [torch.int8, torch.float8_e4m3fn])
def test_dynamic_equals_two_steps(gpu_lib, M, act_dtype):
    N, K = 512, 1024
    x = w4synth.gen_act16(M, K, torch.float16, seed=9).to(DEV)
    e = w4synth.gen_w4a8(M, N, K, group_size=-1, seed=10)
    b = w4.prepack_B(e["w"].to(DEV), e["wtype"], e["layout"], K, N)
    quant = w4.quantize_per_token if act_dtype == torch.int8 else w4.quantize_per_token_fp8
    q, s = quant(x)
    bias = torch.randn(N, device=DEV).half()
    for gated in (False, True):
        r = torch.randn(M, N // 2 if gated else N, device=DEV).half()
        kw = dict(channel_scales=e["s_ch"].to(DEV), bias=bias, act=w4.ACT_GELU_TANH, gated=gated,
                  residual=r)
        two = w4.gemm(q, b, e["wtype"], N, token_scales=s, **kw)
        assert torch.equal(two, w4.gemm_dynamic(x, b, e["wtype"], N, act_dtype=act_dtype, **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,gs,mode", [(1024, 8192, 21760, -1, "int8"),
                                           (600, 8192, 21760, 128, "int8"),
                                           (16, 28672, 4096, 128, "bf16"),
                                           (4096, 8192, 1024, -1, "e4m3")])
def test_large_products_sampled(gpu_lib, M, N, K, gs, mode):
    """The sizes at which the schedules are chosen for speed: rows and
    columns spread over all tiles, against 64-bit sums of the same values."""
    g = torch.Generator(device=DEV).manual_seed(11)
    words = torch.randint(-2**31, 2**31 - 1, (K // 8, N), generator=g, device=DEV, dtype=torch.int32)
    G = 1 if gs == -1 else K // gs
    kw = dict(group_size=gs)
    if mode == "bf16":
        a = torch.randint(-3, 4, (M, K), generator=g, device=DEV).bfloat16()
        kw["scales"] = torch.exp2(torch.randint(-9, -6, (G, N), generator=g, device=DEV).float()).bfloat16()
        wt, dt = w4.UINT4B8, torch.bfloat16
    else:
        wt, dt = w4.INT4, torch.float16
        if mode == "int8":
            a = torch.randint(-127, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
        else:
            a = torch.randint(-8, 9, (M, K), generator=g, device=DEV).float().to(torch.float8_e4m3fn)
        if G > 1:
            kw["scales"] = torch.randint(1, 17, (G, N), generator=g, device=DEV, dtype=torch.int8)
        kw["token_scales"] = torch.rand(M, generator=g, device=DEV) + 0.5
        kw["channel_scales"] = (torch.rand(N, generator=g, device=DEV) + 0.5) * (
            2.0**-16 if mode == "int8" else 2.0**-11)
    b = w4.prepack_B(words, wt, w4.KN_SEQ, K, N)
    rows = torch.unique(torch.cat([torch.arange(0, M, max(1, M // 37)), torch.tensor([M - 1])]))
    cols = torch.unique(torch.cat([torch.arange(0, N, 514), torch.arange(1, N, 514),
                                   torch.tensor([N - 2, N - 1])]))
    w = words[:, cols.to(DEV)]
    nib = (w[:, None, :] >> torch.arange(0, 32, 4, device=DEV, dtype=torch.int32)[None, :, None]) & 15
    nib = nib.reshape(K, -1).double()
    nib = nib - 8 if wt == w4.UINT4B8 else torch.where(nib >= 8, nib - 16, nib)
    if "scales" in kw:
        nib = nib * kw["scales"][:, cols.to(DEV)].double().repeat_interleave(K // G, 0)
    prod = a[rows.to(DEV)].to(torch.float64) @ nib
    if mode != "bf16":
        prod = prod * kw["token_scales"][rows.to(DEV)].double()[:, None] * \
            kw["channel_scales"][cols.to(DEV)].double()
    prod = prod.cpu().numpy()
    assert cols.numel() % 2 == 0 and bool((cols[0::2] + 1 == cols[1::2]).all())
    for gated in (False, True):
        n = N // 2 if gated else N
        r = torch.randn(M, n, generator=g, device=DEV).to(dt)
        out = w4.gemm(a, b, wt, N, act=w4.ACT_SILU, gated=gated, residual=r, **kw)
        at = cols[0::2] // 2 if gated else cols
        pick = lambda t: t[rows.to(DEV)][:, at.to(DEV)].cpu()
        ref, err = reference(prod, None, "silu", gated, pick(r))
        check(pick(out), ref, err, "bf16" if mode == "bf16" else "f16", (M, N, K, gated))


@pytest.mark.gpu
def test_empty_and_k_zero(gpu_lib):
    N = 136
    b = torch.zeros(1, dtype=torch.uint8, device=DEV)
    s = torch.ones(1, N, dtype=torch.bfloat16, device=DEV)
    bias = torch.randn(N, device=DEV).bfloat16()
    for gated in (False, True):
        n = N // 2 if gated else N
        r = torch.randn(3, n, device=DEV).bfloat16()
        a = torch.empty(3, 0, dtype=torch.bfloat16, device=DEV)
        out = w4.gemm(a, b, w4.UINT4B8, N, scales=s, bias=bias, act=w4.ACT_SILU, gated=gated,
                      residual=r)
        ref, err = reference(np.zeros((3, N)), bias.cpu(), "silu", gated, r.cpu())
        check(out, ref, err, "bf16", gated)
        e = w4.gemm(torch.empty(0, 128, dtype=torch.bfloat16, device=DEV), b, w4.UINT4B8, N,
                    scales=s, act=w4.ACT_SILU, gated=gated)
        assert e.shape == (0, n)


@pytest.mark.gpu
def test_graph_and_another_stream(gpu_lib):
    c = Case("int8", 64, 512, 2048, seed=12)
    a, b, kw = c.device()
    r = torch.randn(64, 512, device=DEV).half()
    ref = w4.gemm(a, b, c.wtype, c.N, act=w4.ACT_SILU, residual=r, **kw)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        out = w4.gemm(a, b, c.wtype, c.N, act=w4.ACT_SILU, residual=r, **kw)
    st.synchronize()
    assert torch.equal(out, ref)
    ws = torch.zeros(w4.workspace_size(64, 512, 2048, torch.int8, -1), dtype=torch.uint8, device=DEV)
    out = r.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.gemm(a, b, c.wtype, c.N, act=w4.ACT_SILU, residual=out, out=out, ws=ws, **kw)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    assert w4.check_status(ws) == w4.OK


# ------------------------------------------------------------- refusals (CPU)
P = 0x100000


@pytest.fixture(scope="module")
def lib():
    w4.build()
    return w4.load()


def _call(lib, M=4, N=64, K=64, act=0, gated=0, residual=0, out=0x900000, a_type=0, out_type=0,
          st=0, sc=0, scales=0x300000, wt=w4.UINT4B8, ws=0x400000):
    return lib.w4_gemm_epilogue(P, a_type, M, K, 0x200000, wt, N, scales, a_type, 0, -1, st, sc, 0,
                                act, gated, residual, out, out_type, ws, 1 << 30, None, -1)


BAD = w4.ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw,status", [
    (dict(act=5), BAD), (dict(act=-1), BAD), (dict(gated=1, N=63), BAD),
    (dict(act=2, residual=0x800001), BAD), (dict(residual=0x900002), BAD),
    (dict(residual=0x900000 - 4 * 64 * 2 + 2), BAD), (dict(gated=1, residual=0x900040), BAD),
    (dict(act=2, a_type=w4.S8, wt=w4.INT4, out_type=w4.S32, scales=0), BAD),
    (dict(act=2, out_type=1), BAD),
    (dict(act=2, ws=0), w4.ERR_WORKSPACE), (dict(act=2, K=72), w4.ERR_UNSUPPORTED),
    (dict(act=2, M=0), w4.OK), (dict(act=9, M=0), BAD),
])
def test_epilogue_refusals(lib, kw, status):
    assert _call(lib, **kw) == status


def test_dynamic_epilogue_refusals(lib):
    def call(act=2, gated=0, residual=0, N=64, out=0x900000):
        return lib.w4_gemm_dynamic_epilogue(P, 0, 4, 128, 0x200000, w4.INT4, N, 0, w4.S8, -1,
                                            0x500000, w4.S8, 0, act, gated, residual, out, 0,
                                            0x400000, ctypes.c_size_t(1 << 30), None)
    assert call(act=7) == BAD
    assert call(gated=1, N=63) == BAD
    assert call(residual=0x900002) == BAD
    assert call(residual=0x800001) == BAD


def test_default_rule_fits_in_the_published_workspaces(lib):
    """Whatever schedule the epilogue's own rule takes, its need is within
    w4_gemm_workspace_size and w4_gemm_dynamic_workspace_size (read from the
    WORKSPACE error of a workspace that is too small; host only)."""
    import re
    rng = np.random.default_rng(1)
    need = lambda: int(re.search(r"(\d+) bytes", lib.w4_last_error().decode()).group(1))
    for _ in range(400):
        at = int(rng.choice([w4.F16, w4.BF16, w4.S8, w4.E4M3]))
        M = int(np.exp(rng.uniform(0, np.log(5000))))
        N = 2 * int(np.exp(rng.uniform(0, np.log(30000))))
        K = 128 * int(rng.integers(1, 120))
        gs = -1 if at == w4.E4M3 else int(rng.choice([g for g in (-1, 64, 128, 256) if K % g == 0]))
        w8 = at in (w4.S8, w4.E4M3)
        sg = 0x300000 if at == w4.S8 and gs not in (-1, K) else 0 if w8 else 0x300000
        st = lib.w4_gemm_epilogue(
            P, at, M, K, 0x200000, w4.INT4 if w8 else w4.UINT4B8, N, sg, at, 0, gs,
            0x500000 if w8 else 0, 0x600000 if w8 else 0, 0, w4.ACT_SILU, 1, 0, 0x40000000,
            w4.F16 if w8 else at, 0x400000, 16, None, -1)
        assert st == w4.ERR_WORKSPACE, (M, N, K, at, gs, st, lib.w4_last_error())
        assert need() <= lib.w4_gemm_workspace_size(M, N, K, at, gs), (M, N, K, at, gs)
        if w8:
            st = lib.w4_gemm_dynamic_epilogue(
                P, w4.F16, M, K, 0x200000, w4.INT4, N, sg, w4.S8, gs, 0x600000, at, 0, w4.ACT_SILU,
                1, 0, 0x40000000, 0, 0x400000, 16, None)
            assert st == w4.ERR_WORKSPACE, (M, N, K, at, gs, st, lib.w4_last_error())
            assert need() <= lib.w4_gemm_dynamic_workspace_size(M, N, K, at, gs), (M, N, K, at, gs)


@pytest.mark.gpu
def test_binding_refusals(gpu_lib):
    c = Case("bf16", 4, 64, 128)
    a, b, kw = c.device()
    f = dict(dtype=torch.bfloat16, device=DEV)
    for bad in (dict(residual=torch.zeros(4, 63, **f)), dict(residual=torch.zeros(4, 64, device=DEV)),
                dict(residual=torch.zeros(4, 64, **f), gated=True),
                dict(act=w4.ACT_SILU, out=torch.zeros(4, 32, **f)),
                dict(gated=True, out=torch.zeros(4, 64, **f)),
                dict(act=w4.ACT_SILU, bias=torch.zeros(63, **f)),
                dict(residual=torch.zeros(4, 64, dtype=torch.bfloat16)),
                dict(residual=torch.zeros(4, 128, **f)[:, ::2]),
                dict(act=w4.ACT_SILU, scales=kw["scales"][:, :32].contiguous()),
                dict(act=w4.ACT_SILU, zeros=kw["scales"].float())):
        with pytest.raises(ValueError):
            w4.gemm(a, b, c.wtype, c.N, **{**kw, **bad})
    with pytest.raises(ValueError, match="b_packed"):
        w4.gemm(a, b[:64], c.wtype, c.N, act=w4.ACT_SILU, **kw)
    c8 = Case("int8", 4, 64, 128)
    a8, b8, kw8 = c8.device()
    for name in ("token_scales", "channel_scales"):
        for t in (kw8[name][1:].clone(), kw8[name].half()):
            with pytest.raises(ValueError, match=name):
                w4.gemm(a8, b8, c8.wtype, c8.N, act=w4.ACT_SILU, **{**kw8, name: t})
    with pytest.raises(ValueError, match="channel_scales"):
        w4.gemm_dynamic(torch.zeros(4, 128, dtype=torch.float16, device=DEV), b8, c8.wtype, c8.N,
                        channel_scales=kw8["channel_scales"][1:].clone(), act=w4.ACT_SILU)
    with pytest.raises(w4.W4Error):
        w4.gemm(a, b, c.wtype, c.N, act=9, **kw)


def test_interleave_columns_on_the_host():
    g, u = torch.arange(6).view(2, 3), torch.arange(10, 16).view(2, 3)
    assert w4.interleave_columns(g, u).tolist() == [[0, 10, 1, 11, 2, 12], [3, 13, 4, 14, 5, 15]]
    assert w4.interleave_columns(g, u, dim=0).tolist() == [[0, 1, 2], [10, 11, 12], [3, 4, 5],
                                                          [13, 14, 15]]
    with pytest.raises(ValueError):
        w4.interleave_columns(g, u[:1])


def test_binding_refuses_what_is_no_tensor(lib):
    """Errors of the host's part, before anything of the device's."""
    x = torch.zeros(2, 64, dtype=torch.float16)
    for call in (lambda: w4.rmsnorm(None), lambda: w4.rmsnorm([1.0]), lambda: w4.rmsnorm(x, [1.0]),
                 lambda: w4.rmsnorm(x, None, "eps"), lambda: w4.rmsnorm_quant(x, residual=3),
                 lambda: w4.gemm(None, x, w4.INT4, 64, act=w4.ACT_SILU),
                 lambda: w4.gemm(x, x, w4.INT4, 64, gated=True, bias=1.0),
                 lambda: w4.gemm(x, x, w4.INT4, 2.5, act=w4.ACT_SILU),
                 lambda: w4.gemm_dynamic(x, None, w4.INT4, 64, act=w4.ACT_SILU)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: w4.gemm(x, x, w4.INT4, 64, act=w4.ACT_SILU),
                 lambda: w4.gemm_dynamic(x, x, w4.INT4, 64, residual=x)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


@pytest.mark.gpu
def test_binding_workspace_grows_and_capture_is_refused(gpu_lib):
    """The stream's cached workspace is taken as it is when it is large
    enough, replaced when not, and a call under capture wants its own."""
    small, large = Case("int8", 4, 64, 128), Case("int8", 300, 1032, 4096)
    with torch.cuda.stream(torch.cuda.Stream()):
        key = (torch.device(DEV).index or 0, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        w4._ws_cache.pop(key, None)  # (a pooled stream another test has used)
        sizes = []
        for c in (small, large, small):
            a, b, kw = c.device()
            torch.cuda.current_stream().synchronize()
            out = w4.gemm(a, b, c.wtype, c.N, act=w4.ACT_RELU, **kw)
            sizes.append(w4._ws_cache[key].numel())
            plain = w4.gemm(a, b, c.wtype, c.N, ws=torch.zeros(
                w4.workspace_size(c.M, c.N, c.K, a.dtype, kw["group_size"]), dtype=torch.uint8,
                device=DEV), act=w4.ACT_RELU, **kw)
            assert torch.equal(out, plain)
        assert sizes[0] < sizes[1] == sizes[2]
        ws = w4._ws_cache.pop(key)  # (the stream and its workspace go with this test)
        torch.cuda.current_stream().synchronize()
        assert w4.check_status(ws) == w4.OK
    a, b, kw = small.device()
    ws = torch.zeros(w4.workspace_size(4, 64, 128, a.dtype, kw["group_size"]), dtype=torch.uint8,
                     device=DEV)
    ref = w4.gemm(a, b, small.wtype, 64, act=w4.ACT_RELU, ws=ws, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(RuntimeError, match="capture"):
            w4.gemm(a, b, small.wtype, 64, act=w4.ACT_RELU, **kw)
        out = w4.gemm(a, b, small.wtype, 64, act=w4.ACT_RELU, ws=ws, **kw)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("gs,groups", [(128, 0), (128, 1), (-1, 1), (-1, 0)])
def test_k_zero_with_the_scales_of_no_group(gpu_lib, gs, groups):
    """A product over no K reads no scale: an array of K / group_size = 0 groups
    is as good as one of one group, with an epilogue as without."""
    N = 136
    b = torch.zeros(1, dtype=torch.uint8, device=DEV)
    a = torch.empty(3, 0, dtype=torch.bfloat16, device=DEV)
    s = torch.ones(groups, N, dtype=torch.bfloat16, device=DEV)
    r = torch.randn(3, N, device=DEV).bfloat16()
    z = torch.empty_like(s)
    for kw in (dict(scales=s), dict(scales=s, zeros=z)):
        plain = w4.gemm(a, b, w4.UINT4B8, N, group_size=gs, **kw)
        assert torch.equal(plain, torch.zeros_like(r))
        out = w4.gemm(a, b, w4.UINT4B8, N, group_size=gs, residual=r, **kw)
        assert torch.equal(out, r)
