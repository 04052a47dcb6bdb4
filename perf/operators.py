"""The operators around the 4-bit-weight products, measured: the root-mean-square norm that makes a
product's activations (residual added, 16-bit or 8-bit output with one scale per token) and the
product with bias, activation (plain or gated) and residual in its epilogue.

Each case has a plain form (elementary torch operations in 32 bits) and the framework's call.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
F16, BF16 = "fp16", "bf16"
DT = {F16: torch.float16, BF16: torch.bfloat16}
# symmetric int8: 127 steps to the row's largest magnitude; E4M3: its largest value
TOP = {"int8": 127.0, "e4m3": 448.0}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def _norm(name, M, K, dtype, out, residual):
    return {"name": name, "op": "norm", "M": M, "K": K, "dtype": dtype, "out": out,
            "residual": residual}


def _gemm(name, mode, M, N, K, group, act="none", gated=False, bias=False, residual=False,
          zeros=False):
    return {"name": name, "op": "gemm", "mode": mode, "M": M, "N": N, "K": K, "group": group,
            "act": act, "gated": gated, "bias": bias, "residual": residual, "zeros": zeros}


def listed():
    return [
        # one decoded token, hidden size of Llama-3-8B, before a 16-bit-activation product
        _norm("norm bf16 M=1", 1, 4096, BF16, "same", True),
        # a decode batch before an int8-activation product, hidden size of Llama-3-70B
        _norm("norm int8 M=16", 16, 8192, F16, "int8", True),
        # a ragged batch of short odd rows: no 16-byte loads
        _norm("norm e4m3 odd", 777, 1111, F16, "e4m3", False),
        # a prefill chunk at the longest row of the W4A8 sweep, fp8 activations
        _norm("norm e4m3 M=1024", 1024, 21760, F16, "e4m3", True),
        # a long prefill, hidden size of Llama-3-70B, int8 activations
        _norm("norm int8 M=16384", 16384, 8192, F16, "int8", True),
        # one decoded token through Llama-3-8B's gate and up projections, gated in the epilogue
        _gemm("gemm bf16 gated M=1", BF16, 1, 28672, 4096, 128, "silu", gated=True, zeros=True),
        # a decode batch through Llama-3-8B's down projection, back onto the residual stream
        _gemm("gemm bf16 res M=16", BF16, 16, 4096, 14336, 128, residual=True, zeros=True),
        # the W4A8 sweep's shape at a decode batch, a layer with bias and GELU
        _gemm("gemm int8 gelu M=32", "int8", 32, 8192, 21760, -1, "gelu", bias=True),
        # a ragged small batch, fp16 activations, every part of the epilogue at once
        _gemm("gemm fp16 all M=77", F16, 77, 2056, 4096, 64, "relu", bias=True, residual=True),
        # the W4A8 sweep's shape with group scales, onto the residual stream
        _gemm("gemm int8 g128 M=1000", "int8", 1000, 8192, 21760, 128, residual=True),
        # the same with fp8 activations and GELU (tanh form)
        _gemm("gemm e4m3 M=1024", "e4m3", 1024, 8192, 21760, -1, "gelu_tanh", bias=True),
        # a prefill chunk through Llama-3-70B's gate and up projections
        _gemm("gemm bf16 gated M=4096", BF16, 4096, 57344, 8192, 128, "silu", gated=True,
              zeros=True),
    ]


def _size(rng, lo, hi, step=1):
    """A multiple of step between lo and hi, spread over its logarithm."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = max(lo, n // step * step)
    return n if n != 3072 else n + step


def draw(rng):
    if rng.random() < 0.45:
        K = _size(rng, 128, 28672, 8 if rng.random() < 0.7 else 1)
        M = _size(rng, 1, min(16384, 16384 * 8192 // K))
        c = _norm("", M, K, rng.choice((F16, BF16)), rng.choice(("same", "int8", "e4m3")),
                  rng.random() < 0.7)
    else:
        mode = rng.choice((F16, BF16, BF16, "int8", "int8", "e4m3"))
        K = _size(rng, 512, 28672, 128)
        N = _size(rng, 256, min(57344, 57344 * 8192 // K), 16)
        M = _size(rng, 1, 4096)
        group = -1 if mode == "e4m3" else rng.choice((-1, 128))
        gated = rng.random() < 0.4
        c = _gemm("", mode, M, N, K, group, rng.choice(ACTS[1:]) if gated else rng.choice(ACTS),
                  gated, bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                  zeros=mode in (F16, BF16) and rng.random() < 0.5)
    del c["name"]
    return c


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * std

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=g, device=DEV) * (hi - lo) + lo

    s = dict(case)
    M, K = case["M"], case["K"]
    if case["op"] == "norm":
        dt = DT[case["dtype"]]
        # activations with a few large channels, as a transformer's residual stream has
        spread = 1 + 20 * (uniform(0, 1, K) < 0.002)
        s["x"] = normal(M, K).to(dt)
        s["r"] = (normal(M, K, std=2.0) * spread).to(dt) if case["residual"] else None
        s["w"] = uniform(0.2, 1.8, K).to(dt)
        return s
    mode, N = case["mode"], case["N"]
    G = 1 if case["group"] == -1 else K // case["group"]
    od = DT.get(mode, torch.float16)
    # scales that give products of unit size, where the activations bend
    unit = 1 / (4.6 * math.sqrt(K))
    s["wq"] = torch.randint(-2**31, 2**31 - 1, (K // 8, N), generator=g, device=DEV,
                            dtype=torch.int32)
    s["scales"] = s["zeros"] = s["st"] = s["sc"] = None
    if mode in DT:
        s["a"] = normal(M, K).to(od)
        s["scales"] = uniform(0.5 * unit, 1.5 * unit, G, N).to(od)
        if case["zeros"]:  # pre-scaled zero-points
            z = torch.randint(6, 10, (G, N), generator=g, device=DEV)
            s["zeros"] = (z * s["scales"].float()).to(od)
    else:
        if mode == "int8":
            s["a"] = torch.randint(-127, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
            size = 73.0
        else:
            s["a"] = normal(M, K, std=100.0).clamp(-448, 448).to(torch.float8_e4m3fn)
            size = 100.0
        if G > 1:
            s["scales"] = torch.randint(1, 17, (G, N), generator=g, device=DEV, dtype=torch.int8)
            size *= 9.5
        s["st"] = uniform(0.5, 1.5, M) / size
        s["sc"] = uniform(0.5, 1.5, N) * unit
    n_out = N // 2 if case["gated"] else N
    s["bias"] = normal(N, std=0.5).to(od) if case["bias"] else None
    s["r"] = normal(M, n_out).to(od) if case["residual"] else None
    if own:  # a program lays its weights out once, when it loads them
        import int4_weight_mixed_gb300 as w4
        s["wtype"] = w4.INT4 if s["st"] is not None else w4.UINT4 if case["zeros"] else w4.UINT4B8
        s["b"] = w4.prepack_B(s["wq"], s["wtype"], w4.KN_SEQ, K, N)
    return s


def run(s):
    if s["op"] == "norm":
        return _norm_own(s) if own else _norm_plain(s)
    return _gemm_own(s) if own else _gemm_plain(s)


def _norm_own(s):
    import int4_weight_mixed_gb300 as w4
    if s["out"] == "same":
        r = w4.rmsnorm(s["x"], s["w"], EPS, residual=s["r"])
        return {"y": r[0], "h": r[1]} if s["residual"] else {"y": r}
    act = torch.int8 if s["out"] == "int8" else torch.float8_e4m3fn
    r = w4.rmsnorm_quant(s["x"], s["w"], EPS, residual=s["r"], act_dtype=act)
    return dict(zip(("codes", "scale", "h"), r))


def _norm_plain(s):
    # The 8-bit codes stand for multiples of the token's scale: with hw = h * w and A its row's
    # largest magnitude, y / scale = hw * top / A, which needs no statistic of the norm.  Each
    # step is one rounding in 32 bits, so the codes are the same whole numbers on both sides.
    x = s["x"].float()
    h = x + s["r"].float() if s["residual"] else x
    rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    w = s["w"].float()
    if s["out"] == "same":
        out = {"y": (h * rstd * w).to(s["x"].dtype)}
    else:
        hw = h * w
        A = hw.abs().amax(-1, keepdim=True)
        q = hw * (TOP[s["out"]] / A)
        out = {"codes": torch.round(q).to(torch.int8) if s["out"] == "int8"
               else q.to(torch.float8_e4m3fn),
               "scale": (rstd * (A / TOP[s["out"]])).squeeze(-1)}
    if s["residual"]:
        out["h"] = h.to(s["x"].dtype)
    return out


def _gemm_own(s):
    import int4_weight_mixed_gb300 as w4
    act = {"none": w4.ACT_NONE, "relu": w4.ACT_RELU, "silu": w4.ACT_SILU, "gelu": w4.ACT_GELU,
           "gelu_tanh": w4.ACT_GELU_TANH}[s["act"]]
    return {"out": w4.gemm(s["a"], s["b"], s["wtype"], s["N"], scales=s["scales"],
                           zeros=s["zeros"], group_size=s["group"], token_scales=s["st"],
                           channel_scales=s["sc"], bias=s["bias"], act=act, gated=s["gated"],
                           residual=s["r"])}


def _activate(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _gemm_plain(s):
    # value j of a word sits at bits 4j; int4 is two's complement, uint4 with zero-points its
    # stored value, uint4b8 its stored value less 8
    K, N = s["K"], s["N"]
    shifts = torch.arange(0, 32, 4, device=DEV, dtype=torch.int32)
    q = ((s["wq"][:, None, :] >> shifts[None, :, None]) & 15).view(K, N)
    if s["st"] is not None:
        q = (q ^ 8) - 8
    elif s["zeros"] is None:
        q = q - 8
    w = q.float()
    if s["scales"] is not None:
        G = s["scales"].shape[0]
        w = w.view(G, K // G, N) * s["scales"].float()[:, None]
        if s["zeros"] is not None:
            w = w - s["zeros"].float()[:, None]
        w = w.view(K, N)
    v = s["a"].float() @ w
    if s["st"] is not None:
        v = v * s["st"][:, None] * s["sc"]
    if s["bias"] is not None:
        v = v + s["bias"].float()
    # gated: the even columns are the gate, the odd ones what it multiplies
    v = _activate(v[:, 0::2], s["act"]) * v[:, 1::2] if s["gated"] else _activate(v, s["act"])
    if s["r"] is not None:
        v = v + s["r"].float()
    return {"out": v.to(DT.get(s["mode"], torch.float16))}


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "norm":
        e = M * K
        out = 2 * e if case["out"] == "same" else e + 4 * M
        return {"bytes": 2 * e + 2 * K + out + (4 * e if case["residual"] else 0), "flops": 5 * e}
    N = case["N"]
    G = 1 if case["group"] == -1 else K // case["group"]
    n_out = N // 2 if case["gated"] else N
    if case["mode"] in DT:
        side = 2 * M * K + 2 * G * N * (2 if case["zeros"] else 1)
    else:
        side = M * K + 4 * M + 4 * N + (G * N if G > 1 else 0)
    return {"bytes": K * N // 2 + side + 2 * M * n_out + (2 * N if case["bias"] else 0)
            + (2 * M * n_out if case["residual"] else 0), "flops": 2 * M * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return _norm_exact(s) if case["op"] == "norm" else _gemm_exact(s)


def _norm_exact(s):
    h = s["x"].double()
    if s["residual"]:
        h.add_(s["r"].double())
    y = h / (h.square().sum(1) / s["K"] + EPS).sqrt()[:, None]
    y *= s["w"].double()
    if s["out"] == "same":
        out = {"y": y}
    else:
        scale = y.abs().max(1).values / TOP[s["out"]]
        out = {"codes": None, "scale": scale}
        if s["out"] == "e4m3":  # the E4M3 value nearest to y / scale: steps of 2^-3 of its binade
            t = y / scale[:, None]
            step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0**-6))) - 3)
            out["codes"] = torch.round(t / step) * step
    if s["residual"]:
        out["h"] = h
    return out


def _gemm_exact(s):
    K, N, M = s["K"], s["N"], s["M"]
    a = s["a"].to(torch.float64)
    out = torch.empty(M, N // 2 if s["gated"] else N, dtype=torch.float64, device=DEV)
    wide = max(2, min(N, (1 << 28) // K // 2 * 2))
    for n0 in range(0, N, wide):  # a block of columns at a time
        n1 = min(N, n0 + wide)
        # bytes of a word in memory order hold its values two by two, the lower nibble first
        byte = s["wq"][:, n0:n1].contiguous().view(torch.uint8).view(K // 8, n1 - n0, 4)
        byte = byte.permute(0, 2, 1).reshape(K // 2, n1 - n0)
        w = torch.empty(K, n1 - n0, dtype=torch.float64, device=DEV)
        w[0::2] = (byte % 16).double()
        w[1::2] = torch.div(byte, 16, rounding_mode="floor").double()
        if s["st"] is not None:
            w[w >= 8] -= 16
        elif s["zeros"] is None:
            w -= 8
        if s["scales"] is not None:
            rep = K // s["scales"].shape[0]
            w *= s["scales"][:, n0:n1].double().repeat_interleave(rep, 0)
            if s["zeros"] is not None:
                w -= s["zeros"][:, n0:n1].double().repeat_interleave(rep, 0)
        v = torch.mm(a, w)
        if s["st"] is not None:
            v *= torch.outer(s["st"].double(), s["sc"][n0:n1].double())
        if s["bias"] is not None:
            v += s["bias"][n0:n1].double()
        up = None
        if s["gated"]:
            v, up = v[:, ::2], v[:, 1::2]
        if s["act"] == "relu":
            v = v.clamp_min(0)
        elif s["act"] == "silu":
            v = v * torch.special.expit(v)
        elif s["act"] == "gelu":
            v = v * torch.special.ndtr(v)
        elif s["act"] == "gelu_tanh":  # (1 + tanh(u)) / 2 is the logistic function of 2u
            v = v * torch.special.expit(math.sqrt(8 / math.pi) * (v + 0.044715 * v**3))
        if up is not None:
            v = v * up
            n0, n1 = n0 // 2, n1 // 2
        out[:, n0:n1] = v
    if s["r"] is not None:
        out += s["r"].double()
    return {"out": out}
