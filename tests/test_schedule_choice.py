"""Which schedule a product takes by default, with and without an epilogue."""
import math
import random

import pytest
import torch

import int4_weight_mixed_gb300 as w4
from fake_cuda import build

P = 0x10000000  # (never dereferenced: nothing runs)


@pytest.fixture(scope="module")
def rec(tmp_path_factory):
    return build(tmp_path_factory.mktemp("recorded"))


def _launched(rec, M, N, K, a_type, gs=-1, **ep):
    """The kernels of a product, with an epilogue if `ep` has one."""
    w8 = a_type in (w4.S8, w4.E4M3)
    scales = 0 if w8 and gs == -1 else 2 * P
    d = dict(bias=0, act=0, gated=0, residual=0, out=8 * P, ch=6 * P if w8 else 0)
    d.update(ep)
    rec.reset()
    st = rec.lib.w4_gemm_epilogue(
        P, a_type, M, K, 3 * P, w4.INT4 if w8 else w4.UINT4B8, N, scales, a_type, 0, gs,
        5 * P if w8 else 0, d["ch"], d["bias"], d["act"], d["gated"], d["residual"], d["out"],
        w4.F16 if w8 else a_type, 0x40000000, 1 << 40, None, -1)
    assert st == w4.OK, rec.lib.w4_last_error()
    return " ".join(k for _, k in rec.launches())


def test_overrides_of_one_kind_leave_the_other(rec):
    """An override for products without an epilogue does not touch those with
    one, and the reverse; the kernels that are launched follow."""
    lib = rec.lib
    index = {lib.w4_schedule_name(i).decode(): i for i in range(lib.w4_num_schedules())}
    shape = (64, 4096, 4096, w4.BF16, 128)
    plain, epilogue = lib.w4_default_schedule(*shape), lib.w4_default_epilogue_schedule(*shape)
    key = (w4.BF16, 33, 64, 4096, 4096, 128)
    other = index["tc256p_dp"]
    assert other not in (plain, epilogue)
    assert lib.w4_override_schedule(*key, other) == w4.OK
    assert lib.w4_default_schedule(*shape) == other
    assert lib.w4_default_epilogue_schedule(*shape) == epilogue
    pair = "Lb1ELb1E"  # tc_gemm_kernel<mode, MMA2, PAIR, LEAN, ..>
    M, N, K, at, gs = shape
    assert pair in _launched(rec, M, N, K, at, gs)
    assert pair not in _launched(rec, M, N, K, at, gs, act=w4.ACT_SILU)
    assert lib.w4_override_epilogue_schedule(*key, index["tc16_sk"]) == w4.OK
    assert lib.w4_default_schedule(*shape) == other
    assert lib.w4_default_epilogue_schedule(*shape) == index["tc16_sk"]
    assert lib.w4_override_schedule(*key, -1) == w4.OK      # removed: the other stays
    assert lib.w4_default_schedule(*shape) == plain
    assert lib.w4_default_epilogue_schedule(*shape) == index["tc16_sk"]
    assert lib.w4_override_epilogue_schedule(*key, index["ds8_sk"]) == w4.OK  # cannot run 64 rows
    assert lib.w4_default_epilogue_schedule(*shape) == epilogue
    assert lib.w4_override_epilogue_schedule(*key, -1) == w4.OK
    assert lib.w4_override_epilogue_schedule(7, 1, 2, 8, 64, -1, 1) == w4.ERR_INVALID_ARGUMENT
    assert lib.w4_override_epilogue_schedule(1, 1, 2, 8, 64, -1, 99) == w4.ERR_INVALID_ARGUMENT
    # the built-in entries hold for both
    big = (4096, 57344, 8192, w4.BF16, 128)
    assert lib.w4_default_epilogue_schedule(*big) == lib.w4_default_schedule(*big) == other


def test_the_binding_names_the_kind():
    shape = (64, 4096, 14336, torch.bfloat16, 128)
    plain, epilogue = w4.default_schedule(*shape), w4.default_schedule(*shape, epilogue=True)
    try:
        w4.override_schedule(torch.bfloat16, 64, 64, 4096, 14336, 128, "tc256_dp", epilogue=True)
        assert w4.default_schedule(*shape) == plain
        name = w4.schedule_names()[w4.default_schedule(*shape, epilogue=True)]
        assert name == "tc256_dp"
    finally:
        w4.override_schedule(torch.bfloat16, 64, 64, 4096, 14336, 128, None, epilogue=True)
    assert w4.default_schedule(*shape, epilogue=True) == epilogue


@pytest.mark.gpu
def test_autotune_of_an_epilogue_is_its_own(gpu_lib):
    """Tuning a product with an epilogue leaves the plain product's choice,
    the reverse too, and does not add into a residual that is the output."""
    dev, M, N, K = "cuda:0", 48, 1024, 2048
    g = torch.Generator(device=dev).manual_seed(1)
    b = w4.prepack_B(torch.randint(-2**31, 2**31 - 1, (K // 8, N), generator=g, device=dev,
                                   dtype=torch.int32), w4.UINT4B8, w4.KN_SEQ, K, N)
    a = torch.randn(M, K, generator=g, device=dev).bfloat16()
    s = torch.full((K // 128, N), 2.0**-7, device=dev).bfloat16()
    h = torch.randn(M, N, generator=g, device=dev).bfloat16()
    before = h.clone()
    names = w4.schedule_names()
    pick = lambda e: names[w4.default_schedule(M, N, K, torch.bfloat16, 128, epilogue=e)]
    plain, epilogue = pick(False), pick(True)
    kw = dict(scales=s, group_size=128, reps=3)
    try:
        times = w4.autotune(a, b, w4.UINT4B8, N, residual=h, out=h, **kw)
        assert torch.equal(h, before)
        assert pick(True) == min(times, key=times.get) and pick(False) == plain
        w4.override_schedule(torch.bfloat16, M, M, N, K, 128, None, epilogue=True)
        times = w4.autotune(a, b, w4.UINT4B8, N, **kw)
        assert pick(False) == min(times, key=times.get) and pick(True) == epilogue
    finally:
        for e in (False, True):
            w4.override_schedule(torch.bfloat16, M, M, N, K, 128, None, epilogue=e)


def test_an_epilogue_rounds_no_weight_that_the_product_does_not():
    """W4A16: the decode schedules take the weights as they are and scale sums
    in fp32, the tensor-core ones round each dequantized weight to 16 bits.  A
    product that runs on the former runs there with an epilogue too."""
    names = w4.schedule_names()
    rng = random.Random(3)
    w4.load()
    shapes = [(24, 57344, 8192), (18, 18256, 896), (17, 8960, 512)]
    for _ in range(600):
        shapes.append((rng.randint(1, 40), 8 * int(math.exp(rng.uniform(2, math.log(7168)))),
                       128 * int(math.exp(rng.uniform(1, math.log(224))))))
    decode = 0
    for M, N, K in shapes:
        for dt in (torch.float16, torch.bfloat16):
            for gs in (-1, 128):
                plain, ep = (names[w4.default_schedule(M, N, K, dt, gs, epilogue=e)]
                             for e in (False, True))
                if not plain.startswith("tc"):
                    assert not ep.startswith("tc"), (M, N, K, dt, gs, plain, ep)
                    decode += 1
    assert decode > 1000


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(17, 8960, 512), (18, 18256, 896), (19, 14576, 19584)])
def test_an_epilogue_keeps_the_products_accuracy(gpu_lib, M, N, K):
    """bf16 products of 17 to 32 rows with scales of many bits, whose product
    with a weight bf16 would round.  No weight is rounded, so what is left is
    the output's one rounding (half an ulp of bf16, at most 2^-8 of it) and the
    scales' and sums' fp32 arithmetic, far below."""
    dev = "cuda:0"
    g = torch.Generator(device=dev).manual_seed(4)
    wq = torch.randint(-2**31, 2**31 - 1, (K // 8, N), generator=g, device=dev, dtype=torch.int32)
    b = w4.prepack_B(wq, w4.UINT4B8, w4.KN_SEQ, K, N)
    a = torch.randn(M, K, generator=g, device=dev).bfloat16()
    s = ((torch.rand(K // 128, N, generator=g, device=dev) + 0.5) / (4.6 * K**0.5)).bfloat16()
    r = torch.randn(M, N, generator=g, device=dev).bfloat16()
    out = w4.gemm(a, b, w4.UINT4B8, N, scales=s, group_size=128, residual=r)
    C = 256
    sh = torch.arange(0, 32, 4, device=dev, dtype=torch.int32)
    q = ((wq[:, None, :C] >> sh[None, :, None]) & 15).reshape(K, C).double() - 8
    w = q * s[:, :C].double().repeat_interleave(128, 0)
    ref = a.double() @ w + r[:, :C].double()
    terms = a.double().abs() @ w.abs()
    err = (out[:, :C].double() - ref).abs()
    # rounded weights would be off by up to 2^-9 of the terms' sum, about
    # 2^-9 sqrt(K) / K of it in the mean square; fp32 sums by K 2^-24
    bound = 2.0**-8 * ref.abs() + (K + 64) * 2.0**-24 * terms
    assert bool((err <= bound).all()), (err / bound).max().item()


UNALIGNED = {"out": dict(out=8 * P + 2), "residual": dict(residual=9 * P + 2),
             "bias": dict(bias=9 * P + 2), "channel scales": dict(ch=6 * P + 4)}


@pytest.mark.parametrize("what", list(UNALIGNED))
@pytest.mark.parametrize("mode,M,N,K,gs", [
    (w4.S8, 24, 4096, 14336, -1), (w4.S8, 32, 57344, 8192, -1), (w4.S8, 17, 8960, 512, 128),
    (w4.E4M3, 24, 8192, 21760, -1), (w4.E4M3, 18, 1024, 512, -1), (w4.BF16, 24, 57344, 8192, 128),
    (w4.F16, 31, 2048, 4096, -1), (w4.S8, 3, 4096, 4096, -1), (w4.E4M3, 9, 4096, 4096, -1)])
def test_arrays_off_a_boundary_stay_off_the_cuda_cores(rec, mode, M, N, K, gs, what):
    """Up to 32 rows there is a schedule whose epilogue goes by element."""
    if what == "channel scales" and mode in (w4.F16, w4.BF16):
        return
    got = _launched(rec, M, N, K, mode, gs, act=w4.ACT_SILU, **UNALIGNED[what])
    assert "simt" not in got and "tc_gemm" not in got, got
    assert "ds_gemm" in got or "gv_gemm" in got


def test_dynamic_products_off_a_boundary(rec):
    """The same inside the call that quantizes, within its workspace."""
    for act_type in (w4.S8, w4.E4M3):
        for M, N, K in ((24, 4096, 14336), (24, 57344, 8192), (18, 1024, 512), (5, 4096, 4096)):
            rec.reset()
            ws = rec.lib.w4_gemm_dynamic_workspace_size(M, N, K, act_type, -1)
            st = rec.lib.w4_gemm_dynamic_epilogue(
                P, w4.F16, M, K, 3 * P, w4.INT4, N, 0, w4.S8, -1, 6 * P, act_type, 0, w4.ACT_SILU,
                0, 9 * P + 2, 8 * P, 0, 0x40000000, ws, None)
            assert st == w4.OK, rec.lib.w4_last_error()
            got = " ".join(k for _, k in rec.launches())
            assert "simt" not in got and ("ds_gemm" in got or "gv_gemm" in got), got
