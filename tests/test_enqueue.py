"""What a call enqueues, seen by a recording CUDA runtime (CPU), and two host
threads on one stream (GPU)."""
import threading

import pytest
import torch

import int4_weight_mixed_gb300 as w4
from fake_cuda import build

P = 0x10000000  # (never dereferenced: nothing runs)
WS = 0x40000000


@pytest.fixture(scope="module")
def rec(tmp_path_factory):
    return build(tmp_path_factory.mktemp("recorded"))


def _epilogue(lib, M, N, K, a_type, gs=-1, residual=0, act=w4.ACT_SILU, gated=0, out=8 * P, bias=0,
              ch=6 * P, ws=WS, schedule=-1):
    w8 = a_type in (w4.S8, w4.E4M3)
    scales = 0 if w8 and gs == -1 else 2 * P
    return lib.w4_gemm_epilogue(
        P, a_type, M, K, 3 * P, w4.INT4 if w8 else w4.UINT4B8, N, scales, a_type, 0, gs,
        5 * P if w8 else 0, ch if w8 else 0, bias, act, gated, residual, out,
        w4.F16 if w8 else a_type, ws, 1 << 32, None, schedule)


def _plain(lib, M, N, K, a_type, gs=-1):
    w8 = a_type in (w4.S8, w4.E4M3)
    return lib.w4_gemm(P, a_type, M, K, 3 * P, w4.INT4 if w8 else w4.UINT4B8, N,
                       0 if w8 and gs == -1 else 2 * P, a_type, 0, gs, 5 * P if w8 else 0,
                       6 * P if w8 else 0, 8 * P, w4.F16 if w8 else a_type, WS, 1 << 32, None)


def _dynamic(lib, M, N, K, act_type=w4.S8):
    return lib.w4_gemm_dynamic_epilogue(P, w4.F16, M, K, 3 * P, w4.INT4, N, 0, w4.S8, -1, 6 * P,
                                        act_type, 0, w4.ACT_SILU, 0, 0, 8 * P, 0, WS, 1 << 32, None)


# calls of several launches: split tiles with an epilogue, the int8 staging
# launch, the streamed schedule, the quantizer before the product
CALLS = {
    "split tiles, epilogue": lambda lib: _epilogue(lib, 64, 4096, 14336, w4.BF16, 128),
    "staged int8": lambda lib: _plain(lib, 128, 1024, 4096, w4.S8),
    "streamed": lambda lib: _plain(lib, 8, 8192, 21760, w4.S8),
    "quantized int8": lambda lib: _dynamic(lib, 64, 4096, 14336),
    "quantized fp8": lambda lib: _dynamic(lib, 3, 4096, 14336, w4.E4M3),
}


@pytest.mark.parametrize("kind", list(CALLS))
def test_launches_of_a_call_stay_together(rec, kind):
    """Two host threads with one workspace on one stream: what a call leaves
    in the workspace for its next launch is not overwritten by the other
    thread's, so no launch of another call comes between a call's own."""
    call, calls = CALLS[kind], 4
    rec.reset()
    assert call(rec.lib) == w4.OK
    alone = [k for _, k in rec.launches()]
    assert len(alone) >= 2, alone
    rec.reset(pause_us=2000)
    start, status = threading.Barrier(2), []

    def work():
        start.wait()
        for _ in range(calls):
            status.append(call(rec.lib))

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert status == [w4.OK] * 2 * calls
    got = rec.launches()
    assert len(got) == 2 * calls * len(alone)
    for i in range(0, len(got), len(alone)):
        part = got[i:i + len(alone)]
        assert [k for _, k in part] == alone and len({t for t, _ in part}) == 1, part


@pytest.mark.gpu
@pytest.mark.parametrize("mode,M,N,K,gs", [("bf16", 64, 4096, 2048, 128), ("int8", 64, 1024, 4096, -1),
                                           ("e4m3", 40, 2048, 4096, -1), ("int8", 8, 1024, 8192, -1)])
def test_two_host_threads_on_one_stream(gpu_lib, mode, M, N, K, gs):
    """Both threads take the stream's cached workspace: each call's result is
    the one it has alone, bit for bit."""
    dev = "cuda:0"
    g = torch.Generator(device=dev).manual_seed(2)
    b = w4.prepack_B(torch.randint(-2**31, 2**31 - 1, (K // 8, N), generator=g, device=dev,
                                   dtype=torch.int32), w4.INT4, w4.KN_SEQ, K, N)

    def operands():
        a = torch.randn(M, K, generator=g, device=dev)
        if mode == "bf16":
            s = (torch.rand(K // gs, N, generator=g, device=dev) + 0.5) / 256
            return a.bfloat16(), dict(scales=s.bfloat16(), group_size=gs)
        a = (a * 30).clamp(-127, 127)
        return a.to(torch.int8 if mode == "int8" else torch.float8_e4m3fn), dict(
            token_scales=torch.rand(M, generator=g, device=dev) / 4096,
            channel_scales=torch.rand(N, generator=g, device=dev) / 64)

    jobs = []
    for _ in range(2):
        a, kw = operands()
        r = torch.randn(M, N, generator=g, device=dev).to(torch.bfloat16 if mode == "bf16"
                                                          else torch.float16)
        for extra in (dict(residual=r), dict(act=w4.ACT_SILU), {}):
            jobs.append((a, dict(kw, **extra), w4.gemm(a, b, w4.INT4, N, **kw, **extra)))
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(2), []

    def work(mine):
        start.wait()
        outs = [(w4.gemm(a, b, w4.INT4, N, **kw), ref) for _ in range(40) for a, kw, ref in mine]
        wrong.extend(i for i, (out, ref) in enumerate(outs) if not torch.equal(out, ref))

    threads = [threading.Thread(target=work, args=(jobs[i::2],)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
