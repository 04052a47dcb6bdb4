"""The norm, the gated product and the product onto the residual stream used
together, as examples/mlp_block.py does: against the same block in fp32.

Both sides quantise the same two activations to int8.  A code may round to the
other side where fp32 values differ (the gated activations are rounded to
fp16, 2^-11 of each, before they are quantised: a step of amax / 127 moves
with probability of order 2^-11 * 127 / 4), so the difference is held in the
2-norm: fp16 roundings (2^-11 each of the activations, the stream and the
output) and a share p < 0.1 of activations off by one step, a step being
under 4 % of their size, give less than sqrt(3 * 2^-22 + 0.1 * 0.04^2) = 1.3e-2
of the down product."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 7, 40, 300])
@pytest.mark.parametrize("hidden,ffn", [(256, 512), (1024, 1408)])
def test_block_matches_fp32(gpu_lib, tokens, hidden, ffn):
    import mlp_block
    weights = mlp_block.random_weights(hidden, ffn, seed=tokens)
    block = mlp_block.MlpBlock(*weights)
    norm, gate, up, down, sg, su, sd = weights
    plain = [mlp_block.dequantized(*p) for p in ((gate, sg), (up, su), (down, sd))]
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").half()
    h = torch.randn(tokens, hidden, generator=g, device="cuda").half()
    stream = h.clone()
    out = block(x, stream)
    assert out is stream
    ref = mlp_block.plain_block(x, h, norm, *plain)
    down_part = ref - (h.float() + x.float())
    off = (out.float() - ref).norm() / down_part.norm()
    assert off < 1.3e-2 + 2.0**-11 * float(ref.norm() / down_part.norm()), float(off)


def test_block_in_a_graph(gpu_lib):
    """The three calls captured once and replayed on new inputs."""
    import mlp_block
    w4 = gpu_lib
    block = mlp_block.MlpBlock(*mlp_block.random_weights(512, 1024))
    x, h = (torch.randn(8, 512, device="cuda").half() for _ in range(2))
    ref = block(x, h.clone())
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    stream = h.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q, s, _ = w4.rmsnorm_quant(x, block.norm, block.eps, residual=stream, residual_out=stream)
        a = w4.gemm(q, block.gate_up, w4.INT4, 2048, token_scales=s,
                    channel_scales=block.s_gate_up, act=w4.ACT_SILU, gated=True, ws=ws)
        w4.gemm_dynamic(a, block.down, w4.INT4, 512, channel_scales=block.s_down, residual=stream,
                        out=stream, ws=ws)
    for seed in (1, 2):
        x.copy_(torch.randn(8, 512, generator=torch.Generator().manual_seed(seed)))
        stream.copy_(h)
        ref = block(x, h.clone())
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(stream, ref)
    assert w4.check_status(ws) == w4.OK
