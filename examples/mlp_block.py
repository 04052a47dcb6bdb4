"""A transformer's MLP block on 4-bit weights with int8 activations, three
calls on the residual stream:

    norm      h += x; codes, scales = the norm of h, per token in 8 bits
    gate, up  a = SiLU(codes . gate) * (codes . up)      (one gated product)
    down      h += a quantised per token . down          (residual in place)

python examples/mlp_block.py [tokens [hidden [ffn]]]

makes a block of that size with random weights (default: Llama-3-8B's, 4096
and 14336), runs it, compares it with the same block in plain torch operations
in fp32 and prints the time of both.
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import int4_weight_mixed_gb300 as w4  # noqa: E402


class MlpBlock:
    """Weights [K/8, N] of packed int4 words (K packed, KN_SEQ) with one fp32
    scale per column; norm [hidden] fp16."""

    def __init__(self, norm, gate, up, down, s_gate, s_up, s_down, eps=1e-5):
        self.hidden, self.ffn, self.eps = gate.shape[0] * 8, gate.shape[1], eps
        self.norm = norm
        # gate and up columns side by side: one product feeds the gated epilogue
        self.gate_up = w4.prepack_B(w4.interleave_columns(gate, up), w4.INT4, w4.KN_SEQ,
                                    self.hidden, 2 * self.ffn)
        self.s_gate_up = w4.interleave_columns(s_gate, s_up)
        self.down = w4.prepack_B(down, w4.INT4, w4.KN_SEQ, self.ffn, self.hidden)
        self.s_down = s_down

    def __call__(self, x, h):
        """x [tokens, hidden]: what the layer before adds to the residual
        stream h (fp16, updated in place and returned)."""
        codes, scales, h = w4.rmsnorm_quant(x, self.norm, self.eps, residual=h, residual_out=h)
        a = w4.gemm(codes, self.gate_up, w4.INT4, 2 * self.ffn, token_scales=scales,
                    channel_scales=self.s_gate_up, act=w4.ACT_SILU, gated=True)
        return w4.gemm_dynamic(a, self.down, w4.INT4, self.hidden, channel_scales=self.s_down,
                               residual=h, out=h)


def random_weights(hidden, ffn, seed=0, device="cuda"):
    """Arguments of MlpBlock with unit-size products."""
    g = torch.Generator(device=device).manual_seed(seed)

    def weight(K, N):
        words = torch.randint(-2**31, 2**31 - 1, (K // 8, N), generator=g, device=device,
                              dtype=torch.int32)
        scale = torch.rand(N, generator=g, device=device) + 0.5
        return words, scale / (4.6 * K**0.5)

    (gate, sg), (up, su), (down, sd) = weight(hidden, ffn), weight(hidden, ffn), weight(ffn, hidden)
    norm = (torch.rand(hidden, generator=g, device=device) + 0.5).half()
    return norm, gate, up, down, sg, su, sd


def dequantized(words, scale):
    """[K, N] fp32 weights of packed int4 words."""
    shifts = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    q = (words[:, None, :] >> shifts[None, :, None]) & 15
    return (q - 16 * (q >= 8)).reshape(-1, words.shape[1]).float() * scale


def quantized(y):
    """y as int8 codes and scales stand for it, in fp32."""
    s = y.abs().amax(-1, keepdim=True) / 127
    return torch.round(y / s) * s


def plain_block(x, h, norm, gate, up, down, eps=1e-5):
    """The block in fp32, with the same two quantisations of activations;
    gate, up and down are dequantized weights."""
    h = h.float() + x.float()
    y = quantized(h * torch.rsqrt((h * h).mean(-1, keepdim=True) + eps) * norm.float())
    a = torch.nn.functional.silu(y @ gate) * (y @ up)
    return h + quantized(a) @ down


def main(tokens=64, hidden=4096, ffn=14336):
    weights = random_weights(hidden, ffn)
    block = MlpBlock(*weights)
    norm, gate, up, down, sg, su, sd = weights
    plain = [dequantized(*p) for p in ((gate, sg), (up, su), (down, sd))]
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").half()
    h = torch.randn(tokens, hidden, generator=g, device="cuda").half()
    ref = plain_block(x, h, norm, *plain)
    got = block(x, h.clone()).float()
    off = ((got - ref).norm() / ref.norm()).item()
    print(f"{tokens} tokens, hidden {hidden}, ffn {ffn}: relative difference {off:.1e}")
    for name, run in (("block", lambda: block(x, h)),
                      ("plain fp32", lambda: plain_block(x, h, norm, *plain))):
        for _ in range(3):
            run()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(20):
            run()
        b.record()
        b.synchronize()
        print(f"{name}: {a.elapsed_time(b) / 20 * 1e3:.1f} us")
    return off


if __name__ == "__main__":
    main(*(int(v) for v in sys.argv[1:4]))
