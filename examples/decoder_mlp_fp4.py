"""A decoder block's MLP on 4-bit operands, end to end on one GPU:

    x' = x + norm(y)             the attention block's output joins the stream
    u  = norm(x') as 4-bit       wq.block_norm, one kernel
    h  = silu(gate) * up         wq.gemm_fp4 on the interleaved gate / up weight
    h4 = h as 4-bit              wq.quantize
    y' = h4 . down^T             wq.gemm_fp4
    z, v = x' + norm(y'), norm(z)   wq.block_norm: ready for the next block

Weights are quantised once from bf16; the sizes are those of the 3B decoder
whose projections the library's benchmark sweeps (width 3072, MLP 8192).

    python examples/decoder_mlp_fp4.py --rows 128 --fmt nvfp4
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_bit_w4a16_gb300 as wq  # noqa: E402


def interleave(gate, up):
    """One weight of 2 F rows from a gate and an up weight of F rows, in groups of 8 rows (wq_gemm_fused)."""
    F, K = gate.shape
    return torch.stack((gate.view(F // 8, 8, K), up.view(F // 8, 8, K)), dim=1).reshape(2 * F, K)


class Mlp:
    """The block's weights as 4-bit operands and its norms' weights."""

    def __init__(self, gate, up, down, norms, fmt):
        self.fmt = fmt
        self.gate_up = wq.quantize(interleave(gate, up).contiguous(), fmt)
        self.down = wq.quantize(down, fmt)
        self.post_attn, self.pre_mlp, self.post_mlp, self.pre_next = norms

    def __call__(self, x, y):
        """x: the residual stream (rows, d), y: the attention block's output.  Returns (x'', the next block's input)."""
        x, u = wq.block_norm(x, self.pre_mlp, branch=y, post_weight=self.post_attn, fmt=self.fmt)
        h = wq.gemm_fp4(u, self.gate_up, gated=True)
        y = wq.gemm_fp4(wq.quantize(h, self.fmt), self.down)
        return wq.block_norm(x, self.pre_next, branch=y, post_weight=self.post_mlp)


def reference(x, y, gate, up, down, norms):
    """The same block in fp32 torch on the weights that were quantised."""
    def norm(v, w):
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-5) * w.float()

    x = x.float() + norm(y.float(), norms[0])
    u = norm(x, norms[1])
    h = torch.nn.functional.silu(u @ gate.float().t()) * (u @ up.float().t())
    x = x + norm(h @ down.float().t(), norms[2])
    return x, norm(x, norms[3])


def inputs(rows, d, ffn, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g, device="cuda")

    weights = [(r(ffn, d) / d ** 0.5).bfloat16(), (r(ffn, d) / d ** 0.5).bfloat16(), (r(d, ffn) / ffn ** 0.5).bfloat16()]
    norms = [(1 + 0.1 * r(d)).bfloat16() for _ in range(4)]
    return r(rows, d).bfloat16(), r(rows, d).bfloat16(), weights, norms


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=128)
    ap.add_argument("--d", type=int, default=3072)
    ap.add_argument("--ffn", type=int, default=8192)
    ap.add_argument("--fmt", choices=("nvfp4", "mxfp4"), default="nvfp4")
    a = ap.parse_args()
    x, y, weights, norms = inputs(a.rows, a.d, a.ffn)
    mlp = Mlp(*weights, norms, a.fmt)
    z, v = mlp(x, y)
    zr, vr = reference(x, y, *weights, norms)
    for name, got, want in (("stream", z, zr), ("next input", v, vr)):
        print(f"{name}: relative difference from fp32 weights and activations "
              f"{float((got.float() - want).norm() / want.norm()):.4f}")
    # the five launches as one graph
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        mlp(x, y)
        with torch.cuda.graph(graph, stream=side):
            mlp(x, y)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    start.record()
    for _ in range(50):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"{a.rows} rows, {a.d} wide, MLP {a.ffn}, {a.fmt}: {start.elapsed_time(end) / 50 * 1e3:.1f} us a block")
    if wq.wq_get_device_error() != wq.WQ_OK:
        raise SystemExit("a bounded device-side wait ran out")


if __name__ == "__main__":
    main()
