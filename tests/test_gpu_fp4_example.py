"""The 4-bit decoder MLP of examples/: the block's calls together.

Against fp32 weights and activations the difference is that of 4-bit
quantisation: e2m1 rounds a value by at most a quarter of itself, uniformly
distributed some 0.1 of its size (rms), in both operands of both products, so
their outputs are within 0.3, and the stream, to which the normed output adds
one part in about three, within 0.25.  Against the same quantisation done step
by step in fp64 it is rounding alone."""
import os
import sys

import numpy as np
import pytest
import torch

import weight_only_bit_w4a16_gb300 as wq
from oracle import fp4

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decoder_mlp_fp4 as ex  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("rows", [1, 5, 128, 300])
def test_block_is_near_the_fp32_block(fmt, rows):
    x, y, weights, norms = ex.inputs(rows, 512, 1024)
    z, v = ex.Mlp(*weights, norms, fmt)(x, y)
    zr, vr = ex.reference(x, y, *weights, norms)
    assert wq.wq_get_device_error() == wq.WQ_OK
    for got, want in ((z, zr), (v, vr)):
        assert float((got.float() - want).norm() / want.norm()) < 0.25


def test_block_step_by_step():
    """Each call of the block on the fp64 oracle, fed with the call before's own outputs."""
    fmt, rows, d, ffn = "nvfp4", 37, 256, 512
    x, y, (gate, up, down), norms = ex.inputs(rows, d, ffn)
    h64 = lambda t: t.double().cpu().numpy()
    x1, u = wq.block_norm(x, norms[1], branch=y, post_weight=norms[0], fmt=fmt, layout="rows")
    wx, wu = fp4.block_norm(h64(x), h64(y), None, h64(norms[1]), None, True, h64(norms[0]), None, 1.0, 1.0, "rms", 1e-5)
    assert (np.abs(h64(x1) - wx) <= 2.0 ** -8 * np.abs(wx) + 2.0 ** -16).all()
    uv = fp4.values(fp4.unpack(u.packed.cpu().numpy()), u.scales.cpu().numpy(), fmt)
    # 4-bit u: within half a step of e2m1's widest spacing (2 of 6) and the scale's rounding (1 / 16) of its group's top
    top = np.repeat(np.abs(wu).reshape(rows, -1, 16).max(-1), 16, axis=1)
    assert (np.abs(uv - wu) <= top * (1 / 6 + 1 / 16 + 0.01)).all()
    W = ex.interleave(gate, up).contiguous()
    wv = torch.empty_like(W)
    w4 = wq.quantize(W, fmt, values=wv)
    u4 = wq.fp4_operand(u.packed, u.scales, fmt)
    h = wq.gemm_fp4(u4, w4, gated=True, out_dtype="fp32")
    C, S = fp4.product(uv, h64(wv))
    import oracle
    want, T = oracle.epilogue(C, S, None, None, True, "fp32")
    assert (np.abs(h64(h) - want) <= T).all()
