"""The attention half of a decoder block of examples/: its calls together, each against its fp64 definition on what the
call before it gave."""
import os
import sys

import numpy as np
import pytest
import torch

import weight_only_bit_w4a16_gb300 as wq
from oracle import heads as ref
from test_gpu_prefix_attention import compare, f64

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decoder_attention as ex  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sequences,prefix", [(1, 70), (5, 300), (40, 130)])
def test_steps_of_a_block(sequences, prefix):
    """Three steps: the new keys and values are in the cache, and the attention is that of the cache it leaves."""
    D, heads, kv, d = 128, 8, 2, 256
    block = ex.Attention(d, heads, kv, D, prefix, sequences, 96, page=32, seed=sequences)
    g = torch.Generator(device="cuda").manual_seed(5)
    lens = torch.randint(1, 80, (sequences,), generator=g, device="cuda").int()
    x = torch.randn(sequences, d, generator=g, device="cuda").bfloat16()
    for step in range(3):
        before = f64(block.cache.k)
        y, a = block(x, lens)
        torch.cuda.synchronize()
        assert wq.wq_get_device_error() == wq.WQ_OK
        # the projection's heads again, by the same calls
        _, u = wq.block_norm(x, block.norm)
        qkv = wq.gemm_prepacked(u, block.qkv, workspace="auto").view(sequences, -1, D)
        q, k, v = qkv.split((heads, kv, kv), dim=1)
        at = (lens - 1).cpu().numpy()
        pos = at + prefix
        freq = [500000.0 ** -(i / (D // 2)) for i in range(D // 2)]
        tables = block.tables.cpu().numpy()
        kc, vc = f64(block.cache.k), f64(block.cache.v)
        want = ref.rotate(ref.head_norm(f64(k), f64(block.k_norm), None, "rms", 1e-6), [pos], freq, [0] * (D // 2), "halves")
        changed = np.zeros(kc.shape[:2], dtype=bool)
        for b in range(sequences):
            page, slot = tables[b, at[b] // 32], at[b] % 32
            changed[page, slot] = True
            assert (np.abs(kc[page, slot] - want[b]) <= 2.0 ** -8 * np.abs(want[b]) + 2.0 ** -16).all()
            assert (vc[page, slot] == f64(v)[b]).all()
        assert (kc[~changed] == before[~changed]).all()
        q2, _ = wq.head_rope(q, k, table=block.table, positions=lens - 1 + prefix, q_weight=block.q_norm,
                             k_weight=block.k_norm)
        starts = np.arange(sequences + 1)
        compare(a, None, ref.attention(f64(q2), kc, vc, tables, lens.tolist(), block.prefix_pages.cpu().numpy(), prefix,
                                       starts, D ** -0.5))
        # the output projection on the attention's own output, and the residual
        want = wq.gemm_prepacked(a.view(sequences, -1), block.o, workspace="auto", out_dtype="fp32").double() + x.double()
        assert ((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -16 * (want.abs() + x.double().abs())).all()
        x, lens = y, lens + 1


def test_a_step_as_a_graph():
    """A captured step follows new inputs and lengths."""
    block = ex.Attention(256, 8, 2, 128, 200, 9, 64, page=16, seed=3)
    x = torch.randn(9, 256, device="cuda").bfloat16()
    lens = torch.full((9,), 10, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        block(x, lens)
        with torch.cuda.graph(graph, stream=side):
            y, a = block(x, lens)
    torch.cuda.synchronize()
    for step in range(3):
        x.copy_(torch.randn(9, 256, device="cuda"))
        lens += 7
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone(), a.clone()
        want = block(x, lens)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
