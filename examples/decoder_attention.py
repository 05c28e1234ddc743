"""A decoder block's attention half on 4-bit weights, for a batch that shares a prefix, end to end on one GPU:

    u   = norm(x)                          wq.block_norm
    qkv = u . [q k v]^T                    wq.gemm_prepacked, one int4 weight of all heads
    q, k = norm, rotation; k, v -> cache   wq.head_rope, one kernel
    a   = attention(q, prefix and own)     wq.prefix_attention, the prefix read once for the batch
    x'  = x + a . o^T                      wq.gemm_prepacked with the residual

One step takes one new token of each sequence (or several, checked together).  The heads are those of the 3B decoder
whose projections the library's benchmark sweeps, with fewer of them.

    python examples/decoder_attention.py --sequences 32 --prefix 4096
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_bit_w4a16_gb300 as wq  # noqa: E402


def int4_weight(g, n, k):
    """Random int4 weights of groups of 128, prepacked (codes, zero points and scales as a checkpoint holds them)."""
    packed = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    zeros = torch.randint(6, 10, (n, k // 128), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((0.5 + torch.rand(n, k // 128, generator=g, device="cuda")) / (4.6 * k ** 0.5)).bfloat16()
    return wq.prepack(packed, scales, zeros, "int4")


class Attention:
    """A block's weights, and a paged cache with a prefix in it."""

    def __init__(self, d, heads, kv_heads, head_dim, prefix, sequences, longest, page=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.head_dim, self.page = heads, kv_heads, head_dim, page
        self.qkv = int4_weight(g, (heads + 2 * kv_heads) * head_dim, d)
        self.o = int4_weight(g, d, heads * head_dim)
        self.norm, self.q_norm, self.k_norm = ((1 + 0.1 * torch.randn(n, generator=g, device="cuda")).bfloat16()
                                               for n in (d, head_dim, head_dim))
        self.table = wq.rope_table(head_dim, theta=500000.0)
        self.prefix = prefix
        each, shared = (longest + page - 1) // page, (prefix + page - 1) // page
        pages = shared + sequences * each
        store = torch.randn(2, pages, page, kv_heads, head_dim, generator=g, device="cuda").bfloat16()
        self.cache = wq.KVCache(store[0], store[1])
        order = torch.randperm(pages, generator=g, device="cuda").int()
        self.prefix_pages = order[:shared].contiguous()
        self.tables = order[shared:].view(sequences, each).contiguous()
        torch.cuda.synchronize()   # the weights are written before a call may read them ahead

    def __call__(self, x, lens):
        """x: the residual stream of the new tokens (sequences, d); lens: each sequence's own keys, the new one's among
        them (int32).  Returns (x', the attention's output)."""
        tokens, D = x.shape[0], self.head_dim
        at = lens - 1
        slots = (self.tables.gather(1, (at // self.page).long().unsqueeze(1))[:, 0] * self.page + at % self.page).int()
        _, u = wq.block_norm(x, self.norm)
        qkv = wq.gemm_prepacked(u, self.qkv, workspace="auto").view(tokens, -1, D)
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), dim=1)
        q, _ = wq.head_rope(q, k, v, table=self.table, positions=at + self.prefix, q_weight=self.q_norm,
                            k_weight=self.k_norm, cache=self.cache, slots=slots)
        a = wq.prefix_attention(q, self.cache, lens, self.tables, prefix_pages=self.prefix_pages, prefix_len=self.prefix)
        return wq.gemm_prepacked(a.view(tokens, -1), self.o, residual=x, workspace="auto"), a


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--sequences", type=int, default=32)
    ap.add_argument("--prefix", type=int, default=4096)
    ap.add_argument("--own", type=int, default=500)
    ap.add_argument("--d", type=int, default=2048)
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--kv-heads", type=int, default=4)
    a = ap.parse_args()
    block = Attention(a.d, a.heads, a.kv_heads, 128, a.prefix, a.sequences, a.own)
    x = torch.randn(a.sequences, a.d, device="cuda").bfloat16()
    lens = torch.randint(1, a.own + 1, (a.sequences,), device="cuda").int()
    block(x, lens)
    # the step as one graph
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        block(x, lens)
        with torch.cuda.graph(graph, stream=side):
            block(x, lens)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    start.record()
    for _ in range(50):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"{a.sequences} sequences on a prefix of {a.prefix}, {a.heads} / {a.kv_heads} heads: "
          f"{start.elapsed_time(end) / 50 * 1e3:.1f} us a step")
    if wq.wq_get_device_error() != wq.WQ_OK:
        raise SystemExit("a bounded device-side wait ran out")


if __name__ == "__main__":
    main()
