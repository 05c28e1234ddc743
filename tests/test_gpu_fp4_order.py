"""Calls whose inputs the call before them on the stream writes, launched back
to back: the kernels start under their predecessor, so a load that ran ahead
of its completion would read what was there before.  The same calls with a
synchronisation after each one give the expected bits; every buffer is
overwritten with NaN patterns before a chain, so a value left by an earlier
chain does not pass for the right one."""
import pytest
import torch

import weight_only_bit_w4a16_gb300 as wq

pytestmark = pytest.mark.gpu

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


class Chain:
    """Calls on buffers of their own: same() runs them once with a synchronisation after each call and then, several
    times, without any."""

    def __init__(self):
        self.calls, self.bufs = [], []

    def buf(self, shape, dtype):
        t = torch.empty(shape, dtype=dtype, device="cuda")
        self.bufs.append(t)
        return t

    def add(self, call):
        self.calls.append(call)

    def run(self, sync):
        for t in self.bufs:
            t.view(-1).view(U8).fill_(0xFF)
        torch.cuda.synchronize()
        for c in self.calls:
            c()
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return [t.view(-1).view(U8).clone() for t in self.bufs]

    def same(self, times=6):
        want = self.run(True)
        for _ in range(times):
            assert all(torch.equal(a, b) for a, b in zip(want, self.run(False)))
        assert wq.wq_get_device_error() == wq.WQ_OK


def tiled(c, rows, K, fmt):
    return c.buf((rows, K // 2), U8), c.buf(wq.wq_fp4_scale_bytes(rows, K, wq.FORMATS[fmt], wq.WQ_SCALES_TILED), U8)


def weights(n, N, K, fmt, seed):
    g = torch.Generator().manual_seed(seed)
    return [wq.quantize(torch.randn(N, K, generator=g).cuda() / K ** 0.5, fmt) for _ in range(n)]


@pytest.mark.parametrize("fmt,scaled", [("nvfp4", False), ("nvfp4", True), ("mxfp4", False)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("off", [0, 3])
@pytest.mark.parametrize("M", [4, 300])
def test_quantise_what_the_product_before_wrote(fmt, scaled, dtype, off, M):
    """gemm_fp4 -> quantize -> gemm_fp4 ..., x aligned and not; the tensor scale, too, is the output of the call right
    before the quantisation."""
    d, N = 512, 512 + 32
    W = weights(3, N, d, fmt, M)
    one = [wq.quantize(torch.full((1, 32), v, device="cuda"), fmt) for v in (0.02, 0.5)]
    c = Chain()
    x = torch.randn(M, N, generator=torch.Generator().manual_seed(M)).to(dtype).cuda()
    for i in range(9):
        t = None
        if scaled:
            t = c.buf((1, 1), F32)
            c.add(lambda t=t, i=i: wq.gemm_fp4(one[0], one[1] if i % 2 else one[0], out=t))
        q, y, v = tiled(c, M, d, fmt), c.buf((M, N), dtype), c.buf((M, d), BF16)
        c.add(lambda x=x, q=q, v=v, t=t: wq.quantize(x[:, off:off + d], fmt, out=q, values=v,
                                                      scale=None if t is None else t.view(1)))
        c.add(lambda q=q, y=y, t=t, i=i: wq.gemm_fp4(
            wq.Fp4(*q, M, d, fmt, scale=None if t is None else t.view(1)), W[i % 3], out=y))
        x = y
    c.same()


@pytest.mark.parametrize("M,N,pair,split", [(4, 512, None, None), (40, 520, None, None), (300, 512, "128", "1"),
                                            (300, 516, "128", "1"), (300, 512, "64", "2")])
def test_epilogue_of_what_the_calls_before_wrote(M, N, pair, split, monkeypatch):
    """Bias, residual and both tensor scales of a product are written by the calls just before it."""
    if pair:
        monkeypatch.setenv("WQ_FP4_PAIR", pair)
        monkeypatch.setenv("WQ_FP4_SPLIT", split)
    d, fmt = 512, "nvfp4"
    W = weights(2, N, d, fmt, N)
    one = wq.quantize(torch.full((1, d), 0.05, device="cuda"), fmt)
    g = torch.Generator().manual_seed(N)
    rows, vec = torch.randn(M, N, generator=g).to(BF16).cuda(), torch.randn(1, N, generator=g).to(BF16).cuda()
    a = wq.quantize(torch.randn(M, d, generator=g).cuda(), fmt)
    c = Chain()
    for i in range(6):
        ta, tb = c.buf((1, 1), F32), c.buf((1, 1), F32)
        res, bias, y = c.buf((M, N), BF16), c.buf((1, N), BF16), c.buf((M, N), BF16)
        c.add(lambda t=ta: wq.gemm_fp4(one, one, out=t))
        c.add(lambda t=tb: wq.gemm_fp4(one, one, out=t))
        c.add(lambda bias=bias: wq.block_norm(vec, None, out=bias))
        c.add(lambda res=res, rows=rows: wq.block_norm(rows, None, out=res))
        c.add(lambda ta=ta, tb=tb, res=res, bias=bias, y=y, w=W[i % 2]: wq.gemm_fp4(
            wq.Fp4(a.packed, a.scales, M, d, fmt, scale=ta.view(1)), wq.Fp4(w.packed, w.scales, N, d, fmt, scale=tb.view(1)),
            out=y, bias=bias.view(N), residual=res))
        rows = y
    c.same()


@pytest.mark.parametrize("rows,d", [(3, 512), (20, 16416), (9600, 1056)])
def test_norms_of_what_the_calls_before_wrote(rows, d):
    """The tensor scale of a norm's 4-bit output and its inputs are written by the calls just before it."""
    fmt = "nvfp4"
    one = wq.quantize(torch.full((1, 32), 0.1, device="cuda"), fmt)
    x = torch.randn(rows, d, generator=torch.Generator().manual_seed(d)).to(BF16).cuda()
    c = Chain()
    for i in range(3):
        u, xo, q, t = c.buf((rows, d), BF16), c.buf((rows, d), BF16), tiled(c, rows, d, fmt), c.buf((1, 1), F32)
        c.add(lambda x=x, u=u: wq.block_norm(x, None, out=u))
        c.add(lambda t=t: wq.gemm_fp4(one, one, out=t))
        c.add(lambda x=x, u=u, xo=xo, q=q, t=t: wq.block_norm(x, None, branch=u, x_out=xo, out=q, fmt=fmt, scale=t.view(1)))
        x = xo
    c.same(3)
