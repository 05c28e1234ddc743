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


# -- weights that are written on the stream, then read ahead two calls later ------------------
def overlap_chain(c, kind, fmt, write, A, N, K, ready):
    """write(W) -> a product with WQ_LAUNCH_OVERLAP on other weights -> one on the weights just written: the caller's
    promise, that the preceding kernel does not write the weights, holds for both."""
    other = wq.quantize(torch.randn(64, K, generator=torch.Generator().manual_seed(1)).cuda(), fmt,
                        layout="tiled" if kind == "gemm_fp4" else "rows")
    small = wq.quantize(A, fmt) if kind == "gemm_fp4" else A
    torch.cuda.synchronize()
    for _ in range(4):
        layout = wq.WQ_SCALES_TILED if kind == "gemm_fp4" else wq.WQ_SCALES_ROWS
        p, s = c.buf((N, K // 2), U8), c.buf(wq.wq_fp4_scale_bytes(N, K, wq.FORMATS[fmt], layout), U8)
        y0, y1 = c.buf((A.shape[0], 64), F32), c.buf((A.shape[0], N), F32)
        write(c, p, s, "tiled" if kind == "gemm_fp4" else "rows")
        if kind == "gemm_fp4":
            B = wq.Fp4(p, s, N, K, fmt)
            # (a W4A16 call between: it starts its dependents before its predecessor has completed)
            gw = wq.quantize(torch.randn(64, K, generator=torch.Generator().manual_seed(2)).cuda(), fmt, layout="rows")
            c.add(lambda y0=y0, gw=gw: wq.gemm(A, gw.packed, gw.scales, None, fmt, out=y0, out_dtype="fp32",
                                               overlap=True, inputs_ready=ready))
            c.add(lambda B=B, y1=y1: wq.gemm_fp4(small, B, out=y1, overlap=True))
        else:
            G = K // (16 if fmt == "nvfp4" else 32)
            c.add(lambda y0=y0: wq.gemm(A, other.packed, other.scales, None, fmt, out=y0, out_dtype="fp32",
                                        overlap=True, inputs_ready=ready))
            c.add(lambda p=p, s=s, y1=y1, G=G: wq.gemm(A, p, s.view(N, G), None, fmt, out=y1, out_dtype="fp32",
                                                       overlap=True, inputs_ready=ready))
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["gemm", "gemm_fp4"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("N,K", [(64, 512), (8192, 3072), (20000, 512)])
@pytest.mark.parametrize("ready", [False, True])
@pytest.mark.parametrize("M", [1, 16])
def test_quantised_weights_read_ahead_two_calls_later(kind, fmt, N, K, ready, M):
    g = torch.Generator(device="cuda").manual_seed(N)
    W = torch.randn(N, K, generator=g, device="cuda")
    A = torch.randn(M, K, generator=g, device="cuda").to(BF16)
    c = Chain()
    overlap_chain(c, kind, fmt, lambda c, p, s, layout: c.add(lambda: wq.quantize(W, fmt, out=(p, s), layout=layout)),
                  A, N, K, ready)
    c.same(20)


@pytest.mark.parametrize("kind", ["gemm", "gemm_fp4"])
@pytest.mark.parametrize("N,K", [(64, 512), (8192, 3072), (300, 16416), (20000, 64)])
def test_normed_weights_read_ahead_two_calls_later(kind, N, K):
    """The same for 4-bit codes that a norm writes, by each of its kernels."""
    fmt = "nvfp4"
    g = torch.Generator(device="cuda").manual_seed(N)
    W = torch.randn(N, K, generator=g, device="cuda").to(BF16)
    A = torch.randn(4, K, generator=g, device="cuda").to(BF16)
    c = Chain()
    overlap_chain(c, kind, fmt,
                  lambda c, p, s, layout: c.add(lambda: wq.block_norm(W, None, fmt=fmt, layout=layout, out=(p, s))),
                  A, N, K, False)
    c.same(20)


@pytest.mark.parametrize("M,N,K,pair,split", [(4, 600, 1024, "0", None), (4, 20000, 1024, "0", None),
                                              (300, 500, 1024, "128", "1"), (100, 200, 2048, "64", "3")])
@pytest.mark.parametrize("overlap", [False, True])
def test_waits_do_not_count_the_call_before(M, N, K, pair, split, overlap, monkeypatch):
    """A product behind a long call that lets it start early: the bounds of its waits begin when that call has
    completed.  The call before is a norm of one row, which one SM takes over a millisecond for; the bound of the
    epilogue's wait is 0.3 ms (WQ_FP4_WAIT_NS), many times what the product takes."""
    monkeypatch.setenv("WQ_FP4_PAIR", pair)
    if split:
        monkeypatch.setenv("WQ_FP4_SPLIT", split)
    g = torch.Generator(device="cuda").manual_seed(M)
    A = wq.quantize(torch.randn(M, K, generator=g, device="cuda"), "nvfp4")
    B = wq.quantize(torch.randn(N, K, generator=g, device="cuda"), "nvfp4")
    want = wq.gemm_fp4(A, B, out_dtype="fp32")
    x = torch.ones((1, 1 << 26), dtype=BF16, device="cuda")
    u, got = torch.empty_like(x), torch.empty_like(want)
    wq.block_norm(x, None, out=u)
    torch.cuda.synchronize()
    monkeypatch.setenv("WQ_FP4_WAIT_NS", "300000")
    wq.gemm_fp4(A, B, out=got)
    torch.cuda.synchronize()
    assert wq.wq_get_device_error() == wq.WQ_OK and torch.equal(got, want)
    got.zero_()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    wq.block_norm(x, None, out=u)
    wq.gemm_fp4(A, B, out=got, overlap=overlap)
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) > 1.0
    assert wq.wq_get_device_error() == wq.WQ_OK and torch.equal(got, want)
