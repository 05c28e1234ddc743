"""wq_gemm_fp4 against the fp64 product of the values its operands stand for.

Tolerance: the library's gate, |C - C_exact| <= 1e-3 S + 1e-6 with
S = sum |a b| (fp32 output; bf16 adds 2^-8 |C_exact|), as for wq_gemm; and for
fp32 output a tighter one of the arithmetic itself: every product of two codes
and two scales is exact in fp32, and the sum of K products in chunks of 64
loses at most 2^-23 of S a chunk (truncated alignment included), so
|C - C_exact| <= (K / 64 + 2) 2^-23 S + 2^-126."""
import numpy as np
import pytest
import torch

import oracle
import weight_only_bit_w4a16_gb300 as wq
from oracle import fp4

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Operand:
    """Random codes and scales: the values (fp64, host) and the library's handle."""

    def __init__(self, rows, K, fmt, seed, t=None):
        rng = np.random.default_rng(seed)
        G = K // fp4.GROUP[fmt]
        self.code = rng.integers(0, 16, size=(rows, K)).astype(np.uint8)
        if fmt == "nvfp4":
            self.byte = rng.integers(0x20, 0x50, size=(rows, G)).astype(np.uint8)
            self.byte[rng.random((rows, G)) < 0.05] = 0
            self.byte[rng.random((rows, G)) < 0.05] = 3          # subnormal scales
        else:
            self.byte = rng.integers(120, 133, size=(rows, G)).astype(np.uint8)
        self.scale = None if t is None else torch.tensor([t], dtype=torch.float32, device="cuda")
        tv = 1.0 if t is None else float(np.float32(t))
        self.values = fp4.values(self.code, self.byte, fmt, tv)
        self.h = wq.fp4_operand(dev(fp4.pack(self.code)), dev(self.byte), fmt, scale=self.scale)


def check(C, ref, S, K, what=""):
    got = C.double().cpu().numpy()
    out = "fp32" if C.dtype == torch.float32 else "bf16"
    err = np.abs(got - ref)
    tol = oracle.tolerance(ref, S, out)
    if out == "fp32":
        tol = np.minimum(tol, (K / 64 + 2) * 2.0 ** -23 * S + 2.0 ** -126)
    assert (err <= tol).all(), f"{what}: {int((err > tol).sum())}/{err.size}, worst {np.max(err - tol):.3e}"


def product(M, N, K, fmt, out="fp32", seed=0, ta=None, tb=None):
    A, B = Operand(M, K, fmt, seed, ta), Operand(N, K, fmt, seed + 1, tb)
    C = wq.gemm_fp4(A.h, B.h, out_dtype=out)
    torch.cuda.synchronize()
    assert wq.wq_get_device_error() == wq.WQ_OK
    ref, S = fp4.product(A.values, B.values)
    check(C, ref, S, K, f"{fmt} {M}x{N}x{K}")
    return C


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 128, 129, 200, 257, 520])
@pytest.mark.parametrize("N,K", [(256, 256), (136, 96), (1001, 2080), (16, 32), (1, 64), (300, 1056)])
def test_shapes(fmt, M, N, K):
    product(M, N, K, fmt, "fp32" if (M + N) % 2 else "bf16", seed=M)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("K", list(range(32, 577, 32)) + [1024, 4096, 4128])
@pytest.mark.parametrize("M", [3, 140])
def test_every_partial_step(fmt, K, M):
    product(M, 144, K, fmt, seed=K)


@pytest.mark.parametrize("M,N", [(40, 3000), (3000, 40), (1025, 2049), (64, 8192), (700, 5000)])
def test_many_tiles(M, N):
    product(M, N, 544, "nvfp4", "bf16", seed=N)


@pytest.mark.parametrize("M", [5, 100])
def test_tensor_scales(M):
    for ta, tb in ((0.03, None), (None, 4.0), (1e-3, 0.7)):
        A, B = Operand(M, 320, "nvfp4", 1, ta), Operand(96, 320, "nvfp4", 2, tb)
        C = wq.gemm_fp4(A.h, B.h, out_dtype="fp32")
        ref, S = fp4.product(A.values, B.values)
        err = np.abs(C.double().cpu().numpy() - ref)
        assert (err <= (320 / 64 + 5) * 2.0 ** -23 * S).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M", [1, 9, 64, 100, 300])
@pytest.mark.parametrize("parts", ["bias", "residual", "gated", "all"])
@pytest.mark.parametrize("N", [160, 1008])
def test_epilogues(fmt, M, parts, N):
    K = 672
    A, B = Operand(M, K, fmt, M), Operand(N, K, fmt, M + 7)
    rng = np.random.default_rng(M)
    gated = parts in ("gated", "all")
    from weight_only_bit_w4a16_gb300 import synth
    bias = synth.bf16_bits(rng.normal(size=N).astype(np.float32)) if parts in ("bias", "all") else None
    res = synth.bf16_bits(rng.normal(size=(M, N // 2 if gated else N)).astype(np.float32)) \
        if parts in ("residual", "all") else None
    tb = lambda b: None if b is None else dev(b.view(np.int16)).view(torch.bfloat16)
    for out in ("fp32", "bf16"):
        C = wq.gemm_fp4(A.h, B.h, out_dtype=out, bias=tb(bias), residual=tb(res), gated=gated)
        torch.cuda.synchronize()
        ref, S = fp4.product(A.values, B.values)
        want, T = oracle.epilogue(ref, S, bias, res, gated, out)
        err = np.abs(C.double().cpu().numpy() - want)
        assert (err <= T).all(), f"{int((err > T).sum())}/{err.size}, worst {np.max(err - T):.3e}"


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_one_hot_rows_pick_weights(fmt):
    """Row m of A holds one 1.0 at k = m: C is the transposed weights, exactly."""
    K, N = 256, 72
    B = Operand(N, K, fmt, 4)
    code = np.zeros((K, K), dtype=np.uint8)
    code[np.arange(K), np.arange(K)] = 2
    byte = np.full((K, K // fp4.GROUP[fmt]), 0x38 if fmt == "nvfp4" else 127, dtype=np.uint8)
    for M in (K, 40):
        A = wq.fp4_operand(dev(fp4.pack(code[:M])), dev(byte[:M]), fmt)
        C = wq.gemm_fp4(A, B.h, out_dtype="fp32")
        assert np.array_equal(C.double().cpu().numpy(), B.values.T[:M])


def test_scales_of_every_exponent():
    """e8m0 scales far from 1 in both operands: exact powers of two."""
    K, fmt = 64, "mxfp4"
    A, B = Operand(24, K, fmt, 1), Operand(40, K, fmt, 2)
    for ea, eb in ((20, 230), (200, 60), (127, 127), (70, 70)):
        a, b = np.full((24, 2), ea, dtype=np.uint8), np.full((40, 2), eb, dtype=np.uint8)
        C = wq.gemm_fp4(wq.fp4_operand(A.h.packed, dev(a), fmt), wq.fp4_operand(B.h.packed, dev(b), fmt),
                        out_dtype="fp32")
        ref, _ = fp4.product(fp4.values(A.code, a, fmt), fp4.values(B.code, b, fmt))
        assert np.array_equal(C.double().cpu().numpy(), ref)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M", [6, 150])
def test_nan_scales_stay_in_their_row_and_column(fmt, M):
    K, N = 288, 200
    A, B = Operand(M, K, fmt, 1), Operand(N, K, fmt, 2)
    clean = wq.gemm_fp4(A.h, B.h, out_dtype="fp32")
    nan = 0x7F if fmt == "nvfp4" else 0xFF
    a, b = A.byte.copy(), B.byte.copy()
    a[3, -1], b[7, 0] = nan, nan
    C = wq.gemm_fp4(wq.fp4_operand(A.h.packed, dev(a), fmt), wq.fp4_operand(B.h.packed, dev(b), fmt), out_dtype="fp32")
    bad = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    bad[3], bad[:, 7] = True, True
    assert C[bad].isnan().all() and torch.equal(C[~bad], clean[~bad])


@pytest.mark.parametrize("M", [3, 130])
def test_unwritten_scale_rows_do_not_matter(M):
    """Tiled scale bytes of rows past the last one may be anything."""
    K, N, fmt = 160, 130, "nvfp4"
    A, B = Operand(M, K, fmt, 1), Operand(N, K, fmt, 2)
    want = wq.gemm_fp4(A.h, B.h)
    for o, rows in ((A, M), (B, N)):
        live = dev(fp4.tile(np.ones((-(-rows // 128) * 128, 12), dtype=np.uint8) *
                            (np.arange(-(-rows // 128) * 128) < rows)[:, None].astype(np.uint8))).bool()
        o.h.scales[~live] = 0x7F
    assert torch.equal(wq.gemm_fp4(A.h, B.h), want)


def test_quantised_activations_chain():
    """quantize -> gemm_fp4 equals the product of the quantised values."""
    x = torch.randn(37, 512, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    w = torch.randn(96, 512, generator=torch.Generator().manual_seed(1)).cuda()
    for fmt in ("nvfp4", "mxfp4"):
        xv, wv = torch.empty_like(x), torch.empty((96, 512), dtype=torch.bfloat16, device="cuda")
        C = wq.gemm_fp4(wq.quantize(x, fmt, values=xv), wq.quantize(w, fmt, values=wv), out_dtype="fp32")
        ref, S = fp4.product(xv.double().cpu().numpy(), wv.double().cpu().numpy())
        check(C, ref, S, 512, fmt)


def test_empty_and_no_k():
    for M, N in ((0, 32), (5, 0)):
        A = wq.quantize(torch.ones((M, 64), dtype=torch.bfloat16, device="cuda"), "nvfp4")
        B = wq.quantize(torch.ones((N, 64), dtype=torch.bfloat16, device="cuda"), "nvfp4")
        assert wq.gemm_fp4(A, B).shape == (M, N)
    for M in (3, 100):   # K = 0: the epilogue of zero
        A = wq.quantize(torch.ones((M, 0), dtype=torch.bfloat16, device="cuda"), "mxfp4")
        B = wq.quantize(torch.ones((40, 0), dtype=torch.bfloat16, device="cuda"), "mxfp4")
        bias = torch.randn(40, device="cuda").to(torch.bfloat16)
        C = wq.gemm_fp4(A, B, bias=bias)
        assert torch.equal(C, bias[None].expand(M, 40))
    assert wq.wq_get_device_error() == wq.WQ_OK


def test_repeatable_and_on_another_stream():
    A, B = Operand(48, 4096, "nvfp4", 1), Operand(640, 4096, "nvfp4", 2)
    want = wq.gemm_fp4(A.h, B.h, out_dtype="fp32")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [wq.gemm_fp4(A.h, B.h, out_dtype="fp32") for _ in range(5)]
    side.synchronize()
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g, want)


def test_refusals():
    A, B = Operand(4, 64, "nvfp4", 1).h, Operand(8, 64, "nvfp4", 2).h
    X = Operand(8, 64, "mxfp4", 2).h
    bf = torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda")
    rows = wq.Fp4(A.packed, A.scales, 4, 64, "nvfp4", layout="rows")
    short = wq.Fp4(A.packed, A.scales[:16], 4, 64, "nvfp4")
    for a, b, kw in ((A, X, {}), (rows, B, {}), (short, B, {}), (A, B, dict(out=bf[:2])), (A, B, dict(bias=bf[0, :4])),
                     (A, B, dict(residual=bf.float())), (A, B, dict(out=bf.half()))):
        with pytest.raises(ValueError):
            wq.gemm_fp4(a, b, **kw)
    with pytest.raises(wq.WQError):
        wq.gemm_fp4(A, B, gated=True)          # N = 8 is no multiple of 16
    X.scale = torch.ones(1, device="cuda")
    with pytest.raises(wq.WQError):
        wq.gemm_fp4(Operand(4, 64, "mxfp4", 1).h, X)


# -- the kernel of CTA pairs, forced (WQ_FP4_PAIR: a tile's columns) ------------------
@pytest.mark.parametrize("bn", [64, 128, 192, 256])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N,K", [(1, 64, 32), (130, 264, 96), (256, 256, 256), (257, 512, 1056), (600, 1000, 2080),
                                   (520, 776, 64), (1500, 3000, 320)])
def test_pairs(bn, fmt, M, N, K, monkeypatch):
    monkeypatch.setenv("WQ_FP4_PAIR", str(bn))
    product(M, N, K, fmt, "fp32" if (M + K) % 64 else "bf16", seed=bn)


@pytest.mark.parametrize("bn,out", [(128, "bf16"), (256, "bf16"), (64, "fp32"), (128, "fp32"), (256, "fp32")])
@pytest.mark.parametrize("parts", ["bias", "residual", "gated", "all"])
@pytest.mark.parametrize("N", [160, 1008, 2064])
def test_pair_epilogues(bn, out, parts, N, monkeypatch):
    monkeypatch.setenv("WQ_FP4_PAIR", str(bn))
    M, K, fmt = 300, 672, "nvfp4"
    A, B = Operand(M, K, fmt, M), Operand(N, K, fmt, M + 7)
    rng = np.random.default_rng(M)
    gated = parts in ("gated", "all")
    from weight_only_bit_w4a16_gb300 import synth
    bias = synth.bf16_bits(rng.normal(size=N).astype(np.float32)) if parts in ("bias", "all") else None
    res = synth.bf16_bits(rng.normal(size=(M, N // 2 if gated else N)).astype(np.float32)) \
        if parts in ("residual", "all") else None
    tb = lambda b: None if b is None else dev(b.view(np.int16)).view(torch.bfloat16)
    C = wq.gemm_fp4(A.h, B.h, out_dtype=out, bias=tb(bias), residual=tb(res), gated=gated)
    torch.cuda.synchronize()
    assert wq.wq_get_device_error() == wq.WQ_OK
    ref, S = fp4.product(A.values, B.values)
    want, T = oracle.epilogue(ref, S, bias, res, gated, out)
    err = np.abs(C.double().cpu().numpy() - want)
    assert (err <= T).all(), f"{int((err > T).sum())}/{err.size}, worst {np.max(err - T):.3e}"


@pytest.mark.parametrize("K", [256, 4096])
def test_pair_tiles_in_turn(K, monkeypatch):
    """More tiles than pairs: both accumulators in turn, with short and long k, the same bits as the other kernel's
    where the sums are exact (MXFP4 scales of 1)."""
    M, N, fmt = 2600, 3328, "mxfp4"
    A, B = Operand(M, K, fmt, 1), Operand(N, K, fmt, 2)
    one = lambda o: wq.fp4_operand(o.h.packed, torch.full_like(dev(o.byte), 127), fmt)
    A, B = one(A), one(B)
    monkeypatch.setenv("WQ_FP4_PAIR", "0")
    want = wq.gemm_fp4(A, B, out_dtype="fp32")
    for bn in (64, 128, 192, 256):
        monkeypatch.setenv("WQ_FP4_PAIR", str(bn))
        for _ in range(3):
            assert torch.equal(wq.gemm_fp4(A, B, out_dtype="fp32"), want)
    assert wq.wq_get_device_error() == wq.WQ_OK


# -- stages of a tile shared by 1 to 4 pairs (WQ_FP4_SPLIT) ---------------------------
@pytest.mark.parametrize("split", [1, 2, 3, 4])
@pytest.mark.parametrize("bn", [64, 128, 192, 256])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N,K", [(1, 64, 1024), (257, 264, 1056), (520, 777, 2080), (300, 129, 4096)])
def test_split_pairs(split, bn, fmt, M, N, K, monkeypatch):
    monkeypatch.setenv("WQ_FP4_PAIR", str(bn))
    monkeypatch.setenv("WQ_FP4_SPLIT", str(split))
    C = product(M, N, K, fmt, "fp32" if (M + N) % 2 else "bf16", seed=bn)
    A, B = Operand(M, K, fmt, bn), Operand(N, K, fmt, bn + 1)
    again = wq.gemm_fp4(A.h, B.h, out_dtype=C.dtype)
    assert torch.equal(C, again)          # a fixed order of summation


@pytest.mark.parametrize("split", [1, 3])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("parts", ["bias", "residual", "gated", "all"])
@pytest.mark.parametrize("N", [160, 1008, 272])
def test_split_epilogues(split, out, parts, N, monkeypatch):
    monkeypatch.setenv("WQ_FP4_PAIR", "128")
    monkeypatch.setenv("WQ_FP4_SPLIT", str(split))
    M, K, fmt = 300, 1440, "mxfp4"
    A, B = Operand(M, K, fmt, M), Operand(N, K, fmt, M + 7)
    rng = np.random.default_rng(M)
    gated = parts in ("gated", "all")
    from weight_only_bit_w4a16_gb300 import synth
    bias = synth.bf16_bits(rng.normal(size=N).astype(np.float32)) if parts in ("bias", "all") else None
    res = synth.bf16_bits(rng.normal(size=(M, N // 2 if gated else N)).astype(np.float32)) \
        if parts in ("residual", "all") else None
    tb = lambda b: None if b is None else dev(b.view(np.int16)).view(torch.bfloat16)
    C = wq.gemm_fp4(A.h, B.h, out_dtype=out, bias=tb(bias), residual=tb(res), gated=gated)
    torch.cuda.synchronize()
    assert wq.wq_get_device_error() == wq.WQ_OK
    ref, S = fp4.product(A.values, B.values)
    want, T = oracle.epilogue(ref, S, bias, res, gated, out)
    err = np.abs(C.double().cpu().numpy() - want)
    assert (err <= T).all(), f"{int((err > T).sum())}/{err.size}, worst {np.max(err - T):.3e}"


@pytest.mark.parametrize("M", [4, 40, 300])
@pytest.mark.parametrize("overlap", [False, True])
def test_chain_of_dependent_calls(M, overlap):
    """norm -> product -> norm -> product ..., each call's input the one before's output, gives what synchronised
    calls give: launches overlap, results do not."""
    d, N = 512, 512
    g = torch.Generator().manual_seed(M)
    W = [wq.quantize(torch.randn(N, d, generator=g).cuda() / 23, "nvfp4") for _ in range(3)]
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    x0 = torch.randn(M, d, generator=g).to(torch.bfloat16).cuda()

    def chain(sync):
        x, y, outs = x0, None, []
        for i in range(12):
            x, u = wq.block_norm(x, w, branch=y, fmt="nvfp4", x_out=torch.empty_like(x))
            y = wq.gemm_fp4(u, W[i % 3], overlap=overlap)
            if sync:
                torch.cuda.synchronize()
            outs.append((x, y))
        torch.cuda.synchronize()
        return outs

    torch.cuda.synchronize()
    want = chain(True)
    for _ in range(3):
        for (a, b), (c, e) in zip(want, chain(False)):
            assert torch.equal(a, c) and torch.equal(b, e)
    assert wq.wq_get_device_error() == wq.WQ_OK


@pytest.mark.parametrize("M,N,K,bn,split", [(4, 600, 1024, 0, 0), (4, 20000, 1024, 0, 0), (300, 500, 1024, 128, 1),
                                            (2600, 3328, 1024, 256, 1), (2600, 3328, 1024, 128, 1),
                                            (100, 200, 2048, 64, 3)])
def test_a_wait_that_runs_out(M, N, K, bn, split, monkeypatch):
    """The failure path, without a fault or a hang: with the epilogue's wait for its sums bounded at 0 ns
    (WQ_FP4_WAIT_NS, read at launch) every CTA's epilogue gives up at once; the copies and matrix instructions drain
    under their own bounds, the status comes back, and the next call is right."""
    A, B = Operand(M, K, "nvfp4", 1), Operand(N, K, "nvfp4", 2)
    monkeypatch.setenv("WQ_FP4_PAIR", str(bn))
    monkeypatch.setenv("WQ_FP4_SPLIT", str(split))
    assert wq.wq_get_device_error() == wq.WQ_OK
    want = wq.gemm_fp4(A.h, B.h, out_dtype="fp32")
    monkeypatch.setenv("WQ_FP4_WAIT_NS", "0")
    wq.gemm_fp4(A.h, B.h, out_dtype="fp32")
    torch.cuda.synchronize()
    assert wq.wq_get_device_error() == wq.WQ_ERR_DEVICE_TIMEOUT
    assert wq.wq_get_device_error() == wq.WQ_OK
    monkeypatch.delenv("WQ_FP4_WAIT_NS")
    for _ in range(2):
        assert torch.equal(wq.gemm_fp4(A.h, B.h, out_dtype="fp32"), want)
    assert wq.wq_get_device_error() == wq.WQ_OK
