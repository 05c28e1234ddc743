"""wq_fp4_quantize and wq_fp4_tile_scales against the fp64 oracle.

bf16 input without a tensor scale: codes and scales are the exactly rounded
ones (a bf16 value over an e4m3 scale, or over 6, is a tie or further than
2^-12 of itself from one; the kernel's quotients are within 2^-22).  fp32 input
or a tensor scale: the quotients a / (6 t) and x / (s t) carry a relative error
of at most 2^-21 (two roundings of the divisor and two of the quotient, 2^-24
each, and the reciprocal's), so a scale or code may be the neighbour where the
exact quotient lies within that of a tie."""
import numpy as np
import pytest
import torch

import weight_only_bit_w4a16_gb300 as wq
from oracle import fp4

pytestmark = pytest.mark.gpu

REL = 2.0 ** -21


def host(t):
    return t.cpu().numpy()


def run(x, fmt, layout="rows", scale=None, values=False):
    rows, K = x.shape
    G = K // fp4.GROUP[fmt]
    nb = wq.wq_fp4_scale_bytes(rows, K, wq.FORMATS[fmt], wq.LAYOUTS[layout])
    packed = torch.full((rows, K // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((nb,), 0xEE, dtype=torch.uint8, device="cuda")
    vals = torch.full((rows, K), 777.0, dtype=torch.bfloat16, device="cuda") if values else None
    q = wq.quantize(x, fmt, scale=scale, out=(packed, scales), values=vals, layout=layout)
    torch.cuda.synchronize()
    assert q.packed is packed and q.K == K and q.rows == rows
    s = host(scales)
    return fp4.unpack(host(packed)), s.reshape(rows, G) if layout == "rows" else s, vals


def same_codes(a, b):
    """Equal up to the sign of a zero."""
    return np.array_equal(np.where(a == 8, 0, a), np.where(b == 8, 0, b))


def bf16_rows(rows, K, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g) * scale
    x[:, ::7] *= 20
    return x.to(torch.bfloat16).cuda()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("rows,K", [(1, 32), (1, 64), (2, 96), (3, 1056), (127, 160), (129, 2080), (300, 512)])
def test_bf16_is_exact(fmt, rows, K):
    x = bf16_rows(rows, K, rows + K)
    code, byte = fp4.quantize(host(x.double()), fmt)
    c, s, v = run(x, fmt, values=True)
    assert np.array_equal(s, byte)
    assert same_codes(c, code)
    assert np.array_equal(host(v.double()), fp4.values(code, byte, fmt))   # exact in bf16


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_every_bf16_value(fmt):
    """All bf16 patterns, each as the largest of its group and each divided by scales of every mantissa: exact ties
    of every kind are among them.  Groups with an infinity or a NaN get the NaN scale and codes 0."""
    bits = np.arange(65536, dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16).reshape(-1, 1).repeat(1, 32)
    with np.errstate(all="ignore"):
        m = torch.tensor([1.0, 0.5, 0.25, 0.75, 0.125, 0.375, 0.625, 0.875, 0.3, 0.7, 0.9, 0.01, 0.0, -1.0, -0.5, -0.2])
        x = (x.double() * torch.cat([m, m]).double()).to(torch.bfloat16).cuda()
    h = host(x.double())
    code, byte = fp4.quantize(h, fmt)
    c, s, v = run(x, fmt, values=True)
    assert np.array_equal(s, byte)
    assert same_codes(c, code)
    want = fp4.values(code, byte, fmt)
    got = host(v.double())
    assert np.array_equal(np.isnan(got), np.isnan(want))
    # values below bf16's normal range round; all others are exact
    ok = np.isfinite(want) & (np.abs(want) >= 2.0 ** -126)
    assert np.array_equal(got[ok], want[ok])
    small = np.isfinite(want) & ~ok
    assert (np.abs(got[small] - want[small]) <= 2.0 ** -134).all()


def test_every_tie_of_every_scale():
    """x = (midpoint) * s for every e4m3 scale s whose products are bf16 numbers, with 6 s in the group."""
    rows = []
    for s in fp4.E4M3[1:]:
        mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * s
        rows.append(np.concatenate([[6 * s], mids, -mids, [0.0]]))
    x = np.array(rows)
    x = np.concatenate([x, x], axis=1)
    t = torch.from_numpy(x).to(torch.bfloat16)
    assert np.array_equal(t.double().numpy(), x)
    code, byte = fp4.quantize(x, "nvfp4")
    assert np.array_equal(byte[:, 0], np.arange(1, 127))
    c, s, _ = run(t.cuda(), "nvfp4")
    assert np.array_equal(s, byte) and same_codes(c, code)


def allowed(q, table):
    return fp4.nearest(q * (1 - REL), table), fp4.nearest(q * (1 + REL), table)


@pytest.mark.parametrize("rows,K,t,pad", [(1, 32, None, 0), (65, 1056, None, 5), (200, 512, 3e-4, 0), (33, 64, 7.7, 3),
                                          (40, 96, 1e-30, 0), (17, 2080, 0.01, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_tensor_scale_and_fp32(rows, K, t, pad, dtype):
    g = torch.Generator().manual_seed(rows)
    wide = torch.randn(rows, K + pad, generator=g) * (1.0 if t is None else 900.0 * t)
    if dtype == "bf16":
        wide = wide.to(torch.bfloat16)
    x = wide.cuda()[:, :K]
    scale = None if t is None else torch.tensor([t], dtype=torch.float32, device="cuda")
    tv = 1.0 if t is None else float(scale.double().item())
    h = host(x.double())
    c, s, v = run(x, "nvfp4", scale=scale, values=True)
    a = np.abs(h).reshape(rows, -1, 16).max(-1)
    lo, hi = allowed(a / (6 * tv), fp4.E4M3)
    assert ((s == lo) | (s == hi)).all()
    step = np.repeat(fp4.step_of(s, "nvfp4", tv), 16, axis=1)   # the kernel's own scales
    q = np.divide(np.abs(h), step, out=np.zeros_like(h), where=step > 0)
    lo, hi = allowed(q, fp4.E2M1)
    assert (((c & 7) == lo) | ((c & 7) == hi)).all()
    assert (((c >> 3) == np.signbit(h)) | ((c & 7) == 0)).all()
    want = fp4.values(c, s, "nvfp4", tv)
    assert (np.abs(host(v.double()) - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23) + 2.0 ** -134).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,off", [(8, 0), (3, 0), (16, 8), (5, 1)])
def test_strided_rows(fmt, dtype, pad, off):
    """A column slice of a wider tensor, aligned or not, gives what a copy of it gives."""
    wide = (torch.randn(70, 96 + pad + off, generator=torch.Generator().manual_seed(3)) * 2).to(dtype).cuda()
    x = wide[:, off:off + 96]
    c, s, _ = run(x, fmt)
    c2, s2, _ = run(x.contiguous(), fmt)
    assert np.array_equal(c, c2) and np.array_equal(s, s2)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("rows,K", [(1, 32), (5, 96), (128, 64), (129, 160), (257, 1056)])
def test_tiled_scales(fmt, rows, K):
    """The tiled order holds the same bytes, groups past the last one 0; wq_fp4_tile_scales makes the same of
    row-major scales, rows past the last one included."""
    x = bf16_rows(rows, K, 5)
    _, s, _ = run(x, fmt)
    c, tiled, _ = run(x, fmt, layout="tiled")
    want = fp4.tile(s)
    G = K // fp4.GROUP[fmt]
    live = fp4.tile(np.ones((rows, -(-G // 4) * 4), dtype=np.uint8)) == 1
    assert np.array_equal(tiled[live], want[live])
    packed = torch.zeros((rows, K // 2), dtype=torch.uint8, device="cuda")
    o = wq.fp4_operand(packed, torch.from_numpy(s.copy()).cuda(), fmt)
    torch.cuda.synchronize()
    assert np.array_equal(host(o.scales), want) and o.packed is packed


def test_tile_scales_drops_the_nvfp4_sign():
    s = torch.randint(0, 256, (40, 8), dtype=torch.uint8, generator=torch.Generator().manual_seed(1)).cuda()
    packed = torch.zeros((40, 64), dtype=torch.uint8, device="cuda")
    assert np.array_equal(host(wq.fp4_operand(packed, s, "nvfp4").scales), fp4.tile(host(s) & 0x7F))
    packed = torch.zeros((40, 128), dtype=torch.uint8, device="cuda")
    assert np.array_equal(host(wq.fp4_operand(packed, s, "mxfp4").scales), fp4.tile(host(s)))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_rows_layout_feeds_the_w4a16_calls(fmt):
    """Weights quantised here are weights of wq.dequant, wq.gemm and wq.prepack."""
    W = bf16_rows(48, 256, 8, 0.5)
    values = torch.empty_like(W)
    q = wq.quantize(W, fmt, values=values, layout="rows")
    assert torch.equal(wq.dequant(q.packed, q.scales, None, fmt), values)
    A = bf16_rows(3, 256, 9)
    C = wq.gemm(A, q.packed, q.scales, None, fmt, out_dtype="fp32")
    P = wq.gemm_prepacked(A, wq.prepack(q.packed, q.scales, None, fmt), out_dtype="fp32")
    ref, S = fp4.product(host(A.double()), host(values.double()))
    for c in (C, P):
        assert (np.abs(host(c.double()) - ref) <= 1e-3 * S + 1e-6).all()


def test_another_stream_and_empty():
    x = bf16_rows(64, 128, 2)
    want, ws, _ = run(x, "nvfp4")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q = wq.quantize(x, "nvfp4", layout="rows")
    q2 = wq.quantize(x, "nvfp4", layout="rows", stream=side)
    side.synchronize()
    assert np.array_equal(fp4.unpack(host(q.packed)), want) and np.array_equal(host(q2.scales), ws)
    for rows, K in ((0, 64), (3, 0)):
        q = wq.quantize(torch.empty((rows, K), dtype=torch.bfloat16, device="cuda"), "mxfp4")
        assert q.packed.shape == (rows, K // 2)


def test_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    one = torch.ones(1, device="cuda")
    with pytest.raises(ValueError):
        wq.quantize(x, "int4")
    with pytest.raises(ValueError):
        wq.quantize(x.half(), "nvfp4")
    with pytest.raises(ValueError):
        wq.quantize(x.t(), "nvfp4")
    with pytest.raises(ValueError):
        wq.quantize(x, "nvfp4", scale=torch.ones(1))
    with pytest.raises(ValueError):
        wq.quantize(x, "nvfp4", layout="columns")
    with pytest.raises(ValueError):
        wq.quantize(x, "nvfp4", out=(torch.empty(4, dtype=torch.uint8, device="cuda"),) * 2)
    with pytest.raises(ValueError):
        wq.quantize(x, "nvfp4", values=torch.empty((4, 32), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(wq.WQError):
        wq.quantize(x[:, :48], "nvfp4")
    with pytest.raises(wq.WQError):
        wq.quantize(x, "mxfp4", scale=one)
