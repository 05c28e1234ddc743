"""Values at the ends of the range in the 4-bit calls, against their formulas
in 64 bits.

Four ways through the product: rows_kernel with whole and with shared tiles,
pair_kernel with whole and with shared tiles."""
import numpy as np
import pytest
import torch

import weight_only_bit_w4a16_gb300 as wq
from oracle import fp4

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

#: (K, WQ_FP4_PAIR, WQ_FP4_SPLIT); M and N below give rows_kernel whole tiles for K = 32, shared ones for K = 2048
PATHS = {"rows": (32, "0", None), "rows shared": (2048, "0", None), "pair": (96, "128", "1"),
         "pair shared": (512, "128", "2")}


def path(name, monkeypatch):
    K, pair, split = PATHS[name]
    monkeypatch.setenv("WQ_FP4_PAIR", pair)
    if split:
        monkeypatch.setenv("WQ_FP4_SPLIT", split)
    return K


def pairs_of(gates, ups):
    """A bias of interleaved gate / up rows (groups of 8) that pairs every gate with every up, and the two."""
    g, u = (a.reshape(-1) for a in np.meshgrid(gates, ups, indexing="ij"))
    n = -(-len(g) // 8) * 8
    g, u = np.resize(g, n), np.resize(u, n)
    return np.stack((g.reshape(-1, 8), u.reshape(-1, 8)), axis=1).reshape(-1), g, u


@pytest.mark.parametrize("way", list(PATHS))
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("M", [3, 40])
def test_gates_of_every_size(way, out, M, monkeypatch):
    """silu(x) = x / (1 + e^-x) of gates from 2^-100 to the largest, infinite and NaN ones, times small and large ups:
    0 past the exponential's range, NaN of -inf (as the quotient is), +inf of +inf.

    The gate is the bias of a product of zeros.  Relative error below 2^-20 with fp32 output (2^-17 with bf16, which
    adds its own rounding, 2^-8).  Where the factor 1 / (1 + e^-x) leaves the normal range, below 2^-126, it may be
    taken for 0: from x = -87.3 on, where |x| 2^-126 is at most 89 2^-126 until the exponential itself overflows
    at -88.8, and the true value is below that too."""
    K = path(way, monkeypatch)
    mags = [2.0 ** -100, 1e-20, 0.01, 0.5, 1.0, 5.0, 17.0, 20.0, 60.0, 80.0, 85.0, 86.0, 86.5, 87.0, 87.5, 88.0, 88.5,
            89.0, 90.0, 100.0, 120.0, 200.0, 1e3, 1e5, 1e10, 1e20, 1e30, 1e37, 1e38, 3.3e38, np.inf]
    ups = [1.0, -0.75, 1e-20, 1e20, -1e20, 1e38, -3e38, 0.0]
    gates = torch.tensor(mags + [-m for m in mags] + [0.0, np.nan], dtype=F32).to(BF16).double().numpy()
    ups = torch.tensor(ups, dtype=F32).to(BF16).double().numpy()
    bias, g, u = pairs_of(gates, ups)
    N = len(bias)
    zero = lambda rows: wq.quantize(torch.zeros((rows, K), dtype=BF16, device="cuda"), "nvfp4")
    got = wq.gemm_fp4(zero(M), zero(N), out_dtype=out, bias=torch.from_numpy(bias).to(BF16).cuda(), gated=True)
    torch.cuda.synchronize()
    assert wq.wq_get_device_error() == wq.WQ_OK
    got = got.double().cpu().numpy()
    assert (got.view(np.int64) == got[:1].view(np.int64)).all()   # every row the same
    got = got[0]
    with np.errstate(all="ignore"):
        s = g / (1.0 + np.exp(-g))
        want = s * u
        big = float(torch.finfo(F32 if out == "fp32" else BF16).max)
        rel = 2.0 ** -20 if out == "fp32" else 2.0 ** -17
        tol = np.abs(u) * (rel * np.abs(s) + 89 * 2.0 ** -126) + 2.0 ** -148
        tol = tol + (0.0 if out == "fp32" else 2.0 ** -8 * np.abs(want) + 2.0 ** -133)
        over = np.isinf(want) | (np.abs(want) - tol > big)
        near = ~over & (np.abs(want) + tol > big)   # may round either way
        assert not near.any()
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[over], np.sign(want[over]) * np.inf)
        ok = ~over & ~np.isnan(want)
        bad = ok & ~(np.abs(got - want) <= tol)
    assert not bad.any(), [(g[i], u[i], got[i], want[i]) for i in np.flatnonzero(bad)[:5]]


REL = 2.0 ** -21   # of the quantiser's quotients (fp32 input, or a tensor scale)


def check_codes(x, packed, scales, t):
    """Codes and row-major scales of x (fp64) with the tensor scale t: the rounded ones, or, where the exact quotient
    is within REL of a tie, a neighbour.  Returns the codes."""
    c, s = fp4.unpack(packed.cpu().numpy()), scales.cpu().numpy().reshape(x.shape[0], -1)
    a = np.abs(x).reshape(x.shape[0], -1, 16).max(-1)
    near = lambda q, table: (fp4.nearest(q * (1 - REL), table), fp4.nearest(q * (1 + REL), table))
    lo, hi = near(a / (6 * t), fp4.E4M3)
    assert ((s == lo) | (s == hi)).all()
    step = np.repeat(fp4.step_of(s, "nvfp4", t), 16, axis=1)
    q = np.divide(np.abs(x), step, out=np.zeros_like(x), where=step > 0)
    lo, hi = near(q, fp4.E2M1)
    assert (((c & 7) == lo) | ((c & 7) == hi)).all()
    assert (((c >> 3) == np.signbit(x)) | ((c & 7) == 0)).all()
    return c


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("t", [2.0 ** -100, 1e-20, 1e-3, 1.0])
def test_codes_saturate_with_their_sign(dtype, off, t):
    """Values whose quotient by the step passes fp32's range, beside values of the same group that do not saturate,
    one that is zero and one that is minus zero."""
    tv = float(np.float32(t))
    step = 448.0 * tv
    big = [1e12, -1e12, 2e38, -2e38, 3.3e38, -3.3e38, 1e30, -1e25, 40 * step, -41 * step, 7 * step, -6 * step]
    small = [3 * step, -1.5 * step, 0.5 * step, -4 * step, 0.2 * step, -0.24 * step, 0.0, -0.0, 2 * step, -step]
    g = np.random.default_rng(3)
    rows = []
    for b in big:
        for _ in range(4):
            row = g.permutation(np.concatenate([g.choice(big, 8), g.choice(small, 16), [b] * 8]))
            rows.append(row)
        rows.append([b] * 32)
    wide = torch.zeros((len(rows), 32 + off), dtype=dtype)
    wide[:, off:] = torch.tensor(np.array(rows)).to(dtype)
    x = wide.cuda()[:, off:]
    h = x.double().cpu().numpy()
    v = torch.empty((len(rows), 32), dtype=BF16, device="cuda")
    q = wq.quantize(x, "nvfp4", scale=torch.tensor([t], dtype=F32, device="cuda"), values=v, layout="rows")
    c = check_codes(h, q.packed, q.scales, tv)
    want = fp4.values(c, q.scales.cpu().numpy(), "nvfp4", tv)
    assert (np.abs(v.double().cpu().numpy() - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23) + 2.0 ** -134).all()


@pytest.mark.parametrize("rows,d", [(5, 64), (4, 512), (3, 1024), (2, 16416), (9700, 1056)])
@pytest.mark.parametrize("t", [2.0 ** -100, 1e-3])
def test_normed_codes_saturate_with_their_sign(rows, d, t):
    """The 4-bit output of a norm whose weights take u from 1e-3 to 1e38, each of its kernels."""
    g = torch.Generator().manual_seed(d)
    x = torch.randn(rows, d, generator=g).to(BF16).cuda()
    w = torch.logspace(-3, 37.5, d)[torch.randperm(d, generator=g)].to(BF16).cuda()
    u = wq.block_norm(x, w, out_dtype="fp32")[1]
    scale = torch.tensor([t], dtype=F32, device="cuda")
    q = wq.block_norm(x, w, fmt="nvfp4", layout="rows", scale=scale)[1]
    p = wq.quantize(u, "nvfp4", layout="rows", scale=scale)
    assert torch.equal(q.packed, p.packed) and torch.equal(q.scales, p.scales)
    n = min(rows, 50)
    check_codes(u[:n].double().cpu().numpy(), q.packed[:n], q.scales[:n], float(np.float32(t)))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("off", [0, 1])
def test_tensor_scale_of_zero(dtype, off):
    """max |x| / (6 * 448) of an all-zero tensor is 0: its codes and scales are 0, what they stand for is 0, and a product
    with it is the epilogue of 0.  Codes of other tensors are 0 under it too, and nothing is NaN but a group that is
    not finite."""
    x = torch.zeros((20, 96 + off), dtype=dtype, device="cuda")[:, off:]
    t = (x.abs().amax().float() / (6 * 448)).reshape(1)
    v = torch.full((20, 96), 7.0, dtype=BF16, device="cuda")
    q = wq.quantize(x, "nvfp4", scale=t, values=v, layout="rows")
    assert not q.packed.any() and not q.scales.any() and torch.equal(v, torch.zeros_like(v))
    for rows, M in ((20, 5), (5, 300)):
        A = wq.quantize(torch.randn(M, 96, device="cuda").to(BF16), "nvfp4")
        B = wq.quantize(x[:rows], "nvfp4", scale=t)
        bias = torch.randn(rows, device="cuda").to(BF16)
        assert torch.equal(wq.gemm_fp4(A, B, bias=bias), bias[None].expand(M, rows))
        assert not wq.gemm_fp4(B, A, out_dtype="fp32").any()
    y = torch.randn(4, 96 + off, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()[:, off:]
    y[1, 40] = float("nan")
    v = torch.full((4, 96), 7.0, dtype=BF16, device="cuda")
    q = wq.quantize(y, "nvfp4", scale=t, values=v, layout="rows")
    assert not (fp4.unpack(q.packed.cpu().numpy()) & 7).any()
    bad = torch.zeros_like(v, dtype=torch.bool)
    bad[1, 32:48] = True
    assert torch.equal(v.isnan(), bad) and not v[~bad].any()
    assert torch.equal(q.scales.view(4, 6) == 0x7F, bad[:, ::16])


@pytest.mark.parametrize("rows,d", [(5, 64), (4, 512), (3, 1024), (2, 16416), (9700, 1056)])
def test_norm_with_a_tensor_scale_of_zero(rows, d):
    z = torch.zeros((rows, d), dtype=BF16, device="cuda")
    t = torch.zeros(1, device="cuda")
    q = wq.block_norm(z, None, branch=z, post=True, fmt="nvfp4", layout="rows", scale=t)[1]
    assert not q.packed.any() and not q.scales.any()


@pytest.mark.parametrize("way", list(PATHS))
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("ea,eb", [(-75, -75), (-100, -40), (-40, -100), (90, 90), (100, -100), (-100, 100), (60, 40)])
@pytest.mark.parametrize("size,ma,mb", [(1.0, 1.0, 1.0), (60.0, 1.7, 1.3)])
def test_tensor_scales_whose_product_leaves_the_range(way, out, gated, ea, eb, size, ma, mb, monkeypatch):
    """t_A t_B below fp32's normal range or past its end, while t_A t_B sum is in it; rows of zeros stay zeros.

    Tolerance: fp32 sums of K products, 2^-23 S for each chunk of 64 and four more roundings, 2^-148 where the result
    is subnormal; bf16 adds 2^-8.  Gated: the gates are so small, or so large, that silu(x) is x / 2 or x or 0 to within
    its own rounding, a factor of 2^-20 (2^-17) more."""
    K = path(way, monkeypatch)
    M, N = 20, 96
    g = torch.Generator().manual_seed(K)
    ta, tb = (float(np.float32(m * 2.0 ** e)) for m, e in ((ma, ea), (mb, eb)))
    a, b = ((size * torch.randn(r, K, generator=g)).to(BF16) for r in (M, N))
    a[3], b[8:16] = 0.0, 0.0
    av, bv = torch.empty((M, K), dtype=BF16, device="cuda"), torch.empty((N, K), dtype=BF16, device="cuda")
    A, B = wq.quantize(a.cuda(), "nvfp4", values=av), wq.quantize(b.cuda(), "nvfp4", values=bv)
    A.scale, B.scale = (torch.tensor([t], dtype=F32, device="cuda") for t in (ta, tb))
    got = wq.gemm_fp4(A, B, out_dtype=out, gated=gated)
    torch.cuda.synchronize()
    got = got.double().cpu().numpy()
    ref, S = fp4.product(av.double().cpu().numpy(), bv.double().cpu().numpy())
    f = ta * tb
    rel = (K / 64 + 5) * 2.0 ** -23
    big = 2.0 ** 128
    with np.errstate(all="ignore"):
        y, e = ref * f, S * f * rel + 2.0 ** -148
        y32 = np.where(np.abs(y) >= big, np.sign(y) * np.inf, y)   # the fp32 result before the gate
        if gated:
            v, w = y32.reshape(M, -1, 2, 8), e.reshape(M, -1, 2, 8)
            gate, up = (v[:, :, i].reshape(M, -1) for i in (0, 1))
            eg, eu = (w[:, :, i].reshape(M, -1) for i in (0, 1))
            s = gate / (1 + np.exp(-gate))
            y = s * up
            es = 1.1 * eg + np.abs(s) * (2.0 ** -20 if out == "fp32" else 2.0 ** -17) + 89 * 2.0 ** -126
            e = es * np.abs(up) + eu * np.abs(s) + es * eu + 2.0 ** -148
        if out == "bf16":
            e = e + 2.0 ** -8 * np.abs(y) + 2.0 ** -133
        nan = np.isnan(y)
        over = ~nan & (np.abs(y) - e > big)
        sure = ~nan & ~over & np.isfinite(e) & (np.abs(y) + e < big * (1 - 2.0 ** -9))
        assert np.isnan(got[nan]).all()
        assert np.array_equal(got[over], np.sign(y[over]) * np.inf)
        assert (np.abs(got[sure] - y[sure]) <= e[sure]).all()
    assert not got[3].any()
    if not gated:
        assert not got[:, 8:16].any()
