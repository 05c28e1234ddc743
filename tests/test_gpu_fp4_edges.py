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
