"""Sizes at the end of the 32-bit range are refused by the host, before anything
reaches CUDA: past 2^31 - 65536 the kernels' indices could wrap."""
import ctypes

import pytest

import weight_only_bit_w4a16_gb300 as wq

FAKE = 0x10000   # aligned, never dereferenced
UNS = wq.WQ_ERR_UNSUPPORTED
END = 2 ** 31 - 1
MAX = 2 ** 31 - 65536


@pytest.mark.parametrize("rows,d", [(1, END), (END, 1), (END, 8), (1, MAX + 1), (MAX + 1, 32), (2, END - 8191)])
@pytest.mark.parametrize("out_type", [wq.WQ_NORM_OUT_NONE, wq.WQ_NORM_OUT_BF16, wq.WQ_NORM_OUT_F32])
def test_norms(rows, d, out_type):
    n = wq.wq_norm(rows=rows, d=d, x=FAKE, ldx=d, x_out=FAKE, ldxo=d, out=FAKE, ldo=d, out_type=out_type,
                   residual_scale=1.0, eps=1e-5)
    assert wq.wq_block_norm(ctypes.byref(n), None) == UNS


@pytest.mark.parametrize("rows,d", [(1, END - 31), (MAX + 1, 32)])
def test_norms_with_4_bit_output(rows, d):
    n = wq.wq_norm(rows=rows, d=d, x=FAKE, ldx=d, out=FAKE, out_type=wq.WQ_NORM_OUT_NVFP4, out_scales=FAKE,
                   out_scale_layout=1, residual_scale=1.0, eps=1e-5)
    assert wq.wq_block_norm(ctypes.byref(n), None) == UNS


@pytest.mark.parametrize("M,N,K", [(1, END, 0), (END, 1, 0), (17, END, 0), (1, END, 32), (END, 1, 32), (1, 1, END - 31),
                                   (MAX + 1, 16, 0), (16, MAX + 1, 0)])
def test_products(M, N, K):
    assert wq.wq_gemm_fp4(FAKE, FAKE, None, FAKE, FAKE, None, FAKE, M, N, K, 0, None, None, 0) == UNS
