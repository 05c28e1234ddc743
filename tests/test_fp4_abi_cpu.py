"""The 4-bit entry points' argument checks on a machine without a GPU: every
refusal happens before anything reaches CUDA."""
import ctypes

import pytest

import weight_only_bit_w4a16_gb300 as wq
from oracle import fp4

FAKE = 0x10000   # aligned, never dereferenced
OK, INV, UNS, ALN = wq.WQ_OK, wq.WQ_ERR_INVALID_ARG, wq.WQ_ERR_UNSUPPORTED, wq.WQ_ERR_ALIGN


def test_scale_bytes():
    import numpy as np
    for fmt, code in (("nvfp4", 0), ("mxfp4", 1)):
        for rows, K in ((1, 32), (128, 64), (129, 96), (300, 1056)):
            G = K // fp4.GROUP[fmt]
            assert wq.wq_fp4_scale_bytes(rows, K, code, wq.WQ_SCALES_ROWS) == rows * G
            assert wq.wq_fp4_scale_bytes(rows, K, code, wq.WQ_SCALES_TILED) == fp4.tile(
                np.zeros((rows, G), dtype=np.uint8)).size
            for layout in wq.LAYOUTS:
                assert wq._fp4_scale_bytes(rows, K, fmt, layout) == wq.wq_fp4_scale_bytes(rows, K, code,
                                                                                          wq.LAYOUTS[layout])
    for bad in ((0, 32, 0, 0), (4, 0, 0, 0), (4, 48, 0, 0), (4, 64, 2, 0), (4, 64, 0, 2), (-1, 64, 0, 0)):
        assert wq.wq_fp4_scale_bytes(*bad) == 0


@pytest.mark.parametrize("args,expect", [
    # x, x_type, ldx, rows, K, format, tensor_scale, packed, scales, layout, values
    ((FAKE, 0, 64, 0, 64, 0, None, FAKE, FAKE, 1, None), OK),            # no rows
    ((FAKE, 0, 0, 4, 0, 0, None, FAKE, FAKE, 1, None), OK),              # no columns
    ((FAKE, 0, 64, -1, 64, 0, None, FAKE, FAKE, 1, None), INV),
    ((FAKE, 2, 64, 4, 64, 0, None, FAKE, FAKE, 1, None), INV),           # type
    ((FAKE, 0, 63, 4, 64, 0, None, FAKE, FAKE, 1, None), INV),           # stride below K
    ((FAKE, 0, 64, 4, 64, 3, None, FAKE, FAKE, 1, None), INV),           # format
    ((FAKE, 0, 64, 4, 64, 2, None, FAKE, FAKE, 1, None), UNS),           # int4
    ((FAKE, 0, 64, 4, 64, 0x100, None, FAKE, FAKE, 1, None), INV),       # a flag is not a format
    ((FAKE, 0, 64, 4, 48, 0, None, FAKE, FAKE, 1, None), UNS),           # K % 32
    ((FAKE, 0, 64, 4, 64, 1, FAKE, FAKE, FAKE, 1, None), UNS),           # MXFP4 has no tensor scale
    ((FAKE, 0, 64, 4, 64, 0, None, FAKE, FAKE, 2, None), INV),           # layout
    ((None, 0, 64, 4, 64, 0, None, FAKE, FAKE, 1, None), INV),
    ((FAKE, 0, 64, 4, 64, 0, None, None, FAKE, 1, None), INV),
    ((FAKE, 0, 64, 4, 64, 0, None, FAKE, None, 1, None), INV),
    ((FAKE + 1, 0, 64, 4, 64, 0, None, FAKE, FAKE, 1, None), ALN),
    ((FAKE + 2, 1, 64, 4, 64, 0, None, FAKE, FAKE, 1, None), ALN),       # fp32 elements
    ((FAKE, 0, 64, 4, 64, 0, FAKE + 2, FAKE, FAKE, 1, None), ALN),
    ((FAKE, 0, 64, 4, 64, 0, None, FAKE + 8, FAKE, 1, None), ALN),
    ((FAKE, 0, 64, 4, 64, 0, None, FAKE, FAKE + 8, 1, None), ALN),       # tiled scales
    ((FAKE, 0, 64, 4, 64, 0, None, FAKE, FAKE, 1, FAKE + 8), ALN),       # values
])
def test_quantize_checks(args, expect):
    assert wq.wq_fp4_quantize(*args, None) == expect


@pytest.mark.parametrize("args,expect", [
    ((FAKE, FAKE, 0, 64, 0), OK), ((FAKE, FAKE, 4, 0, 0), OK), ((None, FAKE, 4, 64, 0), INV),
    ((FAKE, None, 4, 64, 0), INV), ((FAKE, FAKE + 8, 4, 64, 0), ALN), ((FAKE, FAKE, 4, 48, 0), UNS),
    ((FAKE, FAKE, 4, 64, 2), UNS), ((FAKE, FAKE, 4, -64, 0), INV),
])
def test_tile_scales_checks(args, expect):
    assert wq.wq_fp4_tile_scales(*args, None) == expect


def norm(**kw):
    base = dict(rows=4, d=64, kind=0, post=0, x=FAKE, ldx=64, x_type=0, branch_type=0, branch=FAKE, ldb=64, gate=None,
                gate_rows=0, eps=1e-5, residual_scale=1.0, branch_scale=1.0, weight=FAKE, x_out=FAKE, ldxo=64,
                out=FAKE, ldo=64, out_type=wq.WQ_NORM_OUT_BF16)
    base.update(kw)
    return wq.wq_block_norm(ctypes.byref(wq.wq_norm(**base)), None)


FP4 = dict(out_type=wq.WQ_NORM_OUT_NVFP4, out_scales=FAKE, out_scale_layout=1)


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=0), OK), (dict(d=0, ldx=0, ldb=0, ldxo=0, ldo=0), OK),
    (dict(rows=-1), INV), (dict(d=-1), INV), (dict(kind=2), INV), (dict(post=2), INV), (dict(x_type=2), INV),
    (dict(branch_type=-1), INV), (dict(out_type=5), INV), (dict(out_type=-1), INV),
    (dict(branch=None, post=1), INV), (dict(branch=None, gate=FAKE, gate_rows=1), INV),
    (dict(post_weight=FAKE), INV), (dict(post_bias=FAKE), INV),
    (dict(gate=FAKE, gate_rows=0), INV), (dict(gate=FAKE, gate_rows=3), INV), (dict(gate=FAKE, gate_rows=8), INV),
    (dict(x=None), INV), (dict(out=None), INV), (dict(out_type=0, x_out=None), INV),
    (dict(ldx=63), INV), (dict(ldb=63), INV), (dict(ldxo=63), INV), (dict(ldo=63), INV),
    (dict(x=FAKE + 1), ALN), (dict(x=FAKE + 2, x_type=1), ALN), (dict(branch=FAKE + 1), ALN),
    (dict(gate=FAKE + 1, gate_rows=1), ALN), (dict(weight=FAKE + 1), ALN), (dict(bias=FAKE + 1), ALN),
    (dict(x_out=FAKE + 1), ALN), (dict(out=FAKE + 1), ALN), (dict(out=FAKE + 2, out_type=wq.WQ_NORM_OUT_F32), ALN),
    (dict(FP4, d=48), UNS), (dict(FP4, out_scales=None), INV), (dict(FP4, out_scale_layout=2), INV),
    (dict(FP4, out=FAKE + 8), ALN), (dict(FP4, out_scales=FAKE + 8), ALN), (dict(FP4, out_tensor_scale=FAKE + 2), ALN),
    (dict(FP4, out_type=wq.WQ_NORM_OUT_MXFP4, out_tensor_scale=FAKE), UNS),
])
def test_block_norm_checks(kw, expect):
    assert norm(**kw) == expect


def test_block_norm_null():
    assert wq.wq_block_norm(None, None) == INV


def test_tensor_helpers_refuse_cpu_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        wq.quantize(x, "nvfp4")
    with pytest.raises(ValueError):
        wq.block_norm(x, None)
    with pytest.raises(ValueError):
        wq.fp4_operand(torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 4), dtype=torch.uint8), "nvfp4")


def mm(*args, epi=None, path=0):
    return wq.wq_gemm_fp4(*args, epi, None, path)


@pytest.mark.parametrize("change,expect", [
    # arguments: a_packed, a_scales, a_t, b_packed, b_scales, b_t, C, M, N, K, format
    ({7: 0}, OK), ({8: 0}, OK), ({7: -1}, INV), ({8: -1}, INV), ({9: -32}, INV), ({9: 48}, UNS),
    ({10: 2}, UNS), ({10: 3}, INV), ({10: 0x200}, INV), ({0: None}, INV), ({1: None}, INV), ({3: None}, INV),
    ({4: None}, INV), ({6: None}, INV), ({0: FAKE + 8}, ALN), ({1: FAKE + 8}, ALN), ({3: FAKE + 8}, ALN),
    ({4: FAKE + 8}, ALN), ({6: FAKE + 8}, ALN), ({2: FAKE + 2}, ALN), ({5: FAKE + 2}, ALN),
    ({2: FAKE, 10: 1}, UNS), ({5: FAKE, 10: 1}, UNS),
])
def test_gemm_fp4_checks(change, expect):
    args = [FAKE, FAKE, None, FAKE, FAKE, None, FAKE, 4, 32, 64, 0]
    for i, v in change.items():
        args[i] = v
    assert mm(*args) == expect


def test_gemm_fp4_path_and_epilogue_checks():
    args = [FAKE, FAKE, None, FAKE, FAKE, None, FAKE, 4, 24, 64, 0]
    assert mm(*args, path=wq.WQ_PATH_GEMV) == UNS
    assert mm(*args, path=9) == INV and mm(*args, path=0x400) == INV
    assert mm(*args, epi=ctypes.byref(wq.wq_epilogue(None, None, 1))) == UNS   # N = 24
    assert mm(*args, epi=ctypes.byref(wq.wq_epilogue(None, None, 2))) == INV
    assert mm(*args, epi=ctypes.byref(wq.wq_epilogue(FAKE + 1, None, 0))) == ALN
    args[7] = 0
    assert mm(*args, path=wq.WQ_PATH_TC | wq.WQ_LAUNCH_OVERLAP | wq.WQ_LAUNCH_INPUTS_READY) == OK


def test_packed_norm_struct_is_the_ctypes_struct():
    """block_norm packs wq_norm with the struct module: same size, same bytes."""
    assert wq._NORM_STRUCT.size == ctypes.sizeof(wq.wq_norm)
    vals = list(range(1, 28))
    n = wq.wq_norm(**{f: v for (f, _), v in zip(wq.wq_norm._fields_, vals)})
    assert bytes(n) == wq._NORM_STRUCT.pack(*vals)


def test_packed_quant_and_gemm_structs_are_the_ctypes_structs():
    assert wq._QUANT_STRUCT.size == ctypes.sizeof(wq.wq_fp4_quant)
    assert bytes(wq.wq_fp4_quant(*range(1, 12))) == wq._QUANT_STRUCT.pack(*range(1, 12))
    assert wq._GEMM_STRUCT.size == ctypes.sizeof(wq.wq_fp4_gemm)
    g = wq.wq_fp4_gemm(*range(1, 12), wq.wq_epilogue(12, 13, 1), 15)
    assert bytes(g) == wq._GEMM_STRUCT.pack(*range(1, 14), 1, 15)


def test_null_structs():
    assert wq.lib().wq_fp4_quantize(None, None) == INV
    assert wq.lib().wq_gemm_fp4(None, None) == INV
