"""Pins of the fp64 oracle of the 4-bit operators (CPU): hand-worked groups,
torch's own 8-bit casts, brute force, and the tiled scale order."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import fp4


def test_e4m3_values_are_torch_s():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, fp4.E4M3)


def test_nearest_e4m3_is_torch_s_cast():
    rng = np.random.default_rng(0)
    v = np.exp(rng.uniform(math.log(1e-4), math.log(440), 20000)).astype(np.float32)
    mid = ((fp4.E4M3[:-1] + fp4.E4M3[1:]) / 2).astype(np.float32)   # exact ties
    v = np.concatenate([v, mid, fp4.E4M3.astype(np.float32)])
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp4.nearest(v, fp4.E4M3), want)


@pytest.mark.parametrize("v,code", [(0.25, 0), (0.26, 1), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6),
                                    (5.01, 7), (6.0, 7), (100.0, 7), (0.0, 0)])
def test_e2m1_ties_go_to_the_even_code(v, code):
    assert fp4.nearest(np.array([v]), fp4.E2M1)[0] == code


def test_nvfp4_group_by_hand():
    """max 12: s = 12 / 6 = 2 (e4m3 0x40); 12 -> 6 (code 7), -1 -> -0.5 (code 9), 5 -> 2.5, the tie of 2 and 3,
    which goes to 2 (code 4); 7 -> 3.5, the tie of 3 and 4, to 4 (code 6)."""
    x = np.zeros((1, 16))
    x[0, :4] = [12, -1, 5, 7]
    code, byte = fp4.quantize(x, "nvfp4")
    assert byte.tolist() == [[0x40]] and code[0, :5].tolist() == [7, 9, 4, 6, 0]
    assert fp4.values(code, byte, "nvfp4")[0, :4].tolist() == [12, -1, 4, 8]


def test_mxfp4_group_by_hand():
    """max 12: floor(log2 12) = 3, E = 1 (byte 128); 12 / 2 = 6 (code 7); 15 / 2 = 7.5 would saturate."""
    x = np.zeros((1, 32))
    x[0, :3] = [12, -1, 15]
    code, byte = fp4.quantize(x, "mxfp4")
    assert byte.tolist() == [[128]] and code[0, :3].tolist() == [7, 9, 7]
    x[:] = 0
    assert fp4.quantize(x, "mxfp4")[1].tolist() == [[0]]
    x[0, 5] = 2.0 ** -140
    assert fp4.quantize(x, "mxfp4")[1].tolist() == [[0]]


def test_not_finite_groups_and_saturation():
    x = np.ones((2, 32))
    x[0, 3], x[1, 20] = np.inf, np.nan
    code, byte = fp4.quantize(x, "nvfp4")
    assert byte.tolist() == [[0x7F, fp4.nearest(1 / 6, fp4.E4M3)], [fp4.nearest(1 / 6, fp4.E4M3), 0x7F]]
    assert not code[0, :16].any() and np.isnan(fp4.values(code, byte, "nvfp4")[1, 16:]).all()
    assert fp4.quantize(x, "mxfp4")[1].tolist() == [[0xFF], [0xFF]]
    big = np.full((1, 16), 1e6)
    code, byte = fp4.quantize(big, "nvfp4")
    assert byte[0, 0] == 126 and (code == 7).all()


def test_quantize_by_brute_force_in_rationals():
    rng = np.random.default_rng(1)
    x = (rng.normal(size=(3, 32)) * 3).astype(np.float32)
    for fmt in ("nvfp4", "mxfp4"):
        code, byte = fp4.quantize(x, fmt)
        step = np.repeat(fp4.step_of(byte, fmt), fp4.GROUP[fmt], axis=1)
        for i in np.ndindex(x.shape):
            q = abs(Fraction(float(x[i]))) / Fraction(float(step[i]))
            best = min(range(8), key=lambda c: (abs(Fraction(float(fp4.E2M1[c])) - q), c % 2))
            assert code[i] & 7 == best and (code[i] >> 3) == (x[i] < 0)


def test_pack_and_tile_orders():
    code = np.arange(32, dtype=np.uint8).reshape(1, 32) % 16
    assert fp4.pack(code)[0, 0] == 0x10 and np.array_equal(fp4.unpack(fp4.pack(code)), code)
    byte = np.arange(130 * 6, dtype=np.int64).reshape(130, 6).astype(np.uint8)
    t = fp4.tile(byte)
    assert t.size == 2 * 2 * 512
    assert t[16 * 1 + 4 * 2 + 3] == byte[65, 3]            # row 65 = 2 * 32 + 1
    assert t[512 + 16 * 31 + 4 * 3 + 1] == byte[127, 5]    # second block of groups
    assert t[1024 + 16 * 1 + 0] == byte[129, 0]            # second block of rows
    assert t[512 + 2] == 0                                 # group 6 of row 0: none
    # the same by array reshapes
    full = np.zeros((256, 8), dtype=np.uint8)
    full[:130, :6] = byte
    assert np.array_equal(full.reshape(2, 4, 32, 2, 4).transpose(0, 3, 2, 1, 4).reshape(-1), t)


def test_norms_are_torch_s():
    rng = np.random.default_rng(2)
    x, b = rng.normal(size=(4, 24)), rng.normal(size=(4, 24))
    w, c = rng.normal(size=24), rng.normal(size=24)
    tx, tw, tc = torch.from_numpy(x), torch.from_numpy(w), torch.from_numpy(c)
    ln = torch.nn.functional.layer_norm(tx, (24,), tw, tc, 1e-5).numpy()
    assert np.allclose(fp4.norm(x, w, c, "layer", 1e-5), ln, rtol=1e-12, atol=1e-12)
    rms = torch.nn.functional.rms_norm(tx, (24,), tw, 1e-5).numpy()
    assert np.allclose(fp4.norm(x, w, None, "rms", 1e-5), rms, rtol=1e-12, atol=1e-12)
    g = rng.normal(size=(2, 24))
    xn, u = fp4.block_norm(x, b, g, w, None, True, w, c, 0.5, 2.0, "rms", 1e-6)
    by_hand = 0.5 * x + 2.0 * np.concatenate([g[:1], g[:1], g[1:], g[1:]]) * fp4.norm(b, w, c, "rms", 1e-6)
    assert np.allclose(xn, by_hand) and np.allclose(u, fp4.norm(by_hand, w, None, "rms", 1e-6))
