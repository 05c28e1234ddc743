"""The 4-bit operators in fp64 on the CPU, from their definitions: quantisation
to NVFP4 / MXFP4, the values of codes and scales, the product of two 4-bit
operands and the norms between two blocks.  Plain and slow; shares no code
with the library.

Rounding to a 4-bit or 8-bit float is a search in the sorted list of that
type's values, ties to the even code, so no arithmetic of the type itself is
repeated here."""
from __future__ import annotations

import numpy as np

GROUP = {"nvfp4": 16, "mxfp4": 32}

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3(b):
    e, m = b >> 3, b & 7
    return m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)


#: the finite values of e4m3 by their codes 0 .. 126
E4M3 = np.array([_e4m3(b) for b in range(127)])


def nearest(v, table):
    """Index of the entry of the sorted table nearest to each v >= 0, ties to
    the even index, values past the end to the last entry."""
    v = np.asarray(v, dtype=np.float64)
    hi = np.clip(np.searchsorted(table, v, side="left"), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = v - table[lo], table[hi] - v
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def scale_bytes(x, fmt, t=1.0):
    """The scale byte of each group of x (rows, K), and the value of a unit
    code under it (NaN for a group that is not finite)."""
    rows, K = x.shape
    g = np.abs(np.asarray(x, dtype=np.float64)).reshape(rows, K // GROUP[fmt], GROUP[fmt])
    bad = ~np.isfinite(g).all(-1)
    a = np.where(bad, 0.0, np.where(np.isfinite(g), g, 0.0).max(-1))
    if fmt == "nvfp4":
        byte = nearest(a / (6.0 * float(t)), E4M3)
        step = E4M3[byte] * float(t)
        byte = np.where(bad, 0x7F, byte)
    else:
        m, e = np.frexp(a)                    # a = m 2^e, m in [1/2, 1): floor(log2 a) = e - 1
        E = np.where(a > 0, np.maximum(e - 1 - 2, -127), -127)
        byte = np.where(bad, 0xFF, E + 127)
        step = np.exp2(E.astype(np.float64))
    return byte.astype(np.uint8), np.where(bad, np.nan, step)


def quantize(x, fmt, t=1.0):
    """(codes (rows, K), scale bytes) of x; the code of a value that rounds to
    zero has its sign."""
    byte, step = scale_bytes(x, fmt, t)
    s = np.repeat(step, GROUP[fmt], axis=1)
    ok = np.isfinite(s) & (s > 0)
    q = np.abs(np.where(ok, x, 0.0).astype(np.float64)) / np.where(ok, s, 1.0)
    code = nearest(q, E2M1) | np.where(np.signbit(x) & ok, 8, 0)
    return code.astype(np.uint8), byte


def pack(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    out = np.empty((packed.shape[0], 2 * packed.shape[1]), dtype=np.uint8)
    out[:, 0::2] = packed & 15
    out[:, 1::2] = packed >> 4
    return out


def step_of(byte, fmt, t=1.0):
    """The value of a unit code under each scale byte."""
    byte = np.asarray(byte)
    if fmt == "nvfp4":
        b = byte & 0x7F
        return np.where(b == 0x7F, np.nan, E4M3[np.minimum(b, 126)]) * float(t)
    return np.where(byte == 0xFF, np.nan, np.exp2(byte.astype(np.float64) - 127.0))


def values(code, byte, fmt, t=1.0):
    v = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]
    return v * np.repeat(step_of(byte, fmt, t), GROUP[fmt], axis=1)


def tile(byte):
    """Row-major scale bytes (rows, groups) in the tiled layout, byte by byte;
    every byte that belongs to no row and group is 0."""
    rows, G = byte.shape
    Gb = -(-G // 4)
    out = np.zeros(-(-rows // 128) * Gb * 512, dtype=np.uint8)
    for r in range(rows):
        for g in range(G):
            block = (r // 128) * Gb + g // 4
            out[512 * block + 16 * (r % 32) + 4 * ((r % 128) // 32) + g % 4] = byte[r, g]
    return out


def product(A, B):
    """C = A . B^T and S = sum |a b|, for values A (M, K), B (N, K)."""
    return A @ B.T, np.abs(A) @ np.abs(B).T


def norm(v, w, c, kind, eps):
    v = np.asarray(v, dtype=np.float64)
    if kind == "layer":
        v = v - v.mean(1, keepdims=True)
    y = v / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    if w is not None:
        y = y * w
    return y if c is None else y + c


def block_norm(x, branch, gate, weight, bias, post, post_weight, post_bias, alpha, beta, kind, eps):
    """(x', u) of the norms between two blocks."""
    x = np.asarray(x, dtype=np.float64) * alpha
    if branch is not None:
        b = np.asarray(branch, dtype=np.float64)
        if post:
            b = norm(b, post_weight, post_bias, kind, eps)
        if gate is not None:
            b = b * np.repeat(gate, b.shape[0] // gate.shape[0], axis=0)
        x = x + beta * b
    return x, norm(x, weight, bias, kind, eps)
