"""The head rotation's and the attention's argument checks on a machine without a GPU (every refusal happens before
anything reaches CUDA), and the rotation's table against exact fractions."""
import ctypes
from fractions import Fraction

import pytest

import weight_only_bit_w4a16_gb300 as wq

FAKE = 0x10000   # aligned, never dereferenced
OK, INV, UNS, ALN = wq.WQ_OK, wq.WQ_ERR_INVALID_ARG, wq.WQ_ERR_UNSUPPORTED, wq.WQ_ERR_ALIGN
CACHE = dict(k=FAKE, v=FAKE, pages=4, page_size=16, page_stride=16 * 2 * 64, slot_stride=2 * 64, head_stride=64)


def test_packed_structs_match_the_c_structs():
    assert ctypes.sizeof(wq.wq_rope) == wq._ROPE_STRUCT.size
    assert ctypes.sizeof(wq.wq_attention) == wq._ATTN_STRUCT.size


def rope(cache=None, **kw):
    base = dict(tokens=4, q_heads=4, kv_heads=2, head_dim=64, type=0, out_type=0, q=FAKE, q_token=256, q_head=64,
                k=FAKE, k_token=128, k_head=64, v=FAKE, v_token=128, v_head=64, norm=1, eps=1e-6, q_weight=FAKE,
                k_weight=FAKE, rotary_dim=64, pairs=0, table=FAKE, positions=FAKE, axis_stride=4, axes=1,
                with_cache=1, q_out=FAKE, q_out_token=256, q_out_head=64, k_out=FAKE, k_out_token=128, k_out_head=64,
                cache=wq.wq_kv_cache(**{**CACHE, **(cache or {})}), slots=FAKE)
    base.update(kw)
    return wq.wq_head_rope(ctypes.byref(wq.wq_rope(**base)), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(tokens=0), OK), (dict(head_dim=0, rotary_dim=0), OK), (dict(q_heads=0, kv_heads=0), OK),
    (dict(tokens=-1), INV), (dict(q_heads=-1), INV), (dict(kv_heads=-1), INV), (dict(head_dim=-1), INV),
    (dict(type=2), INV), (dict(out_type=-1), INV), (dict(norm=3), INV), (dict(norm=-1), INV), (dict(pairs=2), INV),
    (dict(norm=0), INV),                                    # weights without a norm
    (dict(rotary_dim=63), INV), (dict(rotary_dim=66), INV), (dict(rotary_dim=-2), INV),
    (dict(axes=0), INV), (dict(axes=5), INV), (dict(with_cache=2), INV),
    (dict(head_dim=264, rotary_dim=64), UNS), (dict(head_dim=256, rotary_dim=130), UNS),   # 33 lanes
    (dict(tokens=1 << 28), UNS),
    (dict(q=None), INV), (dict(q_out=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(slots=None), INV),
    (dict(table=None), INV), (dict(positions=None), INV),
    (dict(with_cache=0, k_out=None), INV),                  # nowhere for the keys to go
    (dict(q=FAKE + 1), ALN), (dict(k=FAKE + 1), ALN), (dict(v=FAKE + 1), ALN), (dict(q_out=FAKE + 1), ALN),
    (dict(type=1, q=FAKE + 2), ALN), (dict(out_type=1, k_out=FAKE + 2), ALN), (dict(q_weight=FAKE + 1), ALN),
    (dict(table=FAKE + 4), ALN), (dict(positions=FAKE + 2), ALN), (dict(slots=FAKE + 2), ALN),
])
def test_head_rope_checks(kw, expect):
    assert rope(**kw) == expect


@pytest.mark.parametrize("cache,expect", [
    (dict(page_size=0), INV), (dict(pages=-1), INV), (dict(k=None), INV), (dict(v=None), INV),
    (dict(k=FAKE + 1), ALN), (dict(pages=1 << 27, page_size=16), UNS),
])
def test_head_rope_cache_checks(cache, expect):
    assert rope(cache=cache) == expect


def test_null_arguments():
    assert wq.lib().wq_head_rope(None, None) == INV
    assert wq.lib().wq_prefix_attention(None, None) == INV


def attend(cache=None, **kw):
    base = dict(tokens=4, sequences=2, q_heads=4, kv_heads=2, head_dim=64, scale=0.125, q=FAKE, q_token=256, q_head=64,
                out=FAKE, out_token=256, out_head=64, lse=FAKE, q_start=FAKE, seq_lens=FAKE, tables=FAKE,
                table_stride=3, table_pages=3, prefix_len=20, prefix_pages=FAKE, prefix_table_pages=2,
                cache=wq.wq_kv_cache(**{**CACHE, **(cache or {})}), workspace=FAKE, workspace_bytes=1 << 40)
    base.update(kw)
    return wq.wq_prefix_attention(ctypes.byref(wq.wq_attention(**base)), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(tokens=0), OK), (dict(q_heads=0), OK), (dict(head_dim=0), OK), (dict(sequences=0), OK),
    (dict(sequences=0, q_start=None), INV),                 # tokens of no sequence
    (dict(tokens=-1), INV), (dict(sequences=-1), INV), (dict(prefix_len=-1), INV), (dict(table_pages=-1), INV),
    (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=float("inf")), INV), (dict(scale=float("nan")), INV),
    (dict(tokens=5, q_start=None), INV),                    # no equal shares
    (dict(head_dim=60), UNS), (dict(head_dim=136), UNS), (dict(kv_heads=3), UNS), (dict(kv_heads=0), UNS),
    (dict(sequences=1025), UNS), (dict(tokens=1 << 23), UNS),
    (dict(q=None), INV), (dict(out=None), INV), (dict(seq_lens=None), INV), (dict(tables=None), INV),
    (dict(prefix_pages=None), INV), (dict(prefix_len=33), INV),   # two pages hold 32 keys
    (dict(table_stride=2), INV), (dict(workspace=None), INV), (dict(workspace_bytes=1024), INV),
    (dict(q=FAKE + 8), ALN), (dict(out=FAKE + 8), ALN), (dict(q_token=260), ALN), (dict(out_head=68), ALN),
    (dict(lse=FAKE + 2), ALN), (dict(q_start=FAKE + 1), ALN), (dict(workspace=FAKE + 128), ALN),
])
def test_prefix_attention_checks(kw, expect):
    assert attend(**kw) == expect


@pytest.mark.parametrize("cache,expect", [
    (dict(page_size=24), UNS), (dict(page_size=8), UNS), (dict(page_size=0), INV), (dict(k=FAKE + 8), ALN),
    (dict(slot_stride=132), ALN), (dict(k=None), INV), (dict(pages=0), INV),
])
def test_prefix_attention_cache_checks(cache, expect):
    assert attend(cache=cache) == expect


def test_workspace_sizes():
    f = wq.wq_prefix_attention_workspace
    assert f(4, 2, 4, 2, 64) > 0
    for bad in ((0, 2, 4, 2, 64), (4, 0, 4, 2, 64), (4, 2, 4, 3, 64), (4, 2, 4, 2, 68), (4, 1025, 4, 2, 64),
                (-1, 2, 4, 2, 64), (4, 2, 4, 0, 64)):
        assert f(*bad) == 0


# ---------------------------------------------------------------------------
# the rotation's table
# ---------------------------------------------------------------------------
def _turn():
    """1 / (2 pi), to 100 digits: Machin's formula in fractions."""
    def arctan(x):
        return sum(Fraction((-1) ** k, (2 * k + 1) * x ** (2 * k + 1)) for k in range(90))
    return 1 / (8 * (4 * arctan(5) - arctan(239)))


def _table(freqs, axes=None):
    n = len(freqs)
    out = (ctypes.c_ulonglong * n)()
    st = wq.wq_rope_table((ctypes.c_double * n)(*freqs), None if axes is None else (ctypes.c_int * n)(*axes), n, out)
    return st, list(out)


def test_table_is_the_exact_fraction_of_a_turn():
    freqs = [1.0, 0.5, 10000.0 ** -0.37, 500000.0 ** -0.984375, 1e-12, 0.0, -0.3, -1e-9, 123456.789, 6.283185307179586,
             3.5e15, 1e18]
    st, table = _table(freqs, [i % 4 for i in range(len(freqs))])
    assert st == OK
    turn = _turn()
    for i, f in enumerate(freqs):
        exact = Fraction(f) * turn
        want = (exact - (exact.numerator // exact.denominator)) * 2 ** 62
        got = table[i] >> 2
        # two roundings to units of 2^-62, and 2^-105 of the whole angle's turns
        tol = 1 + abs(exact) * Fraction(2 ** 62, 2 ** 105)
        off = (got - want) % 2 ** 62
        assert min(off, 2 ** 62 - off) <= tol, (f, float(off))
        assert table[i] & 3 == i % 4


def test_table_refusals():
    assert _table([float("nan")])[0] == INV and _table([float("inf")])[0] == INV
    assert _table([1.0], [4])[0] == INV and _table([1.0], [-1])[0] == INV
    assert wq.wq_rope_table(None, None, 1, None) == INV
    assert wq.wq_rope_table(None, None, -1, None) == INV
    assert wq.wq_rope_table(None, None, 0, None) == OK


def test_rope_table_arguments():
    t = wq.rope_table(8, theta=100.0, device="cpu")
    st, want = _table([100.0 ** -(i / 4) for i in range(4)])
    assert [v % 2 ** 64 for v in t.entries.tolist()] == want and (t.rotary_dim, t.axes) == (8, 1)
    t = wq.rope_table(12, sections=(1, 2, 3), ladder="own", device="cpu")
    assert [v & 3 for v in t.entries.tolist()] == [0, 1, 1, 2, 2, 2] and t.axes == 3
    assert [v % 2 ** 64 >> 2 for v in t.entries.tolist()] == [
        v >> 2 for v in _table([1.0, 1.0, 10000.0 ** -0.5, 1.0, 10000.0 ** -(1 / 3), 10000.0 ** -(2 / 3)])[1]]
    t = wq.rope_table(4, inv_freq=[1.0, 2.0], axis=[1, 0], device="cpu")
    assert [v & 3 for v in t.entries.tolist()] == [1, 0] and t.axes == 2
    assert wq.rope_table(0, device="cpu").entries.numel() == 0
    for bad in (dict(rotary_dim=7), dict(rotary_dim=-2), dict(rotary_dim=8, sections=(1, 2)),
                dict(rotary_dim=8, inv_freq=[1.0]), dict(rotary_dim=4, axis=[0]), dict(rotary_dim=4, ladder="mine"),
                dict(rotary_dim=4, sections=(2,), axis=[0, 0])):
        with pytest.raises(ValueError):
            wq.rope_table(device="cpu", **bad)
    with pytest.raises(wq.WQError):
        wq.rope_table(2, inv_freq=[float("nan")], device="cpu")


def test_tensor_helpers_refuse_cpu_tensors():
    import torch
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        wq.head_rope(x, x)
    with pytest.raises(ValueError):
        wq.KVCache(torch.zeros((2, 16, 4, 64), dtype=torch.bfloat16), torch.zeros((2, 16, 4, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        wq.prefix_attention(x, None, None, None)
