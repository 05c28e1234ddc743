"""Norms and rotation of heads with the write into the cache (wq_head_rope) against the fp64 definition.

Tolerance.  Outputs are rounded once: half a step, 2^-8 of the value in bf16, 2^-24 in fp32.  Before that, fp32: a sum
of D <= 256 terms over lanes is off by at most 13 2^-24 of the sum of magnitudes, a layer norm's deviation by that of
the row's largest value, the root and quotient by 2^-22, the angle by 2^-26 turns (1e-7 rad) and its sine by 2^-23;
the products and the sum of a rotation by three roundings.  All together stay below 2^-19 of the row's largest normed
value (2^-19 = 32 2^-24)."""
import numpy as np
import pytest
import torch

import weight_only_bit_w4a16_gb300 as wq
from oracle import heads as ref

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def dev():
    return torch.device("cuda:0")


def f64(t):
    return t.detach().double().cpu().numpy()


def check(got, want, x, weight, bias, kind, eps, what):
    """got against want; x the unnormed heads."""
    size = np.abs(x).max(axis=-1, keepdims=True)
    if kind is not None:
        y = x - x.mean(axis=-1, keepdims=True) if kind == "layer" else x
        size = size / np.sqrt((y * y).mean(axis=-1, keepdims=True) + eps)
        size = size * (1.0 if weight is None else np.abs(weight).max())
        size = size + (0.0 if bias is None else np.abs(bias).max())
    tol = HALF[got.dtype] * np.abs(want) + 2.0 ** -19 * size + 2.0 ** -133
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), f"{what}: worst {float((err / tol).max())} of the tolerance"


def make(T, Hq, Hkv, D, dtype, seed, pad=0, layout="slices"):
    g = torch.Generator(device=dev()).manual_seed(seed)
    if layout == "slices":    # of one q/k/v array
        x = torch.randn(T, (Hq + 2 * Hkv) * D + pad, generator=g, device=dev()).to(dtype)
        q, k, v = (x[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in
                   ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    else:                     # heads before tokens
        q, k, v = (torch.randn(h, T, D + pad, generator=g, device=dev()).to(dtype)[..., :D].transpose(0, 1)
                   for h in (Hq, Hkv, Hkv))
    w = [(1.0 + 0.2 * torch.randn(D, generator=g, device=dev())).to(torch.bfloat16) for _ in range(4)]
    return q, k, v, w, g


CASES = [
    # tokens, q heads, kv heads, D, R, dtype, norm, bias, pairs, sections, pad, layout
    (1, 4, 1, 128, 128, "bf16", "rms", False, "halves", None, 0, "slices"),
    (1, 1, 1, 8, 8, "bf16", None, False, "halves", None, 0, "slices"),
    (3, 5, 2, 128, 64, "bf16", "layer", True, "adjacent", None, 0, "slices"),
    (17, 7, 1, 64, 64, "fp32", "rms", True, "halves", (10, 12, 10), 0, "heads"),
    (5, 3, 3, 72, 72, "bf16", "rms", False, "halves", (18, 18), 0, "slices"),
    (5, 3, 3, 72, 72, "fp32", "layer", True, "adjacent", (18, 18), 1, "slices"),     # unaligned rows
    (9, 2, 2, 80, 32, "bf16", "rms", False, "halves", None, 3, "slices"),
    (4, 2, 1, 256, 256, "bf16", "rms", False, "adjacent", (60, 34, 34), 0, "slices"),
    (4, 2, 1, 256, 64, "fp32", "layer", False, "halves", None, 0, "heads"),
    (6, 3, 2, 33, 14, "bf16", "layer", True, "halves", None, 0, "slices"),           # sizes that fit no vector
    (6, 3, 2, 33, 32, "fp32", "rms", True, "adjacent", None, 0, "heads"),
    (6, 3, 2, 7, 2, "bf16", "rms", False, "halves", None, 0, "slices"),
    (6, 2, 2, 96, 20, "bf16", "rms", False, "halves", None, 0, "slices"),
    (6, 2, 2, 1, 0, "fp32", "rms", False, "halves", None, 0, "slices"),
    (6, 2, 2, 248, 242, "bf16", "rms", False, "adjacent", None, 0, "slices"),
    (700, 32, 8, 128, 128, "bf16", "rms", False, "halves", None, 0, "slices"),       # several heads a group
    (700, 13, 3, 64, 32, "fp32", "layer", True, "adjacent", (7, 9), 0, "slices"),
    (501, 29, 2, 40, 24, "bf16", "rms", True, "halves", (2, 3, 7), 5, "heads"),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,R,dtype,norm,bias,pairs,sections,pad,layout", CASES)
def test_against_the_definition(T, Hq, Hkv, D, R, dtype, norm, bias, pairs, sections, pad, layout):
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    q, k, v, w, g = make(T, Hq, Hkv, D, dt, D + T, pad, layout)
    axes = 1 if sections is None else len(sections)
    table = wq.rope_table(R, theta=1000.0, sections=sections, ladder="own" if sections else "shared", device=dev()) if R else None
    pos = torch.randint(-5, 300000, (axes, T), generator=g, device=dev()).int()
    axis = [0] * (R // 2) if sections is None else [a for a, p in enumerate(sections) for _ in range(p)]
    freq = ([1000.0 ** -(i / (R // 2)) for i in range(R // 2)] if sections is None
            else [1000.0 ** -(j / p) for p in sections for j in range(p)])
    kw = dict(table=table, positions=pos if axes > 1 else pos[0], norm=norm, eps=1e-5, pairs=pairs)
    use = [None] * 4 if norm is None else [w[0], w[1], w[2] if bias else None, w[3] if bias else None]
    kw.update(q_weight=use[0], k_weight=use[1], q_bias=use[2], k_bias=use[3])
    q2, k2 = wq.head_rope(q, k, **kw)
    # again into the cache, bf16 whatever the inputs are, and outputs of the other type
    page = 16
    pages = (T + page - 1) // page + 1
    store = torch.full((pages, 2, page, Hkv, D), 7.0, dtype=torch.bfloat16, device=dev())
    cache = wq.KVCache(store[:, 0], store[:, 1])
    slots = torch.randperm(pages * page, generator=g, device=dev())[:T].int()
    skip = torch.rand(T, generator=g, device=dev()) < 0.2
    slots[skip] = torch.tensor([-1, pages * page, 2 ** 31 - 1, -2 ** 31], device=dev(), dtype=torch.int32)[
        torch.arange(int(skip.sum()), device=dev()) % 4]
    other = torch.bfloat16 if dt is torch.float32 else torch.float32
    k_other = torch.empty(T, Hkv, D, dtype=other, device=dev())
    q3, k3 = wq.head_rope(q, k, v, cache=cache, slots=slots, out_dtype="bf16" if other is torch.bfloat16 else "fp32",
                          k_out=k_other, **kw)
    torch.cuda.synchronize()
    for x, weight, b, outs in ((q, use[0], use[2], (q2, q3)), (k, use[1], use[3], (k2, k3))):
        x64 = f64(x)
        w64, b64 = (None if t is None else f64(t) for t in (weight, b))
        want = ref.rotate(ref.head_norm(x64, w64, b64, norm, 1e-5), pos.cpu().numpy(), freq, axis, pairs)
        for got in outs:
            check(got, want, x64, w64, b64, norm, 1e-5, f"{got.dtype}")
    kc = store[:, 0].reshape(pages * page, Hkv, D)
    vc = store[:, 1].reshape(pages * page, Hkv, D)
    live = ~skip
    at = slots[live].long()
    assert torch.equal(kc[at], (k2 if dt is torch.bfloat16 else k3)[live].to(torch.bfloat16))
    assert torch.equal(vc[at], v[live].to(torch.bfloat16))
    untouched = torch.ones(pages * page, dtype=torch.bool, device=dev())
    untouched[at] = False
    assert (kc[untouched] == 7.0).all() and (vc[untouched] == 7.0).all()


@pytest.mark.parametrize("T", [1, 300])
def test_in_place_and_heads_first_cache(T):
    """q and k rotated in place; pages of (head, slot) rows; the same bits as apart."""
    q, k, v, w, g = make(T, 8, 2, 128, torch.bfloat16, 3)
    table = wq.rope_table(128, device=dev())
    pos = torch.arange(T, device=dev(), dtype=torch.int32)
    q2, k2 = wq.head_rope(q, k, table=table, positions=pos, q_weight=w[0], k_weight=w[1])
    store = torch.zeros(2, T // 32 + 1, 2, 32, 128, dtype=torch.bfloat16, device=dev())
    cache = wq.KVCache(store[0].transpose(1, 2), store[1].transpose(1, 2))
    slots = torch.arange(T, device=dev(), dtype=torch.int32).flip(0)
    a, b = wq.head_rope(q, k, v, table=table, positions=pos, q_weight=w[0], k_weight=w[1], cache=cache, slots=slots,
                        q_out=q, k_out=k)
    assert a is q and b is k and torch.equal(q, q2) and torch.equal(k, k2)
    rows = cache.k.reshape(-1, 2, 128)[:T].flip(0)
    assert torch.equal(rows, k2)
    assert torch.equal(cache.v.reshape(-1, 2, 128)[:T].flip(0), v)


def test_far_positions():
    """The angle keeps its precision at any position; a position of 0 changes nothing."""
    pos = torch.tensor([0, 1, 2 ** 20 + 1, 2 ** 30 + 12345, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=dev())
    x = torch.randn(6, 2, 64, device=dev())
    q, _ = wq.head_rope(x, x, table=wq.rope_table(64, device=dev()), positions=pos, norm=None)
    assert torch.equal(q[0], x[0])
    freq = [10000.0 ** -(i / 32) for i in range(32)]
    want = ref.rotate(f64(x), [pos.cpu().numpy()], freq, [0] * 32, "halves")
    # fp64's own product pos * freq is off by 2^-53 of up to 2^31
    tol = 2.0 ** -19 * np.abs(f64(x)).max()
    assert np.abs(f64(q) - want).max() <= tol


def test_odd_values_stay_in_their_head():
    """Infinities and NaN in one head leave the others alone, and copied values are copied."""
    q, k, v, w, g = make(40, 4, 4, 64, torch.bfloat16, 9)
    table, pos = wq.rope_table(64, device=dev()), torch.arange(40, device=dev(), dtype=torch.int32)
    want, _ = wq.head_rope(q, k, table=table, positions=pos)
    q = q.clone()
    q[7, 2, 5], q[9, 0] = float("nan"), float("inf")
    v = v.clone()
    v[3, 1] = float("nan")
    cache = wq.KVCache(*torch.zeros(2, 3, 16, 4, 64, dtype=torch.bfloat16, device=dev()))
    got, _ = wq.head_rope(q, k, v, table=table, positions=pos, cache=cache, slots=pos)
    ok = torch.ones(40, 4, dtype=torch.bool, device=dev())
    ok[7, 2] = ok[9, 0] = False
    assert torch.equal(got[ok], want[ok]) and got[7, 2].isnan().all()
    stored = cache.v.reshape(48, 4, 64)[:40]
    assert torch.equal(stored.isnan(), v.isnan()) and torch.equal(stored.nan_to_num(), v.nan_to_num())


def test_zero_heads_and_rows():
    """Rows of zeros: the epsilon keeps them; without queries, without tokens."""
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=dev())
    pos = torch.arange(3, device=dev(), dtype=torch.int32)
    table = wq.rope_table(64, device=dev())
    for norm in ("rms", "layer"):
        q, k = wq.head_rope(x, x, table=table, positions=pos, norm=norm)
        assert (q == 0).all() and (k == 0).all()
    k0 = torch.randn(3, 2, 64, device=dev()).to(torch.bfloat16)
    q, k = wq.head_rope(x[:, :0], k0, table=table, positions=pos)
    _, want = wq.head_rope(k0, k0, table=table, positions=pos)
    assert q.shape == (3, 0, 64) and torch.equal(k, want)
    q, k = wq.head_rope(x[:0], x[:0], table=table, positions=pos[:0])
    assert q.shape == (0, 2, 64)


def test_captured_on_another_stream():
    """Replays follow new positions and slots."""
    q, k, v, w, g = make(8, 4, 2, 128, torch.bfloat16, 4)
    table = wq.rope_table(128, device=dev())
    pos = torch.arange(8, device=dev(), dtype=torch.int32)
    slots = torch.arange(8, device=dev(), dtype=torch.int32)
    cache = wq.KVCache(*torch.zeros(2, 2, 16, 2, 128, dtype=torch.bfloat16, device=dev()))
    out = torch.empty_like(q, memory_format=torch.contiguous_format)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        wq.head_rope(q, k, v, table=table, positions=pos, cache=cache, slots=slots, q_out=out)
    for step in range(3):
        pos += 100
        slots += 2
        graph.replay()
        want, kw = wq.head_rope(q, k, table=table, positions=pos)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert torch.equal(cache.k.reshape(32, 2, 128)[slots.long()], kw)


@pytest.mark.parametrize("bad", ["k rows", "positions", "positions type", "slots", "v", "cache heads", "q_out", "weight",
                                 "table", "cpu k", "norm"])
def test_refusals(bad):
    q, k, v, w, g = make(4, 4, 2, 64, torch.bfloat16, 1)
    kw = dict(v=v, table=wq.rope_table(64, device=dev()), positions=torch.zeros(4, dtype=torch.int32, device=dev()),
              slots=torch.zeros(4, dtype=torch.int32, device=dev()), q_weight=w[0],
              cache=wq.KVCache(*torch.zeros(2, 1, 16, 2, 64, dtype=torch.bfloat16, device=dev())))
    if bad == "k rows":
        k = k[:3]
    elif bad == "positions":
        kw["positions"] = kw["positions"][:3]
    elif bad == "positions type":
        kw["positions"] = kw["positions"].long()
    elif bad == "slots":
        kw["slots"] = None
    elif bad == "v":
        kw["v"] = v.float()
    elif bad == "cache heads":
        kw["cache"] = wq.KVCache(*torch.zeros(2, 1, 16, 1, 64, dtype=torch.bfloat16, device=dev()))
    elif bad == "q_out":
        kw["q_out"] = torch.empty(4, 4, 128, dtype=torch.bfloat16, device=dev())[..., ::2]
    elif bad == "weight":
        kw["q_weight"] = w[0].float()
    elif bad == "table":
        kw["table"] = wq.rope_table(128, device=dev())
    elif bad == "cpu k":
        k = k.cpu()
    elif bad == "norm":
        kw["norm"] = "batch"
    with pytest.raises(ValueError):
        wq.head_rope(q, k, **kw)
