"""wq_block_norm against the fp64 oracle.

Tolerances.  A row's sums have at most 64 roundings on the way of any term
(32 elements a thread, 5 shuffles, up to 16 or 32 warps; the wide rows' loops
add d / 8192 vectors of 8), so a mean square, a mean of absolute values and
what follows carry a relative error below 2^-17.  With e = 2^-17:
  x'  e (|alpha x| + |beta g| (|N(b)| + |w2| + |c2|)), plus 2^-8 |x'| for a
      bf16 stream;
  u   the error of x', its largest in the row through the statistics, over
      the deviation sigma = sqrt(mean square + eps), times |w| (and 1 + |n| for
      the normed value n), plus e (|u| + |c|), plus 2^-8 |u| for bf16."""
import numpy as np
import pytest
import torch

import weight_only_bit_w4a16_gb300 as wq
from oracle import fp4

pytestmark = pytest.mark.gpu

E = 2.0 ** -17
F32, BF16 = torch.float32, torch.bfloat16


def host(t):
    return None if t is None else t.double().cpu().numpy()


def make(rows, d, seed, stream=BF16, branch=BF16, gate_rows=0, vecs=True, biases=False, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    p = dict(x=(r(rows, d) * 2 + mean).to(stream), branch=None if branch is None else (r(rows, d) + mean).to(branch),
             gate=r(gate_rows, d).to(BF16) if gate_rows else None,
             weight=(1 + 0.1 * r(d)).to(BF16) if vecs else None,
             post_weight=(1 + 0.1 * r(d)).to(BF16) if vecs else None,
             bias=(0.2 * r(d)).to(BF16) if biases else None, post_bias=(0.2 * r(d)).to(BF16) if biases else None)
    return {k: None if v is None else v.cuda() for k, v in p.items()}


def check(p, xn, u, kind, eps, post, alpha, beta):
    h = {k: host(v) for k, v in p.items()}
    wx, wu = fp4.block_norm(h["x"], h["branch"], h["gate"], h["weight"], h["bias"], post, h["post_weight"],
                            h["post_bias"], alpha, beta, kind, eps)
    M = np.abs(alpha * h["x"])
    if h["branch"] is not None:
        b = h["branch"]
        nb = np.abs(b)
        if post:
            nb = np.abs(fp4.norm(b, h["post_weight"], h["post_bias"], kind, eps))
            nb = nb + (1.0 if h["post_weight"] is None else np.abs(h["post_weight"]))
            nb = nb + (0.0 if h["post_bias"] is None else np.abs(h["post_bias"]))
            if kind == "layer":   # b minus its mean: the cancellation
                sd = np.sqrt(((b - b.mean(1, keepdims=True)) ** 2).mean(1, keepdims=True) + eps)
                nb = nb * (1 + np.abs(b).mean(1, keepdims=True) / sd)
        g = 1.0 if h["gate"] is None else np.abs(np.repeat(h["gate"], b.shape[0] // h["gate"].shape[0], axis=0))
        M = M + np.abs(beta) * g * nb
    ex = E * M
    if xn is not None:
        assert xn.dtype == p["x"].dtype
        err = np.abs(host(xn) - wx)
        tol = ex + (2.0 ** -8 * np.abs(wx) if xn.dtype == BF16 else 0)
        assert (err <= tol).all(), f"x': worst {np.max(err - tol):.3e}"
    if u is not None:
        dev = wx - wx.mean(1, keepdims=True) if kind == "layer" else wx
        sigma = np.sqrt((dev ** 2).mean(1, keepdims=True) + eps)
        w = np.ones_like(wx) if h["weight"] is None else np.abs(h["weight"])[None]
        c = 0.0 if h["bias"] is None else np.abs(h["bias"])[None]
        tol = E * (np.abs(wu) + c) + w * (ex + ex.max(1, keepdims=True) * (1 + np.abs(dev / sigma))) / sigma
        if u.dtype == BF16:
            tol = tol + 2.0 ** -8 * np.abs(wu)
        err = np.abs(host(u) - wu)
        assert (err <= tol).all(), f"u: worst {np.max(err - tol):.3e}"


def go(p, kind="rms", eps=1e-5, post=True, alpha=1.0, beta=1.0, out_dtype="fp32", **kw):
    q = dict(p)
    if not post:
        q["post_weight"] = q["post_bias"] = None
    xn, u = wq.block_norm(q["x"], q["weight"], branch=q["branch"], bias=q["bias"], post_weight=q["post_weight"],
                          post_bias=q["post_bias"], post=post, gate=q["gate"], residual_scale=alpha,
                          branch_scale=beta, kind=kind, eps=eps, out_dtype=out_dtype, **kw)
    torch.cuda.synchronize()
    check(q, xn, u, kind, eps, post, alpha, beta)
    return xn, u


#: widths at both sides of every variant's edge, odd ones, and rows on both sides of the few / many rule
WIDTHS = [1, 7, 8, 255, 256, 264, 1000, 1001, 1024, 1032, 2048, 3000, 3072, 3080, 4096, 4104, 8192, 8200, 16384, 16392,
          20001]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("rows", [3, 340])
def test_widths(kind, d, rows):
    p = make(rows, d, d + rows, stream=BF16 if d % 2 else F32, gate_rows=1, biases=True)
    go(p, kind, alpha=0.75, beta=1.5, out_dtype="fp32" if d % 3 else "bf16")


@pytest.mark.parametrize("stream", [BF16, F32])
@pytest.mark.parametrize("branch", [BF16, F32])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate_rows", [0, 1, 4, 24])
def test_parts(stream, branch, post, gate_rows):
    p = make(24, 320, gate_rows, stream, branch, gate_rows)
    go(p, post=post, alpha=0.5, beta=-2.0)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("d", [320, 4096, 17000])
def test_no_branch(kind, d):
    """A pre-norm alone; the stream is stored only where it is asked for."""
    p = make(5, d, 1, branch=None)
    q = dict(p, post_weight=None)
    xn, u = wq.block_norm(q["x"], q["weight"], kind=kind, out_dtype="fp32")
    assert xn is None
    check(q, None, u, kind, 1e-5, False, 1.0, 1.0)
    xo = torch.empty_like(q["x"])
    xn, u = wq.block_norm(q["x"], q["weight"], kind=kind, residual_scale=0.5, x_out=xo, out_dtype="fp32")
    assert xn is xo
    check(q, xn, u, kind, 1e-5, False, 0.5, 1.0)


def test_no_vectors_and_post_without_weight():
    p = make(6, 264, 4, vecs=False)
    go(p)
    go(p, "layer", post=True)


@pytest.mark.parametrize("d", [256, 1000, 4096, 20000])
def test_layer_norm_of_a_large_mean(d):
    """Deviations of 1 around a mean of 100: the variance is summed over deviations."""
    go(make(4, d, 6, stream=F32, branch=F32, mean=100.0), "layer", post=False, beta=0.25)


@pytest.mark.parametrize("d", [64, 1001, 17000])
def test_in_place_and_strides(d):
    """x_out may be x; x, branch, x_out and u may be slices of wider arrays, 16-byte aligned or not."""
    for pad, off in ((0, 0), (8, 8), (3, 1)):
        p = make(9, d, 7, stream=BF16)
        want_x, want_u = go(p, alpha=0.5)

        def wide(t):
            w = torch.zeros((9, d + pad + off), dtype=t.dtype, device="cuda")
            w[:, off:off + d] = t
            return w, w[:, off:off + d]

        (wx, x), (_, b), (wu, u) = wide(p["x"]), wide(p["branch"]), wide(torch.zeros_like(want_u))
        xn, un = wq.block_norm(x, p["weight"], branch=b, post_weight=p["post_weight"], residual_scale=0.5, x_out=x,
                               out=u, eps=1e-5)
        assert xn is x and un is u
        # vector and scalar accesses give the same sums: the same thread holds the same elements
        assert torch.equal(x, want_x) and torch.equal(u, want_u)
        for w in (wx, wu):   # nothing outside the slice is written
            assert not w[:, :off].any() and not w[:, off + d:].any()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("layout", ["rows", "tiled"])
@pytest.mark.parametrize("rows,d", [(1, 32), (5, 96), (130, 416), (2, 1024), (400, 1056), (3, 4096), (310, 3072),
                                    (3, 8192), (2, 16384), (2, 16416), (1, 20000)])
def test_quantised_output_is_that_of_the_fp32_output(fmt, layout, rows, d):
    """The codes and scales of u are those wq.quantize makes of the fp32 u, bit for bit, with a tensor scale too."""
    p = make(rows, d, rows + d, gate_rows=1)
    args = dict(branch=p["branch"], post_weight=p["post_weight"], gate=p["gate"], branch_scale=0.5)
    xn, u = wq.block_norm(p["x"], p["weight"], out_dtype="fp32", **args)
    for t in (None, 0.003) if fmt == "nvfp4" else (None,):
        scale = None if t is None else torch.tensor([t], device="cuda")
        nb = wq.wq_fp4_scale_bytes(rows, d, wq.FORMATS[fmt], wq.LAYOUTS[layout])
        bufs = [(torch.zeros((rows, d // 2), dtype=torch.uint8, device="cuda"),
                 torch.zeros(nb, dtype=torch.uint8, device="cuda")) for _ in range(2)]
        xq, q = wq.block_norm(p["x"], p["weight"], fmt=fmt, layout=layout, scale=scale, out=bufs[0], **args)
        want = wq.quantize(u, fmt, scale=scale, layout=layout, out=bufs[1])
        assert torch.equal(xq, xn)
        assert torch.equal(q.packed, want.packed) and torch.equal(q.scales, want.scales)
        assert q.scale is scale and q.fmt == fmt and q.layout == layout


def test_not_finite_rows_stay_rows():
    """A NaN or an infinity spoils its own row only."""
    p = make(12, 512, 3, stream=F32)
    clean = wq.block_norm(p["x"], p["weight"], branch=p["branch"], out_dtype="fp32")
    p["x"][3, 100], p["branch"][7, 5] = float("nan"), float("inf")
    xn, u = wq.block_norm(p["x"], p["weight"], branch=p["branch"], out_dtype="fp32")
    rows = [r for r in range(12) if r not in (3, 7)]
    assert torch.equal(u[rows], clean[1][rows]) and torch.equal(xn[rows], clean[0][rows])
    assert u[3].isnan().all() and u[7].isnan().any()


def test_zero_rows_and_empty():
    z = torch.zeros((3, 64), dtype=BF16, device="cuda")
    xn, u = wq.block_norm(z, None, branch=z, post=True)
    assert not xn.any() and not u.any()
    for rows, d in ((0, 64), (4, 0)):
        e = torch.empty((rows, d), dtype=BF16, device="cuda")
        xn, u = wq.block_norm(e, None, branch=e)
        assert u.shape == (rows, d) and xn.shape == (rows, d)


def test_another_stream():
    p = make(200, 3072, 5)
    want = wq.block_norm(p["x"], p["weight"], branch=p["branch"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = wq.block_norm(p["x"], p["weight"], branch=p["branch"])
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_refusals():
    x = torch.zeros((6, 64), dtype=BF16, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    for kw in (dict(branch=x[:, :32]), dict(branch=x.half()), dict(gate=x[:4], branch=x), dict(x_out=x.float()),
               dict(out=x[:3]), dict(kind="batch"), dict(fmt="int4"), dict(bias=w[:32]), dict(post_weight=w.float())):
        with pytest.raises(ValueError):
            wq.block_norm(x, w, **kw)
    for kw in (dict(gate=x), dict(post_weight=w), dict(fmt="mxfp4", scale=torch.ones(1, device="cuda"))):
        with pytest.raises(wq.WQError):   # no branch to gate or norm; a tensor scale is NVFP4's
            wq.block_norm(x, w, **kw)
    with pytest.raises(wq.WQError):
        wq.block_norm(x[:, :48], w[:48], fmt="nvfp4")


@pytest.mark.parametrize("stream", [BF16, F32])
@pytest.mark.parametrize("d", [520, 1024, 1528, 2048, 3000, 4096])
@pytest.mark.parametrize("kind,post,gate_rows", [("rms", True, 1), ("rms", False, 0), ("layer", True, 3), ("layer", False, 1)])
def test_many_rows_are_few_rows(stream, d, kind, post, gate_rows):
    """Many rows (blocks that take row after row) give every row the bits it gets among few, and the oracle's values."""
    rows = 12000 if d <= 1024 else 6000
    p = make(rows, d, d, stream=stream, gate_rows=gate_rows, biases=kind == "layer")
    post_w = p["post_weight"] if post else None
    post_b = p["post_bias"] if post else None

    def call(x, b, gate, **kw):
        return wq.block_norm(x, p["weight"], branch=b, bias=p["bias"], post_weight=post_w, post_bias=post_b, gate=gate,
                             residual_scale=0.75, branch_scale=0.5, kind=kind, **kw)

    xn, u = call(p["x"], p["branch"], p["gate"], out_dtype="fp32")
    fmt = "nvfp4" if d % 32 == 0 else None
    q = call(p["x"], p["branch"], p["gate"], fmt=fmt)[1] if fmt else None
    if q is not None:
        want = wq.quantize(u, fmt)
        assert torch.equal(q.packed, want.packed)
    for r0 in (0, rows // 2, rows - 40):
        s = slice(r0, r0 + 40)
        gate = None if p["gate"] is None else p["gate"] if gate_rows == 1 else \
            p["gate"].repeat_interleave(rows // gate_rows, 0)[s].contiguous()
        xs, us = call(p["x"][s], p["branch"][s], gate, out_dtype="fp32")
        assert torch.equal(xs, xn[s]) and torch.equal(us, u[s])
    s = torch.tensor([0, 1, rows // 3, rows - 1])
    sub = {k: v for k, v in p.items()}
    sub["x"], sub["branch"] = p["x"][s], p["branch"][s]
    if p["gate"] is not None and gate_rows > 1:
        sub["gate"] = p["gate"].repeat_interleave(rows // gate_rows, 0)[s]
    if not post:
        sub["post_weight"] = sub["post_bias"] = None
    check(sub, xn[s], u[s], kind, 1e-5, post, 0.75, 0.5)
    # in place
    x = p["x"].clone()
    assert call(x, p["branch"], p["gate"], x_out=x, out_dtype="fp32")[0] is x
    assert torch.equal(x, xn)


#: rows that share a warp: both sides of each number of lanes a row gets, and row counts that leave lanes without one
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("d", [1, 8, 9, 31, 32, 33, 40, 63, 64, 65, 72, 127, 128, 129, 136])
@pytest.mark.parametrize("rows", [1, 2, 31, 33, 515])
def test_short_rows(kind, d, rows):
    p = make(rows, d, d * rows, stream=F32 if d % 2 else BF16, gate_rows=rows if d % 3 else 1, biases=True)
    go(p, kind, alpha=0.75, beta=1.5, out_dtype="bf16" if d % 3 else "fp32")
    go(dict(p, branch=None, gate=None), kind, post=False, alpha=0.5, x_out=torch.empty_like(p["x"]))


@pytest.mark.parametrize("d", [8, 31, 64, 120])
def test_short_rows_are_rows_alone(d):
    """A row gets the bits that it gets alone, whatever rows share its warp: one is NaN, one infinite, one zero."""
    p = make(37, d, d, stream=F32)
    p["x"][5], p["x"][6], p["x"][7] = float("nan"), float("inf"), 0.0
    p["branch"][7] = 0.0
    xn, u = wq.block_norm(p["x"], p["weight"], branch=p["branch"], post_weight=p["post_weight"], out_dtype="fp32")
    for r in range(37):
        xr, ur = wq.block_norm(p["x"][r:r + 1], p["weight"], branch=p["branch"][r:r + 1], post_weight=p["post_weight"],
                               out_dtype="fp32")
        assert torch.equal(xr.view(torch.int32), xn[r:r + 1].view(torch.int32))
        if r not in (5, 6):   # (which NaN a NaN row holds is not stated)
            assert torch.equal(ur, u[r:r + 1])
            assert ur.isfinite().all()
        else:
            assert u[r].isnan().any()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("layout", ["rows", "tiled"])
@pytest.mark.parametrize("rows,d", [(1, 32), (37, 32), (3, 64), (130, 64), (5, 96), (33, 128), (31, 160)])
def test_short_rows_quantised(fmt, layout, rows, d):
    p = make(rows, d, rows + d, gate_rows=rows)
    args = dict(branch=p["branch"], post_weight=p["post_weight"], gate=p["gate"], branch_scale=0.5)
    u = wq.block_norm(p["x"], p["weight"], out_dtype="fp32", **args)[1]
    nb = wq.wq_fp4_scale_bytes(rows, d, wq.FORMATS[fmt], wq.LAYOUTS[layout])
    bufs = [(torch.zeros((rows, d // 2), dtype=torch.uint8, device="cuda"),
             torch.zeros(nb, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    q = wq.block_norm(p["x"], p["weight"], fmt=fmt, layout=layout, out=bufs[0], **args)[1]
    want = wq.quantize(u, fmt, layout=layout, out=bufs[1])
    assert torch.equal(q.packed, want.packed) and torch.equal(q.scales, want.scales)
