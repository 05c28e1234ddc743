"""wq_block_norm with many rows, where a block takes row after row: every width
class of that kernel, each with full and partial vectors a thread, whatever
the device's number of SMs.

A row gets the bits that it gets among few rows (the one-row-a-block kernel,
whose tests are in test_gpu_block_norm.py), and the oracle's values within the
tolerances derived there."""
import ctypes

import pytest
import torch
from test_gpu_block_norm import check, make

import weight_only_bit_w4a16_gb300 as wq

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16

#: both ends of each class: up to 1024, 1536, 2048, 3072, 4096, 6144 and 8192 elements
WIDTHS = [520, 1024, 1032, 1528, 1536, 1544, 2048, 2056, 3072, 3080, 4096, 4104, 6136, 6144, 6152, 8184, 8192]
WIDTHS_32 = [544, 1024, 1056, 1536, 1568, 2048, 2080, 3072, 3104, 4096, 4128, 6144, 6176, 8192]
FEW = 40


def many(d):
    """Rows from which on the kernel is taken: eight vectors for each of 1024 threads an SM; and a few more than a
    multiple of the blocks, so that the last turn is not full."""
    vecs = d // 8
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = -(-8 * 1024 * sms // vecs) + 3
    assert rows * vecs >= 8 * 1024 * sms and FEW * vecs < 8 * 1024 * sms
    return rows


def call(p, s=slice(None), gate=None, **kw):
    """block_norm of the rows s."""
    args = dict(bias=p["bias"], gate=gate, residual_scale=0.75, kind=p["kind"])
    if p["branch"] is not None:
        args.update(branch=p["branch"][s], post_weight=p["post_weight"], post_bias=p["post_bias"], post=p["post"],
                    branch_scale=0.5)
    return wq.block_norm(p["x"][s], p["weight"], **args, **kw)


def gate_of(p, s=None):
    g = p["gate"]
    if g is None or g.shape[0] == 1 or s is None:
        return g
    return g.repeat_interleave(p["x"].shape[0] // g.shape[0], 0)[s].contiguous()


def make_many(d, kind, post, gates, stream, branch=True, vecs=True):
    rows = many(d)
    if gates == "sequence":
        rows = -(-rows // 3) * 3
    gate_rows = {"none": 0, "channel": 1, "sequence": 3, "element": rows}[gates]
    p = make(rows, d, d, stream=stream, branch=BF16 if branch else None, gate_rows=gate_rows, vecs=vecs,
             biases=kind == "layer")
    if not post:
        p["post_weight"] = p["post_bias"] = None
    p.update(kind=kind, post=post)
    return p, rows


def pieces(rows):
    return [slice(r, r + FEW) for r in (0, rows // 2, rows - FEW)]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("stream", [BF16, F32])
@pytest.mark.parametrize("kind,post,gates", [("rms", True, "channel"), ("layer", True, "sequence"),
                                             ("rms", False, "element"), ("layer", False, "none")])
def test_rows_among_many_and_few(d, stream, kind, post, gates):
    p, rows = make_many(d, kind, post, gates, stream)
    i = torch.tensor([0, 1, rows // 3, rows - 1])
    sub = {k: p[k] for k in ("weight", "bias", "post_weight", "post_bias")}
    sub.update(x=p["x"][i], branch=p["branch"][i], gate=gate_of(p, i))
    for out in ("bf16", "fp32"):
        xn, u = call(p, gate=p["gate"], out_dtype=out)
        for s in pieces(rows):
            xs, us = call(p, s, gate_of(p, s), out_dtype=out)
            assert torch.equal(xs, xn[s]) and torch.equal(us, u[s])
        check(sub, xn[i], u[i], kind, 1e-5, post, 0.75, 0.5)


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("stream", [BF16, F32])
def test_no_branch_and_no_vectors(d, stream):
    p, rows = make_many(d, "rms", False, "none", stream, branch=False)
    xo = torch.empty_like(p["x"])
    xn, u = call(p, x_out=xo)
    alone = call(p)
    assert xn is xo and alone[0] is None and torch.equal(alone[1], u)
    for s in pieces(rows):
        xs, us = call(p, s, x_out=torch.empty_like(xo[s]))
        assert torch.equal(xs, xn[s]) and torch.equal(us, u[s])
    p, rows = make_many(d, "layer", True, "channel", stream, vecs=False)
    p["bias"] = p["post_bias"] = None
    xn, u = call(p, gate=p["gate"])
    for s in pieces(rows):
        xs, us = call(p, s, gate_of(p, s))
        assert torch.equal(xs, xn[s]) and torch.equal(us, u[s])


@pytest.mark.parametrize("d", [520, 1536, 6152])
def test_stream_only(d):
    """WQ_NORM_OUT_NONE: x' alone is stored, in place."""
    p, rows = make_many(d, "rms", True, "channel", BF16)
    want = call(p, gate=p["gate"])[0]
    x = p["x"].clone()
    n = wq.wq_norm(rows=rows, d=d, kind=0, post=1, x=x.data_ptr(), ldx=d, branch=p["branch"].data_ptr(), ldb=d,
                   gate=p["gate"].data_ptr(), gate_rows=1, eps=1e-5, residual_scale=0.75, branch_scale=0.5,
                   post_weight=p["post_weight"].data_ptr(), x_out=x.data_ptr(), ldxo=d, out_type=wq.WQ_NORM_OUT_NONE)
    assert wq.wq_block_norm(ctypes.byref(n), torch.cuda.current_stream().cuda_stream) == wq.WQ_OK
    assert torch.equal(x, want)


@pytest.mark.parametrize("d", WIDTHS_32)
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("branch", [True, False])
def test_quantised_output_is_that_of_the_fp32_output(d, fmt, branch):
    """Codes and scales of u are those wq.quantize makes of the fp32 u, and of the same rows among few."""
    p, rows = make_many(d, "rms", branch, "element" if branch else "none", BF16 if d % 64 else F32, branch=branch)
    xn, u = call(p, gate=p["gate"], out_dtype="fp32")
    s = slice(rows - FEW, rows)
    for layout in ("rows", "tiled"):
        def buffers():
            nb = wq.wq_fp4_scale_bytes(rows, d, wq.FORMATS[fmt], wq.LAYOUTS[layout])
            return (torch.zeros((rows, d // 2), dtype=torch.uint8, device="cuda"),
                    torch.zeros(nb, dtype=torch.uint8, device="cuda"))

        for t in (None, 0.003) if fmt == "nvfp4" else (None,):
            scale = None if t is None else torch.tensor([t], device="cuda")
            xq, q = call(p, gate=p["gate"], fmt=fmt, layout=layout, scale=scale, out=buffers())
            want = wq.quantize(u, fmt, scale=scale, layout=layout, out=buffers())
            assert torch.equal(q.packed, want.packed) and torch.equal(q.scales, want.scales)
            assert xq is None if not branch else torch.equal(xq, xn)
            f = call(p, s, gate_of(p, s), fmt=fmt, layout="rows", scale=scale)[1]
            assert torch.equal(f.packed, q.packed[s])
            if layout == "rows":
                assert torch.equal(f.scales.view(-1), q.scales.view(rows, -1)[s].reshape(-1))


@pytest.mark.parametrize("d", [1032, 4104, 8192])
def test_strided_rows_and_in_place(d):
    """16-byte aligned slices of wider arrays, x' in place: the same bits, and nothing outside the slices."""
    p, rows = make_many(d, "rms", True, "channel", BF16)
    want = call(p, gate=p["gate"])
    wide = {k: torch.zeros((rows, d + 24), dtype=BF16, device="cuda") for k in ("x", "branch", "u")}
    for k in ("x", "branch"):
        wide[k][:, 8:8 + d] = p[k]
    q = dict(p, x=wide["x"][:, 8:8 + d], branch=wide["branch"][:, 8:8 + d])
    xn, u = call(q, gate=p["gate"], x_out=q["x"], out=wide["u"][:, 8:8 + d])
    assert torch.equal(xn, want[0]) and torch.equal(u, want[1])
    for w in wide.values():
        assert not w[:, :8].any() and not w[:, 8 + d:].any()
