"""The 4-bit (W4A4) operators, measured: quantisation to microscaled 4-bit floats, the product of two such
operands, the norms between two blocks, and a norm -> quantise -> product chain.

`own` false: plain torch operations in 32 bits.  `own` true: the calls a user makes of the library.
"""
import math

import torch

own = False

GROUP = {"nvfp4": 16, "mxfp4": 32}
EPS = 1e-5


def dev():
    return torch.device("cuda")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoded token's activations before the down projection
        dict(name="quantize token", op="quantize", fmt="nvfp4", rows=1, K=8192, dtype="bf16", pad=0, scaled=False),
        # a ragged batch, a slice of a wider activation tensor
        dict(name="quantize ragged slice", op="quantize", fmt="mxfp4", rows=777, K=1056, dtype="bf16", pad=40,
             scaled=False),
        # an output embedding turned into 4-bit weights, with a tensor scale
        dict(name="quantize weights", op="quantize", fmt="nvfp4", rows=128256, K=3072, dtype="fp32", pad=0,
             scaled=True),
        # a gate or up projection of one token
        dict(name="product token", op="product", fmt="nvfp4", M=1, N=8192, K=3072, out="bf16", epi="none"),
        # a down projection of a decode batch, added to the residual stream
        dict(name="product batch", op="product", fmt="mxfp4", M=16, N=3072, K=8192, out="fp32", epi="residual"),
        # odd sizes: rows of C that are not 16-byte aligned, a partial k step, a bias
        dict(name="product ragged", op="product", fmt="nvfp4", M=333, N=1001, K=2080, out="bf16", epi="bias"),
        # an attention projection over a prompt
        dict(name="product prefill", op="product", fmt="mxfp4", M=2048, N=3072, K=3072, out="bf16", epi="none"),
        # large and bound by the matrix units
        dict(name="product large", op="product", fmt="nvfp4", M=8192, N=8192, K=8192, out="bf16", epi="none"),
        # one token between two blocks
        dict(name="norm token", op="norm", kind="rms", rows=1, d=3072, stream="bf16", post=True, gate="channel",
             bias=False),
        # a prompt between two blocks, fp32 residual stream, a gate for each element
        dict(name="norm prompt", op="norm", kind="rms", rows=8192, d=3072, stream="fp32", post=True, gate="token",
             bias=False),
        # layer norms of an odd width, gates for each sequence of the batch
        dict(name="norm ragged", op="norm", kind="layer", rows=1000, d=1001, stream="bf16", post=False, gate="batch",
             bias=True),
        # a decode batch: norms between blocks, quantised, then the gate / up product of the next block
        dict(name="norm and gate/up", op="chain", fmt="nvfp4", rows=128, d=3072, N=16384, gated=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "norm", "chain"])
    fmt = rng.choice(["nvfp4", "mxfp4"])
    if op == "quantize":
        K = 32 * _log(rng, 1, 512)
        rows = max(1, min(_log(rng, 1, 65536), (1 << 28) // K))
        return dict(op=op, fmt=fmt, rows=rows, K=K, dtype=rng.choice(["bf16", "fp32"]),
                    pad=rng.choice([0, 0, 8, 40, 3]), scaled=fmt == "nvfp4" and rng.random() < 0.5)
    if op == "product":
        K = 32 * _log(rng, 1, 512)
        N = _log(rng, 8, 32768)
        if rng.random() < 0.6:
            N = (N + 15) // 16 * 16
        M = max(1, min(_log(rng, 1, 8192), (1 << 38) // (N * K)))
        epi = rng.choice(["none", "none", "bias", "residual", "gated"])
        if epi == "gated":
            N = (N + 15) // 16 * 16
        return dict(op=op, fmt=fmt, M=M, N=N, K=K, out=rng.choice(["bf16", "bf16", "fp32"]), epi=epi)
    if op == "norm":
        d = _log(rng, 16, 16384)
        if rng.random() < 0.6:
            d = (d + 7) // 8 * 8
        rows = max(1, min(_log(rng, 1, 32768), (1 << 26) // d))
        gate = rng.choice(["none", "channel", "batch", "token"])
        if gate == "batch":
            rows = (rows + 7) // 8 * 8
        return dict(op=op, kind=rng.choice(["rms", "rms", "layer"]), rows=rows, d=d,
                    stream=rng.choice(["bf16", "fp32"]), post=rng.random() < 0.6, gate=gate,
                    bias=rng.random() < 0.3)
    d = 32 * _log(rng, 4, 256)
    N = 16 * _log(rng, 4, 1024)
    return dict(op=op, fmt=fmt, rows=_log(rng, 1, 2048), d=d, N=N, gated=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=dev(), dtype=torch.float32)


def _mma_layout(scales):
    """Row-major scale bytes (rows, groups) in the order the 4-bit product takes: 512-byte blocks of 128 rows x 4
    groups, row r's four bytes at 16 (r mod 32) + 4 (r / 32)."""
    R, G = scales.shape
    Rb, Gb = (R + 127) // 128, (G + 3) // 4
    full = torch.zeros((Rb * 128, Gb * 4), dtype=torch.uint8, device=scales.device)
    full[:R, :G] = scales
    return full.view(Rb, 4, 32, Gb, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _operand(g, rows, K, fmt):
    """A 4-bit operand as a user holds it: normal values quantised (codes, scale bytes by rows and in the product's
    order)."""
    x = _normal(g, rows, K).to(torch.bfloat16)
    code, byte = _quantize_plain(x.float(), fmt, None)
    packed = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
    return dict(packed=packed, scales=byte, tiled=_mma_layout(byte), rows=rows, K=K, fmt=fmt)


def _bf16(t):
    return t.to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    s = dict(case)
    s["table"] = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                              dtype=torch.float32, device=dev())
    op = case["op"]
    if op == "quantize":
        rows, K = case["rows"], case["K"]
        wide = _normal(g, rows, K + case["pad"])
        # activations have a few loud channels
        wide[:, ::97] *= 8.0
        if case["dtype"] == "bf16":
            wide = _bf16(wide)
        s["x"] = wide[:, :K]
        s["t"] = None
        if case["scaled"]:
            s["x"].mul_(0.02)
            s["t"] = (s["x"].abs().amax().float() / (6.0 * 448.0)).reshape(1)
        G = K // GROUP[case["fmt"]]
        s["codes"] = torch.empty((rows, K // 2), dtype=torch.uint8, device=dev())
        s["tiled"] = torch.empty((rows + 127) // 128 * ((G + 3) // 4) * 512, dtype=torch.uint8, device=dev())
        s["values"] = torch.empty((rows, K), dtype=torch.bfloat16, device=dev())
    elif op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        s["A"] = _operand(g, M, K, case["fmt"])
        s["B"] = _operand(g, N, K, case["fmt"])
        s["tb"] = None
        if case["fmt"] == "nvfp4":   # weights with a tensor scale
            s["tb"] = torch.rand(1, generator=g, device=dev()) * 0.02 + 0.01
        cols = N // 2 if case["epi"] == "gated" else N
        s["bias"] = _bf16(_normal(g, N)) if case["epi"] == "bias" else None
        s["residual"] = _bf16(_normal(g, M, cols)) if case["epi"] == "residual" else None
        s["gated"] = case["epi"] == "gated"
        s["C"] = torch.empty((M, cols), dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16, device=dev())
    else:
        chain = op == "chain"
        rows, d = case["rows"], case["d"]
        f32 = not chain and case["stream"] == "fp32"
        x = _normal(g, rows, d) * 3.0
        s["x"] = x if f32 else _bf16(x)
        s["branch"] = _bf16(_normal(g, rows, d) * (1.0 + torch.rand(rows, 1, generator=g, device=dev())))
        gate = "channel" if chain else case["gate"]
        grows = {"none": 0, "channel": 1, "batch": 8, "token": rows}[gate]
        s["gate"] = _bf16(torch.tanh(_normal(g, grows, d))) if grows else None
        s["weight"] = _bf16(1.0 + 0.1 * _normal(g, d))
        s["post_weight"] = _bf16(1.0 + 0.1 * _normal(g, d)) if chain or case["post"] else None
        with_bias = not chain and case["bias"]
        s["bias"] = _bf16(0.1 * _normal(g, d)) if with_bias else None
        s["post_bias"] = _bf16(0.1 * _normal(g, d)) if with_bias and case["post"] else None
        s["x_out"] = torch.empty_like(s["x"])
        if chain:
            s["B"] = _operand(g, case["N"], d, case["fmt"])
            G = d // GROUP[case["fmt"]]
            s["codes"] = torch.empty((rows, d // 2), dtype=torch.uint8, device=dev())
            s["tiled"] = torch.empty((rows + 127) // 128 * ((G + 3) // 4) * 512, dtype=torch.uint8, device=dev())
            cols = case["N"] // 2 if case["gated"] else case["N"]
            s["C"] = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev())
        else:
            s["u"] = torch.empty((rows, d), dtype=torch.bfloat16, device=dev())
    return s


# ---------------------------------------------------------------------------
# the plain forms, 32 bits
# ---------------------------------------------------------------------------
def _e2m1_code(v):
    """Codes of the nearest e2m1 values (ties to even, saturating): bit 3 the sign."""
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return (code + (v < 0) * 8).to(torch.uint8)


def _quantize_plain(x, fmt, t):
    """(codes, scale bytes) of float32 x."""
    rows, K = x.shape
    grp = x.reshape(rows, -1, GROUP[fmt])
    a = grp.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        t = 1.0 if t is None else t
        s8 = (a / (6.0 * t)).clamp(max=448.0).to(torch.float8_e4m3fn)
        byte = s8.view(torch.uint8)
        step = s8.float() * t
    else:
        # the exponent of the largest power of two not above a, less the 2 of e2m1's own
        e = (a.contiguous().view(torch.int32) >> 23) - 2
        e = e.clamp(min=0)
        byte = e.to(torch.uint8)
        step = torch.ldexp(torch.ones_like(a), e - 127)
    v = torch.where(step > 0, grp / step, torch.zeros_like(grp))
    return _e2m1_code(v).reshape(rows, K), byte.reshape(rows, -1)


def _values_plain(table, code, byte, fmt, t=None):
    """float32 values of codes (through the 16 values of a code) and scale bytes."""
    rows, K = code.shape
    if fmt == "nvfp4":
        step = byte.view(torch.float8_e4m3fn).float()
        step = step if t is None else step * t
    else:
        step = torch.ldexp(torch.ones_like(byte, dtype=torch.float32), byte.to(torch.int32) - 127)
    return (table[code.to(torch.int32)].view(rows, -1, GROUP[fmt]) * step.unsqueeze(-1)).view(rows, K)


def _unpack(p):
    return torch.stack((p & 15, p >> 4), dim=-1).view(p.shape[0], -1)


def _operand_plain(s, o):
    return _values_plain(s["table"], _unpack(o["packed"]), o["scales"], o["fmt"])


def _gated_plain(y):
    M, N = y.shape
    v = y.view(M, N // 16, 2, 8)
    gate, up = v[:, :, 0], v[:, :, 1]
    return (gate / (1.0 + torch.exp(-gate)) * up).reshape(M, N // 2)


def _norm_plain(v, w, c, kind):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    y = v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS) * w.float()
    return y if c is None else y + c.float()


def _scales_of(s):
    """(residual scale, branch scale): a residual sum kept at unit size."""
    return 0.96875, 0.25


def _block_plain(s, kind):
    b = s["branch"].float()
    if s["post_weight"] is not None:
        b = _norm_plain(b, s["post_weight"], s["post_bias"], kind)
    if s["gate"] is not None:
        g = s["gate"].float()
        rows = b.shape[0]
        b = (b.view(g.shape[0], rows // g.shape[0], -1) * g.unsqueeze(1)).view(rows, -1)
    alpha, beta = _scales_of(s)
    x = alpha * s["x"].float() + beta * b
    return x, _norm_plain(x, s["weight"], s["bias"], kind)


def _run_plain(s):
    op = s["op"]
    if op == "quantize":
        code, byte = _quantize_plain(s["x"].float(), s["fmt"], s["t"])
        return _values_plain(s["table"], code, byte, s["fmt"], s["t"]).to(torch.bfloat16)
    if op == "product":
        y = _operand_plain(s, s["A"]) @ _operand_plain(s, s["B"]).t()
        if s["tb"] is not None:
            y = y * s["tb"]
        if s["bias"] is not None:
            y = y + s["bias"].float()
        if s["gated"]:
            y = _gated_plain(y)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(s["C"].dtype)
    if op == "norm":
        x, u = _block_plain(s, s["kind"])
        return x.to(s["x"].dtype), u.to(torch.bfloat16)
    x, u = _block_plain(s, "rms")
    code, byte = _quantize_plain(u, s["fmt"], None)
    y = _values_plain(s["table"], code, byte, s["fmt"]) @ _operand_plain(s, s["B"]).t()
    if s["gated"]:
        y = _gated_plain(y)
    return x.to(s["x"].dtype), y.to(torch.bfloat16)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _run_own(s):
    import weight_only_bit_w4a16_gb300 as wq

    op = s["op"]
    if op == "quantize":
        wq.quantize(s["x"], s["fmt"], scale=s["t"], out=(s["codes"], s["tiled"]), values=s["values"])
        return s["values"]
    if op == "product":
        a, b = s["A"], s["B"]
        A = wq.Fp4(a["packed"], a["tiled"], a["rows"], a["K"], a["fmt"])
        B = wq.Fp4(b["packed"], b["tiled"], b["rows"], b["K"], b["fmt"], scale=s["tb"])
        return wq.gemm_fp4(A, B, out=s["C"], bias=s["bias"], residual=s["residual"], gated=s["gated"])
    alpha, beta = _scales_of(s)
    if op == "norm":
        return wq.block_norm(s["x"], s["weight"], branch=s["branch"], bias=s["bias"], post_weight=s["post_weight"],
                             post_bias=s["post_bias"], gate=s["gate"], residual_scale=alpha, branch_scale=beta,
                             kind=s["kind"], eps=EPS, x_out=s["x_out"], out=s["u"])
    x, u = wq.block_norm(s["x"], s["weight"], branch=s["branch"], post_weight=s["post_weight"], gate=s["gate"],
                         residual_scale=alpha, branch_scale=beta, kind="rms", eps=EPS, x_out=s["x_out"],
                         out=(s["codes"], s["tiled"]), fmt=s["fmt"])
    b = s["B"]
    B = wq.Fp4(b["packed"], b["tiled"], b["rows"], b["K"], b["fmt"])
    return x, wq.gemm_fp4(u, B, out=s["C"], gated=s["gated"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _fp4_bytes(rows, K, fmt):
    return rows * K / 2 + rows * K / GROUP[fmt]


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["K"]
        return dict(bytes=n * (4 if case["dtype"] == "fp32" else 2) + _fp4_bytes(case["rows"], case["K"], case["fmt"]) + 2 * n,
                    flops=4.0 * n)
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        cols = N // 2 if case["epi"] == "gated" else N
        b = _fp4_bytes(M, K, case["fmt"]) + _fp4_bytes(N, K, case["fmt"]) + M * cols * (4 if case["out"] == "fp32" else 2)
        b += 2 * N if case["epi"] == "bias" else 2 * M * cols if case["epi"] == "residual" else 0
        return dict(bytes=b, flops=2.0 * M * N * K)
    rows, d = case["rows"], case["d"]
    if op == "norm":
        w = 4 if case["stream"] == "fp32" else 2
        gate = {"none": 0, "channel": 1, "batch": 8, "token": rows}[case["gate"]]
        vecs = 1 + case["post"] + case["bias"] * (1 + case["post"])
        return dict(bytes=rows * d * (2 * w + 2 + 2) + 2 * d * (gate + vecs), flops=12.0 * rows * d)
    cols = case["N"] // 2 if case["gated"] else case["N"]
    return dict(bytes=rows * d * (2 + 2 + 2) + 6 * d + _fp4_bytes(case["N"], d, case["fmt"]) + 2 * rows * cols,
                flops=2.0 * rows * d * case["N"] + 16.0 * rows * d)


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------
def _floor_log2(v):
    return torch.floor(torch.frexp(v)[1].to(torch.float64) - 1.0)


def _round_to_grid(v, low, bits):
    """v >= 0 to the nearest binary float of `bits` fraction bits and least exponent `low`, ties to even."""
    e = torch.where(v > 0, _floor_log2(v), torch.full_like(v, float(low))).clamp(min=low)
    unit = torch.exp2(e - bits)
    return torch.round(v / unit) * unit


def _quantized_exact(x, fmt, t):
    rows, K = x.shape
    grp = x.reshape(rows, K // GROUP[fmt], GROUP[fmt])
    top = grp.abs().max(dim=-1, keepdim=True).values
    if fmt == "nvfp4":
        unit = 1.0 if t is None else t.double()
        scale = _round_to_grid((top / (6.0 * unit)).clamp(max=448.0), -6, 3) * unit
    else:
        scale = torch.exp2((torch.where(top > 0, _floor_log2(top), torch.full_like(top, -127.0)) - 2.0).clamp(min=-127.0))
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    q = _round_to_grid((grp.abs() / safe), 0, 1).clamp(max=6.0)
    return (torch.sign(grp) * q * scale).reshape(rows, K)


def _held_exact(o):
    p = o["packed"].to(torch.int64)
    code = torch.empty((o["rows"], o["K"]), dtype=torch.int64, device=p.device)
    code[:, 0::2] = p % 16
    code[:, 1::2] = p // 16
    mag = code % 8
    frac, ex = (mag % 2).double(), (mag // 2).double()
    v = torch.where(mag < 2, 0.5 * frac, (1.0 + 0.5 * frac) * torch.exp2(ex - 1.0))
    v = torch.where(code >= 8, -v, v)
    b = o["scales"].to(torch.int64)
    if o["fmt"] == "nvfp4":
        e, m = (b // 8) % 16, (b % 8).double()
        sc = torch.where(e == 0, m / 8.0 * 2.0 ** -6, (1.0 + m / 8.0) * torch.exp2(e.double() - 7.0))
    else:
        sc = torch.exp2(b.double() - 127.0)
    return v * sc.repeat_interleave(GROUP[o["fmt"]], dim=1)


def _silu_pairs_exact(y):
    j = torch.arange(y.shape[1] // 2, device=y.device)
    gate = y[:, j // 8 * 16 + j % 8]
    return gate * torch.sigmoid(gate) * y[:, j // 8 * 16 + 8 + j % 8]


def _normed_exact(v, w, c, kind):
    n = v.shape[1]
    if kind == "layer":
        v = v - (v.sum(dim=1) / n)[:, None]
    y = v * torch.rsqrt((v * v).sum(dim=1) / n + EPS)[:, None] * w.double()[None, :]
    return y + c.double()[None, :] if c is not None else y


def _between_exact(s, kind):
    b = s["branch"].double()
    if s["post_weight"] is not None:
        b = _normed_exact(b, s["post_weight"], s["post_bias"], kind)
    if s["gate"] is not None:
        b = b * s["gate"].double().repeat_interleave(b.shape[0] // s["gate"].shape[0], dim=0)
    alpha, beta = _scales_of(s)
    x = s["x"].double() * alpha + b * beta
    return x, _normed_exact(x, s["weight"], s["bias"], kind)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        rows = case["rows"]
        # by slabs of rows, as a large weight in 64 bits is many times its size
        step = max(1, (1 << 26) // case["K"])
        got = torch.empty((rows, case["K"]), dtype=torch.float64, device=dev())
        for r in range(0, rows, step):
            got[r:r + step] = _quantized_exact(s["x"][r:r + step].double(), case["fmt"], s["t"])
        return got
    if op == "product":
        y = torch.matmul(_held_exact(s["A"]), _held_exact(s["B"]).T)
        if s["tb"] is not None:
            y *= s["tb"].double()
        if s["bias"] is not None:
            y += s["bias"].double()[None, :]
        if s["gated"]:
            y = _silu_pairs_exact(y)
        if s["residual"] is not None:
            y += s["residual"].double()
        return y
    if op == "norm":
        return _between_exact(s, case["kind"])
    x, u = _between_exact(s, "rms")
    y = torch.matmul(_quantized_exact(u, case["fmt"], None), _held_exact(s["B"]).T)
    return x, _silu_pairs_exact(y) if case["gated"] else y
