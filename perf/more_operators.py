"""The operators between the q/k/v projection and the output projection, measured: norms of query and key heads with
the position rotation (one axis or several) and the write into the cache, attention of a batch that shares a prefix,
and a decode step of both.

`own` false: plain torch operations in 32 bits (angles in 64).  `own` true: the calls a user makes of the library.
"""
import math

import torch

own = False

EPS = 1e-6


def dev():
    return torch.device("cuda")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoded token far into its context: norms, rotation, k and v into the cache
        dict(name="rotate token", op="rotate", tokens=1, kv=8, group=4, D=128, R=128, norm="rms", bias=False,
             dtype="bf16", pairs="halves", sections="", ladder="shared", theta=500000.0, far=130000, page=64, pad=0),
        # a decode batch, seven query heads to a key head, half of each head rotated, q, k and v slices of one array
        dict(name="rotate batch", op="rotate", tokens=129, kv=4, group=7, D=128, R=64, norm="none", bias=False,
             dtype="bf16", pairs="halves", sections="", ladder="shared", theta=10000.0, far=8000, page=16, pad=1),
        # a prompt into the cache
        dict(name="rotate prompt", op="rotate", tokens=8192, kv=8, group=4, D=128, R=128, norm="rms", bias=False,
             dtype="bf16", pairs="halves", sections="", ladder="shared", theta=500000.0, far=0, page=64, pad=1),
        # frames of a video and their text: three axes (time, height, width) that share one ladder of frequencies
        dict(name="rotate video", op="rotate", tokens=6007, kv=4, group=7, D=128, R=128, norm="rms", bias=False,
             dtype="bf16", pairs="halves", sections="16,24,24", ladder="shared", theta=1000000.0, far=2000, page=0, pad=0),
        # patches of an image in an encoder: two axes with a ladder each, layer norms, 32-bit activations, odd head size
        dict(name="rotate patches", op="rotate", tokens=1521, kv=16, group=1, D=72, R=72, norm="layer", bias=True,
             dtype="fp32", pairs="adjacent", sections="18,18", ladder="own", theta=10000.0, far=0, page=0, pad=0),
        # two short chats on one short system prompt: latency
        dict(name="attend pair", op="attend", B=2, qlo=1, qhi=1, kv=8, group=4, D=128, prefix=512, lo=5, hi=64, page=16),
        # a decode batch on a shared document
        dict(name="attend batch", op="attend", B=16, qlo=1, qhi=1, kv=8, group=4, D=128, prefix=8192, lo=100, hi=1000,
             page=64),
        # a wide decode batch of agents on one long instruction, with contexts of their own
        dict(name="attend agents", op="attend", B=64, qlo=1, qhi=1, kv=8, group=4, D=128, prefix=32768, lo=200, hi=3000,
             page=128),
        # drafted tokens checked together: a few queries a sequence, odd sizes throughout
        dict(name="attend draft", op="attend", B=13, qlo=1, qhi=5, kv=4, group=5, D=80, prefix=1999, lo=5, hi=700,
             page=48),
        # questions on a whole book, eight query heads to a key head
        dict(name="attend long", op="attend", B=64, qlo=1, qhi=1, kv=8, group=8, D=128, prefix=131072, lo=64, hi=1024,
             page=256),
        # prompts of a batch read after the shared prefix: causal over their own tokens
        dict(name="attend prompts", op="attend", B=8, qlo=100, qhi=600, kv=8, group=4, D=128, prefix=8192, lo=0, hi=300,
             page=64),
        # a decode step: rotate and store the new tokens, then attend
        dict(name="rotate and attend", op="step", B=32, qlo=1, qhi=1, kv=8, group=4, D=128, prefix=4096, lo=100, hi=800,
             page=64, R=128, norm="rms", bias=False, dtype="bf16", pairs="halves", sections="", ladder="shared",
             theta=500000.0, far=0, pad=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rotation(rng, D):
    R = rng.choice([D, D, D, D // 2, 2 * max(1, round(0.2 * D))])
    sections, ladder = "", "shared"
    kind = rng.choice(["one", "one", "two", "three"])
    if kind != "one" and R >= 12:
        n = R // 2
        a = rng.randint(1, n - 2)
        parts = [a, n - a] if kind == "two" else [a, (n - a + 1) // 2, (n - a) // 2]
        sections = ",".join(str(p) for p in parts if p > 0)
        ladder = rng.choice(["shared", "own"])
    return dict(R=R, norm=rng.choice(["rms", "rms", "layer", "none"]), bias=rng.random() < 0.25,
                pairs=rng.choice(["halves", "halves", "adjacent"]), sections=sections, ladder=ladder,
                theta=rng.choice([100.0, 10000.0, 500000.0]), far=rng.choice([0, 1000, 100000, 1000000]),
                pad=rng.choice([0, 1]))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "attend", "attend", "attend", "step"])
    if op == "rotate":
        D = rng.choice([64, 72, 80, 96, 128, 128, 160, 256])
        kv, group = _log(rng, 1, 16), _log(rng, 1, 12)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        top = (1 << 25) // (kv * (group + 2) * D)
        return dict(op=op, tokens=max(1, min(_log(rng, 1, 16384), top)), kv=kv, group=group, D=D, dtype=dtype,
                    page=rng.choice([0, 16, 48, 64, 256]) if dtype == "bf16" else 0, **_draw_rotation(rng, D))
    D = rng.choice([64, 72, 80, 96, 128, 128])
    kv, group = _log(rng, 1, 16), _log(rng, 1, 12)
    B = _log(rng, 1, 128)
    case = dict(op=op, B=B, qlo=1, qhi=1, kv=kv, group=group, D=D, prefix=_log(rng, 16, 131072), lo=0, hi=0,
                page=rng.choice([16, 32, 48, 64, 128, 256, 1024]))
    if op == "attend":
        kind = rng.choice(["tokens", "tokens", "draft", "prompts"])
        if kind == "draft":
            case["qhi"] = rng.randint(2, 8)
        elif kind == "prompts":
            case["qlo"] = _log(rng, 1, 200)
            case["qhi"] = case["qlo"] + _log(rng, 1, 1000)
            case["prefix"] = min(case["prefix"], 16384)
    case["lo"] = _log(rng, 1, 1000)
    case["hi"] = case["lo"] + _log(rng, 1, 4000)
    if op == "step":
        case.update(_draw_rotation(rng, D), dtype="bf16")
        case["far"] = 0
    # within the cost of the largest listed cases
    while work(case)["flops"] > 2e11 or work(case)["bytes"] > 5e8:
        if case["B"] > 1 and (case["qhi"] > 8 or case["prefix"] < 4096):
            case["B"] = (case["B"] + 1) // 2
        else:
            case["prefix"] = (case["prefix"] + 1) // 2
            case["lo"] = (case["lo"] + 1) // 2
            case["hi"] = case["lo"] + (case["hi"] + 1) // 2
    return case


def _ragged(n, lo, hi, salt):
    """n lengths spread over lo .. hi, the ends among them."""
    out = [lo + (i * 2654435761 + salt * 40503) % 4294967296 * (hi - lo + 1) // 4294967296 for i in range(n)]
    if n > 1:
        out[n // 2], out[n - 1] = lo, hi
    return out


def _lengths(case):
    """Queries of each sequence, and its own keys (the new tokens' among them)."""
    q = _ragged(case["B"], case["qlo"], case["qhi"], 1)
    return q, [n + m for n, m in zip(q, _ragged(case["B"], case["lo"], case["hi"], 2))]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=dev(), dtype=torch.float32)


def _bf16(t):
    return t.to(torch.bfloat16)


def _axes(case):
    """For each rotated pair its axis and its frequency (Python floats, 64 bits)."""
    n = case["R"] // 2
    parts = [int(p) for p in case["sections"].split(",")] if case["sections"] else [n]
    axis, freq = [], []
    for a, p in enumerate(parts):
        for j in range(p):
            axis.append(a)
            freq.append(case["theta"] ** (-(j / p if case["ladder"] == "own" else len(freq) / n)))
    return axis, freq, len(parts)


def _rotation_inputs(s, g, tokens, positions):
    D, kv, heads = s["D"], s["kv"], s["kv"] * s["group"]
    f32 = s["dtype"] == "fp32"
    # q, k and v side by side, as one projection writes them; a few loud channels
    qkv = _normal(g, tokens, (heads + 2 * kv) * D + 8 * s["pad"])
    qkv[:, ::61] *= 5.0
    qkv = qkv if f32 else _bf16(qkv)
    s["q"] = qkv[:, :heads * D].view(tokens, heads, D)
    s["k"] = qkv[:, heads * D:(heads + kv) * D].view(tokens, kv, D)
    s["v"] = qkv[:, (heads + kv) * D:(heads + 2 * kv) * D].view(tokens, kv, D)
    normed = s["norm"] != "none"
    # weights above one keep the scores of a trained model's spread
    s["wq"] = _bf16(1.4 + 0.1 * _normal(g, D)) if normed else None
    s["wk"] = _bf16(1.4 + 0.1 * _normal(g, D)) if normed else None
    s["bq"] = _bf16(0.1 * _normal(g, D)) if normed and s["bias"] else None
    s["bk"] = _bf16(0.1 * _normal(g, D)) if normed and s["bias"] else None
    axis, freq, axes = _axes(s)
    s["axis"] = torch.tensor(axis, device=dev())
    s["freq"] = torch.tensor(freq, dtype=torch.float64, device=dev())
    s["positions"] = positions if axes == 1 else torch.stack(
        [positions] + [torch.randint(0, 200, (tokens,), generator=g, device=dev()).int() for _ in range(axes - 1)])
    s["q_out"] = torch.empty((tokens, heads, D), dtype=qkv.dtype, device=dev())
    if own:
        import weight_only_bit_w4a16_gb300 as wq

        s["table"] = wq.rope_table(s["R"], inv_freq=freq, axis=axis, device=dev())


def _cache(g, pages, page, kv, D):
    k = torch.empty((pages, page, kv, D), dtype=torch.bfloat16, device=dev())
    v = torch.empty_like(k)
    for p in range(0, pages, 512):
        k[p:p + 512] = _normal(g, *k[p:p + 512].shape)
        v[p:p + 512] = _normal(g, *v[p:p + 512].shape)
    return k, v


def prepare(case, seed):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    s = dict(case)
    kv, heads, D = s["kv"], s["kv"] * s["group"], s["D"]
    if s["op"] == "rotate":
        T = s["tokens"]
        positions = (s["far"] + torch.arange(T, device=dev())).int()
        _rotation_inputs(s, g, T, positions)
        s["k_out"] = torch.empty((T, kv, D), dtype=s["q"].dtype, device=dev())
        if s["page"]:
            pages = (T + s["page"] - 1) // s["page"] + 2
            s["ck"], s["cv"] = _cache(g, pages, s["page"], kv, D)
            order = torch.randperm(pages, generator=g, device=dev())
            slots = (order[:, None] * s["page"] + torch.arange(s["page"], device=dev())).view(-1)
            s["slots"] = slots[3:3 + T].int()
            if own:
                import weight_only_bit_w4a16_gb300 as wq

                s["cache"] = wq.KVCache(s["ck"], s["cv"])
        return s
    qlens, klens = _lengths(s)
    B, P, page = s["B"], s["prefix"], s["page"]
    T = sum(qlens)
    own_pages = [(n + page - 1) // page for n in klens]
    prefix_pages = (P + page - 1) // page
    pages = prefix_pages + sum(own_pages) + 3
    order = torch.randperm(pages, generator=g, device=dev()).int()
    s["ck"], s["cv"] = _cache(g, pages, page, kv, D)
    s["prefix_pages"] = order[:prefix_pages].contiguous()
    tables = torch.zeros((B, max(own_pages)), dtype=torch.int32)
    host, at = order.cpu(), prefix_pages
    for b, n in enumerate(own_pages):
        tables[b, :n] = host[at:at + n]
        at += n
    s["tables"] = tables.to(dev())
    s["lens"] = torch.tensor(klens, dtype=torch.int32, device=dev())
    starts = [0]
    for n in qlens:
        starts.append(starts[-1] + n)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev())
    s["qmax"], s["kmax"] = max(qlens), max(klens)
    # the sequence of each query token and its place among the sequence's queries
    s["seq"] = torch.repeat_interleave(torch.arange(B, device=dev()), s["starts"].diff())
    s["place"] = torch.arange(T, device=dev()) - s["starts"][s["seq"]]
    s["scale"] = D ** -0.5
    s["out"] = torch.empty((T, heads, D), dtype=torch.bfloat16, device=dev())
    if s["op"] == "step":
        at = s["lens"] - 1
        _rotation_inputs(s, g, T, (at + P).int())
        s["slots"] = (s["tables"].gather(1, (at // page).long().unsqueeze(1))[:, 0] * page + at % page).int()
    else:
        # queries with a common direction, which the prefix's first key answers (the sink of a trained model)
        u = _normal(g, kv, 1, D)
        s["q"] = _bf16(2.0 * _normal(g, T, kv, s["group"], D) + u).view(T, heads, D)
        if P:
            s["ck"][s["prefix_pages"][0], 0] = _bf16(8.0 / math.sqrt(D) * u[:, 0] + 0.3 * _normal(g, kv, D))
    if own:
        import weight_only_bit_w4a16_gb300 as wq

        s["cache"] = wq.KVCache(s["ck"], s["cv"])
        s["workspace"] = wq.prefix_attention_workspace(T, B, heads, kv, D, device=dev())
    return s


# ---------------------------------------------------------------------------
# the plain forms, 32 bits
# ---------------------------------------------------------------------------
def _norm_plain(x, w, b, kind):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    return y if b is None else y + b.float()


def _rotate_plain(s, x):
    """Pairs of the first R values turned by position times frequency (angles in 64 bits)."""
    n = s["R"] // 2
    pos = s["positions"].view(-1, x.shape[0]).double()
    angle = pos[s["axis"]].t() * s["freq"]
    cos, sin = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    if s["pairs"] == "halves":
        a, b, rest = x[..., :n], x[..., n:2 * n], x[..., 2 * n:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1)
    a, b, rest = x[..., 0:2 * n:2], x[..., 1:2 * n:2], x[..., 2 * n:]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), rest), -1)


def _heads_plain(s):
    q = _rotate_plain(s, _norm_plain(s["q"].float(), s["wq"], s["bq"], s["norm"])).to(s["q"].dtype)
    k = _rotate_plain(s, _norm_plain(s["k"].float(), s["wk"], s["bk"], s["norm"])).to(s["q"].dtype)
    return q, k


def _store_plain(s, k):
    pages, page, kv, D = s["ck"].shape
    s["ck"].view(pages * page, kv, D)[s["slots"].long()] = k.to(torch.bfloat16)
    s["cv"].view(pages * page, kv, D)[s["slots"].long()] = s["v"].to(torch.bfloat16)


def _attend_plain(s, q):
    T, heads, D = q.shape
    B, kv, G, P, page = s["B"], s["kv"], s["group"], s["prefix"], s["page"]
    pages = s["ck"].shape[0]
    K, V = (c.view(pages * page, kv, D) for c in (s["ck"], s["cv"]))
    at = torch.arange(page, device=q.device)
    q = q.float().view(T, kv, G, D) * s["scale"]
    # the prefix, all queries at once
    rows = (s["prefix_pages"].long()[:, None] * page + at).view(-1)[:P]
    kp, vp = (c[rows].float().transpose(0, 1) for c in (K, V))                   # (kv, P, D)
    sp = torch.matmul(q.transpose(0, 1).reshape(kv, T * G, D), kp.transpose(1, 2))
    # each sequence's own keys, padded to the longest
    n, L = s["qmax"], s["kmax"]
    rows = (s["tables"].long()[:, :, None] * page + at).view(B, -1)[:, :L]
    ks, vs = (c[rows].float().transpose(1, 2) for c in (K, V))                   # (B, kv, L, D)
    token = (s["starts"][:-1, None] + torch.arange(n, device=q.device)).clamp(max=T - 1)
    qs = q[token].permute(0, 2, 1, 3, 4).reshape(B, kv, n * G, D)
    ss = torch.matmul(qs, ks.transpose(2, 3)).view(B, kv, n, G, L)
    seen = s["lens"][:, None] - s["starts"].diff()[:, None] + torch.arange(1, n + 1, device=q.device)
    hidden = torch.arange(L, device=q.device) >= seen[:, :, None]                # (B, n, L)
    ss = ss.masked_fill(hidden[:, None, :, None, :], float("-inf"))
    ss = ss[s["seq"], :, s["place"]]                                             # (T, kv, G, L)
    sp = sp.view(kv, T, G, P).permute(1, 0, 2, 3)
    top = torch.maximum(sp.amax(-1, keepdim=True), ss.amax(-1, keepdim=True))
    pp, ps = torch.exp(sp - top), torch.exp(ss - top)
    total = pp.sum(-1, keepdim=True) + ps.sum(-1, keepdim=True)
    o = torch.matmul(pp.permute(1, 0, 2, 3).reshape(kv, T * G, P), vp).view(kv, T, G, D).transpose(0, 1)
    padded = torch.zeros((B, n, kv, G, L), device=q.device)
    padded[s["seq"], s["place"]] = ps
    os = torch.matmul(padded.transpose(1, 2).reshape(B, kv, n * G, L), vs).view(B, kv, n, G, D)
    return ((o + os[s["seq"], :, s["place"]]) / total).reshape(T, heads, D).to(torch.bfloat16)


def _run_plain(s):
    if s["op"] == "attend":
        return _attend_plain(s, s["q"])
    q, k = _heads_plain(s)
    if s["op"] == "rotate" and not s["page"]:
        return q, k
    _store_plain(s, k)
    return (q if s["op"] == "rotate" else _attend_plain(s, q)), s["ck"], s["cv"]


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _run_own(s):
    import weight_only_bit_w4a16_gb300 as wq

    def rotate(**to):
        return wq.head_rope(s["q"], s["k"], table=s["table"], positions=s["positions"], pairs=s["pairs"],
                            norm=None if s["norm"] == "none" else s["norm"], eps=EPS, q_weight=s["wq"],
                            k_weight=s["wk"], q_bias=s["bq"], k_bias=s["bk"], q_out=s["q_out"], **to)

    def attend(q):
        return wq.prefix_attention(q, s["cache"], s["lens"], s["tables"], prefix_pages=s["prefix_pages"],
                                   prefix_len=s["prefix"], q_start=s["starts"], scale=s["scale"], out=s["out"],
                                   workspace=s["workspace"])

    if s["op"] == "attend":
        return attend(s["q"])
    if s["op"] == "rotate" and not s["page"]:
        return rotate(k_out=s["k_out"])
    q, _ = rotate(v=s["v"], cache=s["cache"], slots=s["slots"])
    return (q if s["op"] == "rotate" else attend(q)), s["ck"], s["cv"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _rotation_work(case, tokens):
    kv, heads, D = case["kv"], case["kv"] * case["group"], case["D"]
    es = 4 if case["dtype"] == "fp32" else 2
    rows = heads + kv + (kv if case["page"] else 0)
    axes = case["sections"].count(",") + 1
    return 2.0 * es * tokens * rows * D + tokens * (4.0 * axes + (4 if case["page"] else 0)), \
        10.0 * tokens * (heads + kv) * D


def _attention_work(case):
    q, k = _lengths(case)
    kv, heads, D = case["kv"], case["kv"] * case["group"], case["D"]
    keys = case["prefix"] + sum(k)
    seen = sum(n * case["prefix"] + n * (m - n) + n * (n + 1) // 2 for n, m in zip(q, k))
    return 4.0 * sum(q) * heads * D + 4.0 * keys * kv * D, 4.0 * D * heads * seen


def work(case):
    if case["op"] == "rotate":
        b, f = _rotation_work(case, case["tokens"])
    else:
        b, f = _attention_work(case)
        if case["op"] == "step":
            rb, rf = _rotation_work(case, case["B"])
            b, f = b + rb, f + rf
    return dict(bytes=b, flops=f)


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------
def _head_exact(s, x, w, b):
    x = x.double()
    D = x.shape[2]
    if s["norm"] == "layer":
        x = x - (x.sum(dim=2) / D)[:, :, None]
    if s["norm"] != "none":
        x = x * torch.rsqrt((x * x).sum(dim=2) / D + EPS)[:, :, None] * w.double()
        if b is not None:
            x = x + b.double()
    y = x.clone()
    pos = s["positions"].double().reshape(-1, x.shape[0])
    axis, freq, _ = _axes(s)
    n = s["R"] // 2
    for i in range(n):
        lo, hi = (i, i + n) if s["pairs"] == "halves" else (2 * i, 2 * i + 1)
        turn = torch.polar(torch.ones_like(pos[0]), pos[axis[i]] * freq[i])[:, None]
        z = torch.complex(x[:, :, lo], x[:, :, hi]) * turn
        y[:, :, lo], y[:, :, hi] = z.real, z.imag
    return y


def _stored_exact(s, rows):
    """The caches with the new rows; `rows` the keys' values."""
    page = s["page"]
    out = []
    for cache, new in ((s["ck"], rows), (s["cv"], s["v"].double())):
        c = cache.double()
        slot = s["slots"].long()
        c[slot // page, slot % page] = new
        out.append(c)
    return out


def _attend_exact(s, q, ck, cv):
    """By heads: the prefix's weights of all queries against the total of each, then each sequence's own."""
    T, heads, D = q.shape
    kv, G, P, page = s["kv"], s["group"], s["prefix"], s["page"]
    qlens, klens = _lengths(s)
    j = torch.arange(P, device=q.device)
    at = s["prefix_pages"].long()[j // page] if P else j
    out = torch.empty((T, heads, D), dtype=torch.float64, device=q.device)
    for h in range(kv):
        qh = q[:, h * G:(h + 1) * G].double().reshape(T * G, D) / math.sqrt(D)
        kp, vp = (c[at, j % page, h].double() for c in (ck, cv))
        sp = torch.mm(qh, kp.T)
        norm_p = torch.logsumexp(sp, dim=1) if P else torch.full((T * G,), -math.inf, dtype=torch.float64,
                                                                 device=q.device)
        total, parts, t = norm_p.clone(), [], 0
        for b, (n, m) in enumerate(zip(qlens, klens)):
            i = torch.arange(m, device=q.device)
            page_of = s["tables"][b].long()[i // page]
            ks, vs = (c[page_of, i % page, h].double() for c in (ck, cv))
            w = torch.mm(qh[t * G:(t + n) * G], ks.T).view(n, G, m)
            reach = torch.ones((n, m), dtype=torch.bool, device=q.device).tril(m - n)
            w = torch.where(reach[:, None, :], w, torch.full_like(w, -math.inf)).view(n * G, m)
            span = slice(t * G, (t + n) * G)
            total[span] = torch.logaddexp(norm_p[span], torch.logsumexp(w, dim=1))
            parts.append((span, w, vs))
            t += n
        o = torch.mm(torch.exp(sp - total[:, None]), vp)
        for span, w, vs in parts:
            o[span] += torch.mm(torch.exp(w - total[span, None]), vs)
        out[:, h * G:(h + 1) * G] = o.view(T, G, D)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "attend":
        return _attend_exact(s, s["q"], s["ck"], s["cv"])
    q, k = _head_exact(s, s["q"], s["wq"], s["bq"]), _head_exact(s, s["k"], s["wk"], s["bk"])
    if s["op"] == "rotate" and not s["page"]:
        return q, k
    ck, cv = _stored_exact(s, k)
    return (q if s["op"] == "rotate" else _attend_exact(s, q, ck, cv)), ck, cv
