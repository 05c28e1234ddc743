"""Attention over a shared prefix (wq_prefix_attention) against the fp64 definition.

Tolerance, with p the softmax weights, E = max_j scale sum_d |q_d k_jd|: a score is an fp32 sum of up to 128 exact
products, off by at most 128 2^-24 E = 2^-17 E (any order), and so is its weight, relatively, next to 2^-20 for the
powers of two and sums; a weight is rounded to bf16 for the product with v (2^-8 at most); the quotient repeats the
weights' error but for the rounding.  So |out - exact| <= 2^-8 |exact| + (2^-8 + 2 (2^-17 E + 2^-20)) (1 + 2^-6)
sum_j p_j |v_j|, and |lse - exact| <= 2^-17 E + 2^-20 + 2^-22 |exact|."""
import numpy as np
import pytest
import torch

import weight_only_bit_w4a16_gb300 as wq
from oracle import heads as ref

pytestmark = pytest.mark.gpu


def dev():
    return torch.device("cuda:0")


def f64(t):
    return t.detach().double().cpu().numpy()


class Batch:
    """A batch with its cache: pages in random order, garbage (NaN, infinities) in every slot past a length."""

    def __init__(self, qlens, klens, Hq, Hkv, D, prefix, page, seed=0, heads_first=False, pad_tokens=0, uniform=False,
                 scale_q=1.0):
        g = torch.Generator(device=dev()).manual_seed(seed)
        B = len(qlens)
        self.qlens, self.klens, self.prefix, self.page = list(qlens), list(klens), prefix, page
        need = [(n + page - 1) // page for n in klens]
        npre = (prefix + page - 1) // page
        pages = npre + sum(need) + 2
        shape = (2, pages, Hkv, page, D) if heads_first else (2, pages, page, Hkv, D)
        store = torch.randn(shape, generator=g, device=dev()).to(torch.bfloat16)
        if heads_first:
            store = store.transpose(2, 3)
        self.cache = wq.KVCache(store[0], store[1])
        order = torch.randperm(pages, generator=g, device=dev()).int()
        self.prefix_pages = order[:npre].contiguous() if npre else None
        width = max(need + [0]) + 1
        self.tables = torch.full((B, width), 1 << 30, dtype=torch.int32, device=dev())
        at = npre
        bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device=dev()).to(torch.bfloat16)
        for b, n in enumerate(need):
            self.tables[b, :n] = order[at:at + n]
            at += n
        spans = [(self.tables[b], n) for b, n in enumerate(klens)] + ([(order[:npre], prefix)] if npre else [])
        for table, n in spans:
            if n % page:
                p = int(table[n // page])
                for i, s in enumerate(range(n % page, page)):
                    self.cache.k[p, s] = bad[i % 3]
                    self.cache.v[p, s] = bad[(i + 1) % 3]
        for p in order[at:]:
            self.cache.k[p] = bad[0]
            self.cache.v[p] = bad[1]
        starts = np.concatenate(([0], np.cumsum(qlens))).astype(np.int32)
        self.q_start = None if uniform else torch.from_numpy(starts).to(dev())
        self.starts = starts
        self.T = int(starts[-1]) + pad_tokens
        self.q = (scale_q * torch.randn(self.T, Hq, D, generator=g, device=dev())).to(torch.bfloat16)
        self.lens = torch.tensor(klens, dtype=torch.int32, device=dev())

    def call(self, **kw):
        args = dict(prefix_pages=self.prefix_pages, prefix_len=self.prefix, q_start=self.q_start)
        args.update(kw)
        return wq.prefix_attention(self.q, self.cache, self.lens, self.tables, **args)

    def reference(self, scale=None):
        k, v = f64(self.cache.k), f64(self.cache.v)
        return ref.attention(f64(self.q), k, v, self.tables.cpu().numpy(), self.klens,
                             None if self.prefix_pages is None else self.prefix_pages.cpu().numpy(), self.prefix,
                             self.starts, self.q.shape[2] ** -0.5 if scale is None else scale)


def compare(out, lse, want, what=""):
    o, l, spread, reach = want
    live = ~np.isnan(l)
    E = reach[..., None]
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2 * (2.0 ** -17 * E + 2.0 ** -20)) * (1 + 2.0 ** -6) * spread
    err = np.abs(f64(out) - o)
    bad = ~(err <= tol) & live[..., None]
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside; worst {np.nanmax(err[live] - tol[live])}"
    if lse is not None:
        got = f64(lse)
        none = live & np.isinf(l)
        assert (got[none] == -np.inf).all()
        some = live & np.isfinite(l)
        tol = 2.0 ** -17 * reach + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(some, l, 0.0))
        assert (np.abs(got[some] - l[some]) <= tol[some]).all(), f"{what}: lse"


def run(b, scale=None, what=""):
    lse = torch.full((b.T, b.q.shape[1]), 5.0, device=dev())
    out = torch.full_like(b.q, 3.0)
    got = b.call(scale=scale, out=out, lse=lse)
    torch.cuda.synchronize()
    assert wq.wq_get_device_error() == wq.WQ_OK
    assert got is out
    compare(out, lse, b.reference(scale), what)
    end = int(b.starts[-1])
    assert (out[end:] == 3.0).all() and (lse[end:] == 5.0).all()   # rows behind the last sequence
    return out, lse


@pytest.mark.parametrize("group,kv", [(1, 3), (4, 2), (5, 1), (7, 2), (8, 1), (12, 1), (16, 2)])
@pytest.mark.parametrize("D", [128, 64, 80, 8])
def test_single_tokens(group, kv, D):
    run(Batch([1] * 5, [1, 17, 16, 100, 333], group * kv, kv, D, 77, 16, seed=group + D), what=f"{group} {kv} {D}")


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 127, 128, 129, 1000, 4097])
@pytest.mark.parametrize("B", [1, 9, 40])
def test_prefix_lengths(prefix, B):
    run(Batch([1] * B, [(37 * i) % 90 + 1 for i in range(B)], 8, 2, 128, prefix, 64, seed=prefix + B))


@pytest.mark.parametrize("page", [16, 32, 48, 112, 128, 256, 1024])
@pytest.mark.parametrize("B,D", [(3, 128), (30, 72)])
def test_page_sizes(page, B, D):
    run(Batch([1] * B, [(53 * i) % 300 + 1 for i in range(B)], 4, 2, D, 777, page, seed=page, heads_first=page % 32 == 0))


@pytest.mark.parametrize("qlens,klens,prefix", [
    ([2, 1, 5, 3], [2, 40, 100, 7], 60),              # drafts: a few tokens each
    ([0, 3, 0, 0, 2, 0], [9, 50, 0, 1, 2, 0], 40),    # sequences without tokens
    ([1, 1, 2], [0, 0, 0], 33),                       # no keys of their own
    ([3, 2, 1], [1, 2, 0], 0),                        # more tokens than keys: the first see none at all
    ([1, 1], [0, 0], 0),                              # no key anywhere
    ([100], [100], 0),                                # a prompt without a prefix
    ([33, 70, 129, 5], [33, 90, 400, 5], 300),        # prompts, causal
    ([257, 1, 64], [300, 1, 64], 1),
    ([600], [1000], 150),
    ([300, 250], [10, 0], 0),                         # whole row tiles that see no key
    ([1, 1, 1, 200], [5, 300, 0, 200], 100),          # single tokens beside a prompt
    ([40, 1, 30, 2], [40, 77, 300, 9], 500),
])
@pytest.mark.parametrize("group,D", [(4, 128), (3, 64)])
def test_several_tokens(qlens, klens, prefix, group, D):
    run(Batch(qlens, klens, 2 * group, 2, D, prefix, 32, seed=len(qlens) + prefix, pad_tokens=3))


@pytest.mark.parametrize("small,large,kv", [(10, 60, 2), (1, 140, 1), (32, 33, 3)])
def test_small_and_large_prompts_share_runs(small, large, kv):
    """Units of one and of two row tiles follow each other in a run, over many turns of the ring."""
    B = 24
    run(Batch([small if i % 2 else large for i in range(B)], [small + i if i % 2 else large + i for i in range(B)], 4 * kv,
              kv, 64, 2300, 32, seed=small))


@pytest.mark.parametrize("group,kv,D", [(4, 8, 128), (12, 3, 64), (6, 5, 128), (1, 32, 72)])
@pytest.mark.parametrize("prefix,longest", [(300, 100), (0, 9000), (5000, 9000)])
def test_many_rows_of_few_tokens_each(group, kv, D, prefix, longest):
    """More than 8192 rows, joined by warps; one sequence's keys in many parts; tokens without a key, and none."""
    qlens = [(5 * i) % 9 for i in range(80)]
    klens = [(7 * i) % 50 + (3 if i % 5 else 0) for i in range(80)]
    klens[11] = longest
    assert sum(qlens) * group * kv > 8192
    run(Batch(qlens, klens, group * kv, kv, D, prefix, 16, seed=group, pad_tokens=3), what=f"{group} {kv} {D}")


@pytest.mark.parametrize("tokens,group,kv", [(64, 8, 2), (47, 8, 3), (49, 8, 1), (96, 8, 8), (130, 8, 1), (250, 8, 2),
                                             (255, 8, 1), (260, 8, 1), (120, 12, 11)])
@pytest.mark.parametrize("prefix", [200, 9000])
def test_tiles_of_rows_that_share_keys(tokens, group, kv, prefix):
    """One token a sequence, two to nine tiles of 256 rows a key head, the last from a few rows to all."""
    run(Batch([1] * tokens, [(11 * i) % 70 + 1 for i in range(tokens)], group * kv, kv, 64, prefix, 32, seed=tokens),
        what=f"{tokens} {group}")


@pytest.mark.parametrize("prefix", [1000, 20000])
def test_tiles_of_rows_with_no_own_keys(prefix):
    """Sequences without keys: the prefix alone is on the line."""
    b = Batch([1] * 72, [0] * 72, 32, 4, 128, prefix, 64, seed=9, pad_tokens=2)
    b.qlens = [1] * 72
    run(b)


@pytest.mark.parametrize("B", [65, 300, 1024])
def test_many_sequences(B):
    run(Batch([1] * B, [(29 * i) % 40 for i in range(B)], 2, 1, 64, 50, 16, seed=B))


def test_uniform_tokens_need_no_starts():
    b = Batch([3] * 4, [10, 3, 60, 5], 8, 2, 128, 100, 16, uniform=True)
    out, lse = run(b)
    b.q_start = torch.from_numpy(b.starts).to(dev())
    out2, lse2 = run(b)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_one_sequence_and_long_keys():
    run(Batch([1], [20011], 4, 1, 128, 9001, 64, seed=1))
    run(Batch([1], [1], 1, 1, 128, 30000, 256, seed=2))


@pytest.mark.parametrize("scale_q,scale", [(8.0, None), (1.0, 3.0), (0.0, None), (1.0, 1e-6), (30.0, 1.0)])
@pytest.mark.parametrize("B", [4, 60])
def test_score_ranges(scale_q, scale, B):
    """Peaked, flat and huge scores (a maximum that rises late moves all sums)."""
    b = Batch([1] * B, [40 + i for i in range(B)], 4, 1, 128, 600, 32, seed=5, scale_q=scale_q)
    # keys that grow along the prefix
    for i, p in enumerate(b.prefix_pages.tolist()):
        b.cache.k[p] = b.cache.k[p] * (0.1 + 0.1 * i)
        b.cache.v[p] = b.cache.v[p].nan_to_num(0.0, 0.0, 0.0)
    b.cache.k.nan_to_num_(0.0, 0.0, 0.0)
    run(b, scale)


@pytest.mark.parametrize("T,group", [(4, 4), (50, 4)])
def test_strided_and_in_place(T, group):
    """q a slice of a q/k/v array, out q itself or heads first."""
    Hq, Hkv, D = 2 * group, 2, 128
    b = Batch([1] * T, [20 + i for i in range(T)], Hq, Hkv, D, 200, 16, seed=6)
    want = b.call()
    wide = torch.randn(T, (Hq + 2 * Hkv) * D + 8, device=dev()).to(torch.bfloat16)
    view = wide[:, :Hq * D].unflatten(1, (Hq, D))
    view.copy_(b.q)
    plain, b.q = b.q, view
    out = torch.empty(Hq, T, D, dtype=torch.bfloat16, device=dev()).transpose(0, 1)
    assert torch.equal(b.call(out=out), want)
    before = wide[:, Hq * D:].clone()
    assert torch.equal(b.call(out=view), want)
    assert torch.equal(wide[:, Hq * D:], before)


@pytest.mark.parametrize("group,D,each", [(4, 128, 50), (3, 64, 200), (4, 128, 20)])
def test_prompts_in_place(group, D, each):
    """out is q, with units of many rows: what is stored early is nobody else's query."""
    b = Batch([each] * 7, [each + 30 * i for i in range(7)], 2 * group, 2, D, 2000, 64, seed=61)
    want = b.call()
    got = b.call(out=b.q)
    assert got is b.q and torch.equal(got, want)


def test_starts_that_descend_touch_nothing_else():
    """Against the contract, but memory stays whole: no row outside out is written, and the next call is right."""
    b = Batch([4] * 40, [30 + i for i in range(40)], 8, 2, 128, 300, 16, seed=62, pad_tokens=5)
    want = b.call()
    pool = torch.full((b.T + 64, 8, 128), 3.0, dtype=torch.bfloat16, device=dev())
    ws = wq.prefix_attention_workspace(b.T, 40, 8, 2, 128, dev())
    guard = torch.zeros(ws.numel() + 4096, dtype=torch.uint8, device=dev())
    for starts in ([160 if i % 2 else 0 for i in range(41)], [160 - 4 * i for i in range(41)], [2 ** 31 - 1] * 41,
                   [-2 ** 31] * 41, [0] * 40 + [165]):
        guard.fill_(0x5A)
        b.call(q_start=torch.tensor(starts, dtype=torch.int32, device=dev()), out=pool[32:-32], workspace=guard[:ws.numel()])
        torch.cuda.synchronize()
        assert wq.wq_get_device_error() == wq.WQ_OK
        assert (pool[:32] == 3.0).all() and (pool[-32:] == 3.0).all() and (guard[ws.numel():] == 0x5A).all()
    assert torch.equal(b.call()[:160], want[:160])


@pytest.mark.parametrize("T,tokens", [(3, 1), (70, 1), (6, 60)])
def test_repeats_its_bits_whatever_the_workspace_holds(T, tokens):
    b = Batch([tokens] * T, [tokens + (13 * i) % 200 for i in range(T)], 8, 2, 128, 3000, 64, seed=7)
    ws = wq.prefix_attention_workspace(T * tokens, T, 8, 2, 128, dev())
    want = b.call(workspace=ws)
    for fill in (0, 0xFF, 0x7F):
        ws.fill_(fill)
        assert torch.equal(b.call(workspace=ws), want)


@pytest.mark.parametrize("T", [3, 70])
def test_captured_call_follows_the_lengths(T):
    b = Batch([1] * T, [100] * T, 8, 2, 128, 500, 32, seed=8)
    b.cache.k.nan_to_num_(0.0, 0.0, 0.0)
    b.cache.v.nan_to_num_(0.0, 0.0, 0.0)
    ws = wq.prefix_attention_workspace(T, T, 8, 2, 128, dev())
    out = torch.empty_like(b.q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.call(workspace=ws, out=out)
    for n in (100, 0, 1, 57, 99):
        b.klens = [(n * (i + 1)) % 101 for i in range(T)]
        b.lens.copy_(torch.tensor(b.klens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        compare(out, None, b.reference(), f"length {n}")


def test_two_streams_with_a_workspace_each():
    """Calls at the same time: the results of calls one after the other."""
    batches = [Batch([1] * n, [(31 * i) % 500 for i in range(n)], 8, 2, 128, 6000, 64, seed=n) for n in (20, 64)]
    want = [b.call() for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    spaces = [wq.prefix_attention_workspace(b.T, b.T, 8, 2, 128, dev()) for b in batches]
    outs = [torch.empty_like(b.q) for b in batches]
    torch.cuda.synchronize()
    for _ in range(10):
        for b, s, w, o in zip(batches, streams, spaces, outs):
            b.call(stream=s, workspace=w, out=o)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("qlens,more,prefix", [([2300], 0, 0), ([1290], 500, 40), ([1500, 1, 1100], 3, 200),
                                               ([0, 1100, 0], 7, 0), ([40] * 12 + [1100], 0, 70)])
def test_long_prompts(qlens, more, prefix):
    """Tens of row tiles a sequence, more than a warp looks over at a time."""
    b = Batch(qlens, [n + more for n in qlens], 8, 1, 64, prefix, 64, seed=len(qlens), pad_tokens=1)
    assert max(qlens) * 8 > 32 * 256
    run(b)


@pytest.mark.parametrize("group,kv", [(4, 1), (3, 2), (5, 1)])
@pytest.mark.parametrize("prompt,keys", [(700, 700), (700, 1003), (700, 350), (650, 3), (300, 77)])
def test_one_prompt_among_single_tokens(group, kv, prompt, keys):
    """Hundreds of small row tiles of one sequence, some or all of its tokens without a key of their own."""
    qlens = [1] * 40 + [prompt] + [2] * 50
    assert sum(qlens) * group < 64 * len(qlens)
    klens = [5 + i for i in range(40)] + [keys] + [2 + i for i in range(50)]
    for prefix in (0, 60):
        run(Batch(qlens, klens, group * kv, kv, 64, prefix, 16, seed=keys + prefix, pad_tokens=2))


def test_what_a_call_allocates_is_of_its_stream(monkeypatch):
    """A workspace of the current stream's memory could go to another tensor while the call still runs."""
    b = Batch([1] * 6, [40] * 6, 8, 2, 128, 300, 16, seed=3)
    side = torch.cuda.Stream()
    seen = []
    empty = torch.empty

    def spy(*args, **kw):
        seen.append(torch.cuda.current_stream())
        return empty(*args, **kw)

    torch.cuda.synchronize()
    with monkeypatch.context() as m:
        m.setattr(torch, "empty", spy)
        out = b.call(stream=side)
        q, k = wq.head_rope(b.q, b.q[:, :2], table=None, stream=side)
    torch.cuda.synchronize()
    assert len(seen) == 4 and all(s == side for s in seen)
    compare(out, None, b.reference())


def test_lengths_past_the_table_are_cut_and_negative_ones_are_none():
    b = Batch([1] * 3, [32, 32, 32], 4, 2, 64, 40, 16, seed=11)
    b.tables = b.tables[:, :2].contiguous()
    want = b.call()
    b.lens.copy_(torch.tensor([2 ** 31 - 1, 33, 32], dtype=torch.int32))
    assert torch.equal(b.call(), want)
    b.lens.copy_(torch.tensor([-5, -2 ** 31, 0], dtype=torch.int32))
    b.klens = [0, 0, 0]
    run(b)


@pytest.mark.parametrize("B", [3, 50])
def test_pages_outside_the_cache_read_as_zeros(B):
    b = Batch([1] * B, [64] * B, 4, 2, 128, 64, 16, seed=12)
    b.tables[0, 1] = -1
    b.tables[1, 2] = 1 << 30
    b.prefix_pages[2] = -7
    run(b)


@pytest.mark.parametrize("B,tokens", [(2, 1), (40, 1), (5, 60)])
def test_waits_that_run_out(B, tokens, monkeypatch):
    """The failure path, without a fault or a hang: with the bound of the waits for blocks and scores at 0
    (WQ_ATTN_WAIT_NS, read at launch) every CTA gives up at once; its copies and matrix instructions drain under
    bounds of their own, tensor memory is freed and the timeout is recorded.  The next call is right."""
    b = Batch([tokens] * B, [tokens + 20 + i for i in range(B)], 8, 2, 128, 1500, 32, seed=63)
    assert wq.wq_get_device_error() == wq.WQ_OK
    monkeypatch.setenv("WQ_ATTN_WAIT_NS", "0")
    b.call()
    torch.cuda.synchronize()
    assert wq.wq_get_device_error() == wq.WQ_ERR_DEVICE_TIMEOUT
    assert wq.wq_get_device_error() == wq.WQ_OK
    monkeypatch.delenv("WQ_ATTN_WAIT_NS")
    run(b)


def test_follows_the_writes_before_it():
    """The chain of a decode step on one stream, no synchronisation between: the projection's array is rotated, the keys
    are stored, and the attention reads them."""
    T, Hq, Hkv, D, page = 24, 8, 2, 128, 16
    b = Batch([1] * T, [5 + i for i in range(T)], Hq, Hkv, D, 333, page, seed=13)
    table = wq.rope_table(D, device=dev())
    at = b.lens - 1
    pos = at + b.prefix
    slots = (b.tables.gather(1, (at // page).long().unsqueeze(1))[:, 0] * page + at % page).int()
    big = torch.randn(1 << 24, device=dev())
    for step in range(3):
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, device=dev()).to(torch.bfloat16)
        q, k, v = (qkv[:, x * D:y * D].unflatten(1, (y - x, D)) for x, y in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
        torch.cuda.synchronize()
        big.mul_(1.0)   # the calls queue behind it
        b.q, _ = wq.head_rope(q, k, v, table=table, positions=pos, cache=b.cache, slots=slots)
        out = b.call()
        torch.cuda.synchronize()
        compare(out, None, b.reference())


@pytest.mark.parametrize("bad", ["q type", "cache size", "lens", "tables", "prefix", "starts", "lse", "workspace",
                                 "small workspace", "page size", "out"])
def test_refusals(bad):
    b = Batch([1] * 3, [5, 6, 7], 4, 2, 64, 20, 16)
    kw, err = {}, ValueError
    if bad == "q type":
        b.q = b.q.float()
    elif bad == "cache size":
        b.q = b.q[..., :32].contiguous()
    elif bad == "lens":
        b.lens = b.lens.long()
    elif bad == "tables":
        b.tables = b.tables[:2]
    elif bad == "prefix":
        kw, err = dict(prefix_len=33), wq.WQError
    elif bad == "starts":
        kw = dict(q_start=b.q_start[:3])
    elif bad == "lse":
        kw = dict(lse=torch.empty(3, 4, dtype=torch.bfloat16, device=dev()))
    elif bad == "workspace":
        kw = dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))
    elif bad == "small workspace":
        kw, err = dict(workspace=torch.empty(1024, dtype=torch.uint8, device=dev())), wq.WQError
    elif bad == "page size":
        kv = torch.zeros(2, 4, 24, 2, 64, dtype=torch.bfloat16, device=dev())
        b.cache, err = wq.KVCache(kv[0], kv[1]), wq.WQError
    elif bad == "out":
        kw = dict(out=torch.empty(3, 4, 128, dtype=torch.bfloat16, device=dev())[..., ::2])
    with pytest.raises(err):
        b.call(**kw)
