"""Decode over a paged cache, with and without shared prompts, against a plain 64-bit
implementation."""
import math

import numpy as np
import pytest
import torch

import dynamic_block_sparse_pooled_b200 as fpx
import serve_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


class Case:
    """Caches with garbage (NaN) wherever no request has a token, tables with -1 where unused."""

    def __init__(self, dtype, ctx, hq, hkv, d, page, q_len=1, groups=None, prefix=None, seed=0,
                 gain=2.0, width=None, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.ctx, self.q_len, self.d = dtype, ctx, q_len, d
        n = len(ctx)
        need = [-(-c // page) for c in ctx]
        width = width or max(1, max(need))
        lead = [None] * n
        if groups:
            for gi in range(len(groups) - 1):
                for s in range(groups[gi], groups[gi + 1]):
                    lead[s] = gi
        shared = prefix or []
        num = sum(shared) + sum(max(0, need[s] - (shared[lead[s]] if lead[s] is not None else 0))
                                for s in range(n)) + spare
        order = np.random.default_rng(seed).permutation(num)
        at = 0
        prompts = []
        for x in shared:
            prompts.append([int(p) for p in order[at:at + x]])
            at += x
        table = np.full((n, width), -1, np.int32)
        self.used = {}
        for s in range(n):
            mine = list(prompts[lead[s]]) if lead[s] is not None else []
            while len(mine) < need[s]:
                mine.append(int(order[at]))
                at += 1
            table[s, :len(mine)] = mine[:width]
            for i, p in enumerate(mine):
                self.used[p] = max(self.used.get(p, 0), min(page, max(0, ctx[s] - i * page)))
        for gi, pr in enumerate(prompts):  # a prompt is whole, whoever reads it
            for p in pr:
                self.used[p] = page
        self.table = table
        shape = (num, page, hkv, d)
        self.q = torch.randn(n * q_len, hq, d, generator=g) * gain
        k, v = torch.randn(shape, generator=g), torch.randn(shape, generator=g)
        self.scales = {}
        if dtype == "e4m3":
            ks, vs = (torch.rand(hkv, generator=g) + 0.5 for _ in range(2))
            k, v = (x * 40 for x in (k, v))
            k, v = (x.to(torch.float8_e4m3fn) for x in (k, v))
            self.k64, self.v64 = k.double() * (ks / 40).double()[:, None], v.double() * (vs / 40).double()[:, None]
            self.scales = {"k_scale": (ks / 40).cuda(), "v_scale": (vs / 40).cuda()}
        else:
            k, v = k.to(DT[dtype]), v.to(DT[dtype])
            self.k64, self.v64 = k.double(), v.double()
        qdt = torch.float32 if dtype == "f32" else torch.bfloat16
        self.q = self.q.to(qdt)
        self.q64 = self.q.double()
        dirty = torch.ones(num, page, dtype=torch.bool)
        for p, c in self.used.items():
            dirty[p, :c] = False
        k, v = k.float(), v.float()
        k[dirty], v[dirty] = float("nan"), float("nan")
        self.k, self.v = k.to(DT[dtype]).cuda(), v.to(DT[dtype]).cuda()
        self.qd = self.q.cuda()
        self.ctx_d = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        self.table_d = torch.from_numpy(table).cuda()
        more = {}
        if groups:
            more = dict(group_ptr=torch.tensor(groups, dtype=torch.int32, device="cuda"),
                        prefix_pages=torch.tensor(shared, dtype=torch.int32, device="cuda"))
        self.dp = fpx.decode_problem(self.qd, self.k, self.ctx_d, self.table_d, q_len,
                                     **self.scales, **more)
        self.ws = fpx.decode_workspace(self.dp)

    def run(self, rule=None, **kw):
        self.ws[256:] = 255  # what earlier calls left in a workspace does not matter
        return fpx.decode(self.dp, self.qd, self.k, self.v, self.ws, rule, **kw)

    def check(self, o, lse, **rule):
        k64, v64 = torch.nan_to_num(self.k64), torch.nan_to_num(self.v64)
        table = [[max(int(p), 0) for p in row] for row in self.table]
        ref = R.decode_reference(self.q64, k64, v64, self.ctx, table, self.q_len,
                                 1 / math.sqrt(self.d), **rule)
        R.check(o, lse, ref, "f16" if self.dtype == "e4m3" else "bf16",
                "f32" if self.dtype == "f32" else "bf16", max(self.ctx + [1]), self.d)


RAGGED = [1, 0, 31, 32, 33, 127, 128, 129, 1000, 300, 2]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_ragged_batch(dtype, d, page):
    c = Case(dtype, RAGGED, 4, 2, d, page)
    c.check(*c.run())
    assert fpx.status(c.ws) == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("hq,hkv,q_len", [(1, 1, 1), (7, 1, 1), (6, 2, 3), (16, 1, 1), (17, 1, 1),
                                          (32, 1, 1), (8, 2, 12), (5, 1, 13), (16, 1, 9), (64, 1, 3)])
def test_heads_and_drafts(dtype, hq, hkv, q_len):
    """Row counts around every tile: 1 to 192 rows of a request share keys."""
    c = Case(dtype, [5, 40, 700, 0, 2], hq, hkv, 128, 32, q_len, seed=2)
    c.check(*c.run())
    assert fpx.status(c.ws) == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("rule", [dict(softcap=7.0), dict(slopes=True), dict(window=1),
                                  dict(window=50), dict(softcap=4.0, slopes=True, window=333),
                                  dict(window=2 ** 31 - 1), dict(softcap=1e5), dict(softcap=1e-3)])
@pytest.mark.parametrize("grouped", [False, True])
def test_rules(dtype, rule, grouped):
    groups = dict(groups=[0, 4, 4, 7], prefix=[3, 2, 9]) if grouped else {}
    ctx = [200, 193, 640, 192 + 2, 600, 576 + 2, 1000, 130]
    c = Case(dtype, ctx, 6, 2, 128, 64, 2, seed=4, **groups)
    kw = dict(rule)
    if kw.get("slopes"):
        kw["slopes"] = torch.pow(2.0, -8.0 * torch.arange(1, 7).double() / 6).float()
    dev = dict(kw)
    if dev.get("slopes") is not None:
        dev["slopes"] = dev["slopes"].cuda()
    c.check(*c.run(fpx.score_rule(**dev)), **kw)
    assert fpx.status(c.ws) == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("d,page", [(128, 128), (128, 16), (64, 32)])
@pytest.mark.parametrize("many", [3, 40])
def test_shared_prompts(dtype, d, page, many):
    """Groups of one, of several and none; requests whose context ends inside the shared part or
    that hold nothing; the result does not depend on the grouping."""
    pre = 512 // page
    ctx = [512 + 1 + 7 * i for i in range(many)] + [300, 0, 512] + [70, 0] + [33]
    groups = [0, many + 3, many + 5, many + 5]
    c = Case(dtype, ctx, 8, 2, d, page, groups=groups, prefix=[pre, 48 // page, 2], seed=5)
    out = c.run()
    c.check(*out)
    assert fpx.status(c.ws) == 0
    alone = fpx.decode_problem(c.qd, c.k, c.ctx_d, c.table_d, 1, **c.scales)
    c.check(*fpx.decode(alone, c.qd, c.k, c.v, fpx.decode_workspace(alone)))


PROMPTS = {
    # name: (hq, hkv, page, requests, q_len, prompt pages, rule)
    "two tiles": (8, 2, 128, 50, 1, 9, {}),
    "one tile": (8, 2, 128, 30, 1, 9, {}),
    "one key tile": (4, 1, 64, 20, 1, 1, {}),
    "part of a key tile": (4, 1, 16, 20, 1, 13, {}),
    "odd heads": (21, 3, 32, 37, 2, 30, {}),
    "mqa": (64, 1, 128, 9, 1, 5, {}),
    "mqa 128": (128, 1, 128, 3, 1, 5, {}),
    "mha": (4, 4, 128, 300, 1, 3, {}),
    "window": (8, 2, 64, 40, 3, 20, dict(window=700)),
    "window behind": (8, 2, 64, 40, 1, 20, dict(window=5)),
    "cap": (8, 2, 128, 50, 1, 9, dict(softcap=6.0)),
    "cap far": (8, 2, 128, 30, 1, 9, dict(softcap=0.5)),
    "cap above": (8, 2, 128, 30, 1, 9, dict(softcap=1e5)),
    "bias": (8, 2, 32, 50, 1, 9, dict(slopes=True)),
    "cap bias window": (6, 2, 16, 45, 2, 70, dict(softcap=9.0, slopes=True, window=900)),
}


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", sorted(PROMPTS))
def test_many_rows_behind_a_prompt(dtype, name):
    hq, hkv, page, n, q_len, pages, rule = PROMPTS[name]
    pre = pages * page
    ctx = [pre + q_len + (5 * i) % 90 for i in range(n)]
    ctx[1], ctx[2] = 0, max(pre - 7, 0)  # an unused entry, one that ends inside the prompt
    c = Case(dtype, ctx, hq, hkv, 128, page, q_len, groups=[0, n], prefix=[pages], seed=14)
    kw = dict(rule)
    if kw.get("slopes"):
        kw["slopes"] = torch.pow(2.0, -8.0 * torch.arange(1, hq + 1).double() / hq).float()
    dev = dict(kw)
    if dev.get("slopes") is not None:
        dev["slopes"] = dev["slopes"].cuda()
    out = c.run(fpx.score_rule(**dev))
    c.check(*out, **kw)
    assert fpx.status(c.ws) == 0
    again = c.run(fpx.score_rule(**dev))
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


def test_prompts_beyond_every_context():
    """All contexts end inside the shared pages; what lies behind them is garbage."""
    c = Case("bf16", [100, 77, 0, 33] * 8, 8, 2, 128, 32, groups=[0, 32], prefix=[4], seed=15)
    keep = torch.tensor([100, 77, 0, 33] * 8)
    for s in range(0, 32):  # rows of the prompt's last page behind the longest context
        pg = int(c.table[s, 3])
        c.k[pg, 4:], c.v[pg, 4:] = float("nan"), float("nan")
    c.check(*c.run())
    assert keep.max() == 100 and fpx.status(c.ws) == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_group_of_empty_requests(dtype):
    c = Case(dtype, [0, 0, 40], 4, 1, 128, 16, groups=[0, 2], prefix=[2], seed=6)
    c.check(*c.run())
    assert fpx.status(c.ws) == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_key_spans(dtype):
    """Documents and two-sided spans, among them rows that see nothing."""
    ctx, q_len = [100, 333, 64, 7], 3
    lo = torch.tensor([0, 5, 97, 100, 0, 332, 64, 10, -5, 4, 0, 2])
    hi = torch.tensor([99, 4, 98, 400, 0, 332, 70, 20, -1, 6, 6, 1])
    c = Case(dtype, ctx, 4, 2, 128, 32, q_len, seed=7, groups=[0, 2], prefix=[2])
    rule = fpx.score_rule(0.0, None, 0, lo.int().cuda(), hi.int().cuda())
    c.check(*c.run(rule), lo=lo, hi=hi)
    assert fpx.status(c.ws) == 0


def test_long_context_and_many_workers():
    c = Case("bf16", [9000, 1, 20000], 8, 2, 128, 128, seed=8)
    c.check(*c.run())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_repeats_bit_for_bit_and_on_another_stream(dtype):
    c = Case(dtype, [700, 513, 530, 2000], 8, 2, 128, 128, groups=[0, 3], prefix=[4], seed=9)
    a = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws2 = fpx.decode_workspace(c.dp)
    ws2[256:] = 127
    s.wait_stream(torch.cuda.current_stream())
    b = fpx.decode(c.dp, c.qd, c.k, c.v, ws2, stream=s)
    d = c.run()
    torch.cuda.synchronize()
    for x in (b, d):
        assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])


def test_captured_and_replayed_with_other_lengths():
    ctx = [700, 513, 530, 2000]
    c = Case("bf16", ctx, 8, 2, 128, 128, groups=[0, 3], prefix=[4], seed=10, width=16)
    o, lse = torch.empty_like(c.qd), torch.empty(8, 4, device="cuda")
    c.run(o=o, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(o=o, lse=lse)
    for new in (ctx, [512, 513, 0, 1], [600, 0, 514, 1999]):
        c.ctx_d.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c.ctx = new
        c.check(o, lse)
    assert fpx.status(c.ws) == 0


def test_malformed_groups_are_recorded():
    for groups, prefix in (([0, 3, 2], [1, 1]), ([0, 9], [1]), ([-1, 2], [1]), ([0, 2], [-1])):
        c = Case("bf16", [40, 50, 60], 4, 2, 128, 32, seed=11)
        dp = fpx.decode_problem(c.qd, c.k, c.ctx_d, c.table_d, 1,
                                group_ptr=torch.tensor(groups, dtype=torch.int32, device="cuda"),
                                prefix_pages=torch.tensor(prefix, dtype=torch.int32, device="cuda"))
        ws = fpx.decode_workspace(dp)
        o, lse = fpx.decode(dp, c.qd, c.k, c.v, ws)
        assert fpx.status(ws) == -7
        assert (o == 0).all() and torch.isinf(lse).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_lengths_and_pages_out_of_range_are_recorded(dtype):
    c = Case(dtype, [64, 40], 4, 2, 128, 32, seed=12)
    want = c.run()
    c.ctx_d.copy_(torch.tensor([65, 40], dtype=torch.int32))  # the table holds 64 tokens
    got = c.run()
    assert fpx.status(c.ws) == -7
    fpx.clear_status(c.ws)
    c.ctx_d.copy_(torch.tensor([-3, 40], dtype=torch.int32))
    got = c.run()
    assert fpx.status(c.ws) == -7
    fpx.clear_status(c.ws)
    assert (got[0][0] == 0).all() and torch.equal(got[0][1], want[0][1])
    c.ctx_d.copy_(torch.tensor([64, 40], dtype=torch.int32))
    c.table_d[0, 1] = c.k.shape[0]
    got = c.run()
    assert fpx.status(c.ws) == -7
    fpx.clear_status(c.ws)
    assert torch.equal(got[0][1], want[0][1]) and not torch.isnan(got[0]).any()


def test_cache_beyond_32_bit_offsets():
    """More than 2^31 elements per cache, the pages of the context at its far end."""
    hkv, d, page = 8, 128, 128
    num = 2 ** 31 // (hkv * d * page) + 40
    k, v = (torch.zeros(num, page, hkv, d, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(1)
    pages = [num - 1, 3, num - 5]
    k64, v64 = (torch.zeros(3, page, hkv, d, dtype=torch.float64) for _ in range(2))
    for i, p in enumerate(pages):
        for c, c64 in ((k, k64), (v, v64)):
            x = (torch.randn(page, hkv, d, generator=g) * 2).to(torch.float8_e4m3fn)
            c[p] = x.cuda()
            c64[i] = x.double()
    q = torch.randn(1, 8, d, generator=g).bfloat16()
    one = torch.ones(hkv, device="cuda")
    dp = fpx.decode_problem(q.cuda(), k, torch.tensor([300], dtype=torch.int32, device="cuda"),
                            torch.tensor([pages], dtype=torch.int32, device="cuda"), k_scale=one,
                            v_scale=one)
    ws = fpx.decode_workspace(dp)
    o, lse = fpx.decode(dp, q.cuda(), k, v, ws)
    assert fpx.status(ws) == 0
    ref = R.decode_reference(q.double(), k64, v64, [300], [[0, 1, 2]], 1, 1 / math.sqrt(d))
    R.check(o, lse, ref, "f16", "bf16", 300, d)


@pytest.mark.parametrize("gain", [2.0 ** -100, 2.0 ** 60])
def test_queries_far_from_one(gain):
    """Rows of Q whose values lie far outside fp16's range (the e4m3 path scales each row)."""
    c = Case("e4m3", [90, 33], 4, 2, 128, 32, seed=13)
    c.q = (c.q.double() * gain).bfloat16()
    c.q64, c.qd = c.q.double(), c.q.cuda()
    big = gain > 1
    rule = fpx.score_rule(5.0) if big else None
    c.check(*c.run(rule), **({"softcap": 5.0} if big else {}))


def test_two_calls_at_once():
    """Two problems on two streams, each with its own workspace, give what they give alone."""
    cases = [Case("bf16", [3000 + 13 * i for i in range(40)], 8, 2, 128, 128, groups=[0, 40],
                  prefix=[20], seed=16),
             Case("e4m3", [900 + 131 * i for i in range(20)], 6, 2, 128, 32, 3, seed=17)]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for i, c in enumerate(cases):
            got[i].append(fpx.decode(c.dp, c.qd, c.k, c.v, c.ws, stream=streams[i]))
    torch.cuda.synchronize()
    for i, c in enumerate(cases):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
        assert fpx.status(c.ws) == 0


def test_rule_of_another_size_is_refused():
    c = Case("bf16", [40, 50], 4, 2, 128, 32, seed=18)
    short = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        c.run(fpx.score_rule(key_lo=short, key_hi=short))
    with pytest.raises(ValueError):
        c.run(fpx.score_rule(slopes=torch.zeros(3, device="cuda")))
    with pytest.raises(ValueError):
        c.run(fpx.score_rule(slopes=torch.zeros(4)))
