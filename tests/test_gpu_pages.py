"""Block tables, slot maps and cache writes on the GPU against plain host implementations, and the
serving step as a whole: pages, append, prefill under a rule, decode."""
import math
import random

import numpy as np
import pytest
import torch

import dynamic_block_sparse_pooled_b200 as fpx
import serve_ref as R

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def resize(lens, new, table, free, count, page, num_pages, cap, keep=None, in_place=False):
    ws = fpx.page_workspace(len(lens))
    t, f, c = dev(table), dev(free), dev([count])
    out = c if in_place else torch.full((1,), 99, dtype=torch.int32, device="cuda")
    cu, slots, pos = fpx.page_resize(dev(lens), dev(new), t, f, c, page, num_pages, cap, ws,
                                     keep_pages=None if keep is None else dev(keep), count_out=out)
    code = fpx.status(ws)
    return code, dict(table=t.tolist(), free=f.tolist(), count=int(out), cu=cu.tolist(),
                      slots=slots.tolist(), positions=pos.tolist())


def state(rng, lens, page, width, extra):
    need = [-(-n // page) for n in lens]
    num = sum(need) + extra
    order = list(range(num))
    rng.shuffle(order)
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (width - n))
        at += n
    left = order[at:]
    return table, left + [-7] * (num - len(left)), len(left), num


@pytest.mark.parametrize("num", [1, 2, 33, 1000, 3000])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("in_place", [False, True])
def test_resize_matches_the_host(num, page, in_place):
    rng = random.Random(num * page)
    most = 40 if num >= 1000 else 900
    lens = [rng.choice([0, rng.randint(0, most)]) for _ in range(num)]
    new = [rng.choice([0, n, n + 1, rng.randint(0, most)]) for n in lens]
    width = -(-(most + 1) // page)
    table, free, count, pages = state(rng, lens, page, width, 4 + sum(-(-n // page) for n in new))
    cap = sum(max(0, b - a) for a, b in zip(lens, new)) + 17
    keep = [rng.randint(0, 2) for _ in lens] if num % 2 else None
    code, got = resize(lens, new, table, free, count, page, pages, cap, keep, in_place)
    want = R.page_reference(lens, new, table, free, count, page, pages, cap, keep)
    assert code == 0
    assert got == want


def test_pages_given_back_are_taken_in_the_same_call():
    table = [[5, 3, 1], [0, -1, -1]]
    code, got = resize([48, 10], [16, 48], table, [-9] * 6, 0, 16, 6, 40)
    assert code == 0
    assert got["table"] == [[5, 3, 1], [0, 1, 3]] and got["count"] == 0
    assert got["cu"] == [0, 0, 38] and got["slots"][:8] == [10, 11, 12, 13, 14, 15, 16, 17]
    assert got["slots"][38:] == [-1, -1] and got["positions"][:2] == [10, 11]


@pytest.mark.parametrize("cap", [40, 6000])
@pytest.mark.parametrize("why", ["pages", "tokens", "negative", "long", "overfull", "count"])
def test_refused_calls_change_nothing(why, cap):
    lens, new, page, num_pages, count = [20, 5], [40, 9], 16, 8, 4
    table, free = [[0, 1, -1], [2, -1, -1]], [7, 6, 5, 4, -1, -1, -1, -1]
    code_want = -4
    if why == "pages":
        count = 0
    if why == "tokens":
        cap = 23
    if why == "negative":
        new, code_want = [40, -1], -7
    if why == "long":
        new, code_want = [49, 9], -7
    if why == "overfull":
        lens, new, num_pages, free = [48, 5], [0, 9], 5, free[:5]
    if why == "count":
        count = 9
    code, got = resize(lens, new, table, free, count, page, num_pages, cap)
    assert code == code_want
    assert got == dict(table=table, free=free, count=count, cu=[0, 0, 0], slots=[-1] * cap,
                       positions=[-1] * cap)


def test_a_bad_page_gives_no_slot():
    code, got = resize([10, 0], [20, 3], [[9, -1], [-1, -1]], [1, 3, 0, 0], 2, 16, 4, 13)
    assert code == -7  # page 9 of 4 in the table
    assert got["slots"] == [-1] * 6 + [48, 49, 50, 51] + [16, 17, 18]
    code, got = resize([0], [3], [[-1]], [4], 1, 16, 1, 3)
    assert code == -7 and got["slots"] == [-1] * 3


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("n,hkv,d", [(1, 1, 64), (37, 3, 128), (500, 8, 64), (0, 2, 128)])
@pytest.mark.parametrize("fused", [False, True])
def test_append(dtype, n, hkv, d, fused):
    g = torch.Generator().manual_seed(n + d)
    src = torch.float32 if dtype == "f32" else torch.bfloat16
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[dtype]
    rows = 40 * 16
    x = (torch.randn(max(n, 1), 3, hkv, d, generator=g) * 3).to(src)
    x[0, :, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 1e6]).to(src)
    x = x[:n].cuda()
    k, v = (x[:, 1], x[:, 2]) if fused else (x[:, 1].contiguous(), x[:, 2].contiguous())
    slots = torch.randperm(rows, generator=g)[:n].int()
    if n > 2:
        slots[1] = -1
    kc, vc = (torch.ones(40, 16, hkv, d, device="cuda").to(dt) for _ in range(2))
    scales = {}
    if dtype == "e4m3":
        scales = dict(k_scale=(torch.rand(hkv, generator=g) + 0.1).cuda() / 50,
                      v_scale=(torch.rand(hkv, generator=g) + 0.1).cuda())
    want = [kc.clone(), vc.clone()]
    for c, y, s in ((want[0], k, scales.get("k_scale")), (want[1], v, scales.get("v_scale"))):
        y = y.float()
        if s is not None:
            y = (y / s[:, None]).clamp(-448, 448)
        live = slots >= 0
        c.view(rows, hkv, d)[slots[live].long().cuda()] = y[live.cuda()].to(dt)
    ws = fpx.page_workspace(1)
    fpx.kv_append(k, v, slots.cuda(), kc, vc, ws, **scales)
    assert fpx.status(ws) == 0
    for a, b in ((kc, want[0]), (vc, want[1])):
        a, b = a.float(), b.float()
        assert torch.equal(torch.isnan(a), torch.isnan(b))
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def test_append_beyond_the_cache_is_recorded():
    k = torch.ones(3, 1, 64, device="cuda", dtype=torch.bfloat16)
    kc, vc = (torch.zeros(2, 16, 1, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    ws = fpx.page_workspace(1)
    fpx.kv_append(k, k, dev([31, 32, 0]), kc, vc, ws)
    assert fpx.status(ws) == -7
    assert float(kc.float().sum()) == 128 and float(vc.float().sum()) == 128


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("captured", [False, True])
def test_serving_steps(dtype, captured):
    """Two prompts that begin alike are laid out, appended and prefilled, then four tokens each are
    decoded (one step captured and replayed), one request finishes and a new one takes its pages:
    every step against the 64-bit attention over all tokens so far."""
    hq, hkv, d, page, cap_ = 4, 2, 128, 128, 25.0
    g = torch.Generator().manual_seed(21)
    e4m3 = dtype == "e4m3"
    cdt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    num, width, S = 12, 4, 3
    kc, vc = (torch.full((num, page, hkv, d), float("nan"), device="cuda").to(cdt) for _ in range(2))
    scales = {}
    if e4m3:
        scales = dict(k_scale=torch.full((hkv,), 0.02, device="cuda"),
                      v_scale=torch.full((hkv,), 0.015, device="cuda"))
    table = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    free, count = torch.arange(num, dtype=torch.int32, device="cuda"), dev([num])
    lens = torch.zeros(S, dtype=torch.int32, device="cuda")
    wsp = fpx.page_workspace(S)
    slopes = torch.tensor([0.5, 0.25, 0.02, 0.0])
    slopes_d = slopes.cuda()
    keep = torch.zeros(S, dtype=torch.int32, device="cuda")
    hist_k, hist_v = ([torch.zeros(0, hkv, d, dtype=torch.float64) for _ in range(S)] for _ in range(2))

    def stored(x, s):
        if not e4m3:
            return x.double()
        return (x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).double() * s

    def rows(n):
        return (torch.randn(n, hq, d, generator=g) * 2).bfloat16(), \
            torch.randn(n, hkv, d, generator=g).bfloat16(), torch.randn(n, hkv, d, generator=g).bfloat16()

    # prompts: request 0 has 300 tokens; request 1 the same first 256 and 10 more; 2 is unused
    q0, k0, v0 = rows(300)
    q1, k1, v1 = rows(10)
    new = dev([300, 0, 0])
    cu, slots, pos = fpx.page_resize(lens, new, table, free, count, page, num, 300, wsp)
    fpx.kv_append(k0.cuda(), v0.cuda(), slots, kc, vc, wsp, **scales)
    lens = new
    table[1, :2] = table[0, :2]
    keep[1] = 2
    lens = dev([300, 256, 0])
    new = dev([300, 266, 0])
    cu, slots, pos = fpx.page_resize(lens, new, table, free, count, page, num, 10, wsp, keep)
    assert pos.tolist() == list(range(256, 266))
    fpx.kv_append(k1.cuda(), v1.cuda(), slots, kc, vc, wsp, **scales)
    lens = new
    ks, vs = (float(scales[x][0]) if e4m3 else 1.0 for x in ("k_scale", "v_scale"))
    hist_k[0], hist_v[0] = stored(k0, ks), stored(v0, vs)
    hist_k[1] = torch.cat([hist_k[0][:256], stored(k1, ks)])
    hist_v[1] = torch.cat([hist_v[0][:256], stored(v1, vs)])
    if not e4m3:  # the paged prefill of the first prompt under the same rule
        pf = fpx.problem(q0.cuda(), kc.view(-1, hkv, d), 128)
        ws = fpx.workspace(pf, -1)
        rule = fpx.score_rule(cap_, slopes_d)
        rp, ci, _ = fpx.span_select(pf, rule, ws)
        clean = [torch.nan_to_num(c) for c in (kc, vc)]
        o, lse = fpx.span_prefill(pf, q0.cuda(), *clean, rule, rp, ci, ws,
                                  kv=fpx.paged_kv(table[:1].contiguous(), num))
        assert fpx.status(ws) == 0
        at = torch.arange(300)
        ref = R.attend(q0.double(), hist_k[0], hist_v[0], at, torch.zeros_like(at), at,
                       1 / math.sqrt(d), cap_, slopes)
        R.check(o, lse, ref, "bf16", "bf16", 300, d)
    # decode: a fixed batch of S entries, requests 0 and 1 share two pages
    q, kn, vn = (torch.zeros(S, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    groups = dict(group_ptr=dev([0, 2]), prefix_pages=dev([2]))
    step = torch.zeros(S, dtype=torch.int32, device="cuda")
    now = torch.zeros(S, dtype=torch.int32, device="cuda")
    dp = fpx.decode_problem(q, kc, now, table, **scales, **groups)
    wsd = fpx.decode_workspace(dp)
    rule = fpx.score_rule(cap_, slopes_d)
    o, lse = torch.empty_like(q), torch.empty(hq, S, device="cuda")
    kp, vp = (torch.zeros(S, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cu = torch.empty(S + 1, dtype=torch.int32, device="cuda")
    slots, pos = (torch.empty(S, dtype=torch.int32, device="cuda") for _ in range(2))

    def one_step():
        torch.add(lens, step, out=now)
        fpx.page_resize(lens, now, table, free, count, page, num, S, wsp, keep, cu_new=cu,
                        slots=slots, positions=pos)
        fpx.kv_append(kp, vp, slots, kc, vc, wsp, **scales)
        fpx.decode(dp, q, kc, vc, wsd, rule, o=o, lse=lse)
        lens.copy_(now)

    graph = None
    for it in range(4):
        live = [0, 1] if it < 2 else [0, 2]
        if it == 2:  # request 1 ends: its own page goes back, entry 2 begins with one token
            back = lens.clone()
            back[1] = 0
            fpx.page_resize(lens, back, table, free, count, page, num, 0, wsp, keep)
            lens.copy_(back)
            keep[1] = 0
        qn, kx, vx = rows(S)
        q.copy_(qn)
        step.copy_(dev([1 if s in live else 0 for s in range(S)]))
        kp.zero_()
        vp.zero_()
        for i, s in enumerate(live):
            kp[i], vp[i] = kx[s].cuda(), vx[s].cuda()
            hist_k[s] = torch.cat([hist_k[s], stored(kx[s:s + 1], ks)])
            hist_v[s] = torch.cat([hist_v[s], stored(vx[s:s + 1], vs)])
        if captured and it == 1:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                one_step()
        if graph is not None:
            graph.replay()
        else:
            one_step()
        torch.cuda.synchronize()
        assert fpx.status(wsp) == 0 and fpx.status(wsd) == 0
        for s in live:
            n = hist_k[s].shape[0]
            assert int(lens[s]) == n
            at = torch.tensor([n - 1])
            ref = R.attend(qn[s:s + 1].double(), hist_k[s], hist_v[s], at, torch.zeros_like(at), at,
                           1 / math.sqrt(d), cap_, slopes)
            R.check(o[s:s + 1], lse[:, s:s + 1], ref, "f16" if e4m3 else "bf16", "bf16", n, d)
    assert int(count) == num - 3 - 1  # request 0 holds three pages, entry 2 one


@pytest.mark.parametrize("cap", [8, 6000])
@pytest.mark.parametrize("shape", ["release", "grow", "both"])
def test_one_request_moves_thousands_of_pages(cap, shape):
    """A 131072-token request with pages of 16 ends in a call that adds few tokens, one of 4000 begins,
    or both; the others step by a token."""
    page, width = 16, 8192
    lens, new = [3, 40, 0, 15, 16], [4, 41, 0, 16, 17]
    if shape != "grow":
        lens[0], new[0] = 131072, 0
    if shape != "release":
        lens[2], new[2] = 1, 4000 if cap > 8 else 3
    rng = random.Random(5)
    table, free, count, pages = state(rng, lens, page, width, 300)
    code, got = resize(lens, new, table, free, count, page, pages, cap)
    assert code == 0
    assert got == R.page_reference(lens, new, table, free, count, page, pages, cap)


def test_time_does_not_follow_the_longest_request():
    """8192 pages given back by one request take no longer than by 1024 requests, 8 each, within a
    factor (the threads share the pages, not the requests; a walk by one thread is some 50 times)."""
    page, best = 16, {}
    for num, each in ((1024, 8), (1, 8192)):
        lens, new = dev([each * page] * num), dev([0] * num)
        table = torch.arange(num * each, dtype=torch.int32, device="cuda").view(num, each)
        free, count = torch.zeros(num * each, dtype=torch.int32, device="cuda"), dev([0])
        out, ws = dev([0]), fpx.page_workspace(num)
        bufs = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (num + 1, 1, 1)]
        times = []
        for _ in range(8):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(20):
                fpx.page_resize(lens, new, table, free, count, page, num * each, 1, ws, count_out=out,
                                cu_new=bufs[0], slots=bufs[1], positions=bufs[2])
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        best[num] = min(times)
        assert fpx.status(ws) == 0 and int(out) == num * each and torch.equal(free, table.flatten())
    assert best[1] <= 4 * best[1024], best


@pytest.mark.parametrize("cap", [4, 6000])
@pytest.mark.parametrize("bad", [-1, 6, 2 ** 30])
def test_a_bad_page_given_back_is_recorded(cap, bad):
    code, got = resize([40, 5], [10, 6], [[5, bad, 3], [0, -1, -1]], [4, -7, -7, -7, -7, -7], 1, 16, 6,
                       cap)
    assert code == -7
    assert got["free"][:3] == [4, bad, 3] and got["count"] == 3 and got["slots"][:2] == [5, -1]
