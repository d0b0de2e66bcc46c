"""Attention under a score rule (tanh cap, distance bias, window, documents, prefixes) against a
plain 64-bit implementation, on the tensor-core and the CUDA-core path."""
import math

import numpy as np
import pytest
import torch

import dynamic_block_sparse_pooled_b200 as fpx
import serve_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def make(dtype, lens, hq, hkv, d, gain=2.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = sum(lens)
    q, k, v = (torch.randn(t, h, d, generator=g) * s for h, s in ((hq, gain), (hkv, 1.0), (hkv, 1.0)))
    scales = {}
    if dtype == "e4m3":
        out = []
        for name, x in (("q", q), ("k", k), ("v", v)):
            sc = x.abs().amax(dim=(0, 2)).float() / 448
            y = (x / sc[None, :, None]).to(torch.float8_e4m3fn)
            scales[name + "_scale"] = sc.cuda()
            out.append((y, y.double() * sc.double()[None, :, None]))
    else:
        out = [(x.to(DT[dtype]), x.to(DT[dtype]).double()) for x in (q, k, v)]
    return [x[0].cuda() for x in out], [x[1] for x in out], scales


def cumulative(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


LENS = [300, 0, 1, 129, 640]
T = sum(LENS)
RULES = {
    "causal": {},
    "cap": dict(softcap=20.0),
    "cap_small": dict(softcap=1.5),
    "alibi": dict(alibi=True),
    "window1": dict(window=1),
    "window37": dict(window=37, softcap=30.0),
    "window_all": dict(window=10 ** 9),
    "docs": dict(docs=[0, 7, 7, 200, 300, 301, 430, 500, 1070]),
    "docs_across": dict(docs=[0, 250, 310, 600, 1070], alibi=True),
    "docs_partial": dict(docs=[5, 100, 290, 900], softcap=10.0),
    "prefix": dict(prefix=[120, 3, 1, 129, 500]),
    "docs_prefix": dict(docs=[0, 150, 300, 301, 430, 700, 1070], prefix=[150, 3, -4, 1000, 0, 200],
                        alibi=True, softcap=15.0),
    "prefix_window": dict(prefix=[300, 0, 0, 0, 640], window=50),
}
SHAPES = {
    "tc_gqa2": ("bf16", 4, 2, 128, 128), "tc_odd": ("bf16", 3, 1, 128, 128),
    "tc_mha": ("bf16", 2, 2, 128, 128), "tc_e4m3": ("e4m3", 4, 2, 128, 128),
    "simt_f32": ("f32", 2, 1, 64, 64), "simt_f32_128": ("f32", 2, 2, 128, 16),
    "simt_bf16": ("bf16", 3, 1, 64, 32),
}


def slopes_of(hq):
    return torch.pow(2.0, -8.0 * torch.arange(1, hq + 1).double() / hq).float()


def run(shape, lens, docs=None, prefix=None, softcap=0.0, alibi=False, window=0, gain=2.0, seed=0):
    dtype, hq, hkv, d, block = SHAPES[shape]
    (q, k, v), (q64, k64, v64), scales = make(dtype, lens, hq, hkv, d, gain, seed)
    slopes = slopes_of(hq) if alibi else None
    dev = lambda x, t=torch.int32: None if x is None else torch.tensor(x, dtype=t, device="cuda")  # noqa: E731
    out = fpx.span_path(q, k, v, block, cumulative(lens), dev(docs), dev(prefix), softcap,
                        None if slopes is None else slopes.cuda(), window, **scales)
    lo, hi = R.span_bounds(lens, docs, prefix)
    ref = R.span_reference(q64, k64, v64, lens, lo, hi, 1 / math.sqrt(d), softcap, slopes, window)
    out_type = "f32" if dtype == "f32" else "bf16"
    p_type = "e4m3" if dtype == "e4m3" else "bf16"
    R.check(out["o"], out["lse"], ref, p_type, out_type, max(lens), d)
    return out, lo, hi


@pytest.mark.parametrize("shape", ["tc_gqa2", "simt_f32", "tc_e4m3"])
@pytest.mark.parametrize("rule", sorted(RULES))
def test_rules(shape, rule):
    run(shape, LENS, **RULES[rule])


@pytest.mark.parametrize("shape", ["tc_odd", "tc_mha", "simt_f32_128", "simt_bf16"])
@pytest.mark.parametrize("rule", ["docs_prefix", "window37", "docs_partial"])
def test_shapes(shape, rule):
    run(shape, LENS, **RULES[rule])


@pytest.mark.parametrize("lens", [[1], [128], [127], [257], [1, 1, 1], [0, 5]])
@pytest.mark.parametrize("shape", ["tc_gqa2", "simt_f32"])
def test_lengths(shape, lens):
    run(shape, lens, softcap=5.0, alibi=True, seed=3)


@pytest.mark.parametrize("gain", [0.0, 60.0])
def test_cap_at_its_ends(gain):
    """All-zero scores, and scores far beyond the cap."""
    run("tc_gqa2", [500], softcap=8.0, gain=gain)
    run("simt_f32", [200], softcap=8.0, gain=gain)


@pytest.mark.parametrize("shape", ["tc_gqa2", "simt_f32", "tc_e4m3"])
@pytest.mark.parametrize("cap", [1e-3, 3e3, 1e6])
def test_caps_far_from_the_scores(shape, cap):
    """A cap far above the scores leaves them as they are, one far below makes them signs of it."""
    run(shape, [300, 129], softcap=cap)


@pytest.mark.parametrize("block", [16, 128])
@pytest.mark.parametrize("rule", sorted(RULES))
def test_blocks_listed(rule, block):
    """The CSR lists exactly the blocks that some query of the row sees a key of."""
    spec = RULES[rule]
    hq = 2
    (q, k, _), _, _ = make("f32", LENS, hq, 1, 64)
    pf = fpx.problem(q, k, block, cumulative(LENS))
    ws = fpx.workspace(pf, -1)
    dev = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lo_d, hi_d = fpx.spans(pf, dev(spec.get("docs")), dev(spec.get("prefix")))
    rule_d = fpx.score_rule(window=spec.get("window", 0), key_lo=lo_d, key_hi=hi_d)
    rp, ci, nnz = fpx.span_select(pf, rule_d, ws)
    assert fpx.status(ws) == 0
    lo, hi = R.span_bounds(LENS, spec.get("docs"), spec.get("prefix"))
    assert torch.equal(lo_d.cpu().long(), lo) and torch.equal(hi_d.cpu().long(), hi)
    rp, ci = rp.cpu().numpy(), ci.cpu().numpy()
    want = []
    start = 0
    for n in LENS:
        for i0 in range(0, n, block):
            got = set()
            for i in range(i0, min(i0 + block, n)):
                a = max(int(lo[start + i]), 0)
                if spec.get("window"):
                    a = max(a, i - spec["window"] + 1)
                b = min(int(hi[start + i]), n - 1)
                if a <= b:
                    got |= set(range(a // block, b // block + 1))
            want.append(sorted(got))
        start += n
    want = want * hq
    assert len(rp) == len(want) + 1 and int(nnz) == rp[-1]
    for r, row in enumerate(want):
        assert ci[rp[r]:rp[r + 1]].tolist() == row, r


def test_capacity_is_recorded_and_nothing_is_written():
    (q, k, v), _, _ = make("bf16", [640], 4, 2, 128)
    pf = fpx.problem(q, k, 128)
    ws = fpx.workspace(pf, -1)
    col = torch.full((10,), 77, dtype=torch.int32, device="cuda")
    rule = fpx.score_rule()
    rp, ci, nnz = fpx.span_select(pf, rule, ws, col_idx=col)
    assert fpx.status(ws) == -4
    assert int(nnz) == 4 * 15 and (rp == 0).all() and (ci == 77).all()
    fpx.clear_status(ws)
    o, lse = fpx.span_prefill(pf, q, k, v, rule, rp, ci, ws)
    assert fpx.status(ws) == 0 and (o == 0).all() and torch.isinf(lse).all()


def test_plain_rule_is_the_causal_attention():
    """A rule that changes nothing gives fpx_sparse_prefill's result on a sparse CSR too, up to the
    exponentials (the rule's kernel keeps them all on the MUFU, the other shares them with a polynomial
    of relative error 7.5e-5).  Each of the two is within (2 * 2^-8 + 2^-10) A of the exact value, A
    the same attention of |V| (itself off by that much at most), so they are within twice that of
    each other; their LSEs differ by the exponentials' 7.5e-5 and 32-bit roundings."""
    (q, k, v), _, _ = make("bf16", [900, 260], 4, 2, 128, gain=20.0)
    pf = fpx.problem(q, k, 128, cumulative([900, 260]))
    ws = fpx.workspace(pf, -1)
    rp, ci, _ = fpx.select(pf, fpx.block_scores(pf, q, k, ws), 0.5, ws)
    a, la = fpx.sparse_prefill(pf, q, k, v, rp, ci, ws)
    b, lb = fpx.span_prefill(pf, q, k, v, fpx.score_rule(), rp, ci, ws)
    big, _ = fpx.sparse_prefill(pf, q, k, v.abs(), rp, ci, ws)
    assert fpx.status(ws) == 0
    rel = 2 * 2.0 ** -8 + 2.0 ** -10
    assert ((a.double() - b.double()).abs() <= 2 * rel * (1 + rel) * big.double()).all()
    assert (la - lb).abs().max() <= 1e-4


def test_entries_outside_the_sequence_are_skipped_and_recorded():
    (q, k, v), _, _ = make("bf16", [256], 2, 1, 128)
    pf = fpx.problem(q, k, 128)
    for dtype in ("tc", "simt"):
        if dtype == "simt":
            q, k, v = q.float(), k.float(), v.float()
            pf = fpx.problem(q, k, 128)
        ws = fpx.workspace(pf, -1)
        rp = torch.tensor([0, 1, 4, 5, 8], dtype=torch.int32, device="cuda")
        ci = torch.tensor([0, 0, 1, 2, 0, -1, 0, 1], dtype=torch.int32, device="cuda")
        ok = torch.tensor([0, 1, 3, 4, 6], dtype=torch.int32, device="cuda")
        oc = torch.tensor([0, 0, 1, 0, 0, 1], dtype=torch.int32, device="cuda")
        rule = fpx.score_rule(3.0)
        a, la = fpx.span_prefill(pf, q, k, v, rule, rp, ci, ws)
        assert fpx.status(ws) == -7
        fpx.clear_status(ws)
        b, lb = fpx.span_prefill(pf, q, k, v, rule, ok, oc, ws)
        assert fpx.status(ws) == 0
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_unseen_scores_may_be_anything():
    """NaN and infinite keys that no query sees leave the result as it is."""
    lens = [600]
    (q, k, v), _, _ = make("bf16", lens, 2, 1, 128)
    docs = torch.tensor([0, 200, 290, 600], dtype=torch.int32, device="cuda")
    pf = fpx.problem(q, k, 128)
    ws = fpx.workspace(pf, -1)
    lo, hi = fpx.spans(pf, docs)
    lo[200:290], hi[200:290] = 0, -1  # the middle document's queries see nothing, nobody sees it
    rule = fpx.score_rule(9.0, slopes_of(2).cuda(), 0, lo, hi)
    rp, ci, _ = fpx.span_select(pf, rule, ws)
    want = fpx.span_prefill(pf, q, k, v, rule, rp, ci, ws)
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min):
        k2 = k.clone()
        k2[200:290] = bad
        got = fpx.span_prefill(pf, q, k2, v, rule, rp, ci, ws)
        assert fpx.status(ws) == 0
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert (want[0][200:290] == 0).all() and torch.isinf(want[1][:, 200:290]).all()


def test_paged_equals_packed():
    lens, hq, hkv, d = [300, 0, 129, 640], 4, 1, 128
    (q, k, v), _, _ = make("bf16", lens, hq, hkv, d)
    cu = cumulative(lens)
    pf = fpx.problem(q, k, 128, cu)
    ws = fpx.workspace(pf, -1)
    lo, hi = fpx.spans(pf, None, torch.tensor([200, 0, 0, 640], dtype=torch.int32, device="cuda"))
    rule = fpx.score_rule(11.0, slopes_of(hq).cuda(), 0, lo, hi)
    rp, ci, _ = fpx.span_select(pf, rule, ws)
    a = fpx.span_prefill(pf, q, k, v, rule, rp, ci, ws)
    nb = [-(-n // 128) for n in lens]
    pages = sum(nb) + 2
    perm = np.random.default_rng(0).permutation(pages)
    kc, vc = (torch.zeros(pages, 128, hkv, d, dtype=q.dtype, device="cuda") for _ in range(2))
    table = torch.full((len(lens), max(nb)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(lens):
        for J in range(nb[s]):
            pg = int(perm[at])
            at += 1
            table[s, J] = pg
            x0, x1 = cu[s] + 128 * J, min(cu[s] + 128 * (J + 1), cu[s + 1])
            kc[pg, :x1 - x0], vc[pg, :x1 - x0] = k[x0:x1], v[x0:x1]
    kv = fpx.paged_kv(table.cuda(), pages)
    b = fpx.span_prefill(pf, q, kc, vc, rule, rp, ci, ws, kv=kv)
    assert fpx.status(ws) == 0
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_and_replayed_with_other_spans():
    lens = [700]
    (q, k, v), _, _ = make("bf16", lens, 2, 1, 128)
    pf = fpx.problem(q, k, 128)
    ws = fpx.workspace(pf, -1)
    docs = torch.tensor([0, 300, 700], dtype=torch.int32, device="cuda")
    lo = torch.empty(700, dtype=torch.int32, device="cuda")
    hi = torch.empty_like(lo)
    rule = fpx.score_rule(9.0, None, 0, lo, hi)
    col = torch.empty(fpx.span_capacity(pf), dtype=torch.int32, device="cuda")
    rp = torch.empty(pf.rows + 1, dtype=torch.int32, device="cuda")
    nnz = torch.empty(1, dtype=torch.int64, device="cuda")
    o = torch.empty_like(q)
    lse = torch.empty(2, 700, device="cuda")

    def go():
        fpx.spans(pf, docs, None, lo, hi)
        fpx.span_select(pf, rule, ws, rp, col, nnz)
        fpx.span_prefill(pf, q, k, v, rule, rp, col, ws, o=o, lse=lse)

    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for cut in (300, 1, 555):
        docs.copy_(torch.tensor([0, cut, 700], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone(), lse.clone()
        go()
        assert fpx.status(ws) == 0
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)


def test_default_capacity_and_another_stream():
    """Lists of the default size hold a rule without spans (on or below the diagonal) and one with
    them; outputs allocated for another stream."""
    (q, k, v), (q64, k64, v64), _ = make("bf16", [700], 2, 1, 128)
    pf = fpx.problem(q, k, 128)
    s = torch.cuda.Stream()
    ws = fpx.workspace(pf, -1)
    s.wait_stream(torch.cuda.current_stream())
    plain = fpx.score_rule(window=300)
    rp, ci, nnz = fpx.span_select(pf, plain, ws, stream=s)
    assert ci.numel() == 2 * 21
    o, lse = fpx.span_prefill(pf, q, k, v, plain, rp, ci, ws, stream=s)
    lo, hi = fpx.spans(pf, None, torch.tensor([700], dtype=torch.int32, device="cuda"), stream=s)
    s.wait_stream(torch.cuda.current_stream())
    both = fpx.score_rule(key_lo=lo, key_hi=hi)
    rp2, ci2, _ = fpx.span_select(pf, both, ws, stream=s)
    o2, lse2 = fpx.span_prefill(pf, q, k, v, both, rp2, ci2, ws, stream=s)
    assert fpx.status(ws, s) == 0 and ci2.numel() == 2 * 36
    torch.cuda.synchronize()
    a, b = R.span_bounds([700])
    R.check(o, lse, R.span_reference(q64, k64, v64, [700], a, b, 1 / math.sqrt(128), window=300),
            "bf16", "bf16", 700, 128)
    a, b = R.span_bounds([700], None, [700])
    R.check(o2, lse2, R.span_reference(q64, k64, v64, [700], a, b, 1 / math.sqrt(128)), "bf16",
            "bf16", 700, 128)


def test_path_on_a_side_stream_while_the_current_one_is_busy():
    """The whole path on another stream gives the same bits, with work queued on the current stream
    that its own kernels do not wait for."""
    lens = [700, 129]
    (q, k, v), _, _ = make("bf16", lens, 4, 2, 128)
    docs = torch.tensor([0, 300, 829], dtype=torch.int32, device="cuda")
    want = fpx.span_path(q, k, v, 128, cumulative(lens), docs, None, 20.0, None, 200)
    plain = fpx.prefill(q, k, v, 128, 0.3, cumulative(lens))
    probe = fpx.vs_path(q, k, v, 128, 32, 1e-3, 1e-3, cumulative(lens))
    busy = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(100):
        busy = busy @ busy
    got = fpx.span_path(q, k, v, 128, cumulative(lens), docs, None, 20.0, None, 200, stream=s)
    got_plain = fpx.prefill(q, k, v, 128, 0.3, cumulative(lens), stream=s)
    got_probe = fpx.vs_path(q, k, v, 128, 32, 1e-3, 1e-3, cumulative(lens), stream=s)
    torch.cuda.synchronize()
    for a, b in ((want, got), (plain, got_plain), (probe, got_probe)):
        for name in ("o", "lse", "row_ptr", "nnz"):
            assert torch.equal(a[name], b[name]), name


def test_default_list_of_a_million_tokens():
    """32 heads of 8192 blocks under key spans and a window: the default list takes every block that
    the window reaches (33 of a row, fewer at its start)."""
    t, hq, b = 2 ** 20, 32, 128
    q = torch.empty(1, hq, 128, dtype=torch.bfloat16, device="cuda").expand(t, hq, 128)
    pf = fpx.problem(q, q[:, :8], b)
    ws = fpx.workspace(pf, 1)
    lo, hi = fpx.spans(pf, device="cuda")
    rp, ci, nnz = fpx.span_select(pf, fpx.score_rule(window=32 * b, key_lo=lo, key_hi=hi), ws)
    assert fpx.status(ws) == 0
    n = t // b
    want = torch.clamp(torch.arange(1, n + 1, device="cuda"), max=33)
    assert torch.equal((rp[1:] - rp[:-1]).view(hq, n).long(), want.expand(hq, n))
    assert int(nnz) == hq * int(want.sum()) == int(rp[-1])
    last = ci[int(nnz) - 33:int(nnz)]
    assert torch.equal(last.long(), torch.arange(n - 33, n, device="cuda"))
