"""Refusals of the serving entry points on the host (nothing is launched), their size queries, and
the Python wrappers' checks of tensors.  No GPU needed."""
import ctypes

import numpy as np
import pytest
import torch

import dynamic_block_sparse_pooled_b200 as fpx

A = 0x100000  # 256-aligned fake device address, never dereferenced on the host
BIG = 1 << 40


def problem(seqlens=(300, 1000), hq=4, hkv=2, d=128, block=128, dtype=fpx.BF16):
    cu = np.zeros(len(seqlens) + 1, np.int32)
    cu[1:] = np.cumsum(seqlens)
    p = fpx.Problem()
    p.num_seqs, p.cu_seqlens_h, p.cu_seqlens_d = len(seqlens), cu.ctypes.data, 0x1000
    p.total_tokens, p.hq, p.hkv, p.d, p.block, p.dtype = int(cu[-1]), hq, hkv, d, block, dtype
    p._keep = cu
    return p


def rule(softcap=0.0, window=0, slopes=None, lo=None, hi=None):
    return ctypes.byref(fpx.ScoreRule(softcap, window, slopes, lo, hi))


BAD_RULES = {
    "negative cap": (dict(softcap=-1.0), -1), "nan cap": (dict(softcap=float("nan")), -1),
    "infinite cap": (dict(softcap=float("inf")), -1), "cap below its range": (dict(softcap=1e-30), -1),
    "cap beyond its range": (dict(softcap=1e30), -1), "negative window": (dict(window=-1), -1),
    "lo alone": (dict(lo=A), -1), "hi alone": (dict(hi=A), -1),
    "slopes misaligned": (dict(slopes=A + 2), -3), "lo misaligned": (dict(lo=A + 1, hi=A), -3),
}


@pytest.mark.parametrize("name", sorted(BAD_RULES))
def test_bad_rules(name):
    lib = fpx.load()
    kw, want = BAD_RULES[name]
    p = problem()
    assert lib.fpx_span_select(ctypes.byref(p), rule(**kw), A, A, 10, A, A, BIG, None) == want
    assert lib.fpx_span_prefill(ctypes.byref(p), A, A, A, None, rule(**kw), A, A, A, A, A, BIG,
                                None) == want
    d = decode()
    assert lib.fpx_decode(ctypes.byref(d), A, A, A, rule(**kw), A, A, A, BIG, None) == want


def test_span_arguments():
    lib = fpx.load()
    ref = ctypes.byref(problem())
    r = rule()
    assert lib.fpx_spans(ref, 0, A, None, A, A, None) == -1       # offsets without documents
    assert lib.fpx_spans(ref, 3, None, None, A, A, None) == -1
    assert lib.fpx_spans(ref, -1, A, None, A, A, None) == -1
    assert lib.fpx_spans(ref, 3, A, None, None, A, None) == -1
    assert lib.fpx_spans(ref, 3, A, A + 2, A, A, None) == -3
    assert lib.fpx_spans(None, 0, None, None, A, A, None) == -1
    assert lib.fpx_span_select(ref, None, A, A, 10, A, A, BIG, None) == -1
    assert lib.fpx_span_select(ref, r, None, A, 10, A, A, BIG, None) == -1
    assert lib.fpx_span_select(ref, r, A, None, 10, A, A, BIG, None) == -1
    assert lib.fpx_span_select(ref, r, A, A, -1, A, A, BIG, None) == -1
    assert lib.fpx_span_select(ref, r, A, A, 2 ** 31, A, A, BIG, None) == -1
    assert lib.fpx_span_select(ref, r, A, A, 10, A + 4, A, BIG, None) == -3
    assert lib.fpx_span_select(ref, r, A, A, 10, A, A + 8, BIG, None) == -3
    assert lib.fpx_span_select(ref, r, A, A, 10, A, A, 64, None) == -4
    full = (ref, A, A, A, None, r, A, A, A, A, A, BIG, None)
    for i, bad, want in ((5, None, -1), (1, None, -1), (7, None, -1), (8, A + 8, -3), (10, None, -1),
                         (11, 64, -4)):
        args = list(full)
        args[i] = bad
        assert lib.fpx_span_prefill(*args) == want
    kv = ctypes.byref(fpx.PagedKV(0x3000, 8, 64))
    kv64 = ctypes.byref(fpx.PagedKV(0x3000, 16, 64))
    for kw in (dict(dtype=fpx.F32), dict(d=64), dict(block=64)):  # paged: tensor-core path only
        assert lib.fpx_span_prefill(ctypes.byref(problem(**kw)), A, A, A, kv64, r, A, A, A, A, A, BIG,
                                    None) == -2
    assert lib.fpx_span_prefill(ref, A, A, A, ctypes.byref(fpx.PagedKV(0x3000, 7, 64)), r, A, A, A,
                                A, A, BIG, None) == -1


def decode(**kw):
    f = dict(num_seqs=4, q_len=1, hq=4, hkv=2, d=128, page=128, dtype=fpx.BF16, softmax_scale=0.0,
             k_scale_d=None, v_scale_d=None, ctx_lens_d=A, block_table_d=A, pages_per_seq=8,
             num_pages=64, num_groups=0, group_ptr_d=None, prefix_pages_d=None)
    f.update(kw)
    return fpx.DecodeProblem(*(f[n] for n, _ in fpx.DecodeProblem._fields_))


BAD_DECODES = {
    "no requests": (dict(num_seqs=0), -1), "no queries": (dict(q_len=0), -1),
    "heads": (dict(hq=5), -1), "no kv heads": (dict(hkv=0), -1), "head dim": (dict(d=96), -2),
    "page size": (dict(page=48), -2), "page too small": (dict(page=8), -2),
    "page too large": (dict(page=256), -2), "dtype": (dict(dtype=5), -2),
    "no lengths": (dict(ctx_lens_d=None), -1), "no table": (dict(block_table_d=None), -1),
    "no pages": (dict(num_pages=0), -1), "no table columns": (dict(pages_per_seq=0), -1),
    "negative groups": (dict(num_groups=-1), -1), "groups alone": (dict(num_groups=1), -1),
    "more groups than requests": (dict(num_groups=5, group_ptr_d=A, prefix_pages_d=A), -2),
    "e4m3 without scales": (dict(dtype=fpx.E4M3), -1),
    "scales without e4m3": (dict(k_scale_d=A, v_scale_d=A), -1),
    "scale": (dict(softmax_scale=float("nan")), -1),
    "lengths misaligned": (dict(ctx_lens_d=A + 2), -3),
    "cache rows beyond int32": (dict(num_pages=2 ** 25), -2),
    "positions beyond int32": (dict(pages_per_seq=2 ** 25), -2),
    "outputs beyond int32": (dict(num_seqs=2 ** 20, q_len=2 ** 10), -2),
    "tiles beyond int32": (dict(num_seqs=2 ** 17, pages_per_seq=2 ** 14, num_pages=2 ** 20), -2),
}


@pytest.mark.parametrize("name", sorted(BAD_DECODES))
def test_bad_decode_problems(name):
    lib = fpx.load()
    kw, want = BAD_DECODES[name]
    d = decode(**kw)
    assert lib.fpx_decode_workspace_bytes(ctypes.byref(d)) == 0
    assert lib.fpx_decode(ctypes.byref(d), A, A, A, None, A, A, A, BIG, None) == want


def test_decode_arguments():
    lib = fpx.load()
    d = decode()
    full = (ctypes.byref(d), A, A, A, None, A, A, A, BIG, None)
    for i, bad, want in ((0, None, -1), (1, None, -1), (2, None, -1), (3, None, -1), (5, None, -1),
                         (7, None, -1), (1, A + 8, -3), (2, A + 4, -3), (5, A + 2, -3),
                         (6, A + 2, -3), (7, A + 16, -3),
                         (8, lib.fpx_decode_workspace_bytes(ctypes.byref(d)) - 1, -4)):
        args = list(full)
        args[i] = bad
        assert lib.fpx_decode(*args) == want, (i, bad)


@pytest.mark.parametrize("kw", [dict(), dict(dtype=fpx.F32, d=64), dict(q_len=7, hq=64, hkv=1),
                                dict(num_seqs=1000, num_groups=3, group_ptr_d=A, prefix_pages_d=A),
                                dict(dtype=fpx.E4M3, k_scale_d=A, v_scale_d=A, page=16)])
def test_decode_workspace_holds_every_partial(kw):
    """At least one 32-bit partial of every row that the problem has."""
    d = decode(**kw)
    rows = d.num_seqs * d.q_len * d.hq
    assert fpx.load().fpx_decode_workspace_bytes(ctypes.byref(d)) > rows * (d.d + 2) * 4


def test_page_arguments():
    lib = fpx.load()
    assert lib.fpx_page_workspace_bytes(0) == 0 and lib.fpx_page_workspace_bytes(5) > 0
    full = (4, 16, 64, A, A, None, A, 8, A, A, A, A, A, A, 100, A, BIG, None)
    bads = ((0, 0, -1), (1, 24, -2), (1, 256, -2), (2, 0, -1), (3, None, -1), (4, None, -1),
            (6, None, -1), (7, 0, -1), (8, None, -1), (9, None, -1), (10, None, -1), (11, None, -1),
            (12, None, -1), (13, None, -1), (14, -1, -1), (15, None, -1), (16, 8, -4), (3, A + 2, -3),
            (5, A + 1, -3), (15, A + 8, -3), (2, 2 ** 28, -2), (7, 2 ** 28, -2))
    for i, bad, want in bads:
        args = list(full)
        args[i] = bad
        assert lib.fpx_page_resize(*args) == want, (i, bad)


def test_append_arguments():
    lib = fpx.load()
    row = 2 * 128
    full = (fpx.BF16, 2, 128, 10, A, row, A, row, A, A, A, 160, None, None, A, BIG, None)
    bads = ((0, 9, -2), (1, 0, -1), (2, 96, -2), (3, -1, -1), (4, None, -1), (5, row - 8, -1),
            (5, row + 4, -3), (6, A + 8, -3), (8, None, -1), (8, A + 2, -3), (9, None, -1),
            (10, A + 4, -3), (11, 0, -1), (12, A, -1), (14, None, -1), (14, A + 4, -3), (15, 8, -4),
            (0, fpx.E4M3, -1), (7, 2 ** 62, -1))
    for i, bad, want in bads:
        args = list(full)
        args[i] = bad
        assert lib.fpx_kv_append(*args) == want, (i, bad)
    args = list(full)
    args[3] = 0
    assert lib.fpx_kv_append(*args) == 0  # no tokens: nothing to launch


# ---- the wrappers refuse tensors that the device code would misread --------------------------

def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_rule_wrapper():
    with pytest.raises(TypeError):
        fpx.score_rule(slopes=torch.zeros(4, dtype=torch.float64))
    with pytest.raises(TypeError):
        fpx.score_rule(key_lo=torch.zeros(4, dtype=torch.int64), key_hi=i32(4))
    with pytest.raises(ValueError):
        fpx.score_rule(key_lo=i32(4))
    with pytest.raises(ValueError):
        fpx.score_rule(slopes=torch.zeros(8)[::2])


def decode_args(**kw):
    a = dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16), k=torch.zeros(5, 16, 2, 64, dtype=torch.bfloat16),
             ctx=i32(3), table=i32(3, 2))
    a.update(kw)
    return a["q"], a["k"], a["ctx"], a["table"]


def test_decode_wrapper():
    fpx.decode_problem(*decode_args())
    for kw in (dict(q=torch.zeros(4, 4, 64, dtype=torch.bfloat16)),
               dict(q=torch.zeros(3, 4, 128, dtype=torch.bfloat16)),
               dict(k=torch.zeros(5, 16, 64, dtype=torch.bfloat16)), dict(table=i32(2, 2)),
               dict(table=i32(2, 3).T), dict(ctx=i32(6)[::2])):
        with pytest.raises(ValueError):
            fpx.decode_problem(*decode_args(**kw))
    with pytest.raises(TypeError):
        fpx.decode_problem(*decode_args(ctx=torch.zeros(3, dtype=torch.int64)))
    with pytest.raises(TypeError):
        fpx.decode_problem(*decode_args(k=torch.zeros(5, 16, 2, 64, dtype=torch.float16)))
    with pytest.raises(ValueError):
        fpx.decode_problem(*decode_args(), group_ptr=i32(2))
    with pytest.raises(ValueError):
        fpx.decode_problem(*decode_args(), group_ptr=i32(3), prefix_pages=i32(1))
    dp = fpx.decode_problem(*decode_args())
    q, k, _, _ = decode_args()
    ws = torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(TypeError):
        fpx.decode(dp, q.float(), k, k, ws)
    with pytest.raises(ValueError):
        fpx.decode(dp, q[:2], k, k, ws)
    with pytest.raises(ValueError):
        fpx.decode(dp, q, k, k[:4], ws)
    with pytest.raises(TypeError):
        fpx.decode(dp, q, k, k.float(), ws)
    with pytest.raises(ValueError):
        fpx.decode(dp, q, k, k, ws, fpx.score_rule(slopes=torch.zeros(3)))
    with pytest.raises(ValueError):
        fpx.decode(dp, q, k, k, ws, o=torch.zeros(3, 4, 128, dtype=torch.bfloat16))


def test_page_and_append_wrappers():
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError):
        fpx.page_resize(i32(3), i32(3), i32(2, 4), i32(9), i32(1), 16, 9, 10, ws)
    with pytest.raises(ValueError):
        fpx.page_resize(i32(3), i32(3), i32(3, 4), i32(8), i32(1), 16, 9, 10, ws)
    with pytest.raises(ValueError):
        fpx.page_resize(i32(3), i32(3), i32(3, 4), i32(9), i32(1), 16, 9, 10, ws, slots=i32(9))
    with pytest.raises(TypeError):
        fpx.page_resize(i32(3).long(), i32(3), i32(3, 4), i32(9), i32(1), 16, 9, 10, ws)
    with pytest.raises(TypeError):
        fpx.page_resize(i32(3), i32(3), i32(3, 4), i32(9), i32(1), 16, 9, 10, i32(64))
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    for args in ((k.float(), k, i32(4), c, c), (k, k[:3], i32(4), c, c), (k, k, i32(3), c, c),
                 (k, k, i32(4), c, c[:2]), (k, k, i32(4), c.view(3, 16, 1, 128), c),
                 (torch.zeros(4, 64, 2, dtype=torch.bfloat16).transpose(1, 2), k, i32(4), c, c)):
        with pytest.raises(ValueError):
            fpx.kv_append(*args, ws)
    with pytest.raises(TypeError):
        fpx.kv_append(k, k, i32(4), c.half(), c, ws)


# ---- the paths run on the caller's stream from their first byte on ----------------------------

@pytest.mark.parametrize("path,args", [("prefill", (0.5,)), ("vs_path", (2, 0.5, 0.5)), ("span_path", ())])
def test_paths_make_their_workspace_on_the_stream_they_launch_on(monkeypatch, path, args):
    """The kernels write tables into the workspace: zeros that another stream still has to write
    would land on top of them."""
    inside = []

    class Within:
        def __init__(self, what):
            self.what = what

        def __enter__(self):
            inside.append(self.what)

        def __exit__(self, *_):
            inside.pop()

    class Reached(Exception):
        pass

    mine, seen = object(), []
    monkeypatch.setattr(torch.cuda, "device", lambda d: Within("device"))
    monkeypatch.setattr(torch.cuda, "stream", Within)
    zeros = torch.zeros

    def watched(*a, **kw):
        seen.append(list(inside))
        if kw.get("dtype") is torch.uint8:
            raise Reached  # nothing is launched
        return zeros(*a, **kw)

    q = zeros(300, 2, 128, dtype=torch.bfloat16)
    monkeypatch.setattr(torch, "zeros", watched)
    with pytest.raises(Reached):
        getattr(fpx, path)(q, q, q, 128, *args, stream=mine)
    assert seen and all(mine in s for s in seen)
    assert not inside


@pytest.mark.parametrize("i", [0, 14])
def test_page_counts_whose_strides_would_pass_32_bits(i):
    """Requests or tokens so near 2^31 that a thread's next index would wrap to a negative one and be
    read or written in front of the buffers.  Just below, the next check answers (a workspace that is
    too small): nothing is launched."""
    lib = fpx.load()
    most = 2 ** 31 - 2 ** 20 - 1
    full = [4, 16, 64, A, A, None, A, 1, A, A, A, A, A, A, 100, A, 0, None]
    for n, want in ((most + 1, -2), (2 ** 31 - 1, -2), (most, -4)):
        full[i] = n
        assert lib.fpx_page_resize(*full) == want, n


def test_append_of_the_most_tokens_is_checked_like_any_other():
    """2^31 - 1 tokens: their number plus one does not fit 32 bits.  The workspace is too small, which
    is the last check: nothing is launched."""
    lib = fpx.load()
    row = 2 * 128
    args = [fpx.BF16, 2, 128, 2 ** 31 - 1, A, row, A, row, A, A, A, 160, None, None, A, 8, None]
    assert lib.fpx_kv_append(*args) == -4
    args[5] = 2 ** 60
    assert lib.fpx_kv_append(*args) == -1


def test_host_tensors_are_refused():
    """Calls that are right but for lying in host memory: their addresses never reach a kernel."""
    ws = torch.zeros(4096, dtype=torch.uint8)
    q, c = torch.zeros(3, 4, 128, dtype=torch.bfloat16), torch.zeros(2, 128, 4, 128, dtype=torch.bfloat16)
    pf = fpx.problem(q, q, 128)
    lo, hi = i32(3), i32(3)
    r = fpx.score_rule(key_lo=lo, key_hi=hi)
    dp = fpx.decode_problem(q, c, i32(3), i32(3, 1))
    calls = [lambda: fpx.spans(pf, None, i32(1), lo, hi), lambda: fpx.span_select(pf, r, ws),
             lambda: fpx.span_prefill(pf, q, q, q, r, i32(5), i32(4), ws),
             lambda: fpx.decode(dp, q, c, c, ws),
             lambda: fpx.page_resize(i32(2), i32(2), i32(2, 2), i32(4), i32(1), 16, 4, 8, ws),
             lambda: fpx.kv_append(q, q, i32(3), c, c, ws)]
    for call in calls:
        with pytest.raises(ValueError, match="must be on a GPU"):
            call()


class Elsewhere(torch.Tensor):
    """A tensor that says it lies on GPU 1."""

    def get_device(self):
        return 1


def test_a_problem_on_another_device_is_refused():
    """Offsets, scales, tables and outputs that lie on another device than the call's tensors."""
    away = lambda t: t.as_subclass(Elsewhere)  # noqa: E731
    ws = torch.zeros(4096, dtype=torch.uint8)
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    pf = fpx.problem(q, q, 128, [0, 3])
    pf.cu_d = away(pf.cu_d)
    lo, hi, r = i32(3), i32(3), fpx.score_rule()
    for call in (lambda: fpx.span_select(pf, r, ws),
                 lambda: fpx.span_prefill(pf, q, q, q, r, i32(5), i32(4), ws)):
        with pytest.raises(ValueError, match="cu_seqlens is on"):
            call()
    e = q.to(torch.float8_e4m3fn)
    one = torch.ones(4)
    pf = fpx.problem(e, e, 128, None, 0.0, one, away(one), one)
    with pytest.raises(ValueError, match="k_scale is on"):
        fpx.span_prefill(pf, e, e, e, r, i32(5), i32(4), ws)
    pf = fpx.problem(e, e, 128, None, 0.0, one, one, torch.ones(3))
    with pytest.raises(ValueError, match="v_scale holds 3"):
        fpx.span_prefill(pf, e, e, e, r, i32(5), i32(4), ws)
    pf = fpx.problem(q, q, 128)
    kv = fpx.paged_kv(away(i32(1, 1)), 1)
    c = torch.zeros(1, 128, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="block_table is on"):
        fpx.span_prefill(pf, q, c, c, r, i32(5), i32(4), ws, kv=kv)
    away_csr = (away(i32(5)), away(i32(64)), away(torch.zeros(1, dtype=torch.int64)))
    for k in range(3):
        csr = [i32(5), i32(64), torch.zeros(1, dtype=torch.int64)]
        csr[k] = away_csr[k]
        with pytest.raises(ValueError, match="is on"):
            fpx.span_select(pf, r, ws, *csr)


def test_default_list_of_a_long_layer_is_one_that_the_call_takes():
    """A million tokens, 32 heads: 2^31 entries would hold every block, one more than a call takes; a
    window needs a few million of them."""
    class Layer:
        struct, cu_h = fpx.Problem(), None
    Layer.struct.total_tokens, Layer.struct.hq, Layer.struct.block = 2 ** 20, 32, 128
    assert fpx.span_capacity(Layer) == 2 ** 31 - 1
    lib, p = fpx.load(), problem(seqlens=(2 ** 20,), hq=32, hkv=8)
    # the capacity is taken: what the call refuses is nnz, misaligned
    for cap, want in ((2 ** 31, -1), (2 ** 31 - 1, -3)):
        assert lib.fpx_span_select(ctypes.byref(p), rule(), A, A, cap, A + 4, A, 2 ** 50, None) == want
    Layer.struct.total_tokens, Layer.struct.hq = 700, 2
    assert fpx.span_capacity(Layer) == 2 * 36
