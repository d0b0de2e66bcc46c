"""Attention under a tanh cap where the cap is far above the scores, up to the end of its range.

Q and K are small whole numbers, so every dot product is exact in 32 bits and what is left of a
score's error is known: the roundings of scale / cap, of the product with it, of cap log2 e and of
the coefficients that it is folded into, and of the result (6 in all, counted as 8 half steps of
2^-24), and the tanh polynomials' relative error (the largest, 6.2e-7, is that of the fit to 1/2;
counted as POLY).  A row's LSE is off by at most that of its largest score, a weight by twice that.
On top come the sum over n keys in 32 bits, the exponentials and logarithm (2^-20), and for O the
roundings of P and of O itself as in serve_ref."""
import math

import pytest
import torch

import dynamic_block_sparse_pooled_b200 as fpx
import serve_ref as R

pytestmark = pytest.mark.gpu

POLY = 7e-7
SCALE = 16.0  # scores of some hundreds from dot products of some tens


def whole(n, h, d, most, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, (n, h, d), generator=g).double()


def inputs(n, hq, hkv, shift, seed):
    """q, k, v in 64 bits; the scores lie around shift * SCALE."""
    q, k = whole(n, hq, 128, 2, seed), whole(n, hkv, 128, 1, seed + 1)
    if shift:
        q[..., 0], k[..., 0] = 8.0, shift / 8.0
    v = torch.randn(n, hkv, 128, generator=torch.Generator().manual_seed(seed + 2))
    return q, k, v.bfloat16().double()


def close(o, lse, ref, scores, p_type):
    """scores [Hq, n]: each row's largest |score|."""
    o64, l64, a, _ = ref
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    err = scores.double() * (POLY + 8 * 2.0 ** -24)
    lse_tol = err + o64.shape[0] * 2.0 ** -24 + 2.0 ** -20
    worst = ((lse.double().cpu() - l64).abs() / lse_tol).max().item()
    assert worst <= 1.0, f"LSE off by {worst:.2f} of its tolerance"
    rel = R.P_STEP[p_type] + 2.0 ** -8 + 2.0 ** -10 + torch.expm1(2 * err).T[..., None]
    tol = rel * a + R.P_LEAST[p_type] * ref[3] + 1e-6
    worst = ((o.double().cpu() - o64).abs() / tol).max().item()
    assert worst <= 1.0, f"O off by {worst:.2f} of its tolerance"


def causal(q, k, v, cap):
    n, hq = q.shape[:2]
    at = torch.arange(n)
    ref = R.attend(q, k, v, at, torch.zeros_like(at), at, SCALE, cap)
    s = torch.einsum("nhd,lhd->hnl", q, k.repeat_interleave(hq // k.shape[1], dim=1)) * SCALE
    s = torch.where(at[None, :] <= at[:, None], cap * torch.tanh(s.abs() / cap), torch.zeros(()).double())
    return ref, s.amax(-1)


def prefill(q, k, v, cap, dtype):
    dt = torch.float8_e4m3fn if dtype == "e4m3" else torch.bfloat16
    scales = {}
    if dtype == "e4m3":
        scales = {x + "_scale": torch.ones(t.shape[1], device="cuda") for x, t in (("q", q), ("k", k), ("v", v))}
    dev = [x.float().to(dt).cuda() for x in (q, k, v)]
    out = fpx.span_path(*dev, 128, softcap=cap, softmax_scale=SCALE, **scales)
    return out["o"], out["lse"], dev[2].double().cpu()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("shift", [0, -64, 64])
@pytest.mark.parametrize("cap", [1e4, 1e5, 1e6])
def test_scores_keep_their_relative_precision(dtype, shift, cap):
    """Scores of hundreds (and around +-1024) far below the cap."""
    q, k, v = inputs(640, 2, 1, shift, 5)
    o, lse, v = prefill(q, k, v, cap, dtype)
    ref, top = causal(q, k, v, cap)
    close(o, lse, ref, top, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("shift", [0, -64, 64])
@pytest.mark.parametrize("cap", [1e8, 1e10, 1e15, 1e20])
def test_caps_to_the_end_of_their_range(dtype, shift, cap):
    """The reference that the weights are taken against must be that of the same scores: any other
    one is off by its error times the cap."""
    test_scores_keep_their_relative_precision(dtype, shift, cap)


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("cap", [50.0, 1e5])
def test_a_row_at_the_cap_leaves_its_neighbours_alone(cap, slopes):
    """One row in 32 has scores a thousand times the others': past the cap, where tanh takes
    another form.  The other rows keep their precision."""
    q, k, v = inputs(640, 2, 1, 0, 7)
    q[::32] *= 1024.0
    sl = torch.tensor([0.25, 0.0]) if slopes else None
    at = torch.arange(640)
    ref = R.attend(q, k, v, at, torch.zeros_like(at), at, SCALE, cap, sl)
    _, top = causal(q, k, v, cap)
    if slopes:  # the largest addend of a score that counts: the bias moves no score up
        top = top + 0.25 * 640
    out = fpx.span_path(*(x.bfloat16().cuda() for x in (q, k, v)), 128, softcap=cap,
                        slopes=None if sl is None else sl.cuda(), softmax_scale=SCALE)
    close(out["o"], out["lse"], ref, top, "bf16")


@pytest.mark.parametrize("cap", [50.0, 1e5, 1e20])
def test_decode_behind_a_shared_prompt(cap):
    """The same two on the shared prompt's tensor-core path: 64 requests of 2 heads each, one request
    in 16 with scores a thousand times the others'."""
    S, n, page, hq = 64, 512, 128, 2
    q, k, v = inputs(n, hq, 1, 0, 9)
    q = q[:S].clone()
    if cap < 1e20:
        q[::16] *= 1024.0
    table = torch.arange(n // page, dtype=torch.int32).repeat(S, 1).cuda()
    ctx = torch.full((S,), n, dtype=torch.int32, device="cuda")
    kc, vc = (x.bfloat16().view(n // page, page, 1, 128).cuda() for x in (k, v))
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    dp = fpx.decode_problem(q.bfloat16().cuda(), kc, ctx, table, softmax_scale=SCALE,
                            group_ptr=dev([0, S]), prefix_pages=dev([n // page]))
    ws = fpx.decode_workspace(dp)
    o, lse = fpx.decode(dp, q.bfloat16().cuda(), kc, vc, ws, fpx.score_rule(cap))
    assert fpx.status(ws) == 0
    at, lo = torch.full((S,), n - 1), torch.zeros(S, dtype=torch.int64)
    ref = R.attend(q, k, v, at, lo, at, SCALE, cap)
    s = torch.einsum("nhd,ld->hnl", q, k[:, 0]) * SCALE
    close(o, lse, ref, (cap * torch.tanh(s.abs() / cap)).amax(-1), "bf16")
