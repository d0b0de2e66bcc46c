"""Plain 64-bit references of the serving operators, and the tolerances of their GPU tests.

Tolerances count roundings (a rounding is off by at most half a step: bf16 2^-8, fp16 2^-11, e4m3
2^-4, relative) on the scale of the row's own sum A = sum_j p_j |v_j| (64 bits):
* O: P in its 16- or 8-bit type, plus the output's rounding, plus 2^-10 for the exponentials
  (polynomial 7.5e-5), the scores' 32-bit sums (at most D 2^-24 sum |q k| scale, below 3e-4 on
  these inputs) and tanh (a few 2^-23 of the cap);
* a type with few exponents adds half its smallest step for every key, relative to a row whose
  largest weight is at least 1: B = sum |v_j| / sum exp(s_j - max s) times 2^-25 (fp16) or 2^-10
  (e4m3);
* fp32: n + D sums of 2^-24 each, and 2^-18 for ex2 and the rounding of scores of magnitude < 64;
* LSE: the same relative error of the sum, as an absolute one: 3e-4, fp32 n 2^-24 + 2^-16.
"""
import math

import torch

P_STEP = {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -4, "f16": 2.0 ** -11}
P_LEAST = {"bf16": 0.0, "e4m3": 2.0 ** -10, "f16": 2.0 ** -25}


def attend(q, k, v, at, lo, hi, scale, softcap=0.0, slopes=None):
    """q [n, Hq, D], k and v [L, Hkv, D] in 64 bits; positions at, bounds lo, hi [n] (ints).
    -> O, LSE [Hq, n], A and B of the tolerance (shapes of O and [n, Hq, 1])."""
    n, hq, d = q.shape
    g = hq // k.shape[1]
    kk, vv = (x.repeat_interleave(g, dim=1).permute(1, 0, 2) for x in (k, v))
    x = torch.einsum("nhd,hld->hnl", q, kk) * scale
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    j = torch.arange(k.shape[0], dtype=torch.int64)
    if slopes is not None:
        x = x - slopes.double()[:, None, None] * (at[:, None] - j[None]).abs()[None]
    seen = (j[None] >= lo[:, None]) & (j[None] <= hi[:, None])
    x = torch.where(seen[None], x, torch.full_like(x, -math.inf))
    lse = torch.logsumexp(x, -1) if k.shape[0] else torch.full((hq, n), -math.inf, dtype=torch.float64)
    safe = torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)
    p = torch.where(seen[None], torch.exp(x - safe[..., None]), torch.zeros_like(x))
    o = torch.einsum("hnl,hld->nhd", p, vv)
    a = torch.einsum("hnl,hld->nhd", p, vv.abs())
    if k.shape[0]:
        top = x.amax(-1)
        rel = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top)[..., None]).sum(-1)
    else:
        rel = torch.ones_like(lse)
    total = torch.einsum("hnl,hld->nhd", seen[None].double().expand_as(x).contiguous(), vv.abs())
    b = total / rel.clamp(min=1.0).T[..., None]
    return o, lse, a, b


def check(o, lse, ref, p_type, out_type, keys, d):
    """o, lse: the GPU's; ref: attend()'s (or a list of them along the query axis)."""
    o64, l64, a, b = ref
    o, lse = o.double().cpu(), lse.double().cpu()
    none = torch.isinf(l64)
    assert torch.equal(none, torch.isinf(lse) & (lse < 0)), "rows without a key differ"
    assert not torch.isnan(o).any() and not torch.isnan(lse).any()
    if out_type == "f32":
        rel = (keys + d) * 2.0 ** -24 + 2.0 ** -18
        tol, lse_tol = rel * a + 1e-7, keys * 2.0 ** -24 + 2.0 ** -16
    else:
        tol = (P_STEP[p_type] + 2.0 ** -8 + 2.0 ** -10) * a + P_LEAST[p_type] * b + 1e-6
        lse_tol = 3e-4
    err = (o - o64).abs()
    worst = (err / tol).max().item()
    assert worst <= 1.0, f"O off by {worst:.2f} of its tolerance (abs {err.max().item():.3e})"
    live = ~none
    if live.any():
        e = (lse[live] - l64[live]).abs().max().item()
        assert e <= lse_tol, f"LSE off by {e:.3e}"
    assert (o[none.T] == 0).all()


def span_bounds(lens, docs=None, prefix=None):
    """(lo, hi) of every packed token; docs: (first, last) document offsets list, or None."""
    los, his = [], []
    start = 0
    for s, n in enumerate(lens):
        for i in range(n):
            t = start + i
            if docs is None:
                d0, d1, doc = start, start + n, s
            else:
                doc = [e for e in range(len(docs) - 1) if docs[e] <= t < docs[e + 1]]
                if not doc:
                    los.append(0)
                    his.append(-1)
                    continue
                doc = doc[0]
                d0, d1 = max(docs[doc], start), min(docs[doc + 1], start + n)
            hi = i
            if prefix is not None:
                hi = max(hi, min(d0 + max(prefix[doc], 0), d1) - 1 - start)
            los.append(d0 - start)
            his.append(hi)
        start += n
    return torch.tensor(los, dtype=torch.int64), torch.tensor(his, dtype=torch.int64)


def span_reference(q, k, v, lens, lo, hi, scale, softcap=0.0, slopes=None, window=0, kept=None):
    """Packed batch under a rule; kept(h, s, I) -> list of blocks is not needed for full lists."""
    parts, start = [], 0
    for n in lens:
        sl = slice(start, start + n)
        at = torch.arange(n)
        first = lo[sl].clamp(min=0)
        if window:
            first = torch.maximum(first, at - window + 1)
        parts.append(attend(q[sl], k[sl], v[sl], at, first, hi[sl].clamp(max=n - 1), scale,
                            softcap, slopes))
        start += n
    return (torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts], 1),
            torch.cat([p[2] for p in parts]), torch.cat([p[3] for p in parts]))


def decode_reference(q, k_cache, v_cache, ctx, table, q_len, scale, softcap=0.0, slopes=None,
                     window=0, lo=None, hi=None):
    """Caches [pages, page, Hkv, D] in 64 bits (scales applied), host lists ctx and table."""
    page = k_cache.shape[1]
    parts = []
    for s, n in enumerate(ctx):
        pages = table[s][: -(-n // page)]
        k = k_cache[pages].reshape(-1, *k_cache.shape[2:])[:n] if n else k_cache.new_zeros(0, *k_cache.shape[2:])
        v = v_cache[pages].reshape(-1, *v_cache.shape[2:])[:n] if n else v_cache.new_zeros(0, *v_cache.shape[2:])
        at = torch.arange(n - q_len, n)
        sl = slice(s * q_len, (s + 1) * q_len)
        first = torch.zeros_like(at) if lo is None else lo[sl].clamp(min=0)
        last = at.clone() if hi is None else hi[sl].clamp(max=n - 1)
        if window:
            first = torch.maximum(first, at - window + 1)
        last = torch.where(at < 0, torch.full_like(last, -1), last)
        parts.append(attend(q[sl], k, v, at, first, last, scale, softcap, slopes))
    return (torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts], 1),
            torch.cat([p[2] for p in parts]), torch.cat([p[3] for p in parts]))


def page_reference(lens, new, table, free, count, page, num_pages, cap, keep=None):
    """fpx_page_resize on host lists; None where the call must leave everything as it was."""
    width = len(table[0])
    need = lambda n: -(-n // page)  # noqa: E731
    keep = keep or [0] * len(lens)
    if any(n < 0 or m < 0 or n > width * page or m > width * page for n, m in zip(lens, new)) or \
            min(keep) < 0:
        return None
    table, free = [list(r) for r in table], list(free)
    top = count
    for s, (n, m) in enumerate(zip(lens, new)):
        for i in range(max(need(m), keep[s]), need(n)):
            if top >= num_pages:
                return None
            free[top] = table[s][i]
            top += 1
    take = sum(max(0, need(m) - need(n)) for n, m in zip(lens, new))
    tokens = sum(max(0, m - n) for n, m in zip(lens, new))
    if take > top or tokens > cap or not 0 <= count <= num_pages:
        return None
    cu, slots, pos = [0], [], []
    for s, (n, m) in enumerate(zip(lens, new)):
        for i in range(need(n), need(m)):
            top -= 1
            table[s][i] = free[top]
        for x in range(n, m):
            slots.append(table[s][x // page] * page + x % page)
            pos.append(x)
        cu.append(len(slots))
    pad = [-1] * (cap - tokens)
    return dict(table=table, free=free, count=top, cu=cu, slots=slots + pad, positions=pos + pad)
