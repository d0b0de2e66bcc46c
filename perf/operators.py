"""Timing cases of the serving operators, each with its plain form in elementary torch operations:

  span    attention under a score rule: key spans (causal, documents, prefixes, window), a tanh cap on
          the scores, a bias that grows with distance
  decode  the last tokens of a batch of requests against a paged K / V cache, with groups of requests
          that share their leading pages
  pages   block tables and slot maps from request lengths
  append  K / V rows of new tokens into the paged cache

A list inside a case is a text of comma-separated numbers (one entry per sequence, document, request
or group).
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
ES = {"f32": 4, "bf16": 2, "e4m3": 1}


def ints(text):
    return [int(x) for x in text.split(",")] if text else []


def texts(values):
    return ",".join(str(int(v)) for v in values)


def ceil_div(a, b):
    return -(-a // b)


def spread(total, parts, first):
    """`parts` unequal lengths >= 1 that add up to `total` (a fixed, ragged split)."""
    w = [1.0 + ((first + 7 * i) % 13) for i in range(parts)]
    n = [max(1, int(total * x / sum(w))) for x in w]
    n[-1] += total - sum(n)
    if n[-1] < 1:
        n[max(range(parts), key=lambda i: n[i])] += n[-1] - 1
        n[-1] = 1
    return n


# ---- cases ----------------------------------------------------------------------------------


def span_case(name, dtype, hq, hkv, d, block, lens, docs="", prefix="", softcap=0.0, alibi=False,
              window=0):
    c = {"op": "span", "dtype": dtype, "hq": hq, "hkv": hkv, "d": d, "block": block, "lens": lens,
         "docs": docs, "prefix": prefix, "softcap": softcap, "alibi": alibi, "window": window}
    return dict(c, name=name) if name else c


def decode_case(name, dtype, hq, hkv, d, page, ctx, q_len=1, groups="", prefix_pages="",
                softcap=0.0, alibi=False, window=0):
    c = {"op": "decode", "dtype": dtype, "hq": hq, "hkv": hkv, "d": d, "page": page, "ctx": ctx,
         "q_len": q_len, "groups": groups, "prefix_pages": prefix_pages, "softcap": softcap,
         "alibi": alibi, "window": window}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one whole prompt through a layer that caps its scores
        span_case("span cap 8192", "bf16", 32, 8, 128, 128, "8192", softcap=50.0),
        # packed prompts made of documents, each with a prefix seen in both directions, distance bias
        span_case("span documents prefix alibi", "bf16", 16, 4, 128, 128, "9001,1,4096,777",
                  texts(spread(9001, 5, 3) + [1] + spread(4096, 3, 5) + [777]),
                  "600,0,1500,33,1,0,1024,0,128,700", alibi=True),
        # the small single-precision layer, windowed
        span_case("span window f32 1000", "f32", 2, 1, 64, 64, "1000", texts(spread(1000, 3, 1)),
                  "", softcap=20.0, window=200),
        # one request with a very long context: the latency of a single token
        decode_case("decode one 131072", "bf16", 32, 8, 128, 128, "131072"),
        # an ordinary ragged batch in a layer with cap and window, a padded entry among it
        decode_case("decode ragged cap window", "bf16", 16, 8, 128, 64,
                    texts([1 + (977 * i * i + 131 * i) % 8191 for i in range(63)] + [0]),
                    softcap=30.0, window=4096),
        # many requests behind one long system prompt
        decode_case("decode prefix 32768 x 128", "bf16", 32, 8, 128, 128,
                    texts([32768 + 1 + (37 * i) % 601 for i in range(128)]), groups="128",
                    prefix_pages="256"),
        # an 8-bit cache, drafted tokens (three per request), two shared prompts and a group without
        decode_case("decode e4m3 drafts groups", "e4m3", 24, 8, 128, 32,
                    texts([4096 + 3 + 53 * i for i in range(20)] +
                          [1024 + 3 + 211 * i for i in range(20)] +
                          [3 + 400 * i for i in range(8)]), q_len=3, groups="20,20,8",
                    prefix_pages="128,32,0"),
        # the smallest call: a few short requests in single precision
        decode_case("decode small f32", "f32", 4, 2, 64, 16, "1,37,300", alibi=True),
        # one token more for a handful of requests
        {"name": "pages step 8", "op": "pages", "page": 128, "old": texts(300 + 128 * i for i in range(8)),
         "new": texts(301 + 128 * i for i in range(8))},
        # a large server: prompts arriving, requests stepping, finished ones giving pages back
        {"name": "pages mixed 1024", "op": "pages", "page": 16,
         "old": texts((0 if i % 3 == 0 else (i * 37) % 3001) for i in range(1024)),
         "new": texts(((i * 53) % 900 if i % 3 == 0 else 0 if i % 7 == 1 else (i * 37) % 3001 + 1)
                      for i in range(1024))},
        # the rows of one decode step
        {"name": "append step 64", "op": "append", "dtype": "bf16", "hkv": 8, "d": 128, "page": 128,
         "tokens": 64, "pages": 256},
        # a prompt quantised into an 8-bit cache
        {"name": "append e4m3 16384", "op": "append", "dtype": "e4m3", "hkv": 8, "d": 128, "page": 64,
         "tokens": 16384, "pages": 300},
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["span", "span", "decode", "decode", "decode", "pages", "append"])
    if op == "span":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        hkv = rng.choice([1, 2, 3, 4])
        hq = hkv * rng.choice([1, 2, 3, 4])
        d, block = (128, 128) if dtype == "bf16" and rng.random() < 0.7 else \
            (rng.choice([64, 128]), rng.choice([16, 32, 64, 128]))
        total = log_int(rng, 20, 8192 if d == 128 and block == 128 and dtype == "bf16" else 1500)
        lens = spread(total, rng.randint(1, min(4, total)), rng.randint(0, 50))
        docs, prefix = "", ""
        if rng.random() < 0.6:
            parts = [spread(n, rng.randint(1, min(4, n)), rng.randint(0, 50)) for n in lens]
            flat = [n for p in parts for n in p]
            docs = texts(flat)
            if rng.random() < 0.6:
                prefix = texts(rng.randint(0, n) for n in flat)
        return span_case("", dtype, hq, hkv, d, block, texts(lens), docs, prefix,
                         rng.choice([0.0, 20.0, 50.0]), rng.random() < 0.4,
                         rng.choice([0, 0, log_int(rng, 1, total)]))
    if op == "decode":
        dtype = rng.choice(["bf16", "bf16", "e4m3", "f32"])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 7, 8])
        page = rng.choice([16, 32, 64, 128])
        q_len = rng.choice([1, 1, 1, 2, 5])
        num = log_int(rng, 1, 96)
        longest = log_int(rng, 1, 1500 if dtype == "f32" else min(65536, 400000 // num))
        ctx = [rng.randint(0, longest) for _ in range(num)]
        groups, prefix_pages = "", ""
        if rng.random() < 0.5:
            sizes = spread(num, rng.randint(1, min(3, num)), rng.randint(0, 50))
            shared = [rng.randint(0, ceil_div(longest, page)) for _ in sizes]
            groups, prefix_pages = texts(sizes), texts(shared)
            of = [g for g, n in enumerate(sizes) for _ in range(n)]
            ctx = [shared[of[i]] * page + q_len + n // 4 for i, n in enumerate(ctx)]
        return decode_case("", dtype, hq, hkv, rng.choice([64, 128, 128]), page, texts(ctx), q_len,
                           groups, prefix_pages, rng.choice([0.0, 0.0, 30.0]), rng.random() < 0.3,
                           rng.choice([0, 0, log_int(rng, 1, longest)]))
    if op == "pages":
        num, most = log_int(rng, 1, 1024), log_int(rng, 1, 3000)
        old = [rng.choice([0, rng.randint(0, most)]) for _ in range(num)]
        new = [rng.choice([0, n + 1, n + 1, rng.randint(0, most)]) for n in old]
        return {"op": "pages", "page": rng.choice([16, 32, 64, 128]), "old": texts(old),
                "new": texts(new)}
    tokens, page = log_int(rng, 1, 12000), rng.choice([16, 32, 64, 128])
    return {"op": "append", "dtype": rng.choice(["f32", "bf16", "e4m3"]),
            "hkv": rng.choice([1, 3, 8]), "d": rng.choice([64, 128]), "page": page,
            "tokens": tokens, "pages": ceil_div(tokens, page) + rng.randint(0, 40)}


# ---- what a program has in hand -------------------------------------------------------------


def slopes_of(hq, device):
    """Geometric per-head slopes, 2^(-8 (h + 1) / hq)."""
    return torch.pow(2.0, -8.0 * torch.arange(1, hq + 1, dtype=torch.float64, device=device) / hq).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"span": prepare_span, "decode": prepare_decode, "pages": prepare_pages,
            "append": prepare_append}[case["op"]](case, gen)


def normal(gen, shape, dtype, gain=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * gain).to(dtype)


def cumulative(values):
    return np.concatenate([[0], np.cumsum(np.asarray(values, dtype=np.int64))]).astype(np.int32)


def prepare_span(case, gen):
    dt, lens = DT[case["dtype"]], ints(case["lens"])
    total = sum(lens)
    # logits with a spread of about 3: the cap bends the largest ones
    s = {"case": case,
         "q": normal(gen, (total, case["hq"], case["d"]), dt, 3.0),
         "k": normal(gen, (total, case["hkv"], case["d"]), dt),
         "v": normal(gen, (total, case["hkv"], case["d"]), dt),
         "cu": torch.from_numpy(cumulative(lens)).cuda(),
         "slopes": slopes_of(case["hq"], "cuda") if case["alibi"] else None,
         "doc_cu": torch.from_numpy(cumulative(ints(case["docs"]))).cuda() if case["docs"] else None,
         "prefix": torch.tensor(ints(case["prefix"]), dtype=torch.int32, device="cuda")
         if case["prefix"] else None}
    if own:
        import dynamic_block_sparse_pooled_b200 as fpx
        s["pf"] = fpx.problem(s["q"], s["k"], case["block"], cumulative(lens))
        s["ws"] = fpx.workspace(s["pf"], -1)
        lo = torch.empty(total, dtype=torch.int32, device="cuda")
        hi = torch.empty_like(lo)
        s["rule"] = fpx.score_rule(case["softcap"], s["slopes"], case["window"], lo, hi)
        s["lo"], s["hi"] = lo, hi
        blocks = sum(ceil_div(n, case["block"]) ** 2 for n in lens) * case["hq"]
        s["col_idx"] = torch.empty(blocks, dtype=torch.int32, device="cuda")
    return s


def table_of(pages_each, order, shared_of):
    """Block table rows: `shared_of[s]` = (pages of the prompt the request begins with)."""
    width = max(1, max(pages_each))
    table = np.zeros((len(pages_each), width), np.int32)
    at = 0
    for s, n in enumerate(pages_each):
        lead = shared_of[s][:n]
        table[s, :len(lead)] = lead
        table[s, len(lead):n] = order[at:at + n - len(lead)]
        at += n - len(lead)
    return table


def prepare_decode(case, gen):
    page, ctx, hkv, d = case["page"], ints(case["ctx"]), case["hkv"], case["d"]
    sizes, shared = ints(case["groups"]), ints(case["prefix_pages"])
    pages_each = [ceil_div(n, page) for n in ctx]
    lead = [g for g, n in enumerate(sizes) for _ in range(n)]
    num_pages = sum(shared) + sum(max(0, n - (shared[lead[s]] if lead else 0))
                                  for s, n in enumerate(pages_each)) + 3
    order = torch.randperm(num_pages, generator=gen, device="cuda").cpu().numpy().astype(np.int32)
    cut = np.concatenate([[0], np.cumsum(shared)]).astype(int) if shared else [0]
    prompts = [list(order[cut[g]:cut[g + 1]]) for g in range(len(sizes))]
    table = table_of(pages_each, order[cut[-1]:], [prompts[lead[s]] if lead else []
                                                   for s in range(len(ctx))])
    dt = DT[case["dtype"]]
    qdt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    shape = (num_pages, page, hkv, d)
    e4m3 = case["dtype"] == "e4m3"
    s = {"case": case, "q": normal(gen, (len(ctx) * case["q_len"], case["hq"], d), qdt, 2.0),
         "k": normal(gen, shape, torch.float32, 60.0).clamp_(-448, 448).to(dt) if e4m3
         else normal(gen, shape, dt),
         "v": normal(gen, shape, torch.float32, 60.0).clamp_(-448, 448).to(dt) if e4m3
         else normal(gen, shape, dt),
         "k_scale": (torch.rand(hkv, generator=gen, device="cuda") + 0.5) / 60 if e4m3 else None,
         "v_scale": (torch.rand(hkv, generator=gen, device="cuda") + 0.5) / 60 if e4m3 else None,
         "table": torch.from_numpy(table).cuda(),
         "ctx": torch.tensor(ctx, dtype=torch.int32, device="cuda"),
         "slopes": slopes_of(case["hq"], "cuda") if case["alibi"] else None}
    if own:
        import dynamic_block_sparse_pooled_b200 as fpx
        more = {}
        if sizes:
            more = {"group_ptr": torch.from_numpy(cumulative(sizes)).cuda(),
                    "prefix_pages": torch.tensor(shared, dtype=torch.int32, device="cuda")}
        s["dp"] = fpx.decode_problem(s["q"], s["k"], s["ctx"], s["table"], case["q_len"],
                                     k_scale=s["k_scale"], v_scale=s["v_scale"], **more)
        s["ws"] = fpx.decode_workspace(s["dp"])
        s["rule"] = fpx.score_rule(case["softcap"], s["slopes"], case["window"])
    return s


def prepare_pages(case, gen):
    page, old, new = case["page"], ints(case["old"]), ints(case["new"])
    have = [ceil_div(n, page) for n in old]
    width = max(1, max(ceil_div(max(a, b), page) for a, b in zip(old, new)))
    grow = sum(max(0, ceil_div(b, page) - ceil_div(a, page)) for a, b in zip(old, new))
    num_pages = sum(have) + grow + 5
    order = torch.randperm(num_pages, generator=gen, device="cuda").cpu().numpy().astype(np.int32)
    table = table_of(have, order, [[] for _ in have])
    table = np.concatenate([table, np.zeros((len(old), width - table.shape[1]), np.int32)], axis=1)
    free = np.zeros(num_pages, np.int32)
    left = order[sum(have):]
    free[:len(left)] = left
    tokens = sum(max(0, b - a) for a, b in zip(old, new))
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"case": case, "old": dev(old), "new": dev(new), "table": torch.from_numpy(table).cuda(),
         "free": torch.from_numpy(free).cuda(), "count": dev([len(left)]), "tokens": max(1, tokens),
         "num_pages": num_pages}
    if own:
        import dynamic_block_sparse_pooled_b200 as fpx
        s["ws"] = fpx.page_workspace(len(old))
        s["count_out"] = torch.empty(1, dtype=torch.int32, device="cuda")
    return s


def prepare_append(case, gen):
    shape = (case["pages"], case["page"], case["hkv"], case["d"])
    src = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    dt = DT[case["dtype"]]
    # K and V are two slices of the projection's output, as a layer has them
    kv = normal(gen, (case["tokens"], 2, case["hkv"], case["d"]), src)
    slots = torch.randperm(case["pages"] * case["page"], generator=gen, device="cuda")[:case["tokens"]]
    s = {"case": case, "k_new": kv[:, 0], "v_new": kv[:, 1], "slots": slots.int(),
         "k": torch.zeros(shape, device="cuda").to(dt), "v": torch.zeros(shape, device="cuda").to(dt),
         "k_scale": None, "v_scale": None}
    if case["dtype"] == "e4m3":
        s["k_scale"] = (torch.rand(case["hkv"], generator=gen, device="cuda") + 0.5) / 100
        s["v_scale"] = (torch.rand(case["hkv"], generator=gen, device="cuda") + 0.5) / 100
    if own:
        import dynamic_block_sparse_pooled_b200 as fpx
        s["ws"] = fpx.page_workspace(1)
    return s


# ---- one pass -------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        import dynamic_block_sparse_pooled_b200 as fpx
        return {"span": own_span, "decode": own_decode, "pages": own_pages,
                "append": own_append}[op](fpx, state)
    return {"span": plain_span, "decode": plain_decode, "pages": plain_pages,
            "append": plain_append}[op](state)


def own_span(fpx, s):
    fpx.spans(s["pf"], s["doc_cu"], s["prefix"], s["lo"], s["hi"])
    row_ptr, col_idx, _ = fpx.span_select(s["pf"], s["rule"], s["ws"], col_idx=s["col_idx"])
    o, lse = fpx.span_prefill(s["pf"], s["q"], s["k"], s["v"], s["rule"], row_ptr, col_idx, s["ws"])
    return {"o": o, "lse": lse, "lo": s["lo"], "hi": s["hi"], "row_ptr": row_ptr}


def own_decode(fpx, s):
    o, lse = fpx.decode(s["dp"], s["q"], s["k"], s["v"], s["ws"], s["rule"])
    return {"o": o, "lse": lse}


def own_pages(fpx, s):
    cu, slots, positions = fpx.page_resize(s["old"], s["new"], s["table"], s["free"], s["count"],
                                           s["case"]["page"], s["num_pages"], s["tokens"], s["ws"],
                                           count_out=s["count_out"])
    return {"cu": cu, "slots": slots, "positions": positions, "table": s["table"], "free": s["free"],
            "count": s["count_out"]}


def own_append(fpx, s):
    fpx.kv_append(s["k_new"], s["v_new"], s["slots"], s["k"], s["v"], s["ws"], s["k_scale"],
                  s["v_scale"])
    return {"k": s["k"], "v": s["v"]}


def softmax_rows(scores, seen):
    """(weights, 1 / sum, LSE) of the last axis, in place; a row that sees no key has weights 0."""
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    scores.sub_(top).exp_()
    total = scores.sum(-1, keepdim=True)
    return scores, torch.where(total > 0, 1 / total, torch.zeros_like(total)), (top + total.log()).squeeze(-1)


def plain_span(s):
    case, dev = s["case"], s["q"].device
    total, hq, d = s["q"].shape
    hkv, block = case["hkv"], case["block"]
    g = hq // hkv
    at = torch.arange(total, device=dev)
    seq = torch.searchsorted(s["cu"], at.int(), right=True) - 1
    start, end = s["cu"][seq].long(), s["cu"][seq + 1].long()
    here = at - start
    lo, hi = torch.zeros_like(at), here
    if s["doc_cu"] is not None:
        doc = torch.searchsorted(s["doc_cu"], at.int(), right=True) - 1
        d0 = torch.maximum(s["doc_cu"][doc].long(), start)
        d1 = torch.minimum(s["doc_cu"][doc + 1].long(), end)
        lo = d0 - start
        if s["prefix"] is not None:
            hi = torch.maximum(here, torch.minimum(d0 + s["prefix"][doc].long(), d1) - 1 - start)
    first = torch.maximum(lo, here - case["window"] + 1) if case["window"] else lo
    # [T, T]: token i (row) sees token j
    seen = (seq[:, None] == seq[None, :]) & (here[None, :] >= first[:, None]) & (here[None, :] <= hi[:, None])
    # kept key blocks of every query block: blocks restart at each sequence
    blocks = (s["cu"][1:] - s["cu"][:-1] + block - 1).div(block, rounding_mode="floor").long()
    base = torch.cumsum(blocks, 0) - blocks
    of = base[seq] + here.div(block, rounding_mode="floor")
    count = (total + block - 1) // block + s["cu"].numel()
    pair = torch.zeros(count, count, device=dev)
    rows = torch.zeros(count, total, device=dev).index_add_(0, of, seen.float())
    pair.index_add_(1, of, rows)
    kept = (pair > 0).sum(1)
    ends = torch.cumsum(kept, 0)
    last = base[-1] + blocks[-1]
    per_head = ends[:last]
    row_ptr = (per_head[None, :] + per_head[-1] * torch.arange(hq, device=dev)[:, None]).reshape(-1)
    row_ptr = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), row_ptr]).int()
    q = s["q"].float().view(total, hkv, g, d).permute(1, 2, 0, 3)
    k = s["k"].float().permute(1, 2, 0)[:, None]
    v = s["v"].float().permute(1, 0, 2)[:, None]
    scores = (q @ k).mul_(1 / math.sqrt(d))
    if case["softcap"]:
        scores.div_(case["softcap"]).tanh_().mul_(case["softcap"])
    if s["slopes"] is not None:
        far = (here[:, None] - here[None, :]).abs().float()
        scores.addcmul_(far[None, None], s["slopes"].view(hkv, g, 1, 1), value=-1)
    p, inverse, lse = softmax_rows(scores, seen)
    o = (p @ v) * inverse
    return {"o": o.permute(2, 0, 1, 3).reshape(total, hq, d).to(s["q"].dtype),
            "lse": lse.reshape(hq, total), "lo": lo.int(), "hi": hi.int(), "row_ptr": row_ptr}


def plain_decode(s):
    case, dev = s["case"], s["q"].device
    num, width = s["table"].shape
    page, hkv, q_len, hq, d = case["page"], case["hkv"], case["q_len"], case["hq"], case["d"]
    g = hq // hkv
    j = torch.arange(width * page, device=dev)
    row = s["table"].long()[:, j.div(page, rounding_mode="floor")] * page + j % page
    k = s["k"].view(-1, hkv, d)[row].float().permute(0, 2, 3, 1)
    v = s["v"].view(-1, hkv, d)[row].float().permute(0, 2, 1, 3)
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"].view(-1, 1, 1), v * s["v_scale"].view(-1, 1, 1)
    q = s["q"].float().view(num, q_len, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(num, hkv, g * q_len, d)
    at = s["ctx"].long()[:, None] - q_len + torch.arange(q_len, device=dev)
    seen = (j[None, None, :] <= at[:, :, None])
    if case["window"]:
        seen = seen & (j[None, None, :] > at[:, :, None] - case["window"])
    scores = (q @ k).mul_(1 / math.sqrt(d)).view(num, hkv, g, q_len, -1)
    if case["softcap"]:
        scores.div_(case["softcap"]).tanh_().mul_(case["softcap"])
    if s["slopes"] is not None:
        far = (at[:, :, None] - j[None, None, :]).abs().float()
        scores.addcmul_(far[:, None, None], s["slopes"].view(hkv, g, 1, 1), value=-1)
    p, inverse, lse = softmax_rows(scores, seen[:, None, None])
    o = (p.view(num, hkv, g * q_len, -1) @ v).view(num, hkv, g, q_len, d) * inverse
    return {"o": o.permute(0, 3, 1, 2, 4).reshape(num * q_len, hq, d).to(s["q"].dtype),
            "lse": lse.permute(1, 2, 0, 3).reshape(hq, num * q_len)}


def plain_pages(s):
    page, old, new, dev = s["case"]["page"], s["old"].long(), s["new"].long(), s["old"].device
    table, free = s["table"].clone(), s["free"].clone()
    num, width = table.shape
    have = (old + page - 1).div(page, rounding_mode="floor")
    want = (new + page - 1).div(page, rounding_mode="floor")
    j = torch.arange(width, device=dev)[None, :]
    # pages given back, in the order of requests and of their pages, onto the stack
    back = table[(j >= want[:, None]) & (j < have[:, None])]
    count = s["count"].long()
    at = torch.arange(free.numel(), device=dev)
    free = torch.where((at >= count) & (at < count + back.numel()),
                       torch.cat([back, back.new_zeros(1)])[(at - count).clamp(0, back.numel())], free)
    top = count + back.numel()
    # pages taken from its top, in the same order
    take = (j >= have[:, None]) & (j < want[:, None])
    rank = torch.cumsum(take.reshape(-1), 0).view(num, width) - 1
    table = torch.where(take, free[(top - 1 - rank).clamp(0, free.numel() - 1)], table)
    more = (new - old).clamp(min=0)
    ends = torch.cumsum(more, 0)
    t = torch.arange(s["tokens"], device=dev)
    r = torch.searchsorted(ends, t, right=True).clamp(max=num - 1)
    p = old[r] + t - (ends - more)[r]
    live = t < ends[-1]
    slot = table.long()[r, p.div(page, rounding_mode="floor").clamp(0, width - 1)] * page + p % page
    return {"cu": torch.cat([ends.new_zeros(1), ends]).int(),
            "slots": torch.where(live, slot, torch.full_like(slot, -1)).int(),
            "positions": torch.where(live, p, torch.full_like(p, -1)).int(),
            "table": table, "free": free, "count": (top - take.sum()).int()}


def plain_append(s):
    k, v = s["k_new"].float(), s["v_new"].float()
    if s["k_scale"] is not None:
        k = (k / s["k_scale"].view(-1, 1)).clamp(-448, 448)
        v = (v / s["v_scale"].view(-1, 1)).clamp(-448, 448)
    hkv, d = s["case"]["hkv"], s["case"]["d"]
    at = s["slots"].long()
    s["k"].view(-1, hkv, d)[at] = k.to(s["k"].dtype)
    s["v"].view(-1, hkv, d)[at] = v.to(s["v"].dtype)
    return {"k": s["k"], "v": s["v"]}


# ---- the same from the definition, in 64 bits -------------------------------------------------


def bounds(case):
    """Per sequence: (first, last) visible key of every token, numpy int64."""
    found, at = [], 0
    docs, prefix = ints(case["docs"]), ints(case["prefix"])
    cut, n_doc = 0, 0
    for n in ints(case["lens"]):
        lo, hi = np.zeros(n, np.int64), np.arange(n, dtype=np.int64)
        while docs and n_doc < len(docs) and cut < at + n:  # documents end where sequences end
            a, b = cut - at, cut - at + docs[n_doc]
            lo[a:b] = a
            if prefix:
                hi[a:b] = np.maximum(hi[a:b], min(a + prefix[n_doc], b) - 1)
            cut, n_doc = cut + docs[n_doc], n_doc + 1
        found.append((lo, hi))
        at += n
    return found


def windowed(case, lo, n):
    i = np.arange(n)
    return np.maximum(lo, i - case["window"] + 1) if case["window"] else lo


def attend64(q, k, v, at, lo, hi, case, slopes):
    """One sequence: q [n, hq, d], k and v [L, hkv, d] (64 bits); at, lo, hi [n]."""
    n, hq, d = q.shape
    g = hq // k.shape[1]
    j = torch.arange(k.shape[0], device=q.device)
    seen = (j[None] >= lo[:, None]) & (j[None] <= hi[:, None])
    o, lse = torch.zeros_like(q), torch.full((hq, n), -math.inf, dtype=torch.float64, device=q.device)
    for h in range(hq):
        x = q[:, h] @ k[:, h // g].T / math.sqrt(d)
        if case["softcap"]:
            x = case["softcap"] * torch.tanh(x / case["softcap"])
        if slopes is not None:
            x = x - slopes[h].double() * (at[:, None] - j[None]).abs()
        x = torch.where(seen, x, torch.full_like(x, -math.inf))
        lse[h] = torch.logsumexp(x, -1)
        w = torch.exp(x - torch.where(lse[h] == -math.inf, torch.zeros_like(lse[h]), lse[h])[:, None])
        o[:, h] = w @ v[:, h // g]
    return o, lse


def exact(case, seed):
    global own
    if case["op"] == "pages":
        return None
    keep, own = own, False
    s = prepare(case, seed)
    own = keep
    dev = "cuda"
    if case["op"] == "append":
        at = s["slots"].long()
        out = {}
        for name in ("k", "v"):
            cache = s[name].double().view(-1, case["hkv"], case["d"])
            x = s[name + "_new"].double()
            if case["dtype"] == "e4m3":
                x = (x / s[name + "_scale"].double()[:, None]).clamp(-448, 448)
            cache[at] = x
            out[name] = cache.view(s[name].shape)
        return out
    if case["op"] == "span":
        os, ls, at = [], [], 0
        spans = bounds(case)
        for (lo, hi), n in zip(spans, ints(case["lens"])):
            q, k, v = (s[x][at:at + n].double() for x in "qkv")
            f = torch.from_numpy(windowed(case, lo, n)).to(dev)
            o, lse = attend64(q, k, v, torch.arange(n, device=dev), f, torch.from_numpy(hi).to(dev),
                              case, s["slopes"])
            os.append(o)
            ls.append(lse)
            at += n
        return {"o": torch.cat(os), "lse": torch.cat(ls, 1), "lo": None, "hi": None, "row_ptr": None}
    os, ls = [], []
    page, q_len, table = case["page"], case["q_len"], s["table"].cpu().numpy()
    for r, n in enumerate(ints(case["ctx"])):
        rows = torch.from_numpy(table[r, :ceil_div(n, page)].astype(np.int64)).to(dev)
        k, v = (s[x][rows].reshape(-1, case["hkv"], case["d"])[:n].double() for x in "kv")
        if case["dtype"] == "e4m3":
            k, v = k * s["k_scale"].double()[:, None], v * s["v_scale"].double()[:, None]
        at = torch.arange(n - q_len, n, device=dev)
        lo = at - case["window"] + 1 if case["window"] else torch.zeros_like(at)
        o, lse = attend64(s["q"][r * q_len:(r + 1) * q_len].double(), k, v, at, lo, at, case, s["slopes"])
        os.append(o)
        ls.append(lse)
    return {"o": torch.cat(os), "lse": torch.cat(ls, 1)}


# ---- the work of one pass ---------------------------------------------------------------------


def work(case):
    if case["op"] == "span":
        total, pairs, blocks = sum(ints(case["lens"])), 0, 0
        for (lo, hi), n in zip(bounds(case), ints(case["lens"])):
            pairs += int(np.maximum(0, hi - windowed(case, lo, n) + 1).sum())
            blocks += ceil_div(n, case["block"])
        es = ES[case["dtype"]]
        return {"bytes": total * case["d"] * es * 2 * (case["hq"] + case["hkv"]) + 4 * total * case["hq"]
                + 8 * total + 4 * blocks * case["hq"], "flops": 4 * case["d"] * case["hq"] * pairs}
    if case["op"] == "decode":
        ctx, q_len, page = ints(case["ctx"]), case["q_len"], case["page"]
        sizes, shared = ints(case["groups"]), ints(case["prefix_pages"])
        lead = [g for g, n in enumerate(sizes) for _ in range(n)] or [-1] * len(ctx)
        keys, pairs, first = 0, 0, {}
        for g, n in zip(lead, ctx):
            pre = shared[g] * page if g >= 0 else 0
            lo = max(0, n - q_len - case["window"] + 1) if case["window"] else 0
            keys += max(0, n - max(pre, lo))
            if g >= 0 and n:
                first[g] = min(first.get(g, pre), lo)
            for t in range(q_len):
                i = n - q_len + t
                pairs += max(0, i + 1 - (max(0, i - case["window"] + 1) if case["window"] else 0))
        keys += sum(max(0, shared[g] * page - lo) for g, lo in first.items())
        rows = len(ctx) * q_len * case["hq"]
        es, qs = ES[case["dtype"]], 4 if case["dtype"] == "f32" else 2
        return {"bytes": keys * case["hkv"] * case["d"] * es * 2 + rows * (case["d"] * qs * 2 + 4)
                + 4 * sum(ceil_div(n, page) for n in ctx), "flops": 4 * case["d"] * case["hq"] * pairs}
    if case["op"] == "pages":
        old, new, page = ints(case["old"]), ints(case["new"]), case["page"]
        moved = sum(abs(ceil_div(b, page) - ceil_div(a, page)) for a, b in zip(old, new))
        tokens = sum(max(0, b - a) for a, b in zip(old, new))
        return {"bytes": 4 * (3 * len(old) + 2 * moved + 2 * tokens), "flops": 0}
    src = 4 if case["dtype"] == "f32" else 2
    row = 2 * case["hkv"] * case["d"]
    return {"bytes": case["tokens"] * (row * (src + ES[case["dtype"]]) + 4), "flops": 0}
