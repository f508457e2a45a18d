"""Measured cases of the decode step's state and routing operators.

The operators: the page plan of a step (block tables and slot maps from request lengths), the
8-bit KV cache's write and read-back, attention over that cache, and the routing to experts.
``run`` computes a case either in its plain form (elementary torch operations in fp32, rounded
once at the end) or, with ``own`` set, through the library's public entry points.

Cache layout: kq, vq int8 [pages, Hkv, P, D] and kd, vd float32 [pages, Hkv, P / S]: P tokens a
page, S tokens a scale block; slot = page * P + offset names one token's place.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # One decode step of a batch of 16 sequences: every sequence adds one token, a few start a page.
        {"name": "plan_decode_b16", "op": "plan", "B": 16, "page": 64, "ctx_min": 40, "ctx_max": 9000, "new_min": 1,
         "new_max": 1, "pad": 0, "short": False},
        # Admitting many prompts at once (prefix cached for some): half a million slots to fill.
        {"name": "plan_prompts_b512", "op": "plan", "B": 512, "page": 32, "ctx_min": 0, "ctx_max": 600, "new_min": 1,
         "new_max": 5000, "pad": 1000, "short": False},
        # The write of a single-user decode step: one token, K and V as the fp32 products leave them.
        {"name": "append_token_b1", "op": "append", "B": 1, "Hkv": 8, "D": 128, "page": 64, "block": 16, "ctx_min": 2347,
         "ctx_max": 2347, "new_min": 1, "new_max": 1, "dtype": "fp32"},
        # Speculative verify of 16 sequences: up to 8 tokens each, appended into blocks that hold older tokens.
        {"name": "append_verify_b16", "op": "append", "B": 16, "Hkv": 4, "D": 128, "page": 64, "block": 32, "ctx_min": 100,
         "ctx_max": 2000, "new_min": 2, "new_max": 8, "dtype": "bf16"},
        # A prompt's tokens going into the cache in one call (an odd number of them).
        {"name": "append_prompt_8k", "op": "append", "B": 2, "Hkv": 8, "D": 128, "page": 64, "block": 16, "ctx_min": 0,
         "ctx_max": 0, "new_min": 2101, "new_max": 6090, "dtype": "bf16"},
        # Single-user decode early in a conversation: latency (40 query heads on 8 cached heads).
        {"name": "attend_b1_ctx600", "op": "attend", "B": 1, "Hq": 40, "Hkv": 8, "D": 128, "page": 64, "block": 16,
         "ctx_min": 600, "ctx_max": 600, "n": 1, "window": 0, "dtype": "bf16"},
        # Single-user decode over a long document: the cache stream alone.
        {"name": "attend_b1_ctx130k", "op": "attend", "B": 1, "Hq": 40, "Hkv": 8, "D": 128, "page": 64, "block": 16,
         "ctx_min": 130001, "ctx_max": 130001, "n": 1, "window": 0, "dtype": "bf16"},
        # Batched decode of 16 sequences of very different lengths, activations kept in fp32.
        {"name": "attend_b16_ragged_fp32", "op": "attend", "B": 16, "Hq": 40, "Hkv": 8, "D": 128, "page": 32, "block": 32,
         "ctx_min": 37, "ctx_max": 16000, "n": 1, "window": 0, "dtype": "fp32"},
        # Speculative verify: 8 query tokens a sequence (32 query heads on 4 cached heads).
        {"name": "attend_verify_m8_b16", "op": "attend", "B": 16, "Hq": 32, "Hkv": 4, "D": 128, "page": 64, "block": 16,
         "ctx_min": 500, "ctx_max": 8000, "n": 8, "window": 0, "dtype": "bf16"},
        # One token's routing, 8 of 128 experts by softmax (the routed workload's own sizes).
        {"name": "route_t1_e128", "op": "route", "T": 1, "E": 128, "k": 8, "score": "softmax", "bias": False, "groups": 1,
         "topk_groups": 1, "group_top": 1, "dtype": "fp32"},
        # Batched decode with sigmoid scores, a balance bias and groups of experts.
        {"name": "route_t16_e256_groups", "op": "route", "T": 16, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "topk_groups": 4, "group_top": 2, "dtype": "fp32"},
        # A prompt's tokens, bf16 logits.
        {"name": "route_t8191_e256_groups", "op": "route", "T": 8191, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "topk_groups": 4, "group_top": 2, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "attend", "attend", "attend", "route"])
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([b for b in (1, 4, 16, 32, 64) if b <= page])
    if op == "plan":
        B = _log(rng, 1, 600)
        top = _log(rng, 1, max(1, min(5000, 1000000 // B)))
        return {"op": op, "B": B, "page": page, "ctx_min": 0, "ctx_max": _log(rng, 1, 9000), "new_min": rng.choice([0, 1]),
                "new_max": top, "pad": rng.choice([0, 3, 100]), "short": rng.random() < 0.25}
    if op == "append":
        Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        B = _log(rng, 1, 64)
        top = _log(rng, 1, max(1, min(6000, 8000 // B)))
        return {"op": op, "B": B, "Hkv": Hkv, "D": D, "page": page, "block": block, "ctx_min": 0, "ctx_max": _log(rng, 1, 4000),
                "new_min": 1, "new_max": top, "dtype": rng.choice(["bf16", "fp32"])}
    if op == "attend":
        Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        G = rng.choice([1, 2, 4, 5, 7, 8, 16])
        B = _log(rng, 1, 64)
        top = _log(rng, 16, max(64, min(131072, (1 << 27) // (B * Hkv * D))))
        n = rng.choice([1, 1, 2, 4, 8, 16])
        if n * G * Hkv * B * top > 1 << 27:
            n = 1
        return {"op": op, "B": B, "Hq": G * Hkv, "Hkv": Hkv, "D": D, "page": page, "block": block,
                "ctx_min": rng.choice([0, 1, max(1, top // 20)]), "ctx_max": top, "n": n,
                "window": rng.choice([0, 0, max(1, top // 3)]), "dtype": rng.choice(["bf16", "fp32"])}
    E = rng.choice([8, 64, 128, 160, 256, 512])
    groups = rng.choice([1, 1, 4, 8])
    T = _log(rng, 1, min(8191, (8191 * 256) // E))
    return {"op": op, "T": T, "E": E, "k": rng.choice([1, 2, 4, 6, 8]) if E > 8 else 2, "score": rng.choice(["softmax", "sigmoid"]),
            "bias": rng.random() < 0.5, "groups": groups, "topk_groups": max(1, groups // 2) if E > 8 else groups,
            "group_top": 1 if E // groups < 2 else rng.choice([1, 2]), "dtype": rng.choice(["bf16", "fp32"])}


# ---- sizes that a case fixes ----

def _spread(lo, hi, n, key):
    """n whole numbers from lo to hi, even over their logarithm, in an order that `key` fixes."""
    if n == 1 or lo == hi:
        return np.full(n, hi, np.int64)
    x = np.exp(np.linspace(math.log(lo + 1.0), math.log(hi + 1.0), n)) - 1.0
    return np.random.RandomState(key).permutation(np.rint(x).astype(np.int64))


def _lens(case):
    """(tokens in the cache before the step, tokens that the step adds) for each request."""
    B = case["B"]
    ctx = _spread(case["ctx_min"], case["ctx_max"], B, 1000 + B)
    if case["op"] == "attend":  # there, the lengths are those after the step: n of them are the queries
        new = np.minimum(np.full(B, case["n"], np.int64), ctx)
        return ctx - new, new
    return ctx, _spread(case["new_min"], case["new_max"], B, 2000 + B)


def _pages_of(lens, page):
    return (lens + page - 1) // page


def _read_count(case):
    """Tokens read back after an append: the live tokens of the scale blocks that it touched."""
    ctx, new = _lens(case)
    first = ctx - ctx % case["block"]
    return int(np.where(new > 0, ctx + new - first, 0).sum())


def work(case):
    if case["op"] == "plan":
        ctx, new = _lens(case)
        pages = int((_pages_of(ctx + new, case["page"]) - _pages_of(ctx, case["page"])).sum())
        total = int(new.sum()) + case["pad"]
        return {"bytes": 4 * (3 * case["B"] + 2 * total + 2 * pages), "flops": 2 * total}
    if case["op"] == "append":
        es = 2 if case["dtype"] == "bf16" else 4
        ctx, new = _lens(case)
        T, N, W = int(new.sum()), _read_count(case), case["Hkv"] * case["D"]
        # new values in, their codes out; the read rows' codes in, their values out; the slots
        return {"bytes": 2 * W * (T * (es + 1) + N * (1 + es)) + 4 * (T + N) + 8 * case["Hkv"] * (T + N) // case["block"],
                "flops": 2 * W * (4 * T + N)}
    if case["op"] == "attend":
        es = 2 if case["dtype"] == "bf16" else 4
        ctx, new = _lens(case)
        lens = ctx + new
        w = case["window"] or (1 << 40)
        seen = np.minimum(lens, w + new - 1) * (new > 0)
        pairs = sum(int(np.minimum(c + np.arange(n) + 1, w).sum()) for c, n in zip(ctx, new))
        row = 2 * case["Hkv"] * (case["D"] + 4.0 / case["block"])
        return {"bytes": int(seen.sum() * row) + int(new.sum()) * case["Hq"] * (2 * es * case["D"] + 4),
                "flops": 4 * case["D"] * case["Hq"] * pairs}
    es = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": case["T"] * (case["E"] * es + 8 * case["k"]) + 4 * case["E"] * case["bias"],
            "flops": case["T"] * case["E"] * 24}


# ---- inputs ----

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(1000003 * int(seed) + 17)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _table(have, page_ids, max_pages):
    """Block table [B, max_pages] (-1 where a request has no page) taking the ids in order."""
    at = np.arange(max_pages)[None, :] < have[:, None]
    table = np.full(at.shape, -1, np.int32)
    table[at] = page_ids[: int(have.sum())]
    return table


def _quantised(g, n_pages, case):
    """A cache of normal tokens (channels and tokens of different size), a scale for each block."""
    P, S, Hkv, D = case["page"], case["block"], case["Hkv"], case["D"]
    x = _randn(g, n_pages, Hkv, P, D)
    x *= torch.exp(0.4 * _randn(g, 1, Hkv, 1, D))
    x *= torch.exp(0.3 * _randn(g, n_pages, Hkv, P, 1))
    x = x.view(n_pages, Hkv, P // S, S * D)
    d = x.abs().amax(dim=-1) / 127.0
    x /= d[..., None]
    return x.round_().to(torch.int8).view(n_pages, Hkv, P, D), d


def prepare(case, seed):
    g = _gen(seed)
    rs = np.random.RandomState(int(seed) % (1 << 31))
    st = {"case": dict(case)}
    if case["op"] == "route":
        dt = DTYPES[case["dtype"]]
        st["logits"] = (1.5 * _randn(g, case["T"], case["E"])).to(dt)
        st["bias"] = 0.1 * _randn(g, case["E"]) if case["bias"] else None
        return st
    P = case["page"]
    ctx, new = _lens(case)
    if case["op"] == "plan":
        have, after = _pages_of(ctx, P), _pages_of(ctx + new, P)
        need = int((after - have).sum())
        n_pages = int(after.sum()) + 64
        ids = rs.permutation(n_pages).astype(np.int32)
        n_free = int(0.9 * need) if case["short"] else need + 40
        st.update(ctx=_dev(ctx.astype(np.int32)), new=_dev(new.astype(np.int32)), page=P, tokens=int(new.sum()) + case["pad"],
                  table=_dev(_table(have, ids, int(after.max()) + 2)), free=_dev(np.resize(ids[int(have.sum()):], 7 + n_free)),
                  head=torch.full((1,), 7, dtype=torch.int32, device=DEV))
        return st
    have = _pages_of(ctx + new, P)
    n_pages = int(have.sum()) + 3
    max_pages = int(have.max()) + 1
    table = _table(have, rs.permutation(n_pages).astype(np.int32), max_pages)
    kq, kd = _quantised(g, n_pages, case)
    vq, vd = _quantised(g, n_pages, case)
    # the scales of blocks that hold no token yet are whatever the memory held
    S = case["block"]
    held = ctx if case["op"] == "append" else ctx + new
    at = (np.arange(max_pages * (P // S))[None, :] * S < held[:, None]).reshape(case["B"], max_pages, P // S)
    live = np.zeros((n_pages, P // S), bool)
    live[table[table >= 0]] = at[table >= 0]
    dead = ~_dev(live)[:, None, :]
    kd.masked_fill_(dead, math.nan)
    vd.masked_fill_(dead, math.nan)
    st.update(kq=kq, kd=kd, vq=vq, vd=vd)
    T = int(new.sum())
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    owner = np.repeat(np.arange(case["B"]), new)
    pos = np.arange(T) - cu[owner] + ctx[owner]
    dt = DTYPES[case["dtype"]]
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "append":
        # K and V are columns of the fused projection's rows, next to the queries
        rows = (_randn(g, T, (2 * Hkv + 4) * D) * torch.exp(0.3 * _randn(g, T, 1))).to(dt)
        st["k"] = rows[:, 4 * D:(4 + Hkv) * D].view(T, Hkv, D)
        st["v"] = rows[:, (4 + Hkv) * D:].view(T, Hkv, D)
        st["slots"] = _dev((table[owner, pos // P].astype(np.int64) * P + pos % P).astype(np.int32))
        first = np.where(new > 0, ctx - ctx % S, ctx)
        count = ctx + new - first
        who = np.repeat(np.arange(case["B"]), count)
        at = np.arange(int(count.sum())) - np.repeat(np.cumsum(count) - count, count) + first[who]
        st["read"] = _dev((table[who, at // P].astype(np.int64) * P + at % P).astype(np.int32))
        st["dtype"] = dt
        return st
    st["q"] = (1.5 * _randn(g, T, case["Hq"], D)).to(dt)
    st.update(table=_dev(table), kv_lens=_dev((ctx + new).astype(np.int32)), cu_q=_dev(cu), n=case["n"], window=case["window"],
              scale=D ** -0.5, workspace=torch.zeros(32 << 20, dtype=torch.uint8, device=DEV))
    return st


# ---- the plain forms ----

def _plain_plan(st):
    P, table, T = st["page"], st["table"], st["tokens"]
    ctx, new = st["ctx"].long(), st["new"].long()
    B, max_pages = table.shape
    n_free = st["free"].shape[0]
    have, after = (ctx + P - 1) // P, (ctx + new + P - 1) // P
    upto = torch.cumsum(new, 0)
    fits = (after <= max_pages) & (upto <= T)
    need = torch.where(fits, after - have, 0)
    end = st["head"].long() + torch.cumsum(need, 0)
    ok = fits & ((need == 0) | (end <= n_free))
    col = torch.arange(max_pages, device=DEV)[None, :]
    fresh = ok[:, None] & (col >= have[:, None]) & (col < after[:, None])
    at = (end - need)[:, None] + col - have[:, None]
    table = torch.where(fresh, st["free"][at.clamp(0, n_free - 1)], table)
    cu = torch.cat([upto.new_zeros(1), upto]).clamp(max=T)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    real = b < B
    b = b.clamp(max=B - 1)
    pos = torch.where(real, ctx[b] + t - cu[b], -1)
    page = table[b, (pos // P).clamp(0, max_pages - 1)].long()
    slots = torch.where(real & ok[b], page * P + pos % P, -1)
    head = st["head"].long() + torch.where(ok, need, 0).sum()
    return {"kv_lens": torch.where(ok, ctx + new, 0).int(), "cu_q": cu.int(), "slots": slots.int(), "positions": pos.int(),
            "table": table, "head": head.int()}


def _away(x):
    """Nearest whole number, halves away from zero."""
    t = torch.trunc(x)
    return torch.where((x - t).abs() == 0.5, t + torch.sign(x), torch.round(x))


def _ratio(a, b):
    return torch.where(b == 0, 0.0, a / b)


def _plain_append_plane(x, q, d, slots, read, out_dtype):
    n_pages, Hkv, P, D = q.shape
    nb = d.shape[2]
    S = P // nb
    slots, read = slots.long(), read.long()
    x = x.float()
    blocks = n_pages * nb
    d0 = d.permute(0, 2, 1).reshape(blocks, Hkv)
    tok_block = slots // S
    amax = torch.zeros(blocks, Hkv, device=DEV).scatter_reduce(0, tok_block[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
    first = torch.full((blocks,), S, device=DEV).scatter_reduce(0, tok_block, slots % S, "amin")
    old = torch.where((first > 0)[:, None], d0, 0.0)
    d1 = torch.where((first < S)[:, None], torch.maximum(old, amax / torch.full_like(amax, 127.0)), d0)  # a division, not a product
    # the tokens read back: older ones at the block's new scale, new ones quantised with it
    rb, ro, rp = read // S, read % S, read // P
    codes = q[rp, :, read % P].float()
    dr, dold = d1[rb], old[rb]
    grown = torch.where((dr > dold)[..., None], _away(codes * _ratio(dold, dr)[..., None]), codes)
    source = torch.full((n_pages * P,), -1, device=DEV).scatter(0, slots, torch.arange(slots.shape[0], device=DEV))[read]
    fresh = _away(_ratio(x[source.clamp(min=0)], dr[..., None])).clamp(-127, 127)
    codes = torch.where((ro < first[rb])[:, None, None], grown, fresh)
    return (codes * dr[..., None]).to(out_dtype), d1.view(n_pages, nb, Hkv).permute(0, 2, 1).contiguous()


def _plain_append(st):
    k, kd = _plain_append_plane(st["k"], st["kq"], st["kd"], st["slots"], st["read"], st["dtype"])
    v, vd = _plain_append_plane(st["v"], st["vq"], st["vd"], st["slots"], st["read"], st["dtype"])
    return {"k": k, "v": v, "kd": kd, "vd": vd}


def _plain_rows(q, d, table, live):
    """The cached rows of each request, [B, Hkv, L, D]; zeros where it has no token."""
    B, max_pages = table.shape
    _, Hkv, P, D = q.shape
    nb = d.shape[2]
    page = table.clamp(min=0).long()
    x = q[page].float().view(B, max_pages, Hkv, nb, P // nb, D) * d[page][..., None, None]
    x = x.view(B, max_pages, Hkv, P, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, max_pages * P, D)
    return torch.where(live[:, None, :, None], x, 0.0)


def _plain_attend(st):
    q, table, n, window = st["q"], st["table"], st["n"], st["window"]
    T, Hq, D = q.shape
    B = table.shape[0]
    Hkv, P = st["kq"].shape[1], st["kq"].shape[2]
    G, L = Hq // Hkv, table.shape[1] * P
    lens, cu = st["kv_lens"].long(), st["cu_q"].long()
    count = cu[1:] - cu[:-1]
    key = torch.arange(L, device=DEV)
    live = key[None, :] < lens[:, None]
    row = torch.arange(n, device=DEV)
    at = (cu[:-1, None] + row[None, :]).clamp(max=T - 1)
    x = q[at].float().view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    s = torch.matmul(x, _plain_rows(st["kq"], st["kd"], table, live).transpose(2, 3)) * st["scale"]
    pos = lens[:, None] - count[:, None] + row[None, :]
    seen = (key[None, None, :] <= pos[..., None]) & live[:, None, :]
    if window:
        seen &= key[None, None, :] > pos[..., None] - window
    seen = seen[:, None, :, None, :].expand(B, 1, n, G, L).reshape(B, 1, n * G, L)
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _plain_rows(st["vq"], st["vd"], table, live))
    o = torch.where(l > 0, o / l, 0.0).view(B, Hkv, n, G, D)
    lse = (m + torch.log(l)).view(B, Hkv, n, G)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=B - 1)
    i = t - cu[b]
    return {"out": o[b, :, i].reshape(T, Hq, D).to(q.dtype), "lse": lse[b, :, i].reshape(T, Hq)}


def _exp(x):
    """exp by Cody and Waite's range reduction and the degree-7 Taylor polynomial, every step rounded to fp32:
    the library's own exponential, so that equal scores stay equal and the choice of experts is the same."""
    x = x.clamp(-87.0, 88.0)
    k = torch.round(x * 1.44269504088896341)
    r = (x - k * 0.693359375) - k * -2.12194440e-4
    p = torch.full_like(r, 1.0 / 5040.0)
    p = p * r + 1.0 / 720.0
    p = p * r + 1.0 / 120.0
    p = p * r + 1.0 / 24.0
    p = p * r + 1.0 / 6.0
    p = p * r + 0.5
    p = p * r + 1.0
    p = p * r + 1.0
    return p * ((k.int() + 127) << 23).view(torch.float32)


def _sum_by_lanes(e):
    """Row sums in the routing's stated order: 32 lanes take four neighbouring experts of each 128 in turn, and
    the lanes are joined pairwise at distances 16, 8, 4, 2, 1."""
    T, E = e.shape
    c = -(-E // 128)
    e = torch.nn.functional.pad(e, (0, 128 * c - E)).view(T, c, 32, 4).permute(0, 1, 3, 2).reshape(T, 4 * c, 32)
    a = e[:, 0]
    for j in range(1, 4 * c):
        a = a + e[:, j]
    a = a[:, :16] + a[:, 16:]
    a = a[:, :8] + a[:, 8:]
    a = a[:, :4] + a[:, 4:]
    a = a[:, :2] + a[:, 2:]
    return a[:, :1] + a[:, 1:]


def _ranked(v, k):
    """The k largest of each row, ties to the lowest index."""
    return torch.sort(v, dim=-1, descending=True, stable=True).indices[..., :k]


def _plain_route(st):
    c = st["case"]
    x = st["logits"].float()
    T, E = x.shape
    if c["score"] == "softmax":
        e = _exp(x - x.amax(-1, keepdim=True))
        s = e / _sum_by_lanes(e)
    else:
        s = 1.0 / (1.0 + _exp(-x))
    v = s if st["bias"] is None else s + st["bias"]
    if c["groups"] > 1:
        per = v.view(T, c["groups"], E // c["groups"])
        best = torch.sort(per, dim=-1, descending=True).values
        score = best[..., 0] if c["group_top"] == 1 else best[..., 0] + best[..., 1]
        keep = torch.zeros_like(score, dtype=torch.bool).scatter(1, _ranked(score, c["topk_groups"]), True)
        v = torch.where(keep[..., None], per, -math.inf).view(T, E)
    ids = _ranked(v, c["k"])
    w = s.gather(1, ids)
    total = w.sum(-1, keepdim=True)
    return {"ids": ids.int(), "weights": torch.where(total > 0, w / total, 0.0) * 2.5}


# ---- one pass ----

def run(state):
    op = state["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "append": _plain_append, "attend": _plain_attend, "route": _plain_route}[op](state)
    import block_quantized_decode_quantize_gb300 as memra
    if op == "plan":
        kv_lens, cu_q, slots, positions, head = memra.memra_kv_plan(
            state["ctx"], state["new"], state["page"], state["free"], state["table"], state["tokens"], free_head=state["head"])
        return {"kv_lens": kv_lens, "cu_q": cu_q, "slots": slots, "positions": positions, "table": state["table"], "head": head}
    if op == "append":
        cache = (state["kq"], state["kd"], state["vq"], state["vd"])
        memra.memra_kv_append_q8(state["k"], state["v"], state["slots"], *cache)
        k, v = memra.memra_kv_read_q8(state["read"], *cache, dtype=state["dtype"])
        return {"k": k, "v": v, "kd": state["kd"], "vd": state["vd"]}
    if op == "attend":
        out, lse = memra.memra_kv_attention_q8(
            state["q"], state["kq"], state["kd"], state["vq"], state["vd"], state["table"], state["kv_lens"], state["cu_q"],
            scale=state["scale"], window=state["window"], workspace=state["workspace"])
        return {"out": out, "lse": lse}
    c = state["case"]
    ids, weights = memra.memra_moe_route(state["logits"], c["k"], bias=state["bias"], score=c["score"], n_groups=c["groups"],
                                         topk_groups=c["topk_groups"], group_top=c["group_top"], renormalize=True, scale=2.5)
    return {"ids": ids, "weights": weights}


# ---- the definitions in 64 bits ----

def _exact_plane(x, q, d, slots, read):
    n_pages, Hkv, P, D = q.shape
    S = P // d.shape[2]
    x, d = x.double().cpu().numpy(), d.double().cpu().numpy()
    slots, read, q = slots.cpu().numpy().astype(np.int64), read.cpu().numpy().astype(np.int64), q.cpu().numpy()
    out_d, values = d.copy(), np.empty((read.size, Hkv, D))
    row = {int(r): i for i, r in enumerate(read)}
    start = 0
    while start < slots.size:
        block = slots[start] // S
        stop = start
        while stop < slots.size and slots[stop] // S == block:
            stop += 1
        page, b, first = int(block * S // P), int(block * S % P) // S, int(slots[start] % S)
        new = x[start:stop]
        before = d[page, :, b] if first else np.zeros(Hkv)
        scale = np.maximum(before, np.abs(new).max(axis=(0, 2)) / 127.0)
        out_d[page, :, b] = scale
        for j in range(first):
            c = q[page, :, b * S + j].astype(np.float64) * (before / scale)[:, None]
            values[row[int(block * S + j)]] = np.copysign(np.floor(np.abs(c) + 0.5), c) * scale[:, None]
        c = new / scale[None, :, None]
        c = np.copysign(np.floor(np.abs(c) + 0.5), c) * scale[None, :, None]
        for j in range(start, stop):
            values[row[int(slots[j])]] = c[j - start]
        start = stop
    return torch.from_numpy(values), torch.from_numpy(out_d)


def _exact_attend(st):
    q, table, scale, window = st["q"].double(), st["table"].cpu().numpy(), st["scale"], st["window"]
    T, Hq, D = q.shape
    Hkv, P = st["kq"].shape[1], st["kq"].shape[2]
    S, G = P // st["kd"].shape[2], Hq // Hkv
    lens, cu = st["kv_lens"].cpu().numpy(), st["cu_q"].cpu().numpy()
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(table.shape[0]):
        L, n = int(lens[b]), int(cu[b + 1] - cu[b])
        if L == 0 or n == 0:
            continue
        pages = torch.from_numpy(table[b, : -(-L // P)].astype(np.int64)).to(DEV)
        j = torch.arange(L, device=DEV)
        i = torch.arange(L - n, L, device=DEV)
        hidden = j[None, :] > i[:, None]
        if window:
            hidden |= i[:, None] - j[None, :] >= window
        for h in range(Hkv):
            k = st["kq"][pages, h].reshape(-1, D)[:L].double() * st["kd"][pages, h].reshape(-1).repeat_interleave(S)[:L, None].double()
            v = st["vq"][pages, h].reshape(-1, D)[:L].double() * st["vd"][pages, h].reshape(-1).repeat_interleave(S)[:L, None].double()
            rows = q[int(cu[b]):int(cu[b + 1]), h * G:(h + 1) * G]
            score = torch.einsum("nge,le->ngl", rows, k) * scale
            score.masked_fill_(hidden[:, None, :], -math.inf)
            z = torch.logsumexp(score, dim=-1)
            lse[int(cu[b]):int(cu[b + 1]), h * G:(h + 1) * G] = z
            out[int(cu[b]):int(cu[b + 1]), h * G:(h + 1) * G] = torch.einsum("ngl,le->nge", torch.exp(score - z[..., None]), v)
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers only
    st = prepare(case, seed)
    if case["op"] == "append":
        k, kd = _exact_plane(st["k"], st["kq"], st["kd"], st["slots"], st["read"])
        v, vd = _exact_plane(st["v"], st["vq"], st["vd"], st["slots"], st["read"])
        return {"k": k, "v": v, "kd": kd, "vd": vd}
    if case["op"] == "attend":
        return _exact_attend(st)
    x = st["logits"].double().cpu().numpy()
    T, E = x.shape
    if case["score"] == "softmax":
        e = np.exp(x - x.max(axis=1, keepdims=True))
        s = e / e.sum(axis=1, keepdims=True)
    else:
        s = 1.0 / (1.0 + np.exp(-x))
    v = s if st["bias"] is None else s + st["bias"].double().cpu().numpy()[None]
    size = E // case["groups"]
    weights = np.empty((T, case["k"]))
    for t in range(T):
        order = np.argsort(-v[t], kind="stable")
        if case["groups"] > 1:
            g = v[t].reshape(case["groups"], size)
            top = np.sort(g, axis=1)[:, ::-1][:, : case["group_top"]].sum(axis=1)
            kept = set(np.argsort(-top, kind="stable")[: case["topk_groups"]].tolist())
            order = np.array([e for e in order if e // size in kept])
        w = s[t, order[: case["k"]]]
        weights[t] = 2.5 * w / w.sum()
    return {"ids": None, "weights": torch.from_numpy(weights)}
