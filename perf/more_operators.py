"""Measured cases of the decode step's operators around the cache and the LM head.

The operators: the norm and rotation of queries and keys, the log probabilities of tokens with entropy
and top alternatives, and the cache's pages after they are taken: forking sequences (shared pages,
copy on write, release) and compacting the pool.  ``run`` computes a case either in its plain form
(elementary torch operations in fp32, angles in fp64, rounded once at the end) or, with ``own`` set,
through the library's public entry points.

Cache layout, a layer: kq, vq int8 [pages, Hkv, P, D] and kd, vd float32 [pages, Hkv, P / S].  A copy of
pages moves codes and scales bit for bit, so both come back as they are held and have to be equal.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # One token of single-user decode: 40 query and 8 key heads as the fp32 QKV product leaves them; queries go
        # to attention in bf16, keys to the cache's write in fp32.
        {"name": "rope_t1_fp32", "op": "rope", "T": 1, "Hq": 40, "Hkv": 8, "D": 128, "R": 128, "layout": "halves", "norm": True,
         "base": 1000000.0, "far": 130001, "pad": 0, "dtype": "fp32", "q_dtype": "bf16", "k_dtype": "fp32"},
        # Speculative verify of 16 sequences x 8 tokens: half of each head rotated, neighbouring pairs, some padded rows.
        {"name": "rope_t128_partial_pairs", "op": "rope", "T": 128, "Hq": 32, "Hkv": 4, "D": 128, "R": 64, "layout": "pairs",
         "norm": True, "base": 10000.0, "far": 8000, "pad": 5, "dtype": "bf16", "q_dtype": "bf16", "k_dtype": "bf16"},
        # A prompt's tokens (an odd number of them), bf16 rows of the fused projection.
        {"name": "rope_t8191_bf16", "op": "rope", "T": 8191, "Hq": 40, "Hkv": 8, "D": 128, "R": 128, "layout": "halves",
         "norm": True, "base": 1000000.0, "far": 131071, "pad": 0, "dtype": "bf16", "q_dtype": "bf16", "k_dtype": "bf16"},
        # The LM head's logits of one decoded token: its log probability and 20 alternatives.
        {"name": "logprobs_t1_v151936", "op": "logprobs", "T": 1, "V": 151936, "pad": 0, "top": 20, "masked": 0.0, "dtype": "fp32"},
        # A step of 16 sequences (the largest batch of a product) under a grammar that forbids most tokens.
        {"name": "logprobs_t16_masked", "op": "logprobs", "T": 16, "V": 151936, "pad": 128, "top": 5, "masked": 0.999, "dtype": "fp32"},
        # Scoring a few hundred tokens with a small, odd vocabulary, whose rows start at any alignment.
        {"name": "logprobs_t301_v32003", "op": "logprobs", "T": 301, "V": 32003, "pad": 0, "top": 10, "masked": 0.0, "dtype": "bf16"},
        # Scoring a prompt: logits of 2047 tokens in bf16.
        {"name": "logprobs_t2047_v151936", "op": "logprobs", "T": 2047, "V": 151936, "pad": 0, "top": 5, "masked": 0.0, "dtype": "bf16"},
        # The same in fp32, for no alternatives (perplexity of a text).
        {"name": "logprobs_t640_v151936_fp32", "op": "logprobs", "T": 640, "V": 151936, "pad": 0, "top": 0, "masked": 0.0, "dtype": "fp32"},
        # Four samples of one prompt: fork, own last pages in one layer, and their release at the end.
        {"name": "fork_b1_n4", "op": "fork", "B": 1, "n": 4, "layers": 1, "Hkv": 8, "D": 128, "page": 64, "block": 16,
         "ctx_min": 2347, "ctx_max": 2347},
        # Eight samples of each of 32 prompts over 16 layers.
        {"name": "fork_b32_n8", "op": "fork", "B": 32, "n": 8, "layers": 16, "Hkv": 8, "D": 128, "page": 64, "block": 16,
         "ctx_min": 300, "ctx_max": 9000},
        # A small pool after requests have left it.
        {"name": "compact_p256", "op": "compact", "B": 6, "pages": 256, "layers": 1, "Hkv": 4, "D": 128, "page": 64, "block": 32,
         "ctx_min": 40, "ctx_max": 2000},
        # A large pool, about a third in use, whose tail is to be given back.
        {"name": "compact_p6000", "op": "compact", "B": 48, "pages": 6000, "layers": 2, "Hkv": 8, "D": 128, "page": 64, "block": 16,
         "ctx_min": 500, "ctx_max": 8000},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "logprobs", "logprobs", "logprobs", "fork", "compact"])
    Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
    if op == "rope":
        Hq = Hkv * rng.choice([1, 2, 4, 5, 7, 8, 16])
        return {"op": op, "T": _log(rng, 1, min(8191, 8191 * 48 * 128 // (2 * (Hq + Hkv) * D))), "Hq": Hq, "Hkv": Hkv, "D": D,
                "R": rng.choice([D, D, D // 2, D // 4]), "layout": rng.choice(["halves", "pairs"]), "norm": rng.random() < 0.7,
                "base": rng.choice([10000.0, 500000.0, 1000000.0]), "far": _log(rng, 1, 1000000), "pad": rng.choice([0, 0, 1, 9]),
                "dtype": rng.choice(["bf16", "fp32"]), "q_dtype": rng.choice(["bf16", "fp32"]), "k_dtype": rng.choice(["bf16", "fp32"])}
    if op == "logprobs":
        V = _log(rng, 700, 262144)
        return {"op": op, "T": _log(rng, 1, min(8191, 80000000 // V)), "V": V, "pad": rng.choice([0, 0, 1, 64]),
                "top": rng.choice([0, 1, 5, 10, 20, 32]), "masked": rng.choice([0.0, 0.0, 0.5, 0.99]),
                "dtype": rng.choice(["bf16", "fp32"])}
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([b for b in (1, 4, 16, 32, 64) if b <= page])
    layers = rng.choice([1, 2, 5])
    if op == "fork":
        B = _log(rng, 1, 32)
        return {"op": op, "B": B, "n": _log(rng, 1, min(32, 256 // B)), "layers": layers, "Hkv": Hkv, "D": D, "page": page, "block": block,
                "ctx_min": rng.choice([0, 1, 100]), "ctx_max": _log(rng, 101, 9000)}
    B = _log(rng, 1, 64)
    top = _log(rng, 16, 100000 // B)
    held = sum(int(x) for x in _pages_of(_spread(0, top, B, 1000 + B), page))
    pages = held + _log(rng, 16, 2 * held + 64)
    while pages * layers * Hkv * D * page > 700000000 and layers > 1:
        layers -= 1
    return {"op": op, "B": B, "pages": pages, "layers": layers, "Hkv": Hkv, "D": D, "page": page, "block": block, "ctx_min": 0,
            "ctx_max": top}


# ---- sizes that a case fixes ----

def _spread(lo, hi, n, key):
    """n whole numbers from lo to hi, even over their logarithm, in an order that `key` fixes."""
    if n == 1 or lo == hi:
        return np.full(n, hi, np.int64)
    x = np.exp(np.linspace(math.log(lo + 1.0), math.log(hi + 1.0), n)) - 1.0
    return np.random.RandomState(key).permutation(np.rint(x).astype(np.int64))


def _lens(case):
    return _spread(case["ctx_min"], case["ctx_max"], case["B"], 1000 + case["B"])


def _pages_of(lens, page):
    return (lens + page - 1) // page


def work(case):
    if case["op"] == "rope":
        size = {"bf16": 2, "fp32": 4}
        rows = case["T"] * case["D"]
        real = (case["T"] - case["pad"] if case["T"] > case["pad"] else case["T"]) * case["D"]
        heads = case["Hq"] + case["Hkv"]
        return {"bytes": real * heads * size[case["dtype"]] + rows * (case["Hq"] * size[case["q_dtype"]] + case["Hkv"] * size[case["k_dtype"]])
                + 4 * case["T"] + 8 * case["D"] + 4 * case["R"], "flops": real * heads * 8}
    if case["op"] == "logprobs":
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["T"] * (case["V"] * es + 12 + 8 * case["top"]), "flops": 6 * case["T"] * case["V"]}
    P, lens = case["page"], _lens(case)
    token = 2 * case["layers"] * case["Hkv"] * (case["D"] + 4.0 / case["block"])  # K and V of one token in every layer
    held = int(_pages_of(lens, P).sum())
    if case["op"] == "fork":
        copied, n = int((lens % P).sum()) * case["n"], case["n"]
        return {"bytes": int(2 * copied * token) + 4 * held * (1 + 3 * n) + 24 * n * case["B"], "flops": 4 * held * n}
    moved = held * (1.0 - held / case["pages"])  # pages in use behind the first `held`, on average
    return {"bytes": int(2 * moved * P * token) + 8 * held + 12 * case["pages"], "flops": 8 * case["pages"]}


# ---- inputs ----

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(1000003 * int(seed) + 29)


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _table(have, page_ids, max_pages):
    """Block table [B, max_pages] (-1 where a request has no page) taking the ids in order."""
    at = np.arange(max_pages)[None, :] < have[:, None]
    table = np.full(at.shape, -1, np.int32)
    table[at] = page_ids[: int(have.sum())]
    return table


def _planes(g, case, n_pages):
    """Codes and scales of every layer, [layers, ...]."""
    L, Hkv, P, S, D = case["layers"], case["Hkv"], case["page"], case["block"], case["D"]
    st = {}
    for x in "kv":
        st[x + "q"] = torch.randint(-127, 128, (L, n_pages, Hkv, P, D), generator=g, dtype=torch.int8, device=DEV)
        st[x + "d"] = 0.01 + 0.02 * torch.rand((L, n_pages, Hkv, P // S), generator=g, device=DEV)
    st["caches"] = [(st["kq"][i], st["kd"][i], st["vq"][i], st["vd"][i]) for i in range(L)]
    return st


def prepare(case, seed):
    g = _gen(seed)
    rs = np.random.RandomState(int(seed) % (1 << 31))
    st = {"case": dict(case)}
    if case["op"] == "rope":
        T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
        rows = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device=DEV)
        rows *= torch.exp(0.3 * torch.randn((T, 1), generator=g, device=DEV))
        rows = rows.to(DTYPES[case["dtype"]])
        st["q"] = rows[:, :Hq * D].view(T, Hq, D)
        st["k"] = rows[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        # runs of neighbouring positions, as sequences and prompts have them, anywhere up to `far`
        pos = rs.randint(0, case["far"], max(1, T // 64))[np.arange(T) * max(1, T // 64) // T] + np.arange(T) % 64
        if case["pad"] and T > case["pad"]:
            pos[-case["pad"]:] = -1
        st["positions"] = _dev(pos.astype(np.int32))
        j = np.arange(case["R"] // 2, dtype=np.float64)
        st["inv_freq"] = _dev(case["base"] ** (-2.0 * j / case["R"]))
        st["q_weight"] = st["k_weight"] = None
        if case["norm"]:
            st["q_weight"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)
            st["k_weight"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)
        st["eps"] = 1e-6 if case["norm"] else None
        return st
    if case["op"] == "logprobs":
        T, V = case["T"], case["V"]
        dt = DTYPES[case["dtype"]]
        x = torch.empty((T, V + case["pad"]), dtype=dt, device=DEV)
        peak = 4.0 + 8.0 * torch.rand(T, generator=g, device=DEV)
        for t in range(0, T, 128):  # in parts, for the memory that fp32 takes
            part = 2.2 * torch.randn((min(128, T - t), V + case["pad"]), generator=g, device=DEV)
            if case["masked"]:
                gone = torch.rand(part.shape, generator=g, device=DEV) < case["masked"]
                part.masked_fill_(gone, -math.inf)
            x[t:t + 128] = part
        tokens = torch.randint(0, V, (T,), generator=g, device=DEV)
        likely = torch.rand(T, generator=g, device=DEV) < 0.8  # most text is what the model expects, all of it allowed
        other = 2.2 * torch.randn(T, generator=g, device=DEV)
        x[torch.arange(T, device=DEV), tokens] = torch.where(likely, 6.0 + peak, other).to(dt)
        st["logits"] = x[:, :V]
        st["tokens"] = tokens.int()
        return st
    P, lens = case["page"], _lens(case)
    have = _pages_of(lens, P)
    if case["op"] == "fork":
        C = case["B"] * case["n"]
        n_pages = int(have.sum()) + C + 5
        ids = rs.permutation(n_pages).astype(np.int32)
        st.update(_planes(g, case, n_pages))
        taken = int(have.sum())
        st.update(lens=_dev(lens.astype(np.int32)), table=_dev(_table(have, ids, int(have.max()) + 2)), free=_dev(ids),
                  head=torch.full((1,), taken, dtype=torch.int32, device=DEV), refs=torch.zeros(n_pages, dtype=torch.int32, device=DEV),
                  parents=_dev(np.repeat(np.arange(case["B"]), case["n"]).astype(np.int32)),
                  new=torch.ones(C, dtype=torch.int32, device=DEV))
        return st
    ids = rs.permutation(case["pages"]).astype(np.int32)
    table = _table(have, ids, int(have.max()) + 1)
    if case["B"] > 2:  # one request shares another's full pages
        share = min(int(lens[0]), int(lens[1])) // P
        table[1, :share] = table[0, :share]
    st.update(_planes(g, case, case["pages"]))
    st.update(lens=_dev(lens.astype(np.int32)), table=_dev(table))
    return st


# ---- the plain forms ----

def _plain_turn(x, cos, sin, layout):
    R = 2 * cos.shape[-1]
    head, rest = x[..., :R], x[..., R:]
    if layout == "halves":
        a, b = head[..., :R // 2], head[..., R // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = head[..., 0::2], head[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _plain_rope(st):
    c, pos = st["case"], st["positions"]
    angle = pos.double()[:, None, None] * st["inv_freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()

    def one(x, weight, dtype):
        x = x.float()
        if c["norm"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * weight
        x = _plain_turn(x, cos, sin, c["layout"])
        return torch.where((pos >= 0)[:, None, None], x, 0.0).to(DTYPES[dtype])

    return {"q": one(st["q"], st["q_weight"], c["q_dtype"]), "k": one(st["k"], st["k_weight"], c["k_dtype"])}


def _plain_logprobs(st):
    x, n = st["logits"].float(), st["case"]["top"]
    m = x.amax(-1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    z = e.sum(-1, keepdim=True)
    log_z = torch.log(z)
    out = {"logprobs": (d.gather(1, st["tokens"].long()[:, None]) - log_z)[:, 0],
           "entropy": (log_z - torch.where(e > 0, e * d, 0.0).sum(-1, keepdim=True) / z)[:, 0]}
    if n:
        # value and index in one whole number, so that equal values go to the lowest index
        u = x.view(torch.int32).long()
        key = torch.where(u < 0, -(u & 0x7fffffff), u) * (1 << 20) - torch.arange(x.shape[1], device=DEV)
        ids = torch.topk(key, n, dim=-1, sorted=True).indices
        out["top_ids"] = ids.int()
        out["top_logprobs"] = d.gather(1, ids) - log_z
    return out


def _plain_copy(st, src, dst, tokens):
    """Every page of every layer after the copies: where each page's contents come from, and up to which token."""
    n_pages, S = st["kq"].shape[1], st["case"]["block"]
    real = (src >= 0) & (dst >= 0)
    at = torch.where(real, dst, n_pages).long()
    origin = torch.arange(n_pages + 1, device=DEV).scatter(0, at, src.clamp(min=0).long())[:n_pages]
    upto = torch.zeros(n_pages + 1, dtype=torch.int64, device=DEV).scatter(0, at, tokens.long())[:n_pages]
    P, blocks = st["kq"].shape[3], st["kd"].shape[3]
    moved = (torch.arange(P, device=DEV) < upto[:, None])[None, :, None, :, None]
    scales = (torch.arange(blocks, device=DEV) * S < upto[:, None])[None, :, None, :]
    return {"kq": torch.where(moved, st["kq"][:, origin], st["kq"]), "vq": torch.where(moved, st["vq"][:, origin], st["vq"]),
            "kd": torch.where(scales, st["kd"][:, origin], st["kd"]), "vd": torch.where(scales, st["vd"][:, origin], st["vd"])}


def _plain_fork(st):
    P, free, head, refs = st["case"]["page"], st["free"], st["head"].long(), st["refs"].long()
    n_pages, n_free = refs.shape[0], free.shape[0]
    parent = st["parents"].long()
    lens = st["lens"].long()[parent]
    col = torch.arange(st["table"].shape[1], device=DEV)
    mine = col < ((lens + P - 1) // P)[:, None]
    table = torch.where(mine, st["table"][parent], -1)
    refs = refs + torch.zeros(n_pages + 1, dtype=torch.int64, device=DEV).scatter_add(
        0, torch.where(mine, table, n_pages).flatten().long(), torch.ones(table.numel(), dtype=torch.int64, device=DEV))[:n_pages]
    # copy on write: those that go on inside a page that others hold too, in order, as long as it is shared
    part = (lens % P > 0) & (st["new"] > 0)
    last = (lens // P).clamp(max=col.shape[0] - 1)
    page = torch.where(part, table.gather(1, last[:, None])[:, 0], 0).long()
    i = torch.arange(parent.shape[0], device=DEV)
    before = ((page[None, :] == page[:, None]) & part[None, :] & (i[None, :] < i[:, None])).sum(-1)
    need = part & (before < refs[page])
    at = head + torch.cumsum(need, 0) - need.long()
    fits = need & (at < n_free)
    given = free[at.clamp(max=n_free - 1)]
    src, dst = torch.where(fits, page, -1), torch.where(fits, given, -1)
    tokens = torch.where(fits, lens % P, 0)
    table = torch.where(fits[:, None] & (col == last[:, None]), given[:, None], table)
    refs = refs - torch.zeros_like(refs).scatter_add(0, page, fits.long())
    head_taken = head + fits.sum()
    out = _plain_copy(st, src, dst, tokens)
    # release of every forked row: a page whose last holder goes returns to the list, at its last entry's turn
    entry = torch.arange(table.numel(), device=DEV).view(table.shape)
    at = torch.where(mine, table, n_pages).flatten().long()
    let_go = torch.zeros(n_pages + 1, dtype=torch.int64, device=DEV).scatter_add(0, at, torch.ones_like(at))[:n_pages]
    final = torch.full((n_pages + 1,), -1, device=DEV).scatter_reduce(0, at, entry.flatten(), "amax")
    goes = mine.flatten() & (final[at] == entry.flatten()) & (torch.cat([refs - let_go, refs.new_zeros(1)])[at] < 0)
    count = goes.sum()
    place = torch.where(goes, head_taken - count + torch.cumsum(goes, 0) - 1, n_free)
    free = torch.cat([free, free.new_zeros(1)]).scatter(0, place, table.flatten().int())[:n_free]
    out.update(lens=lens.int(), table=table.int(), src=src.int(), dst=dst.int(), tokens=tokens.int(), refs=(refs - let_go).clamp(min=0).int(),
               free=free, head_taken=head_taken.int(), head=(head_taken - count).int())
    return out


def _plain_compact(st):
    P, n_pages = st["case"]["page"], st["case"]["pages"]
    lens = st["lens"].long()
    mine = torch.arange(st["table"].shape[1], device=DEV) < ((lens + P - 1) // P)[:, None]
    at = torch.where(mine, st["table"], n_pages).long()
    held = torch.zeros(n_pages + 1, dtype=torch.int64, device=DEV).scatter_add(0, at.flatten(), torch.ones_like(at).flatten())[:n_pages]
    used = held > 0
    total = used.sum()
    page = torch.arange(n_pages, device=DEV)
    before = torch.cumsum(used, 0) - used.long()
    moves, most = n_pages // 2, n_pages // 2
    # the highest page in use goes to the lowest one that is not, and so on
    leaves, hole = used & (page >= total), ~used & (page < total)
    src = torch.full((moves + 1,), -1, device=DEV).scatter(0, torch.where(leaves, total - 1 - before, most), page)
    dst = torch.full((moves + 1,), -1, device=DEV).scatter(0, torch.where(hole, page - before, most), page)
    src, dst = src[:moves], dst[:moves]
    number = torch.where(leaves, dst[(total - 1 - before).clamp(0, moves - 1)], page)
    table = torch.where(mine, number[at.clamp(max=n_pages - 1)], -1)
    refs = torch.zeros(n_pages + 1, dtype=torch.int64, device=DEV).scatter(0, torch.where(used, number, n_pages), (held - 1).clamp(min=0))[:n_pages]
    out = _plain_copy(st, src, dst, torch.where(src >= 0, P, 0))
    out.update(table=table.int(), refs=refs.int(), free=page.int(), src=src.int(), dst=dst.int(), head=total.int().view(1))
    return out


# ---- one pass ----

def run(state):
    c = state["case"]
    if not own:
        return {"rope": _plain_rope, "logprobs": _plain_logprobs, "fork": _plain_fork, "compact": _plain_compact}[c["op"]](state)
    import block_quantized_decode_quantize_gb300 as memra
    if c["op"] == "rope":
        q, k = memra.memra_qk_norm_rope(state["q"], state["k"], state["positions"], state["inv_freq"], q_weight=state["q_weight"],
                                        k_weight=state["k_weight"], eps=state["eps"], layout=c["layout"],
                                        q_dtype=DTYPES[c["q_dtype"]], k_dtype=DTYPES[c["k_dtype"]])
        return {"q": q, "k": k}
    if c["op"] == "logprobs":
        logprobs, entropy, ids, top = memra.memra_token_logprobs(state["logits"], state["tokens"], top_n=c["top"])
        out = {"logprobs": logprobs, "entropy": entropy}
        if c["top"]:
            out.update(top_ids=ids, top_logprobs=top)
        return out
    planes = {x: state[x] for x in ("kq", "kd", "vq", "vd")}
    if c["op"] == "fork":
        lens, table = memra.memra_kv_fork(state["parents"], state["lens"], state["table"], c["page"], state["refs"])
        _, src, dst, tokens, taken = memra.memra_kv_unshare(lens, state["new"], c["page"], state["refs"], state["free"], table,
                                                            free_head=state["head"])
        memra.memra_kv_copy_pages(src, dst, state["caches"], tokens=tokens)
        _, head = memra.memra_kv_release(lens, c["page"], table, state["refs"], state["free"], taken)
        return dict(planes, lens=lens, table=table, src=src, dst=dst, tokens=tokens, refs=state["refs"], free=state["free"],
                    head_taken=taken, head=head)
    table, refs, free, src, dst, head = memra.memra_kv_compact(state["lens"], state["table"], c["page"], c["pages"])
    memra.memra_kv_copy_pages(src, dst, state["caches"])
    return dict(planes, table=table, refs=refs, free=free, src=src, dst=dst, head=head)


# ---- the definitions in 64 bits ----

def _exact_rope(st):
    c = st["case"]
    pos = st["positions"].cpu().numpy().astype(np.float64)
    t = torch.from_numpy(np.outer(pos, st["inv_freq"].cpu().numpy())).to(DEV)
    turn = torch.polar(torch.ones_like(t), t)[:, None, :]
    out = {}
    for name, x, w in (("q", st["q"], st["q_weight"]), ("k", st["k"], st["k_weight"])):
        x = x.double()
        if c["norm"]:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + st["eps"]) * w.double()
        R = c["R"]
        pair = torch.complex(x[..., :R // 2], x[..., R // 2:R]) if c["layout"] == "halves" else \
            torch.view_as_complex(x[..., :R].unflatten(-1, (R // 2, 2)).contiguous())
        pair = pair * turn
        x = x.clone()
        if c["layout"] == "halves":
            x[..., :R // 2], x[..., R // 2:R] = pair.real, pair.imag
        else:
            x[..., :R] = torch.view_as_real(pair).flatten(-2)
        x[st["positions"] < 0] = 0.0
        out[name] = x
    return out


def _exact_logprobs(st):
    T, n = st["logits"].shape[0], st["case"]["top"]
    parts = []
    for t in range(0, T, 64):
        x = st["logits"][t:t + 64].double()
        lse = torch.logsumexp(x, -1)
        p = torch.exp(x - lse[:, None])
        h = -torch.where(p > 0, p * (x - lse[:, None]), 0.0).sum(-1)
        lp = x.gather(1, st["tokens"][t:t + 64].long()[:, None])[:, 0] - lse
        top = torch.sort(x, dim=-1, descending=True).values[:, :n] - lse[:, None]
        parts.append((lp, h, top))
    out = {"logprobs": torch.cat([p[0] for p in parts]), "entropy": torch.cat([p[1] for p in parts])}
    if n:
        out.update(top_ids=None, top_logprobs=torch.cat([p[2] for p in parts]))
    return out


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # whole numbers, and contents that are copied bit for bit
    st = prepare(case, seed)
    return _exact_rope(st) if case["op"] == "rope" else _exact_logprobs(st)
