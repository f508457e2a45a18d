"""The cache, attention and plan where they reach their limits: many units to a CTA, long units,
sizes far from 1, overlapping arguments, page numbers out of range.  Against float64 or the
stated integers."""
import numpy as np
import pytest
import torch

from test_gpu_kv_route import attention_case, check_attention, dev, ref_append, ref_plan

pytestmark = pytest.mark.gpu
i32 = torch.int32


@pytest.fixture(scope="module")
def mem():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_decode_quantize_gb300 as m
    from block_quantized_decode_quantize_gb300 import build
    build.build()
    m.lib()
    return m


# ---------------------------------------------------------------------------
# Attention: units of which a CTA takes many, and of many keys.
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows", [64, 128])
def test_attention_wide_many_units_to_a_cta(mem, rows):
    """Several units to a CTA, one or two tiles each: every warp reads some ten segments that one
    of its lanes wrote."""
    B, Hkv, G = 30, 16, 8
    n = rows // G
    rs = np.random.RandomState(61)
    c = attention_case(rs, rs.randint(1, 300, B), [n] * B, G * Hkv, Hkv, 64, 32, 16, "bf16")
    o, l = check_attention(mem, *c)
    for _ in range(5):
        o2, l2 = mem.memra_kv_attention_q8(c[0], *[dev(x) for x in c[1:5]], *[dev(x, i32) for x in c[5:]])
        assert torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("new,G,Hkv", [([8, 0, 0, 5, 2], 16, 8), ([5, 6, 5, 6], 8, 8), ([1, 1, 1, 1, 1], 40, 8), ([1] * 4, 48, 6),
                                       ([9, 1, 1, 1, 30], 8, 16)])
def test_attention_wide_units_of_few_rows(mem, new, G, Hkv):
    """Units whose rows leave some of the softmax warps without any: those must not arrive for a
    tile while the others still make the weights of the one before.  Repeated with a cold cache."""
    rs = np.random.RandomState(62)
    lens = [1540, 2438, 2064, 998, 1637][:len(new)]
    c = attention_case(rs, lens, new, G * Hkv, Hkv, 64, 16, 16, "bf16")
    o, l = check_attention(mem, *c)
    t = [dev(x) for x in c[1:5]] + [dev(x, i32) for x in c[5:]]
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    ws = torch.zeros(mem.KV_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    for i in range(60):
        if i % 2:
            flush.fill_(i)
        o2, l2 = mem.memra_kv_attention_q8(c[0], *t, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(l, l2), i


LONG = [
    # dtype, G, n, D
    ("bf16", 5, 1, 128), ("bf16", 8, 1, 64), ("bf16", 8, 1, 256), ("bf16", 8, 2, 128), ("bf16", 8, 4, 64),
    ("fp32", 5, 1, 128), ("fp32", 8, 1, 64), ("fp32", 8, 1, 256), ("fp32", 8, 2, 128), ("fp32", 8, 4, 64),
]


def long_unit(mem, dtype, G, n, D, L, seed=0):
    """B requests of L tokens whose tables name one page of 1024 tokens over and over, so that
    the 64-bit result needs that page's keys alone; V of one sign.  Units are as many as the
    GPU has CTAs, so a CTA takes most of one by itself. Returns out, what it should be, lse and what
    that should be."""
    B, Hkv, P = 40, 8, 1024
    Hq = G * Hkv
    g = torch.Generator(device="cuda").manual_seed(100 * D + 10 * G + n + seed)
    kq = torch.randint(-127, 128, (1, Hkv, P, D), generator=g, device="cuda", dtype=torch.int8)
    vq = torch.randint(64, 128, (1, Hkv, P, D), generator=g, device="cuda", dtype=torch.int8)
    kd = 0.01 * (1 + torch.rand(1, Hkv, P // 16, generator=g, device="cuda"))
    vd = 0.01 * (1 + torch.rand(1, Hkv, P // 16, generator=g, device="cuda"))
    # scores of a few tenths: sum |q| |k| scale below 1/2, so that 2^-18 of it is 2^-19
    q = (torch.rand(B * n, Hq, D, generator=g, device="cuda") - 0.5).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    scale = 2.0 / D
    table = torch.zeros(B, L // P, dtype=i32, device="cuda")
    lens = torch.full((B,), L, dtype=i32, device="cuda")
    cu = torch.arange(B + 1, dtype=i32, device="cuda") * n
    ws = torch.zeros(mem.KV_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    out, lse = mem.memra_kv_attention_q8(q, kq, kd, vq, vd, table, lens, cu, scale=scale, workspace=ws)
    k = kq[0].double() * kd[0].double().repeat_interleave(16, 1)[..., None]
    v = vq[0].double() * vd[0].double().repeat_interleave(16, 1)[..., None]
    x = torch.einsum("bihgd,hjd->bihgj", q.double().view(B, n, Hkv, G, D), k) * scale
    seen = L - n + 1 + torch.arange(n, device="cuda")                    # keys that query i sees
    j = torch.arange(P, device="cuda")
    count = (seen // P)[:, None] + (j[None, :] < (seen % P)[:, None])    # how often each of the page's
    p = torch.exp(x) * count[None, :, None, None, :]
    l = p.sum(-1)
    want = torch.einsum("bihgj,hjd->bihgd", p, v) / l[..., None]
    return out.double(), want.reshape(B * n, Hq, D), lse.double(), torch.log(l).reshape(B * n, Hq)


@pytest.mark.parametrize("dtype,G,n,D", LONG)
def test_attention_sums_do_not_drift(mem, dtype, G, n, D):
    """A sum over 131072 keys of V of one sign.  Scores are off by at most 2^-18 of their terms'
    sum (below 1/2), weights by 2^-22 (fp32) or 2^-12 (bf16, and the output by 2^-8 more), all
    to either side.  The running sums of a warp take 1024 steps, each rounded to nearest: a walk
    of steps of at most 2^-24, 2^-23 / sqrt(12) * sqrt(1024 / 3) = 6.4e-7 after the last, and six
    times that are 3.8e-6; the strip's own products, cut off, add 2 * 2^-23 at most.  So fp32
    elements are within 2^-17.  A sum that cuts off at every step loses 2 * 1024 half steps on
    average: 3e-5 and more.  In bf16 that hides below the rounding of the output; but the last
    query sees the same page 128 times or once, so that the same number is rounded in both
    cases, and the mean of the difference is that of the sums."""
    out, want, lse, wlse = long_unit(mem, dtype, G, n, D, 131072)
    err = (out - want) / want
    assert float(err.abs().max()) < (2.0 ** -17 if dtype == "fp32" else 2.0 ** -8 + 2.0 ** -10)
    assert float((lse - wlse).abs().max()) < 2.0 ** -17 + 4e-7 * float(wlse.abs().max())
    once = long_unit(mem, dtype, G, n, D, 1024)[0]
    assert abs(float(((out - once) / want)[n - 1::n].mean())) < 2.0 ** -17


@pytest.mark.parametrize("G,D", [(8, 128), (16, 128), (8, 64), (16, 64)])
def test_attention_wide_sums_do_not_drift(mem, G, D):
    """The many-row kernel's sums leave the tensor cores every 65536 keys: 256 tiles of a group,
    8 products each (4 where a lane has half of the keys), of which each may cut 2^-22 off a sum
    that is half of its last value on average: 2048 * 2^-23 = 2^-12 at most, and 2^-11 with the
    estimate's own scatter (about a hundred of its results round elsewhere, a tenth of that).
    Over 2^20 keys without an end they would lose 1.4e-3 (64 rows) and 2.9e-3 (128)."""
    out, want, lse, wlse = long_unit(mem, "bf16", G, 8, D, 1 << 20)
    err = (out - want) / want
    assert float(err.abs().max()) < 2.0 ** -8 + 2.0 ** -10
    assert float((lse - wlse).abs().max()) < 2.0 ** -17 + 4e-7 * float(wlse.abs().max())
    once = long_unit(mem, "bf16", G, 8, D, 1024)[0]
    assert abs(float(((out - once) / want)[7::8].mean())) < 2.0 ** -11


@pytest.mark.parametrize("window", [0, 100000])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 16, 2), (128, 16, 1)])
def test_attention_wide_ranges_of_several_runs(mem, window, D, Hq, Hkv):
    """Ranges that are cut into runs, whole units and parts of them, some of which see nothing in
    their first or last run: requests of up to 150000 keys, as the 8-row kernel has them one query
    at a time."""
    rs = np.random.RandomState(71)
    lens, new = [150000, 70000, 16500, 140000, 5, 90000], [40, 9, 16, 8, 8, 25]
    P = 1024
    n_pages = 80
    table = np.array([[rs.randint(0, n_pages) for _ in range(147)] for _ in lens])
    kq, vq = (torch.randint(-127, 128, (n_pages, Hkv, P, D), generator=torch.Generator().manual_seed(i), dtype=torch.int8).cuda() for i in (1, 2))
    kd, vd = (0.01 * torch.rand(n_pages, Hkv, P // 32, generator=torch.Generator().manual_seed(i)).cuda() for i in (3, 4))
    q = torch.randn(sum(new), Hq, D, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    ws = torch.zeros(mem.KV_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    cu = np.concatenate([[0], np.cumsum(new)])
    reps = 3                                               # enough units for each CTA to have whole ones too
    many = [np.concatenate([np.asarray(x)] * reps) for x in (table, lens)]
    cus = np.concatenate([[0], np.cumsum(new * reps)])
    out, lse = mem.memra_kv_attention_q8(q.repeat(reps, 1, 1), kq, kd, vq, vd, dev(many[0], i32), dev(many[1], i32), dev(cus, i32),
                                         scale=D ** -0.5, window=window, workspace=ws)
    # one query at a time: the lengths up to it, of rows of their own
    one = dev(np.concatenate([np.arange(L - n + 1, L + 1) for L, n in zip(lens, new)]), i32)
    rows = dev(np.repeat(table, new, axis=0), i32)
    want, wlse = mem.memra_kv_attention_q8(q.float(), kq, kd, vq, vd, rows, one, dev(np.arange(len(q) + 1), i32), scale=D ** -0.5,
                                           window=window, workspace=ws)
    assert q.shape[0] == cu[-1]
    for r in range(reps):
        o, l = out[r * len(q):(r + 1) * len(q)].double(), lse[r * len(q):(r + 1) * len(q)]
        assert torch.equal(torch.isneginf(l), torch.isneginf(wlse))
        live = ~torch.isneginf(wlse)
        # scores: 2^-18 of sum |q| |k| scale, below 127 * 0.01 * 128 * 0.8 * 128 ** -0.5 = 12 here: 4.4e-5 either
        # side; values of at most 1.27, off by 2^-12, by twice the scores' error and by what sums lose in
        # a run (2^-12), rounded at 2^-8
        assert float((l - wlse)[live].abs().max()) < 2 * 4.4e-5 + 1e-5
        assert float((o - want.double()).abs().max()) < 1.27 * (2.0 ** -11 + 4 * 4.4e-5) + 2.0 ** -8 * float(want.abs().max())


@pytest.mark.parametrize("dtype,G,n,D", [("bf16", 1, 1, 64), ("bf16", 5, 1, 128), ("bf16", 8, 1, 256), ("bf16", 8, 2, 128),
                                         ("bf16", 8, 4, 64), ("bf16", 16, 16, 128), ("fp32", 8, 1, 128)])
def test_attention_beside_a_heavy_key_of_code_zero(mem, dtype, G, n, D):
    """One key takes nearly all of the weight and has code 0 in every dim of V: the result is what
    the others leave, to their own accuracy.  (The tolerance is that of check_attention with the
    grid's end and without anything for the heavy key's scale.)"""
    q, kq, kd, vq, vd, table, lens, cu = attention_case(np.random.RandomState(35), [300, 90], [n, n], 4 * G, 4, D, 32, 16, dtype)
    for b in range(2):
        page, off = int(table[b, 0]), 7
        vq[page, :, off] = 0
        k = kq[page, :, off].astype(np.float64) * kd[page, :, off // 16, None]
        heavy = 16.0 * D ** 0.5 * k / np.square(k).sum(1, keepdims=True)     # its score: 16
        q[n * b:n * b + n] = torch.from_numpy(np.repeat(heavy, G, axis=0)).to(q.dtype).cuda()
    check_attention(mem, q, kq, kd, vq, vd, table, lens, cu, wide_scales=True)


@pytest.mark.parametrize("n,dtype,D", [(1, "bf16", 128), (1, "fp32", 64), (2, "fp32", 128), (1, "fp32", 256), (60, "bf16", 64)])
@pytest.mark.parametrize("size", [1e-33, 1e-37, 1e-39, 1e-44])
def test_attention_next_to_no_values(mem, n, dtype, D, size):
    """Scales of V so small that 2^8 over them is no fp32 number, alone and before blocks of
    usual ones: nothing infinite, and no trace in the rows of usual ones."""
    q, kq, kd, vq, vd, table, lens, cu = attention_case(np.random.RandomState(31), [700, 90], [n, n], 16, 4, D, 32, 16, dtype)
    least = np.where(np.isfinite(vd), vd * np.float32(size), vd).astype(np.float32)
    mixed = vd.copy()
    mixed[table[0, :9]] = least[table[0, :9]]
    for plane in (least, mixed):
        check_attention(mem, q, kq, kd, vq, plane, table, lens, cu, wide_scales=True, code_unit=n == 1 and dtype == "bf16")


@pytest.mark.parametrize("n,dtype,D", [(1, "bf16", 128), (1, "fp32", 64), (2, "fp32", 128), (1, "bf16", 256)])
@pytest.mark.parametrize("power", [-100, 80])
def test_attention_of_values_scaled_by_a_power_of_two(mem, n, dtype, D, power):
    """Scales of V times a power of two: the result times it.  Factors of parts far below a row's
    largest may be subnormal then (2^-149 of rounding, of up to 2^15 times as much, next to results
    of 2^-100), which can turn a last bit: to one part in 2^23 of the row's largest."""
    c = attention_case(np.random.RandomState(33), [700, 90], [n, n], 16, 4, D, 32, 16, dtype)
    t = [c[0]] + [dev(x) for x in c[1:5]] + [dev(x, i32) for x in c[5:]]
    o, l = mem.memra_kv_attention_q8(*t)
    t[4] = t[4] * 2.0 ** power
    o2, l2 = mem.memra_kv_attention_q8(*t)
    most = o.double().abs().amax(-1, keepdim=True)
    assert bool(((o2.double() * 2.0 ** -power - o.double()).abs() <= 2.0 ** -23 * most).all()) and torch.equal(l, l2)


# ---------------------------------------------------------------------------
# The write: a block whose scale is negative.
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("size", [1e-4, 1.0, 50.0])
def test_append_to_a_block_of_negative_scale(mem, dtype, size):
    """Attention takes scales of either sign; a token written after such a block's own must
    leave the older ones what they stand for: to within half a step of the scale."""
    rs = np.random.RandomState(41)
    P, S, Hkv, D = 32, 16, 2, 64
    kq = rs.randint(-127, 128, (2, Hkv, P, D)).astype(np.int8)
    kd = (-0.01 * (1 + rs.rand(2, Hkv, P // S))).astype(np.float32)
    c = [dev(kq), dev(kd), dev(kq), dev(-kd)]
    x = (size * torch.randn(3, Hkv, D, generator=torch.Generator().manual_seed(2))).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    mem.memra_kv_append_q8(x, x, dev(np.arange(37, 40), i32), *c)
    k, v = mem.memra_kv_read_q8(dev(np.arange(32, 40), i32), *c, dtype=torch.float32)
    step = np.maximum(-kd[1, :, 0], x.float().abs().amax(dim=(0, 2)).cpu().numpy() / 127)
    older = kq[1, :, :5].astype(np.float64) * kd[1, :, :1, None]          # [Hkv, 5, D]
    for got, sign in ((k, 1.0), (v, -1.0)):
        got = got.double().cpu().numpy()
        tol = (0.5 + 1e-4) * step[None, :, None]
        assert (np.abs(got[:5] - sign * older.transpose(1, 0, 2)) <= tol).all()
        assert (np.abs(got[5:] - x.double().cpu().numpy()) <= tol).all()


@pytest.mark.parametrize("S", [1, 4, 16])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_append_over_rejected_drafts(mem, S, dtype):
    """Verify steps that write five drafts and keep one to five of them: the stated rule call by
    call; kept tokens within half a step for each growth of their block's scale; and with S = 1
    what is kept is as if the drafts had never been."""
    rs = np.random.RandomState(43)
    P, Hkv, D, L = 16, 2, 64, 60
    g = torch.Generator().manual_seed(44)
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    kept = torch.randn(L, Hkv, D, generator=g).to(tdt)
    order = rs.permutation(6)
    slot = lambda p: order[p // P] * P + p % P
    zero = np.zeros((6, Hkv, P, D), np.int8), np.zeros((6, Hkv, P // S), np.float32)
    c = [dev(x) for x in zero + zero]
    want, step, at = zero, np.zeros((L, Hkv)), 0
    scale = np.zeros((6, Hkv, P // S), np.float32)
    while at < L - 5:
        n = int(rs.randint(1, 6))
        rows = torch.cat([kept[at:at + n], (3.0 * torch.randn(5 - n, Hkv, D, generator=g)).to(tdt)])
        slots = np.array([slot(p) for p in range(at, at + 5)])
        mem.memra_kv_append_q8(rows.cuda(), rows.cuda(), dev(slots, i32), *c)
        want = ref_append(rows.float().numpy(), slots, *want)
        assert all(np.array_equal(c[i].cpu().numpy(), want[i % 2]) for i in range(4))
        for p in range(at + n):                          # what this call may have moved a kept token by
            i = slot(p)
            d = want[1][i // P, :, i % P // S]
            grown = d > scale[i // P, :, i % P // S]
            step[p] = np.where(p >= at, d, step[p] + np.where(grown, d, 0))
        scale = want[1].copy()
        at += n
    k, v = mem.memra_kv_read_q8(dev([slot(p) for p in range(at)], i32), *c, dtype=torch.float32)
    off = (k.double().cpu() - kept[:at].double()).abs().numpy()
    assert torch.equal(k, v) and (off <= (0.5 + 1e-4) * step[:at, :, None]).all()
    if S == 1:
        clean = [dev(x) for x in zero + zero]
        mem.memra_kv_append_q8(kept[:at].cuda(), kept[:at].cuda(), dev([slot(p) for p in range(at)], i32), *clean)
        k2, _ = mem.memra_kv_read_q8(dev([slot(p) for p in range(at)], i32), *clean, dtype=torch.float32)
        assert torch.equal(k, k2)


# ---------------------------------------------------------------------------
# The plan: lengths in place, arrays that overlap.
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("B,max_new", [(5, 40), (40, 900), (1500, 9), (700, 60)])
@pytest.mark.parametrize("which", ["ctx", "new"])
@pytest.mark.parametrize("head_too", [False, True])
def test_plan_lengths_in_place(mem, B, max_new, which, head_too):
    """kv_lens may be the lengths themselves, with one CTA and with several (above 4096 rows)."""
    rs = np.random.RandomState(B + max_new)
    P, ctx, new = 16, rs.randint(0, 60, B), rs.randint(0, max_new + 1, B)
    have, after = -(-ctx // P), -(-(ctx + new) // P)
    ids = rs.permutation(int(after.sum()) + 9)
    table = np.full((B, int(after.max())), -1, np.int64)
    at = 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += int(have[b])
    free = ids[at:at + int(0.9 * (after - have).sum()) + 2]   # the last requests go without
    T = int(new.sum()) + 3
    want = ref_plan(ctx, new, P, free, table, T, 1)
    c, n, t, h = dev(ctx, i32), dev(new, i32), dev(table, i32), dev([1], i32)
    st = torch.zeros(1, dtype=i32, device="cuda")
    kv, cu, slots, pos, head = mem.memra_kv_plan(c, n, P, dev(free, i32), t, T, free_head=h, kv_lens=c if which == "ctx" else n,
                                                 free_head_out=h if head_too else None, dev_status=st)
    assert kv.data_ptr() == (c if which == "ctx" else n).data_ptr()
    for got, ref in ((kv, want[0]), (cu, want[1]), (slots, want[2]), (pos, want[3]), (t, want[4])):
        assert np.array_equal(got.cpu().numpy(), ref)
    assert int(head) == want[5] and int(st) == want[6] and int(h) == (want[5] if head_too else 1)


def test_plan_refuses_overlaps(mem):
    """Anything written that overlaps something else by a part, or by all where that is not
    allowed, is refused before a launch."""
    def call(**at):
        buf = torch.zeros(64, dtype=i32, device="cuda")
        v = dict(ctx_lens=buf[:3], new_lens=buf[4:7], free_pages=buf[8:16], block_table=buf[16:22].view(3, 2), free_head=buf[24:25],
                 kv_lens=buf[28:31], cu_q=buf[32:36], slots=buf[36:42], positions=buf[42:48], free_head_out=buf[50:51],
                 dev_status=buf[52:53])
        for name, i in at.items():
            v[name] = buf[i:i + v[name].numel()].view(v[name].shape)
        return mem.memra_kv_plan(v.pop("ctx_lens"), v.pop("new_lens"), 16, v.pop("free_pages"), v.pop("block_table"), 6, **v)

    call()
    call(kv_lens=0)
    call(kv_lens=4)
    call(free_head_out=24)
    for at in (dict(kv_lens=1), dict(kv_lens=2), dict(kv_lens=5), dict(kv_lens=14), dict(cu_q=28), dict(cu_q=0), dict(slots=42),
               dict(slots=3), dict(positions=20), dict(free_head_out=28), dict(free_head_out=2), dict(dev_status=24),
               dict(dev_status=50), dict(block_table=14), dict(block_table=20, free_head=25)):
        with pytest.raises(mem.MemraError) as e:
            call(**at)
        assert e.value.status == 1, at


def test_plan_page_numbers_out_of_range(mem):
    """A page number that no slot can name gives no slot: not a valid one of another page, as its
    low 32 bits would."""
    P = 16
    ctx, new = np.array([5, 0, 3, 0]), np.array([20, 33, 2, 16])
    table = np.full((4, 4), -1)
    table[0, 0], table[2, 0] = 7, -4                    # the third request's own page is none
    free = np.array([2 ** 28, 3, 2 ** 27, -1, 2 ** 27 - 2])
    t, st = dev(table, i32), torch.zeros(1, dtype=i32, device="cuda")
    kv, cu, slots, pos, head = mem.memra_kv_plan(dev(ctx, i32), dev(new, i32), P, dev(free, i32), t, 75, dev_status=st)
    want = ref_plan(ctx, new, P, free, table, 75)
    page = np.full(75, -1)
    for b in range(4):
        for i in range(new[b]):
            page[sum(new[:b]) + i] = want[4][b, (ctx[b] + i) // P]
    named = (page >= 0) & (page < (2 ** 31 - 1) // P)
    assert np.array_equal(slots.cpu().numpy(), np.where(named, page * P + want[3] % P, -1))
    assert int(st) == 1 and int(head) == 5
    for got, ref in ((kv, want[0]), (cu, want[1]), (pos, want[3]), (t, want[4])):
        assert np.array_equal(got.cpu().numpy(), ref)
