"""The paged 8-bit KV cache (plan, append, read-back, attention) and the routing to experts
against plain float64 / integer implementations."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mem():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_decode_quantize_gb300 as m
    from block_quantized_decode_quantize_gb300 import build
    build.build()
    m.lib()
    return m


def dev(x, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype).cuda()


# ---------------------------------------------------------------------------
# The page plan.
# ---------------------------------------------------------------------------

def ref_plan(ctx, new, P, free, table, T, head=0):
    """The plan, request by request."""
    table = table.copy()
    B, max_pages = table.shape
    kv, cu = np.zeros(B, np.int64), np.zeros(B + 1, np.int64)
    slots, pos = np.full(T, -1, np.int64), np.full(T, -1, np.int64)
    upto, asked, taken, bits = 0, max(head, 0), 0, 0
    for b in range(B):
        c, n = max(int(ctx[b]), 0), max(int(new[b]), 0)
        have, after = -(-c // P), -(-(c + n) // P)
        first = min(upto, T)
        upto += n
        cu[b + 1] = min(upto, T)
        ok = ctx[b] >= 0 and new[b] >= 0 and after <= max_pages and upto <= T
        if not ok:
            bits |= 1
        else:
            need = after - have
            asked += need
            if need and asked > len(free):
                ok = False
                bits |= 4
            else:
                table[b, have:after] = free[asked - need:asked]
                taken += need
        if ok:
            kv[b] = c + n
        for i in range(first, int(cu[b + 1])):
            p = c + i - first
            pos[i] = np.int64(p).astype(np.int32)    # int32, also where a refused request runs past it
            if ok:
                slots[i] = int(table[b, p // P]) * P + p % P
    return kv, cu, slots, pos, table, max(head, 0) + taken, bits


def check_plan(mem, ctx, new, P, free, table, T, head=0, in_place=False):
    want = ref_plan(ctx, new, P, free, table, T, head)
    i32 = torch.int32
    t = dev(table, i32)
    st = torch.zeros(1, dtype=i32, device="cuda")
    h = dev([head], i32)
    kv, cu, slots, pos, out = mem.memra_kv_plan(
        dev(ctx, i32), dev(new, i32), P, dev(free, i32), t, T, free_head=h,
        free_head_out=h if in_place else None, dev_status=st)
    for name, got, ref in (("kv_lens", kv, want[0]), ("cu_q", cu, want[1]), ("slots", slots, want[2]),
                           ("positions", pos, want[3]), ("table", t, want[4])):
        assert np.array_equal(got.cpu().numpy(), ref), name
    assert int(out) == want[5] and int(st) == want[6]
    if in_place:
        assert out.data_ptr() == h.data_ptr()


@pytest.mark.parametrize("B,P,max_ctx,max_new,pad", [
    (1, 16, 0, 1, 0), (1, 64, 700, 1, 0), (3, 16, 50, 40, 5), (33, 32, 300, 3, 1),
    (257, 64, 100, 1, 0), (1025, 16, 40, 7, 9), (2500, 32, 64, 2, 0), (40, 16, 90, 900, 77),
    (1500, 16, 33, 9, 3), (7, 1024, 5000, 3000, 2)])
@pytest.mark.parametrize("kind", ["fits", "short", "narrow", "cut"])
def test_plan(mem, B, P, max_ctx, max_new, pad, kind):
    rs = np.random.RandomState(B * 7 + P + max_new)
    ctx = rs.randint(0, max_ctx + 1, B)
    new = rs.randint(0, max_new + 1, B)
    have, after = -(-ctx // P), -(-(ctx + new) // P)
    need = int((after - have).sum())
    n_pages = int(after.sum()) + 8
    ids = rs.permutation(n_pages)
    max_pages = int(after.max()) + (1 if kind != "narrow" else 0)
    if kind == "narrow":
        max_pages = max(1, max_pages - 1)
        ctx = np.minimum(ctx, max_pages * P)
        have = -(-ctx // P)
    table = np.full((B, max_pages), -1, np.int64)
    at = 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += int(have[b])
    free = rs.permutation(n_pages)[: need + 3] if kind != "short" else rs.permutation(n_pages)[: 2 + need // 2]
    T = int(new.sum()) + pad
    if kind == "cut":
        T = max(0, int(0.7 * new.sum()))
    check_plan(mem, ctx, new, P, free, table, T, head=2 if kind != "fits" else 0, in_place=kind == "short")


def test_plan_edges(mem):
    # no request; no token; lengths below zero; an empty free list; no pages at all
    check_plan(mem, np.zeros(0, int), np.zeros(0, int), 16, np.arange(3), np.zeros((0, 4), int), 5)
    check_plan(mem, np.array([5, 0]), np.array([0, 0]), 16, np.arange(3), np.full((2, 4), -1), 0)
    check_plan(mem, np.array([-3, 4, 5, -1]), np.array([2, -2, 3, 0]), 16, np.arange(9), np.full((4, 4), 1), 8)
    check_plan(mem, np.array([16, 3]), np.array([1, 1]), 16, np.zeros(0, int), np.full((2, 4), 1), 2)
    check_plan(mem, np.array([0]), np.array([4]), 16, np.arange(4), np.zeros((1, 0), int), 4)
    check_plan(mem, np.array([2 ** 31 - 1]), np.array([2 ** 31 - 1]), 16, np.arange(4), np.zeros((1, 2), int), 4)
    check_plan(mem, np.array([0, 0]), np.array([16, 16]), 16, np.arange(4), np.full((2, 1), -1), 32, head=-5)


def test_plan_steps_in_place(mem):
    """A decode loop on the device: the head and the table advance in place, and every step
    equals the plan of the lengths so far."""
    P, B = 16, 5
    i32 = torch.int32
    ctx = np.array([0, 15, 16, 31, 7])
    free = np.random.RandomState(3).permutation(64)
    table = np.full((B, 8), -1)
    used = 0
    for b in range(B):
        n = -(-ctx[b] // P)
        table[b, :n] = free[used:used + n]
        used += n
    t, head = dev(table, i32), dev([used], i32)
    lens = dev(ctx, i32)
    ones = torch.ones(B, dtype=i32, device="cuda")
    for step in range(40):
        kv, cu, slots, pos, _ = mem.memra_kv_plan(lens, ones, P, dev(free, i32), t, B, free_head=head,
                                                  free_head_out=head)
        want = ref_plan(ctx, np.ones(B, int), P, free, table, B, used)
        table, used = want[4], want[5]
        ctx = ctx + 1
        assert np.array_equal(slots.cpu().numpy(), want[2]) and np.array_equal(t.cpu().numpy(), table)
        assert int(head) == used
        lens = kv


# ---------------------------------------------------------------------------
# The cache's write and read-back.
# ---------------------------------------------------------------------------

def away(x):
    t = np.trunc(x)
    return np.where(np.abs(x - t) == 0.5, t + np.sign(x), np.rint(x)).astype(np.float32)


def ref_append(x, slots, q, d):
    """One plane, run by run, in the stated fp32 operations."""
    q, d = q.copy(), d.copy()
    n_pages, Hkv, P, D = q.shape
    S = P // d.shape[2]
    t = 0
    while t < len(slots):
        if slots[t] < 0 or slots[t] >= n_pages * P:
            t += 1
            continue
        blk = slots[t] // S
        e = t
        while e < len(slots) and slots[e] >= 0 and slots[e] // S == blk:
            e += 1
        page, off = int(slots[t] // P), int(slots[t] % P)
        i, first = off // S, off % S
        run = x[t:e]
        amax = np.abs(run).max(axis=(0, 2)).astype(np.float32)
        old = d[page, :, i] if first else np.zeros(Hkv, np.float32)
        new = np.maximum(old, amax / np.float32(127.0)).astype(np.float32)
        for h in range(Hkv):
            if first and new[h] > old[h]:
                ratio = np.float32(old[h] / new[h])
                rows = q[page, h, i * S:i * S + first]
                q[page, h, i * S:i * S + first] = away(rows.astype(np.float32) * ratio).astype(np.int8)
            c = away(run[:, h] / new[h]) if new[h] else np.zeros_like(run[:, h])
            q[page, h, off:off + e - t] = np.clip(c, -127, 127).astype(np.int8)
            d[page, h, i] = new[h]
        t = e
    return q, d


def pool(rs, n_pages, Hkv, P, D, S):
    q = rs.randint(-127, 128, (n_pages, Hkv, P, D)).astype(np.int8)
    d = np.exp(rs.randn(n_pages, Hkv, P // S)).astype(np.float32) * 0.01
    return q, d


APPEND = [(1, 64, 16, 16, 1, "bf16"), (8, 128, 64, 16, 1, "fp32"), (2, 256, 32, 1, 9, "bf16"),
          (3, 64, 48, 4, 40, "fp32"), (4, 128, 64, 32, 100, "bf16"), (2, 128, 128, 128, 300, "fp32"),
          (1, 256, 16, 2, 77, "fp32"), (8, 128, 32, 16, 2000, "bf16"), (5, 64, 96, 24, 501, "bf16")]


@pytest.mark.parametrize("Hkv,D,P,S,T,dtype", APPEND)
@pytest.mark.parametrize("strided", [False, True])
def test_append_and_read(mem, Hkv, D, P, S, T, dtype, strided):
    rs = np.random.RandomState(T + D + S)
    # requests of uneven lengths whose tokens start at any offset of a page, and rows left out
    runs, left = [], T
    while left:
        n = min(left, int(rs.choice([1, 2, 5, S, S + 3, 2 * P + 1])))
        runs.append((int(rs.randint(0, P)), n))
        left -= n
    slots, page = [], 0
    for first, n in runs:
        pages = -(-(first + n) // P)
        slots += [page * P + first + i for i in range(n)]
        page += pages
    n_pages = page + 2
    slots = np.array(slots, np.int64)
    order = rs.permutation(n_pages)                     # pages need not rise
    slots = order[slots // P] * P + slots % P
    gone = rs.rand(T) < 0.1
    gone[np.concatenate([[True], np.diff(slots // S) != 0])] &= T > 20
    for t in range(1, T):                               # a hole ends a run: leave out its rest too
        if gone[t - 1] and slots[t] // S == slots[t - 1] // S:
            gone[t] = True
    slots = np.where(gone, -1, slots)
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    wide = torch.randn(T, (2 * Hkv + 3) * D, generator=torch.Generator().manual_seed(T)).to(tdt).cuda()
    wide[: max(1, T // 3)] *= 8.0                       # scales that grow and that do not
    if T > 4:
        wide[T // 2] = 0.0
    k = wide[:, D:(1 + Hkv) * D].view(T, Hkv, D)
    v = wide[:, (1 + Hkv) * D:(1 + 2 * Hkv) * D].view(T, Hkv, D)
    if not strided:
        k, v = k.contiguous(), v.contiguous()
    kq, kd = pool(rs, n_pages, Hkv, P, D, S)
    vq, vd = pool(rs, n_pages, Hkv, P, D, S)
    c = [dev(kq), dev(kd), dev(vq), dev(vd)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mem.memra_kv_append_q8(k, v, dev(slots, torch.int32), *c, dev_status=st)
    wkq, wkd = ref_append(k.float().cpu().numpy(), slots, kq, kd)
    wvq, wvd = ref_append(v.float().cpu().numpy(), slots, vq, vd)
    assert int(st) == 0
    for got, want in zip(c, (wkq, wkd, wvq, wvd)):
        assert np.array_equal(got.cpu().numpy(), want)
    # once more: nothing changes
    mem.memra_kv_append_q8(k, v, dev(slots, torch.int32), *c)
    for got, want in zip(c, (wkq, wkd, wvq, wvd)):
        assert np.array_equal(got.cpu().numpy(), want)
    some = np.concatenate([rs.randint(-1, n_pages * P, 50), slots])
    for rdt in (torch.float32, torch.bfloat16):
        rk, rv = mem.memra_kv_read_q8(dev(some, torch.int32), *c, dtype=rdt)
        for got, q, d in ((rk, wkq, wkd), (rv, wvq, wvd)):
            s = some.clip(0)
            val = q[s // P, :, s % P].astype(np.float32) * d[s // P, :, (s % P) // S][:, :, None]
            val = torch.from_numpy(np.where((some >= 0)[:, None, None], val, np.float32(0))).to(rdt)
            assert torch.equal(got.cpu(), val)


@pytest.mark.parametrize("quick", [True, False])
def test_a_single_row_may_have_any_strides(mem, quick, monkeypatch):
    """A view of one row or one head keeps whatever strides it was cut with."""
    if not quick:
        class Slow:
            append = attention = staticmethod(lambda *a: None)
        monkeypatch.setattr(mem, "_fast", Slow)
    rs = np.random.RandomState(3)
    x = torch.randn(1, 3, 64, generator=torch.Generator().manual_seed(3)).cuda()
    odd = torch.as_strided(x[:, 1:], (1, 1, 64), (197, 333, 1))
    c = [dev(t) for t in pool(rs, 2, 1, 16, 64, 16) + pool(rs, 2, 1, 16, 64, 16)]
    want = [t.clone() for t in c]
    slots = dev([16], torch.int32)
    mem.memra_kv_append_q8(x[:, 1:2].clone(), x[:, 1:2].clone(), slots, *want)
    mem.memra_kv_append_q8(odd, x[:, 1:2].clone(), slots, *c)
    assert all(torch.equal(a, b) for a, b in zip(c, want))
    table, lens, cu = dev([[1]], torch.int32), dev([1], torch.int32), dev([0, 1], torch.int32)
    ws = torch.zeros(mem.KV_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    got = [mem.memra_kv_attention_q8(q, *c, table, lens, cu, scale=0.125, workspace=ws) for q in (odd, odd.clone())]
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_append_refuses_slots_beyond_the_pool(mem):
    rs = np.random.RandomState(0)
    kq, kd = pool(rs, 2, 1, 16, 64, 16)
    c = [dev(kq), dev(kd), dev(kq), dev(kd)]
    x = torch.randn(3, 1, 64, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mem.memra_kv_append_q8(x, x, dev([32, 3, 2 ** 31 - 1], torch.int32), *c, dev_status=st)
    want = ref_append(x.cpu().numpy(), np.array([32, 3, 2 ** 31 - 1]), kq, kd)
    assert int(st) == 1
    assert np.array_equal(c[0].cpu().numpy(), want[0]) and np.array_equal(c[1].cpu().numpy(), want[1])
    st.zero_()
    k, v = mem.memra_kv_read_q8(dev([32, 3], torch.int32), *c, dtype=torch.float32, dev_status=st)
    assert int(st) == 1 and bool((k[0] == 0).all()) and bool((v[0] == 0).all()) and bool((k[1] != 0).any())


def test_append_small_values(mem):
    """Blocks of zeros (scale 0), of subnormal size, and of values whose quotients are halves."""
    P = S = 16
    x = torch.zeros(3 * P, 1, 64)
    x[P:2 * P] = torch.randn(P, 1, 64, generator=torch.Generator().manual_seed(1)) * 1e-39
    x[2 * P:] = (torch.arange(P * 64).view(P, 1, 64) % 255 - 127).float() / 2.0
    x[2 * P, 0, 0] = 127.0
    z = np.zeros((3, 1, P, 64), np.int8), np.zeros((3, 1, 1), np.float32)
    c = [dev(z[0]), dev(z[1]), dev(z[0]), dev(z[1])]
    mem.memra_kv_append_q8(x.cuda(), x.cuda(), torch.arange(3 * P, dtype=torch.int32, device="cuda"), *c)
    want = ref_append(x.numpy(), np.arange(3 * P), *z)
    for i in range(4):
        assert np.array_equal(c[i].cpu().numpy(), want[i % 2])


# ---------------------------------------------------------------------------
# Attention.
# ---------------------------------------------------------------------------

def ref_attention(q, kq, kd, vq, vd, table, lens, cu, scale, window):
    """float64, row by row; also the sum of |terms| that the tolerance is taken from."""
    T, Hq, D = q.shape
    n_pages, Hkv, P, _ = kq.shape
    S, G = P // kd.shape[2], Hq // Hkv
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    size, reach = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for b in range(len(lens)):
        L = int(min(lens[b], table.shape[1] * P))
        n = int(cu[b + 1] - cu[b])
        if L <= 0 or n == 0:
            continue
        j = np.arange(L)
        page = table[b, j // P]
        there = (page >= 0) & (page < n_pages)
        pg, off = np.where(there, page, 0), j % P
        k = kq[pg, :, off].astype(np.float64) * kd[pg, :, off // S][:, :, None].astype(np.float64)
        v = vq[pg, :, off].astype(np.float64) * vd[pg, :, off // S][:, :, None].astype(np.float64)
        for i in range(n):
            pos, t = L - n + i, int(cu[b]) + i
            seen = there & (j <= pos)
            if window:
                seen &= j > pos - window
            if not seen.any() or t >= T:
                continue
            for h in range(Hq):
                kk, vv = k[seen, h // G], v[seen, h // G]
                s = scale * kk @ q[t, h]
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                out[t, h] = (p / l) @ vv
                size[t, h] = (p / l) @ np.abs(vv)
                lse[t, h] = m + np.log(l)
                reach[t, h] = (abs(scale) * np.abs(kk) @ np.abs(q[t, h])).max()
    return out, lse, size, reach


def attention_case(rs, lens, new, Hq, Hkv, D, P, S, dtype, peak=1.5):
    have = -(-np.asarray(lens) // P)
    n_pages = int(have.sum()) + 3
    ids = rs.permutation(n_pages)
    table = np.full((len(lens), int(have.max(initial=0)) + 1), -1, np.int64)
    at = 0
    for b, h in enumerate(have):
        table[b, :h] = ids[at:at + h]
        at += int(h)
    kq, kd = pool(rs, n_pages, Hkv, P, D, S)
    vq, vd = pool(rs, n_pages, Hkv, P, D, S)
    live = np.zeros((n_pages, P // S), bool)
    for b, L in enumerate(lens):
        for j in range(0, L, S):
            live[table[b, j // P], (j % P) // S] = True
    for d in (kd, vd):                                   # what no token uses may hold anything
        d[:] = np.where(live[:, None, :], d, rs.choice([np.nan, np.inf, -np.inf], d.shape))
    T = int(np.sum(new))
    q = torch.from_numpy((peak * rs.randn(T, Hq, D)).astype(np.float32))
    q = (q.bfloat16() if dtype == "bf16" else q).cuda()
    cu = np.concatenate([[0], np.cumsum(new)])
    return q, kq, kd, vq, vd, table, np.asarray(lens), cu


def check_attention(mem, q, kq, kd, vq, vd, table, lens, cu, scale=None, window=0, status=0, workspace=None,
                    rows=None, wide_scales=False, code_unit=False):
    D = q.shape[2]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = torch.int32
    out, lse = mem.memra_kv_attention_q8(q, dev(kq), dev(kd), dev(vq), dev(vd), dev(table, i32), dev(lens, i32),
                                         dev(cu, i32), scale=scale, window=window, workspace=workspace,
                                         dev_status=st)
    sc = D ** -0.5 if scale is None else scale
    want, wlse, size, reach = ref_attention(q.double().cpu().numpy(), kq, kd, vq, vd, table, lens, cu, sc, window)
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    if rows is not None:
        got, glse, want, wlse, size, reach = (x[rows] for x in (got, glse, want, wlse, size, reach))
    assert int(st) == status
    none = np.isneginf(wlse)
    assert np.array_equal(none, np.isneginf(glse)) and np.array_equal(got[none], np.zeros_like(got[none]))
    # A score is an fp32 sum of D terms (or of two fp16 halves of q): off by at most 2^-18 of sum
    # |terms|; that moves a weight by as much, relatively.  Weights as fp16 pairs or singles:
    # 2^-11 for bf16 results (next to their own rounding, 2^-9), 2^-19 for fp32 ones.
    ds = 2.0 ** -18 * reach + 1e-6
    e = (2.0 ** -8 + 2.0 ** -10 if q.dtype == torch.bfloat16 else 2.0 ** -18) + 2 * ds
    # ... and on a grid that ends at 2^-33 of the largest weight and scale (a half of it a key)
    floor = np.zeros(got.shape[:2])
    if wide_scales:
        for b in range(len(lens)):
            live = table[b, :-(-min(int(lens[b]), table.shape[1] * kq.shape[2]) // kq.shape[2])]
            live = live[(live >= 0) & (live < len(vd))]
            most = np.nanmax(np.where(np.isfinite(vd[live]), vd[live], 0), axis=(0, 2)) if len(live) else np.zeros(vd.shape[1])
            floor[int(cu[b]):int(cu[b + 1])] = (2.0 ** -33 * 127 * lens[b] * np.repeat(most, q.shape[1] // len(most)))[None, :]
    if code_unit:
        # Codes enter the sum over v as c + 128, and 128 leaves it 16 keys at a time: two fp32 sums
        # (2^-23 each, cut off) of up to 128 of each weight times its scale, 2^-15 of theirs in all.
        ones = ref_attention(q.double().cpu().numpy(), kq, kd, np.ones_like(vq), np.abs(vd), table, lens, cu, sc, window)[0]
        floor = floor + 2.0 ** -15 * ones[..., 0]
    assert (np.abs(got - want) <= e[..., None] * size + floor[..., None] + 1e-7).all()
    fine = ~none
    assert (np.abs(glse - np.where(fine, wlse, 0))[fine] <= (ds + 2e-6 + 4e-7 * np.abs(np.where(fine, wlse, 0)))[fine]).all()
    return out, lse


ATTEND = [
    # lens, new, Hq, Hkv, D, P, S, dtype, window
    ([1], [1], 1, 1, 64, 16, 16, "bf16", 0),
    ([17], [1], 5, 1, 128, 16, 1, "fp32", 0),
    ([600], [1], 40, 8, 128, 64, 16, "bf16", 0),
    ([3001], [1], 8, 1, 128, 64, 64, "fp32", 0),
    ([5000], [1], 8, 2, 256, 32, 4, "bf16", 0),
    ([2048, 1, 333, 0, 64, 65, 1023], [1, 1, 1, 1, 1, 1, 0], 16, 4, 64, 64, 32, "bf16", 0),
    ([300, 20, 4, 900], [8, 8, 8, 3], 8, 4, 128, 16, 16, "fp32", 0),
    ([200, 16, 1000], [16, 16, 5], 32, 4, 128, 128, 16, "bf16", 0),
    ([700, 40], [7, 2], 14, 2, 256, 32, 8, "fp32", 50),
    ([700, 40, 3], [1, 9, 3], 7, 1, 64, 96, 24, "bf16", 1),
    ([130], [130], 4, 2, 128, 48, 16, "bf16", 33),
    ([500, 400], [200, 77], 16, 2, 64, 16, 2, "fp32", 0),
    ([260], [33], 48, 1, 128, 64, 16, "bf16", 0),
    ([9000, 8], [1, 1], 2, 2, 64, 1024, 1024, "bf16", 4000),
]


@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attention(mem, case):
    lens, new, Hq, Hkv, D, P, S, dtype, window = ATTEND[case]
    c = attention_case(np.random.RandomState(case), lens, new, Hq, Hkv, D, P, S, dtype)
    check_attention(mem, *c, window=window)


WIDE = [
    # bf16, more than 32 rows to a cached head, 4096 rows in all: the kernel on tcgen05
    # lens, new, Hq, Hkv, D, P, S, window
    ([500, 130, 17, 0, 300], [40, 30, 30, 20, 30], 32, 8, 128, 64, 16, 0),
    ([2000], [16], 256, 4, 128, 128, 64, 0),
    ([700, 40, 333], [22, 22, 20], 64, 16, 64, 16, 4, 0),
    ([260, 900], [33, 5], 128, 1, 128, 48, 16, 100),
    ([400], [130], 32, 2, 64, 1024, 1024, 33),
    ([60, 300, 1, 2], [100, 9, 8, 8], 48, 6, 128, 32, 1, 0),
    ([3000, 128, 256, 129], [8, 8, 8, 8], 128, 16, 128, 64, 16, 1),
    ([2500, 5, 77], [10, 60, 10], 64, 2, 64, 96, 24, 0),
]


@pytest.mark.parametrize("case", range(len(WIDE)))
def test_attention_wide(mem, case):
    lens, new, Hq, Hkv, D, P, S, window = WIDE[case]
    c = attention_case(np.random.RandomState(50 + case), lens, new, Hq, Hkv, D, P, S, "bf16")
    ws = torch.zeros(mem.KV_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    o, l = check_attention(mem, *c, window=window, workspace=ws)
    o2, l2 = check_attention(mem, *c, window=window, workspace=ws)
    assert torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 0.3])
def test_attention_wide_extremes(mem, scale):
    """Scales of either sign, peaked scores, zero blocks, scales of V far apart, pages out of
    range."""
    q, kq, kd, vq, vd, table, lens, cu = attention_case(np.random.RandomState(77), [900, 450], [40, 40], 64, 8, 128, 32,
                                                        16, "bf16", 4.0)
    rs = np.random.RandomState(78)
    vd *= np.where(rs.rand(*vd.shape) < 0.2, np.float32(1e6), np.float32(1.0)).astype(np.float32)
    vd[table[0, :4]] = 0.0
    kd[table[1, 1], 1, 0] = 0.0
    check_attention(mem, q, kq, kd, vq, vd, table, lens, cu, scale=scale, wide_scales=True)
    bad = table.copy()
    bad[0, 3], bad[0, 9], bad[1, 0] = -1, 10 ** 6, -5
    check_attention(mem, q, kq, kd, vq, vd, bad, lens, cu, scale=scale, status=1, wide_scales=True)


def test_attention_wide_strides_and_unowned_rows(mem):
    q, kq, kd, vq, vd, table, lens, cu = attention_case(np.random.RandomState(79), [400, 200], [60, 60], 40, 8, 128, 64,
                                                        16, "bf16")
    o, l = check_attention(mem, q, kq, kd, vq, vd, table, lens, cu)
    wide = torch.full((125, 44, 128), float("nan"), dtype=q.dtype, device="cuda")
    wide[:120, 3:43] = q
    i32 = torch.int32
    o2, l2 = mem.memra_kv_attention_q8(wide[:, 3:43], dev(kq), dev(kd), dev(vq), dev(vd), dev(table, i32),
                                       dev(lens, i32), dev(cu, i32))
    assert torch.equal(o2[:120], o) and torch.equal(l2[:120], l)
    assert bool((o2[120:] == 0).all()) and bool(torch.isneginf(l2[120:]).all())


def test_attention_wide_gives_up_and_recovers(mem):
    """Every wait of the many-row kernel is bounded: when one runs out the rows become NaN and
    status bit 2 is set, and with a zeroed workspace the next call is as before."""
    rs = np.random.RandomState(80)
    c = attention_case(rs, [900, 700, 64], [60, 60, 60], 32, 4, 128, 64, 16, "bf16")
    t = [c[0]] + [dev(x) for x in c[1:5]] + [dev(x, torch.int32) for x in c[5:]]
    ws = torch.zeros(mem.KV_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = mem.memra_kv_attention_q8(*t, scale=0.1, workspace=ws, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    try:
        mem.memra_debug_set_wait_test(1 << 16, 0)
        out, lse = mem.memra_kv_attention_q8(*t, scale=0.1, workspace=ws, dev_status=st)
        torch.cuda.synchronize()                      # the kernel returned
    finally:
        mem.memra_debug_set_wait_test()
    assert int(st) == 2
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
    ws.zero_()
    st.zero_()
    again = mem.memra_kv_attention_q8(*t, scale=0.1, workspace=ws, dev_status=st)
    assert int(st) == 0
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


@pytest.mark.parametrize("n,dtype", [(1, "bf16"), (1, "fp32"), (40, "bf16")])
def test_attention_negative_scales(mem, n, dtype):
    """A cache from elsewhere may have scales of either sign, or none above zero."""
    c = list(attention_case(np.random.RandomState(97), [300, 170], [n, n], 32, 4, 64, 32, 8, dtype))
    for change in (lambda d: -d, lambda d: np.where(np.arange(d.shape[2]) % 2, d, -d).astype(np.float32)):
        check_attention(mem, c[0], c[1], change(c[2]), c[3], change(c[4]), *c[5:], code_unit=dtype == "bf16")


@pytest.mark.parametrize("n", [2, 60])
def test_attention_rows_before_the_first_request(mem, n):
    c = attention_case(np.random.RandomState(98), [300, 170], [n, n], 32, 4, 64, 32, 8, "bf16")
    q = torch.cat([c[0][:5], c[0], c[0][:3]] if n > 2 else [c[0], c[0][:1], c[0], c[0][:3]])
    out, lse = check_attention(mem, q, *c[1:7], c[7] + 5, scale=0.1, code_unit=True)
    for part in (slice(0, 5), slice(2 * n + 5, None)):
        assert bool((out[part] == 0).all()) and bool(torch.isneginf(lse[part]).all())


def test_attention_many_requests(mem):
    """More requests than a CTA has threads, most of them without a token or a query."""
    rs = np.random.RandomState(81)
    lens = np.where(rs.rand(1300) < 0.9, 0, rs.randint(1, 60, 1300))
    new = np.where(rs.rand(1300) < 0.7, 0, 1)
    c = attention_case(rs, lens, new, 4, 2, 64, 16, 16, "fp32")
    check_attention(mem, *c)
    new = np.where(rs.rand(1300) < 0.9, 0, 40)
    c = attention_case(rs, lens, new, 4, 2, 64, 16, 16, "bf16")
    check_attention(mem, *c)


def test_attention_is_the_same_every_time_and_leaves_its_workspace_fit(mem):
    ws = torch.zeros(mem.KV_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    a = attention_case(np.random.RandomState(5), [4000, 37, 0, 999], [1, 1, 1, 2], 16, 4, 128, 64, 16, "fp32")
    b = attention_case(np.random.RandomState(6), [123, 70], [8, 8], 32, 4, 64, 16, 16, "bf16")
    first = [check_attention(mem, *x, workspace=ws) for x in (a, b)]
    for x, (o, l) in zip((a, b, a), (first[0], first[1], first[0])):
        o2, l2 = check_attention(mem, *x, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(l, l2)


def test_attention_rows_that_see_nothing(mem):
    """More queries than tokens, no tokens, rows that no request owns, requests without rows."""
    rs = np.random.RandomState(9)
    q, kq, kd, vq, vd, table, lens, cu = attention_case(rs, [3, 0, 20], [6, 2, 1], 4, 2, 64, 16, 16, "bf16")
    more = torch.cat([q, torch.full((4, 4, 64), float("nan"), device="cuda", dtype=q.dtype)])
    o, l = check_attention(mem, more[:9], kq, kd, vq, vd, table, lens, cu)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = torch.int32
    o2, l2 = mem.memra_kv_attention_q8(more, dev(kq), dev(kd), dev(vq), dev(vd), dev(table, i32), dev(lens, i32),
                                       dev(cu, i32), dev_status=st)
    assert torch.equal(o2[:9], o) and bool((o2[9:] == 0).all()) and bool(torch.isneginf(l2[9:]).all())


def test_attention_out_of_range_pages_and_lengths(mem):
    rs = np.random.RandomState(11)
    q, kq, kd, vq, vd, table, lens, cu = attention_case(rs, [100, 50], [1, 1], 8, 2, 128, 16, 16, "fp32")
    bad = table.copy()
    bad[0, 2], bad[0, 4] = -1, 10 ** 6
    check_attention(mem, q, kq, kd, vq, vd, bad, lens, cu, status=1)
    full = attention_case(rs, [96, 50], [1, 1], 8, 2, 128, 16, 16, "fp32")
    q, kq, kd, vq, vd, table, lens, cu = full
    check_attention(mem, q, kq, kd, vq, vd, table[:, :6], np.array([1000, 50]), cu, status=1)


def test_attention_extremes(mem):
    """Scores far apart, equal scores, scales that differ by a million from block to block."""
    rs = np.random.RandomState(13)
    for peak, dtype in ((40.0, "fp32"), (0.0, "bf16"), (3.0, "fp32")):
        q, kq, kd, vq, vd, table, lens, cu = attention_case(rs, [700, 90], [2, 1], 10, 2, 128, 32, 16, dtype, peak)
        vd *= np.where(rs.rand(*vd.shape) < 0.2, np.float32(1e6), np.float32(1.0)).astype(np.float32)
        vd[table[0, 0], 0, 0] = 0.0
        kd[table[0, 1], 1, 0] = 0.0
        check_attention(mem, q, kq, kd, vq, vd, table, lens, cu)


@pytest.mark.parametrize("size", [1e-6, 1e6])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_query_sizes(mem, size, dtype):
    """Queries far from 1 (with a scale that brings the scores back)."""
    q, kq, kd, vq, vd, table, lens, cu = attention_case(np.random.RandomState(17), [333], [3], 8, 2, 64, 16, 16, dtype)
    q = (q.float() * size).to(q.dtype)
    check_attention(mem, q, kq, kd, vq, vd, table, lens, cu, scale=0.125 / size)


def test_attention_strides_and_streams(mem):
    c = list(attention_case(np.random.RandomState(19), [400, 41], [3, 1], 10, 2, 128, 64, 16, "bf16"))
    o, l = check_attention(mem, *c)
    wide = torch.zeros(4, 14, 128, dtype=c[0].dtype, device="cuda")
    wide[:, 2:12] = c[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, l2 = check_attention(mem, wide[:, 2:12], *c[1:])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, o2) and torch.equal(l, l2)


def test_attention_long_pool(mem):
    """Pages whose byte offsets pass 2^31 (int8 plane of 4.3 GB, used at its end)."""
    Hkv, P, D = 8, 64, 256
    n_pages = (1 << 32) // (Hkv * P * D) + 4
    q, kq, kd, vq, vd, table, lens, cu = attention_case(np.random.RandomState(23), [300], [1], 16, Hkv, D, P, 16, "bf16")
    small = kq.shape[0]
    big = [torch.zeros((n_pages,) + x.shape[1:], dtype=torch.from_numpy(x).dtype, device="cuda") for x in (kq, kd, vq, vd)]
    for b, x in zip(big, (kq, kd, vq, vd)):
        b[n_pages - small:] = dev(x)
    i32 = torch.int32
    o, l = mem.memra_kv_attention_q8(q, *[dev(x) for x in (kq, kd, vq, vd)], dev(table, i32), dev(lens, i32), dev(cu, i32))
    moved = np.where(table >= 0, table + n_pages - small, -1)
    o2, l2 = mem.memra_kv_attention_q8(q, *big, dev(moved, i32), dev(lens, i32), dev(cu, i32))
    assert torch.equal(o, o2) and torch.equal(l, l2)
    x = torch.randn(5, Hkv, D, device="cuda")
    slots = dev(np.arange(5) + (n_pages - 1) * P + 3, i32)
    mem.memra_kv_append_q8(x, x, slots, *big)
    k, v = mem.memra_kv_read_q8(slots, *big, dtype=torch.float32)
    for got, plane in ((k, (kq, kd)), (v, (vq, vd))):     # the same on the small pool, whose last page it is
        wq, wd = ref_append(x.cpu().numpy(), np.arange(5) + (small - 1) * P + 3, *plane)
        want = wq[-1, :, 3:8].astype(np.float32) * wd[-1, :, 0, None, None]
        assert np.array_equal(got.cpu().numpy(), want.transpose(1, 0, 2))


# ---------------------------------------------------------------------------
# Routing.
# ---------------------------------------------------------------------------

f32 = np.float32


def exp32(x):
    x = np.clip(x, f32(-87.0), f32(88.0)).astype(f32)
    k = np.rint(x * f32(1.44269504088896341)).astype(f32)
    r = (x - k * f32(0.693359375)) - k * f32(-2.12194440e-4)
    p = np.full_like(r, f32(1.0 / 5040.0))
    for c in (1.0 / 720.0, 1.0 / 120.0, 1.0 / 24.0, 1.0 / 6.0, 0.5, 1.0, 1.0):
        p = p * r + f32(c)
    return p * np.ldexp(f32(1.0), k.astype(np.int32)).astype(f32)


def ref_route(x, k, bias, score, ng, tg, gt, renorm, scale):
    """The stated fp32 operations in numpy, token by token."""
    T, E = x.shape
    ids, w = np.zeros((T, k), np.int64), np.zeros((T, k), f32)
    for t in range(T):
        l = np.where(np.isnan(x[t]), -np.inf, np.minimum(x[t], np.finfo(f32).max)).astype(f32)
        dead = np.isneginf(l)
        if score == "softmax":
            with np.errstate(invalid="ignore"):
                e = np.where(dead, f32(0), exp32(np.where(dead, f32(0), l - l.max())))
            lanes = np.zeros((32, 0), f32)
            full = np.zeros(-(-E // 128) * 128, f32)
            full[:E] = e
            lanes = full.reshape(-1, 32, 4)
            z = np.zeros(32, f32)
            for c in range(lanes.shape[0]):
                for j in range(4):
                    z = z + lanes[c, :, j]
            for o in (16, 8, 4, 2, 1):
                z = z + z[np.arange(32) ^ o]
            s = np.where(dead, f32(0), e / np.where(z[0] == 0, f32(1), z[0])).astype(f32)
        else:
            s = np.where(dead, f32(0), f32(1) / (f32(1) + exp32(np.where(dead, f32(0), -l)))).astype(f32)
        v = s if bias is None else (s + bias).astype(f32)
        v = np.where(dead, f32(-np.inf), v)
        if ng > 1:
            g = np.sort(v.reshape(ng, E // ng), axis=1)[:, ::-1][:, :gt].sum(axis=1, dtype=f32)
            keep = np.argsort(-g, kind="stable")[:tg]
            v = np.where(np.isin(np.arange(E) // (E // ng), keep), v, f32(-np.inf))
        ids[t] = np.argsort(-v, kind="stable")[:k]
        c = np.where(np.isneginf(v[ids[t]]), f32(0), s[ids[t]])
        total = f32(0)
        for y in c:
            total = total + y
        w[t] = (c / total if total > 0 else np.zeros_like(c)) * f32(scale) if renorm else c * f32(scale)
    return ids, w


ROUTE = [
    # T, E, k, score, bias, groups, topk_groups, group_top, renorm, dtype
    (1, 1, 1, "softmax", False, 1, 1, 1, True, "fp32"),
    (1, 128, 8, "softmax", False, 1, 1, 1, True, "fp32"),
    (5, 7, 3, "sigmoid", True, 1, 1, 1, False, "bf16"),
    (16, 256, 8, "sigmoid", True, 8, 4, 2, True, "fp32"),
    (33, 160, 6, "softmax", False, 8, 3, 1, True, "bf16"),
    (9, 130, 64, "softmax", True, 1, 1, 1, True, "fp32"),
    (70, 512, 2, "sigmoid", False, 32, 1, 2, False, "bf16"),
    (3, 1024, 33, "softmax", True, 16, 16, 1, True, "fp32"),
    (1000, 64, 6, "softmax", True, 1, 1, 1, True, "bf16"),
    (17, 12, 4, "sigmoid", True, 4, 2, 2, True, "fp32"),
    (8, 9, 2, "sigmoid", True, 3, 1, 2, True, "bf16"),
]


@pytest.mark.parametrize("case", range(len(ROUTE)))
@pytest.mark.parametrize("kind", ["plain", "ties", "masked"])
def test_route(mem, case, kind):
    T, E, k, score, has_bias, ng, tg, gt, renorm, dtype = ROUTE[case]
    g = torch.Generator().manual_seed(100 + case)
    x = 2.0 * torch.randn(T, E, generator=g)
    if kind == "ties":
        x = torch.round(x)
    x = x.bfloat16() if dtype == "bf16" else x
    if kind == "masked":
        x[torch.rand(T, E, generator=g) < 0.6] = float("-inf")
        x[0] = float("-inf")
        x[T // 2, E // 2] = float("nan")
        x[T - 1, E - 1] = float("inf")
        x[T - 1, 0] = torch.finfo(x.dtype).min
    bias = (0.1 * torch.randn(E, generator=g) if kind != "ties" else torch.zeros(E)) if has_bias else None
    want_ids, want_w = ref_route(x.float().numpy(), k, None if bias is None else bias.numpy(), score, ng, tg, gt,
                                 renorm, 2.5)
    ids, w = mem.memra_moe_route(x.cuda(), k, bias=None if bias is None else bias.cuda(), score=score, n_groups=ng,
                                 topk_groups=tg, group_top=gt, renormalize=renorm, scale=2.5)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert np.array_equal(w.cpu().numpy(), want_w)


def test_route_weights_match_float64(mem):
    x = 2.0 * torch.randn(64, 256, generator=torch.Generator().manual_seed(1))
    ids, w = mem.memra_moe_route(x.cuda(), 8)
    p = torch.softmax(x.double(), -1).gather(1, ids.cpu().long())
    # the exponentials and quotients are good to a few fp32 roundings
    assert float((w.cpu().double() - p / p.sum(-1, keepdim=True)).abs().max()) < 2e-6


def test_route_strided_and_unaligned_rows(mem):
    x = torch.randn(12, 131, generator=torch.Generator().manual_seed(2)).cuda()
    for view in (x[:, 1:129], x[:, 3:131], x[::2, :128], x[:, :7]):
        k = min(6, view.shape[1])
        a, b = mem.memra_moe_route(view, k), mem.memra_moe_route(view.contiguous(), k)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_routing_feeds_the_routed_product(mem):
    """ids and gate_w go into the routed FFN as they come."""
    import synth
    E, H, F, k = 16, 256, 64, 4
    w = synth.weights_fp32(E * 2 * F, H, 700, 0, device="cuda")
    gq, gd = mem.memra_quantize_q8_0(w)
    w = synth.weights_fp32(E * H, F, 700, 1, device="cuda")
    dq, dd = mem.memra_quantize_q8_0(w)
    banks = gq.view(E, 2 * F, H), gd.view(E, 2 * F, H // 32), dq.view(E, H, F), dd.view(E, H, F // 32)
    x = synth.activations_bf16(3, H, 700, 2, device="cuda")
    ids, gate = mem.memra_moe_route(torch.randn(3, E, device="cuda"), k)
    y = mem.memra_q8_0_moe_ffn_tokens(*banks, ids, gate, x)
    for t in range(3):
        one = mem.memra_q8_0_moe_ffn(*banks, ids[t], gate[t], x[t])
        assert torch.equal(one, y[t])


# ---------------------------------------------------------------------------
# Refusals of the binding.
# ---------------------------------------------------------------------------

def test_refusals(mem):
    i32 = torch.int32
    kq = torch.zeros(2, 2, 16, 64, dtype=torch.int8, device="cuda")
    kd = torch.zeros(2, 2, 1, device="cuda")
    c = (kq, kd, kq.clone(), kd.clone())
    q = torch.zeros(1, 4, 64, device="cuda")
    tab, lens, cu = dev([[0]], i32), dev([3], i32), dev([0, 1], i32)
    ok = mem.memra_kv_attention_q8(q, *c, tab, lens, cu)
    assert ok[0].shape == (1, 4, 64)
    with pytest.raises(TypeError):
        mem.memra_kv_attention_q8(q.half(), *c, tab, lens, cu)
    with pytest.raises(TypeError):
        mem.memra_kv_attention_q8(q, *c, tab, lens.long(), cu)
    with pytest.raises(ValueError):
        mem.memra_kv_attention_q8(q[:, :3], *c, tab, lens, cu)             # 3 heads on 2
    with pytest.raises(ValueError):
        mem.memra_kv_attention_q8(q.cpu(), *c, tab, lens, cu)
    with pytest.raises(ValueError):
        mem.memra_kv_attention_q8(q, *c, tab, lens, cu, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        mem.memra_kv_attention_q8(q.transpose(1, 2).contiguous().transpose(1, 2), *c, tab, lens, cu)
    with pytest.raises(mem.MemraError) as e:
        mem.memra_kv_attention_q8(q, *c, tab, lens, cu, window=-1)
    assert e.value.status == 1
    wide = torch.zeros(1, 4, 66, device="cuda")
    with pytest.raises(mem.MemraError) as e:
        mem.memra_kv_attention_q8(wide[:, :, 1:65], *c, tab, lens, cu)     # not 16-byte aligned
    assert e.value.status == 2
    with pytest.raises(ValueError):
        mem.memra_kv_append_q8(q[:, :2], q[:, :1], dev([0], i32), *c)
    with pytest.raises(TypeError):
        mem.memra_kv_append_q8(q[:, :2], q[:, :2], dev([0], torch.int64), *c)
    with pytest.raises(TypeError):
        mem.memra_kv_read_q8(dev([0], i32), *c, dtype=torch.float16)
    with pytest.raises(mem.MemraError):
        mem.memra_kv_plan(lens, lens, 24, lens, tab, 1)                    # a page of 24 tokens
    with pytest.raises(ValueError):
        mem.memra_kv_plan(lens, lens, 16, lens, tab[0], 1)
    x = torch.zeros(2, 8, device="cuda")
    for kw, st in ((dict(top_k=0), 1), (dict(top_k=9), 1), (dict(top_k=2, n_groups=3), 1),
                   (dict(top_k=2, n_groups=4, topk_groups=5), 1), (dict(top_k=2, n_groups=8, topk_groups=8, group_top=2), 1),
                   (dict(top_k=5, n_groups=4, topk_groups=2), 1)):
        with pytest.raises(mem.MemraError) as e:
            mem.memra_moe_route(x, **kw)
        assert e.value.status == st, kw
    with pytest.raises(mem.MemraError) as e:
        mem.memra_moe_route(torch.zeros(1, 2048, device="cuda"), 2)
    assert e.value.status == 3
    with pytest.raises(ValueError):
        mem.memra_moe_route(x, 2, score="tanh")
