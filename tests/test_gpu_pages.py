"""Forking, copying on write, copying, releasing and compacting cache pages against plain implementations, one entry after
another.  Whole numbers and bit-exact copies: nothing may differ."""
import numpy as np
import pytest
import torch

from _util import Guarded

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


def dev(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=i32).cuda()


def pages(n, P):
    return -(-int(n) // P)


def valid(n, P, width):
    """(length, whether it is one) of a sequence whose row has `width` entries."""
    n = int(n)
    return (0, False) if n < 0 else (min(n, width * P), n <= width * P)


# ---------------------------------------------------------------------------
# Plain forms.
# ---------------------------------------------------------------------------

def ref_fork(parents, lens, table, P, refs, prefix=None):
    B, W = table.shape
    refs, bits = refs.copy(), 0
    out_lens, out = np.zeros(len(parents), np.int64), np.full((len(parents), W), -1, np.int64)
    for r, p in enumerate(parents):
        if not 0 <= p < B:
            bits |= p != -1
            continue
        n, ok = valid(lens[p], P, W)
        bits |= not ok
        if prefix is not None:
            n = min(n, max(int(prefix[r]), 0))
        out_lens[r] = n
        for i in range(pages(n, P)):
            e = table[p, i]
            if 0 <= e < len(refs):
                refs[e] += 1
                out[r, i] = e
            else:
                bits |= 1
    return out_lens, out, refs, int(bits)


def ref_unshare(lens, new, P, refs, free, table, head):
    refs, table, head = refs.copy(), table.copy(), max(head, 0)
    B, W = table.shape
    src, dst, tokens, add, bits = np.full(B, -1), np.full(B, -1), np.zeros(B, int), np.zeros(B, int), 0
    for b in range(B):
        bits |= new[b] < 0
        add[b] = max(int(new[b]), 0)
        n, ok = valid(lens[b], P, W)
        bits |= not ok
        if not ok or add[b] == 0 or n % P == 0:
            continue
        p = table[b, n // P]
        if not 0 <= p < len(refs):
            bits |= 1
        elif refs[p] > 0:
            if head >= len(free):
                add[b] = 0
                bits |= 4
                continue
            f = free[head]
            head += 1
            refs[p] -= 1
            table[b, n // P] = f
            src[b], dst[b], tokens[b] = p, f, n % P
            bits |= not 0 <= f < len(refs)
    return add, src, dst, tokens, head, refs, table, int(bits)


def ref_release(lens, P, table, refs, free, head, keep=None):
    refs, free, bits = refs.copy(), free.copy(), 0
    B, W = table.shape
    out, given = np.zeros(B, int), []
    for b in range(B):
        n, ok = valid(lens[b], P, W)
        k = 0 if keep is None else int(keep[b])
        bits |= (not ok) | (k < 0)
        k = max(k, 0)
        out[b] = min(n, k)
        for i in range(min(pages(k, P), W), pages(n, P)):
            if 0 <= table[b, i] < len(refs):
                given.append(int(table[b, i]))
            else:
                bits |= 1
    last = {p: at for at, p in enumerate(given)}
    for p in given:
        refs[p] -= 1
    goes = [p for at, p in enumerate(given) if last[p] == at and refs[p] < 0]
    bits |= any(refs[p] < -1 for p in goes)
    for p in goes:
        refs[p] = 0
    for i, p in enumerate(goes):
        at = head - len(goes) + i
        if 0 <= at < len(free):
            free[at] = p
        else:
            bits |= 4
    return out, max(head - len(goes), 0), refs, free, int(bits) | (4 if head > len(free) else 0)


def ref_compact(lens, table, P, n_pages):
    B, W = table.shape
    held, bits = np.zeros(n_pages, int), 0
    for b in range(B):
        n, ok = valid(lens[b], P, W)
        bits |= not ok
        for i in range(pages(n, P)):
            if 0 <= table[b, i] < n_pages:
                held[table[b, i]] += 1
            else:
                bits |= 1
    used = int((held > 0).sum())
    high = [p for p in range(n_pages - 1, used - 1, -1) if held[p]]
    low = [p for p in range(used) if not held[p]]
    src, dst = np.full(n_pages // 2, -1), np.full(n_pages // 2, -1)
    src[:len(high)], dst[:len(low)] = high, low
    number = np.arange(n_pages)
    number[high] = low
    out, refs = np.full((B, W), -1), np.zeros(n_pages, int)
    for b in range(B):
        for i in range(pages(valid(lens[b], P, W)[0], P)):
            if 0 <= table[b, i] < n_pages:
                out[b, i] = number[table[b, i]]
    for p in range(n_pages):
        if held[p]:
            refs[number[p]] = held[p] - 1
    return out, refs, np.arange(n_pages), src, dst, used, int(bits)


def same(got, want, what):
    assert np.array_equal(got.cpu().numpy().reshape(-1), np.asarray(want).reshape(-1)), what


def check_fork(mem, parents, lens, table, P, refs, prefix=None):
    want = ref_fork(parents, lens, table, P, refs, prefix)
    r, st = dev(refs), torch.zeros(1, dtype=i32, device="cuda")
    ol, ot = mem.memra_kv_fork(dev(parents), dev(lens), dev(table), P, r, prefix_lens=None if prefix is None else dev(prefix), dev_status=st)
    for got, ref, what in zip((ol, ot, r, st), want, ("lens", "table", "refs", "status")):
        same(got, ref, what)
    return want


def check_unshare(mem, lens, new, P, refs, free, table, head, in_place=False):
    want = ref_unshare(lens, new, P, refs, free, table, head)
    r, t, st, h, a = dev(refs), dev(table), torch.zeros(1, dtype=i32, device="cuda"), dev([head]), dev(new)
    got = mem.memra_kv_unshare(dev(lens), a, P, r, dev(free), t, free_head=h, free_head_out=h if in_place else None,
                               new_lens_out=a if in_place else None, dev_status=st)
    for g, ref, what in zip(got + (r, t, st), want, ("new", "src", "dst", "tokens", "head", "refs", "table", "status")):
        same(g, ref, what)
    assert not in_place or (got[4].data_ptr() == h.data_ptr() and got[0].data_ptr() == a.data_ptr())
    return want


def check_release(mem, lens, P, table, refs, free, head, keep=None, in_place=False):
    want = ref_release(lens, P, table, refs, free, head, keep)
    l, r, f, st, h = dev(lens), dev(refs), dev(free), torch.zeros(1, dtype=i32, device="cuda"), dev([head])
    got = mem.memra_kv_release(l, P, dev(table), r, f, h, keep_lens=None if keep is None else dev(keep), lens_out=l if in_place else None,
                               free_head_out=h if in_place else None, dev_status=st)
    for g, ref, what in zip(got + (r, f, st), want, ("lens", "head", "refs", "free", "status")):
        same(g, ref, what)
    return want


def check_compact(mem, lens, table, P, n_pages, in_place=False):
    want = ref_compact(lens, table, P, n_pages)
    t, st = dev(table), torch.zeros(1, dtype=i32, device="cuda")
    got = mem.memra_kv_compact(dev(lens), t, P, n_pages, table_out=t if in_place else None, dev_status=st)
    for g, ref, what in zip(got + (st,), want, ("table", "refs", "free", "src", "dst", "head", "status")):
        same(g, ref, what)
    return want


# ---------------------------------------------------------------------------
# A pool with sequences, some of which share pages.
# ---------------------------------------------------------------------------

def pool(rs, B, P, top, extra, share=0.5):
    """lens, table, refs, free list and its position; about `share` of the sequences are forks of an earlier one, which then
    went on by themselves."""
    lens = rs.randint(0, top + 1, B)
    W = pages(max(int(lens.max()), 1), P) + 1
    table = np.full((B, W), -1)
    n_pages = sum(pages(n, P) for n in lens) + extra
    ids = rs.permutation(n_pages)
    refs, at = np.zeros(n_pages, int), 0
    for b in range(B):
        have = pages(lens[b], P)
        k = 0
        if b and rs.rand() < share:
            p = rs.randint(b)
            k = min(have, pages(lens[p], P))
            table[b, :k] = table[p, :k]
            refs[table[p, :k]] += 1
        table[b, k:have] = ids[at:at + have - k]
        at += have - k
    return lens, table, refs, ids, at


SIZES = [(1, 16, 10, 3), (3, 16, 100, 9), (7, 32, 900, 40), (40, 64, 700, 64), (33, 1024, 5000, 7), (300, 16, 400, 100), (1500, 16, 90, 50),
         (2500, 32, 64, 10), (9, 16, 40000, 500)]


@pytest.mark.parametrize("B,P,top,extra", SIZES)
def test_fork(mem, B, P, top, extra):
    rs = np.random.RandomState(B + top)
    lens, table, refs, ids, at = pool(rs, B, P, top, extra)
    parents = rs.randint(0, B, 2 * B + 1)
    parents[::5] = -1
    check_fork(mem, parents, lens, table, P, refs)
    check_fork(mem, parents, lens, table, P, refs, prefix=rs.randint(-3, top + 20, 2 * B + 1))
    check_fork(mem, np.zeros(1000, int), lens, table, P, refs)  # one parent of all


def test_fork_odd_inputs(mem):
    table = np.array([[3, 99, 1], [0, -1, 2], [4, 5, 6]])
    lens, refs = np.array([40, 33, -5]), np.zeros(8, int)
    check_fork(mem, [0, 1, 2, 3, -2, 2 ** 31 - 1, -1], lens, table, 16, refs)
    check_fork(mem, [0], np.array([1000, 0, 0]), table, 16, refs)
    check_fork(mem, [0], np.array([2 ** 31 - 1, 0, 0]), table, 16, refs)
    check_fork(mem, [0, -1], np.zeros(0, int), np.zeros((0, 4), int), 16, refs)
    check_fork(mem, [0], np.array([0]), np.zeros((1, 0), int), 16, refs)
    check_fork(mem, [0], np.array([5]), np.zeros((1, 0), int), 16, refs)
    l, t = mem.memra_kv_fork(dev([]), dev(lens), dev(table), 16, dev(refs))
    assert l.shape == (0,) and t.shape == (0, 3)


@pytest.mark.parametrize("B,P,top,extra", SIZES)
@pytest.mark.parametrize("short", [False, True])
def test_unshare(mem, B, P, top, extra, short):
    rs = np.random.RandomState(B * 3 + top)
    lens, table, refs, ids, at = pool(rs, B, P, top, extra, share=0.8)
    new = rs.randint(0, 3, B)
    free = ids[:at + (extra // 4 if short else extra)]
    check_unshare(mem, lens, new, P, refs, free, table, at, in_place=short)
    # many forks of one sequence, which is among them or not
    parents = rs.randint(0, B, 70)
    parents[:40] = parents[0]
    fl, ft, fr, _ = ref_fork(parents, lens, table, P, refs)
    more = np.concatenate([ids, np.arange(90) % len(refs)])
    check_unshare(mem, fl, np.ones(70, int), P, fr, more[:at + (20 if short else 90)], ft, at)
    both_l, both_t = np.concatenate([fl, lens]), np.concatenate([ft, table])
    check_unshare(mem, both_l, np.ones(70 + B, int), P, fr, more[:at + (20 if short else 90)], both_t, at)


def test_unshare_odd_inputs(mem):
    table = np.array([[3, 99], [3, 1], [3, -1], [2, 0], [3, 4]])
    refs, free = np.array([0, 0, 0, 3, 0, 0, 0, 0]), np.array([7, 6, 88, 5])
    lens = np.array([5, 5, 20, -1, 9])
    check_unshare(mem, lens, np.array([1, -4, 2, 1, 1]), 16, refs, free, table, 0)
    check_unshare(mem, lens, np.ones(5, int), 16, refs, free, table, 2)
    check_unshare(mem, lens, np.ones(5, int), 16, refs, free, table, -3)
    check_unshare(mem, lens, np.ones(5, int), 16, refs, free, table, 9)
    check_unshare(mem, np.array([5, 5, 5, 5, 2 ** 31 - 1]), np.ones(5, int), 16, refs, np.zeros(0, int), table, 0)
    check_unshare(mem, np.array([32, 16, 33, 0, 100]), np.ones(5, int), 16, refs, free, table, 0)
    check_unshare(mem, np.zeros(0, int), np.zeros(0, int), 16, refs, free, np.zeros((0, 2), int), 1)


@pytest.mark.parametrize("B,P,top,extra", SIZES)
def test_release(mem, B, P, top, extra):
    rs = np.random.RandomState(B * 5 + top)
    lens, table, refs, ids, at = pool(rs, B, P, top, extra)
    all_gone = check_release(mem, lens, P, table, refs, ids, at)
    assert all_gone[1] == 0 and not all_gone[2].any() and sorted(all_gone[3]) == sorted(ids)
    check_release(mem, lens, P, table, refs, ids, at, keep=rs.randint(0, top + 5, B), in_place=True)
    check_release(mem, lens, P, table, refs, ids, at, keep=np.where(rs.rand(B) < 0.5, lens, 0))
    check_release(mem, lens, P, table, refs, ids, at, keep=lens)
    check_release(mem, lens, P, table, refs, ids, max(at // 3, 0))      # more than fits below the head
    check_release(mem, lens, P, table, refs, ids[:at // 2], at)         # a head behind the list
    check_release(mem, lens, P, table, np.zeros_like(refs), ids, at)    # given up more often than held


def test_release_odd_inputs(mem):
    table = np.array([[3, 99, 1], [3, -1, 2], [4, 5, 6]])
    refs, free = np.zeros(8, int), np.arange(8)
    check_release(mem, np.array([40, 33, -5]), 16, table, refs, free, 6)
    check_release(mem, np.array([1000, 2 ** 31 - 1, 17]), 16, table, refs, free, 8, keep=np.array([-1, 2 ** 31 - 1, 1]))
    check_release(mem, np.array([48, 0, 17]), 16, table, refs, np.zeros(0, int), 0)
    check_release(mem, np.array([48, 0, 17]), 16, table, refs, free, -2)
    check_release(mem, np.zeros(0, int), 16, np.zeros((0, 3), int), refs, free, 4)
    check_release(mem, np.array([3]), 16, np.zeros((1, 0), int), refs, free, 4)
    check_release(mem, np.array([48]), 16, np.array([[2, 2, 2]]), np.array([0, 0, 2, 0]), np.arange(4), 3)


@pytest.mark.parametrize("B,P,top,extra", SIZES)
def test_compact(mem, B, P, top, extra):
    rs = np.random.RandomState(B * 7 + top)
    lens, table, refs, ids, at = pool(rs, B, P, top, extra)
    n_pages = len(refs)
    want = check_compact(mem, lens, table, P, n_pages)
    assert np.array_equal(np.sort(want[1]), np.sort(refs))
    check_compact(mem, lens, table, P, n_pages, in_place=True)
    gone = np.where(rs.rand(B) < 0.6, 0, lens)
    mid = check_compact(mem, gone, table, P, n_pages)
    again = check_compact(mem, gone, mid[0], P, n_pages)
    assert (again[3] == -1).all() and np.array_equal(again[0], mid[0])  # compact already
    check_compact(mem, np.zeros(B, int), table, P, n_pages)


def test_compact_odd_inputs(mem):
    table = np.array([[3, 99, 1], [3, -1, 2], [4, 5, 6]])
    check_compact(mem, np.array([40, 33, -5]), table, 16, 8)
    check_compact(mem, np.array([1000, 1, 2 ** 31 - 1]), table, 16, 7)
    check_compact(mem, np.array([48, 48, 48]), table, 16, 1)
    check_compact(mem, np.array([48, 48, 48]), table, 16, 0)
    check_compact(mem, np.zeros(0, int), np.zeros((0, 3), int), 16, 9)
    check_compact(mem, np.array([3]), np.zeros((1, 0), int), 16, 2)
    check_compact(mem, np.array([16]), np.array([[1]]), 16, 2)


@pytest.mark.parametrize("B,W,n", [(64, 128, 300), (64, 129, 300), (8192, 1, 9000), (8193, 1, 9000), (8, 40, 16384), (8, 40, 16385), (1, 1, 16384),
                                   (3, 7, 1), (5, 1024, 16383), (1, 8192, 12000)])
def test_tables_and_pools_on_both_sides_of_the_small_ones(mem, B, W, n):
    any_pages(mem, B, W, n)


@pytest.mark.parametrize("B,W,n", [(64, 64, 3000), (4097, 1, 3000), (40, 64, 16384), (40, 64, 16385), (70, 100, 131072), (70, 100, 131073), (64, 1024, 9000),
                                   (65, 1009, 9000), (1, 65536, 70000), (300, 150, 8), (300, 150, 9), (9000, 7, 40000), (2, 1, 100000)])
def test_larger_tables_and_pools(mem, B, W, n):
    any_pages(mem, B, W, n)


def any_pages(mem, B, W, n):
    """Any pages at all in the table, many of them shared, and lengths that end anywhere."""
    rs = np.random.RandomState(B + W + n)
    P = 16
    table, lens = rs.randint(0, n, (B, W)), rs.randint(0, P * W + 1, B)
    lens[0] = P * W
    held = np.zeros(n, int)
    for b in range(B):
        np.add.at(held, table[b, :pages(lens[b], P)], 1)
    refs, used = np.maximum(held - 1, 0), int((held > 0).sum())
    check_compact(mem, lens, table, P, n)
    check_compact(mem, np.where(rs.rand(B) < 0.5, lens, 0), table, P, n, in_place=True)
    gone = check_release(mem, lens, P, table, refs, rs.permutation(n), used)
    assert gone[1] == 0 and not gone[2].any()
    check_release(mem, lens, P, table, refs, rs.permutation(n), used, keep=rs.randint(0, P * W + 1, B), in_place=True)
    check_release(mem, lens, P, table, refs, rs.permutation(n)[:used // 2], used // 3)


# ---------------------------------------------------------------------------
# Copies.
# ---------------------------------------------------------------------------

def cache(rs, n_pages, H, P, D, S):
    g = torch.Generator().manual_seed(int(rs.randint(1 << 30)))
    planes = []
    for _ in range(2):
        planes.append(torch.randint(-128, 128, (n_pages, H, P, D), generator=g, dtype=torch.int8).cuda())
        planes.append(torch.randn(n_pages, H, P // S, generator=g).cuda())
    return tuple(planes)


@pytest.mark.parametrize("H,P,D,S", [(1, 16, 64, 16), (8, 64, 128, 16), (3, 48, 256, 1), (2, 1024, 256, 64), (5, 128, 64, 32)])
@pytest.mark.parametrize("layers", [1, 3, 70])
@pytest.mark.parametrize("cut", [False, True])
def test_copy_pages(mem, H, P, D, S, layers, cut):
    rs = np.random.RandomState(H * P + layers)
    n = 11
    caches = [cache(rs, n, H, P, D, S) for _ in range(layers)]
    before = [tuple(x.clone() for x in c) for c in caches]
    order = rs.permutation(n)
    src, dst = np.array([order[0], order[0], -1, order[1], order[2], order[3]]), np.array([order[4], order[5], order[6], -1, order[2], order[7]])
    tokens = np.array([1, P, 3, 3, 3, P - 5]) if cut else None
    st = torch.zeros(1, dtype=i32, device="cuda")
    mem.memra_kv_copy_pages(dev(src), dev(dst), caches, tokens=None if tokens is None else dev(tokens), dev_status=st)
    assert int(st) == 0
    for c, b in zip(caches, before):
        want = [x.clone() for x in b]
        for i in (0, 1, 5):
            m = P if tokens is None else int(tokens[i])
            for x, old in zip(want, b):
                k = m if x.dim() == 4 else -(-m // S)
                x[dst[i], :, :k] = old[src[i], :, :k]
        assert all(torch.equal(x.view(torch.uint8), w.view(torch.uint8)) for x, w in zip(c, want))


def test_copy_pages_odd_inputs(mem):
    rs = np.random.RandomState(1)
    c = cache(rs, 6, 2, 16, 64, 4)
    before = [x.clone() for x in c]
    for s, d, t in ((6, 0, 3), (0, 6, 3), (-2, 0, 3), (0, 2 ** 31 - 1, 3), (0, 1, 17), (0, 1, -1)):
        st = torch.zeros(1, dtype=i32, device="cuda")
        mem.memra_kv_copy_pages(dev([s, -1]), dev([d, 4]), [c], tokens=dev([t, 2]), dev_status=st)
        mem.memra_kv_copy_pages(dev([s, -1]), dev([d, 4]), [c], tokens=dev([t, 2]))
        assert int(st) == 1 and all(torch.equal(a, b) for a, b in zip(c, before)), (s, d, t)
    mem.memra_kv_copy_pages(dev([0]), dev([1]), [c], tokens=dev([0]))
    mem.memra_kv_copy_pages(dev([]), dev([]), [c])
    assert all(torch.equal(a, b) for a, b in zip(c, before))
    mem.memra_kv_copy_pages(dev([0]), dev([1]), [c])
    assert torch.equal(c[0][1], before[0][0]) and torch.equal(c[3][1], before[3][0]) and torch.equal(c[0][2:], before[0][2:])


def test_copy_pages_far_into_a_pool(mem):
    """Pages whose bytes lie past 2^32, and nothing beside the pages."""
    H, P, D = 4, 64, 128
    n = (1 << 32) // (H * P * D) + 5
    planes = [torch.zeros((n, H, P, D), dtype=torch.int8, device="cuda"), torch.zeros((n, H, 4), device="cuda")] * 1
    v = [torch.zeros_like(planes[0]), torch.zeros_like(planes[1])]
    c = (planes[0], planes[1], v[0], v[1])
    c[0][1], c[2][1], c[1][1], c[3][1] = 5, -7, 0.5, 0.25
    mem.memra_kv_copy_pages(dev([1, n - 1]), dev([n - 2, 3]), [c])
    mem.memra_kv_copy_pages(dev([n - 2]), dev([n // 2]), [c])
    for at in (n - 2, n // 2):
        assert bool((c[0][at] == 5).all()) and bool((c[2][at] == -7).all()) and bool((c[1][at] == 0.5).all())
    assert int(c[0].count_nonzero()) == 3 * H * P * D and int(c[3].count_nonzero()) == 3 * H * 4


# ---------------------------------------------------------------------------
# Together.
# ---------------------------------------------------------------------------

def test_nothing_is_written_beside_the_outputs(mem):
    rs = np.random.RandomState(5)
    lens, table, refs, ids, at = pool(rs, 37, 16, 300, 50)
    W, n = table.shape[1], len(refs)
    g = [Guarded((9,), i32), Guarded((9, W), i32)]
    mem.memra_kv_fork(dev(rs.randint(0, 37, 9)), dev(lens), dev(table), 16, dev(refs), lens_out=g[0].view, table_out=g[1].view)
    u = [Guarded((37,), i32) for _ in range(4)] + [Guarded((1,), i32)]
    mem.memra_kv_unshare(dev(lens), dev(np.ones(37)), 16, dev(refs), dev(ids), dev(table), free_head=dev([at]), new_lens_out=u[0].view,
                         src=u[1].view, dst=u[2].view, tokens=u[3].view, free_head_out=u[4].view)
    r = [Guarded((37,), i32), Guarded((1,), i32), Guarded((n,), i32), Guarded((n,), i32)]
    r[2].view.copy_(dev(refs))
    r[3].view.copy_(dev(ids))
    mem.memra_kv_release(dev(lens), 16, dev(table), r[2].view, r[3].view, dev([at]), lens_out=r[0].view, free_head_out=r[1].view)
    c = [Guarded((37, W), i32), Guarded((n,), i32), Guarded((n,), i32)]
    mem.memra_kv_compact(dev(lens), dev(table), 16, n, table_out=c[0].view, refs_out=c[1].view, free_out=c[2].view)
    torch.cuda.synchronize()
    assert all(x.intact() for x in g + u + r + c)


def test_fork_and_give_up_leaves_everything_as_it_was(mem):
    """The free list and the counts return to what they were, page for page, however often."""
    rs = np.random.RandomState(6)
    lens, table, refs, ids, at = pool(rs, 12, 16, 200, 100, share=0.3)
    l, t, r, f, h = dev(lens), dev(table), dev(refs), dev(ids), dev([at])
    parents, ones = dev(rs.randint(0, 12, 30)), torch.ones(30, dtype=i32, device="cuda")
    st = torch.zeros(1, dtype=i32, device="cuda")
    for _ in range(3):
        fl, ft = mem.memra_kv_fork(parents, l, t, 16, r, dev_status=st)
        _, src, dst, tokens, taken = mem.memra_kv_unshare(fl, ones, 16, r, f, ft, free_head=h, dev_status=st)
        assert int(taken) > at
        gone, head = mem.memra_kv_release(fl, 16, ft, r, f, taken, dev_status=st)
        same(head, [at], "head")
        same(r, refs, "refs")
        same(f, ids, "free list")
        assert not bool(gone.any())
    assert int(st) == 0


@pytest.mark.parametrize("graph", [False, True])
def test_a_random_life_of_a_pool(mem, graph):
    """Steps of forks, writes, releases and a compaction: no page is ever both free and held, counts are those of the tables,
    and every sequence reads back what its own history wrote (scale blocks of one token: a value does not change by later ones)."""
    rs = np.random.RandomState(11)
    P, H, D, B, n_pages, W = 16, 1, 64, 12, 160, 12
    c = (torch.zeros(n_pages, H, P, D, dtype=torch.int8, device="cuda"), torch.zeros(n_pages, H, P, device="cuda"),
         torch.zeros(n_pages, H, P, D, dtype=torch.int8, device="cuda"), torch.zeros(n_pages, H, P, device="cuda"))
    lens, table = torch.zeros(B, dtype=i32, device="cuda"), torch.full((B, W), -1, dtype=i32, device="cuda")
    refs, free, head = torch.zeros(n_pages, dtype=i32, device="cuda"), dev(rs.permutation(n_pages)), dev([0])
    st = torch.zeros(1, dtype=i32, device="cuda")
    history = [[] for _ in range(B)]
    parents, keep, new = (torch.zeros(B, dtype=i32, device="cuda") for _ in range(3))
    marks = torch.zeros(B * 20, device="cuda")

    def reshuffle():
        """The next generation: row r goes on from parents[r], cut to keep[r] tokens; the old rows are given up."""
        fl, ft = mem.memra_kv_fork(parents, lens, table, P, refs, prefix_lens=keep, dev_status=st)
        mem.memra_kv_release(lens, P, table, refs, free, head, lens_out=lens, free_head_out=head, dev_status=st)
        lens.copy_(fl)
        table.copy_(ft)

    def write():
        rows = B * 20
        ok, src, dst, tokens, _ = mem.memra_kv_unshare(lens, new, P, refs, free, table, free_head=head, free_head_out=head, dev_status=st)
        mem.memra_kv_copy_pages(src, dst, [c], tokens=tokens, dev_status=st)
        _, _, slots, pos, _ = mem.memra_kv_plan(lens, ok, P, free, table, rows, free_head=head, free_head_out=head, kv_lens=lens, dev_status=st)
        k = marks[:, None, None].expand(rows, H, D).contiguous()
        mem.memra_kv_append_q8(k, k, slots, *c, dev_status=st)

    calls = {"reshuffle": reshuffle, "write": write}
    if graph:
        saved = [x.clone() for x in (lens, table, refs, free, head) + c]
        for name, call in list(calls.items()):
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                call()
            torch.cuda.current_stream().wait_stream(side)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call()
            calls[name] = g.replay
        for x, s in zip((lens, table, refs, free, head) + c, saved):
            x.copy_(s)
        st.zero_()
    for step in range(25):
        if step % 3 == 2:
            p = rs.randint(-1, B, B)
            cut = rs.randint(0, 140, B)
            parents.copy_(dev(p))
            keep.copy_(dev(cut))
            calls["reshuffle"]()
            history = [history[a][:b] if a >= 0 else [] for a, b in zip(p, cut)]
        add = np.minimum(rs.randint(0, 20, B), [W * P - len(h) for h in history])
        new.copy_(dev(add))
        values = rs.randint(1, 100, B * 20).astype(np.float32)
        marks.copy_(torch.from_numpy(values))
        calls["write"]()
        at = 0
        for b in range(B):
            history[b] = history[b] + values[at:at + add[b]].tolist()
            at += add[b]
        if step % 8 == 7:
            t2, r2, f2, src, dst, h2 = mem.memra_kv_compact(lens, table, P, n_pages, dev_status=st)
            mem.memra_kv_copy_pages(src, dst, [c], dev_status=st)
            same(r2.sort().values, refs.sort().values.cpu().numpy(), "refs")
            table.copy_(t2), refs.copy_(r2), free.copy_(f2), head.copy_(h2)
        assert int(st) == 0
        L, tb = lens.tolist(), table.cpu().numpy()
        assert L == [len(h) for h in history]
        held = np.zeros(n_pages, int)
        for b in range(B):
            np.add.at(held, tb[b, :pages(L[b], P)], 1)
        assert np.array_equal(np.maximum(held - 1, 0), refs.cpu().numpy())
        unused = free[int(head):].cpu().numpy()
        assert sorted(unused) == np.flatnonzero(held == 0).tolist()
        slots = np.concatenate([tb[b, np.arange(L[b]) // P] * P + np.arange(L[b]) % P for b in range(B)] + [np.zeros(0)]).astype(int)
        k, v = mem.memra_kv_read_q8(dev(slots), *c, dtype=torch.float32)
        want = np.array([x for h in history for x in h])
        # a code of 127 at scale x / 127, each rounded once: within 2 * 2^-24
        assert np.allclose(k[:, 0, 0].cpu().numpy(), want, rtol=2.0 ** -22) and torch.equal(k, v) and bool((k == k[..., :1]).all())


def test_refusals(mem):
    rs = np.random.RandomState(2)
    lens, table, refs, ids, at = pool(rs, 5, 16, 100, 9)
    l, t, r, f, h = dev(lens), dev(table), dev(refs), dev(ids), dev([at])
    c = cache(rs, 6, 2, 16, 64, 4)
    five = dev(np.zeros(5))
    with pytest.raises((TypeError, ValueError)):
        mem.memra_kv_fork(five.long(), l, t, 16, r)
    with pytest.raises((TypeError, ValueError)):
        mem.memra_kv_fork(five, l, t[:4], 16, r)
    with pytest.raises((TypeError, ValueError)):
        mem.memra_kv_fork(five, l, t, 16, r, prefix_lens=five[:3])
    with pytest.raises((TypeError, ValueError)):
        mem.memra_kv_unshare(l, five[:4], 16, r, f, t)
    with pytest.raises((TypeError, ValueError)):
        mem.memra_kv_release(l, 16, t, r, f, dev([1, 2]))
    with pytest.raises((TypeError, ValueError)):
        mem.memra_kv_copy_pages(five, five[:4], [c])
    with pytest.raises(ValueError, match="differ"):
        mem.memra_kv_copy_pages(five, five, [c, cache(rs, 7, 2, 16, 64, 4)])
    with pytest.raises((TypeError, ValueError)):
        mem.memra_kv_copy_pages(five, five, [c[:3]])
    with pytest.raises(ValueError):
        mem.memra_kv_compact(l, t, 16, -1)
    for call, status in ((lambda: mem.memra_kv_fork(five, l, t, 20, r), 1), (lambda: mem.memra_kv_fork(five, l, t, 2048, r), 3),
                         (lambda: mem.memra_kv_fork(five, l, t, 16, r, lens_out=l), 1),
                         (lambda: mem.memra_kv_fork(five, l, t, 16, r, table_out=t), 1),
                         (lambda: mem.memra_kv_unshare(l, five, 16, r, f, t, src=l), 1),
                         (lambda: mem.memra_kv_release(l, 16, t, r, r, h), 1),
                         (lambda: mem.memra_kv_compact(l, t, 16, 9, refs_out=(x := dev(np.zeros(9))), free_out=x), 1),
                         (lambda: mem.memra_kv_compact(l, t, 16, 2 ** 30), 3)):
        with pytest.raises(mem.MemraError) as e:
            call()
        assert e.value.status == status
