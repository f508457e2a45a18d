"""Token log probabilities, entropy and top alternatives against 64-bit arithmetic.

Tolerances.  Relative to the largest logit m, a term e^d has d off by 2^-24 |d|, its product with log2 e by as much again, and the
exponential by 2^-22: with W = sum e^d |d| / Z, Z is off by (2 W + 4) 2^-24 from these, and by 2^-24 for every addition that a term
takes part in: V / 256 in a lane (256 threads, the fewest, on a row), 5 exchanges, up to 32 warps in turn and 5 more, and the
rescalings, 12 at most each way.  So ln Z is off by (V / 256 + 2 W + 80) 2^-24 =: E; a log probability by E + 3 * 2^-24 |lp| (two
roundings of its own and the subtraction x - m, which |lp| bounds from above); the entropy by E and the same relative error of the
sum W: (1 + W) E + 3 * 2^-24 H."""
import math

import numpy as np
import pytest
import torch

from _util import Guarded

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HUGE = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module")
def mem():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_decode_quantize_gb300 as m
    from block_quantized_decode_quantize_gb300 import build
    build.build()
    m.lib()
    return m


def reference(x, tokens, n):
    """Rows as numpy, 64 bits: lp, H, ids, top, W."""
    x = x.double().cpu().numpy()
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, HUGE))
    T, V = x.shape
    lp, H, W = np.zeros(T), np.zeros(T), np.zeros(T)
    ids, top = np.zeros((T, n), np.int64), np.zeros((T, n))
    for t in range(T):
        order = np.lexsort((np.arange(V), -x[t]))[:n] if n else np.zeros(0, int)
        ids[t] = order
        m = x[t].max()
        if m == -np.inf:
            lse, d = 0.0, np.full(V, -np.inf)
        else:
            d = x[t] - m
            e = np.exp(d)
            rest = e.sum() - 1.0
            if rest < 1e-6:                              # keep the digits of a sum that is next to 1
                rest = np.delete(e, d.argmax()).sum()
            lse = np.log1p(rest)
            W[t] = -np.where(e > 0, e * np.where(e > 0, d, 0.0), 0.0).sum() / (1.0 + rest)
            H[t] = lse + W[t]
        top[t] = d[order] - lse
        tok = -1 if tokens is None else int(tokens[t])
        lp[t] = 0.0 if tok == -1 else d[tok] - lse if 0 <= tok < V else -np.inf
    return lp, H, ids, top, W


def near(got, want, tol, what):
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got), np.isneginf(want)), what + ": -inf"
    ok = np.isfinite(want)
    err = np.abs(got[ok] - want[ok])
    assert np.isfinite(got[ok]).all() and (err <= tol[ok]).all(), "%s: off by %g, tolerance %g" % (what, err.max(), tol[ok][err.argmax()])


def check(mem, x, tokens, n, status=0, **kw):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lp, H, ids, top = mem.memra_token_logprobs(x, tokens, top_n=n, dev_status=st, **kw)
    T, V = x.shape
    w_lp, w_H, w_ids, w_top, W = reference(x, None if tokens is None else tokens.cpu().numpy(), n)
    E = (V / 256 + 2 * W + 80) * 2.0 ** -24
    assert int(st) == status
    assert np.array_equal(ids.cpu().numpy(), w_ids), "ids"
    with np.errstate(invalid="ignore"):
        if tokens is not None:
            near(lp, w_lp, E + 3 * 2.0 ** -24 * np.abs(w_lp), "logprobs")
        near(H, w_H, (1 + W) * E + 3 * 2.0 ** -24 * w_H, "entropy")
        near(top, w_top, E[:, None] + 3 * 2.0 ** -24 * np.abs(w_top), "top")
    return lp, H, ids, top


def rows(T, V, dtype, seed=0, pad=0, scale=3.0):
    g = torch.Generator().manual_seed(seed * 1000 + V)
    x = (scale * torch.randn(T, V + pad, generator=g)).to(DT[dtype]).cuda()
    tok = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
    return x[:, :V], tok


@pytest.mark.parametrize("V", [1, 2, 5, 8, 31, 32, 33, 255, 256, 257, 513, 1000, 4097, 16384, 16385, 32003, 50257])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,n", [(1, 1), (3, 20), (5, 32), (2, 0)])
def test_sizes(mem, V, dtype, T, n):
    x, tok = rows(T, V, dtype)
    check(mem, x, tok, min(n, V))


@pytest.mark.parametrize("T,V,n", [(1, 151936, 20), (16, 151936, 5), (37, 151937, 32), (160, 32003, 10), (700, 9000, 3), (2, 1048576, 32)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_over_clusters(mem, T, V, n, dtype):
    """Every number of CTAs to a row, and the largest vocabulary."""
    x, tok = rows(T, V, dtype, pad=3)
    check(mem, x, tok, n)


@pytest.mark.parametrize("T", [9, 10, 19, 20, 37, 39, 75, 77, 151, 153])
def test_on_both_sides_of_the_rule(mem, T):
    x, tok = rows(T, 40000, "bf16", seed=T)
    check(mem, x, tok, 8)


@pytest.mark.parametrize("offset", range(9))
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_that_start_anywhere(mem, offset, dtype):
    """Rows at every alignment of their type, with NaN before and behind them."""
    T, V = 4, 1237
    buf = torch.full((offset + T * (V + 5) + 16,), float("nan"), dtype=DT[dtype], device="cuda")
    x, tok = rows(T, V, dtype, seed=offset)
    view = buf[offset:offset + T * (V + 5)].view(T, V + 5)[:, :V]
    view.copy_(x)
    check(mem, view, tok, 7)


def patterns(T, V, seed):
    g = torch.Generator().manual_seed(seed)
    base = 2.0 * torch.randn(T, V, generator=g)
    i = torch.arange(V).float()
    yield "equal", torch.full((T, V), 1.25)
    yield "rising", (i / V * 20).expand(T, V).clone()
    yield "falling", (-i / V * 20).expand(T, V).clone()
    yield "few values", torch.randint(0, 3, (T, V), generator=g).float()
    yield "zeros of both signs", torch.where(torch.rand(T, V, generator=g) < 0.5, 0.0, -0.0)
    x = torch.full((T, V), -math.inf)
    x[:, 3 % V] = 0.5
    yield "one left", x
    x = torch.full((T, V), -math.inf)
    for j in (V - 1, V // 2, V // 3):
        x[:, j] = base[:, j]
    yield "few left", x
    x = torch.full((T, V), -math.inf)
    x[:, V // 4:V // 4 + V // 2] = base[:, V // 4:V // 4 + V // 2]
    yield "a range left", x
    yield "none left", torch.full((T, V), -math.inf)
    x = base.clone()
    x[:, ::7] = math.nan
    yield "NaN", x
    yield "all NaN", torch.full((T, V), math.nan)
    x = base.clone()
    x[:, V // 2] = math.inf
    yield "inf", x
    x = base.clone()
    x[:, ::3] = -3.3e38
    yield "lowest values", x
    yield "all lowest", torch.full((T, V), -3.3e38)
    yield "wide", base * 1e30
    x = base.clone()
    x[:, ::256] += 30.0                                  # the largest all lie in the same place of their segments
    yield "strided", x
    x = base.clone()
    x[:, (V // 8192) * 4096:(V // 8192) * 4096 + 300] += 30.0   # or all in one or two of them
    yield "clustered", x
    x = base.clone()
    x[:, 5 % V] = 60.0
    yield "certain", x


@pytest.mark.parametrize("V", [40, 700, 6000, 16385, 70001])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [4, 32])
def test_patterns(mem, V, dtype, n):
    for i, (name, x) in enumerate(patterns(2, V, V)):
        x = x.to(DT[dtype]).cuda()
        tok = torch.tensor([3 % V, V - 1], dtype=torch.int32, device="cuda")
        try:
            check(mem, x, tok, n)
        except AssertionError as e:
            raise AssertionError("%s: %s" % (name, e))


@pytest.mark.parametrize("T", [303, 304, 305, 607, 608, 609, 1217])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_on_both_sides_of_the_threads_rule(mem, T, dtype):
    x, tok = rows(T, 1900, dtype, seed=T)
    check(mem, x, tok, 6)


@pytest.mark.parametrize("T", [310, 620])
@pytest.mark.parametrize("V,n", [(15359, 5), (15360, 5), (30719, 10), (30720, 10)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_on_both_sides_of_the_rule_for_what_is_read_again(mem, T, V, n, dtype):
    x, tok = rows(T, V, dtype, seed=n, pad=1)
    check(mem, x, tok, n)


@pytest.mark.parametrize("dtype,V", [("bf16", 30719), ("bf16", 30720), ("bf16", 32768), ("bf16", 32769), ("fp32", 16384), ("fp32", 16385)])
@pytest.mark.parametrize("T", [2, 200, 400, 700])
def test_on_both_sides_of_the_rule_for_segments(mem, dtype, V, T):
    """Rows at odd places, and in some of them many elements that are equal or lie close together."""
    for n in (20, 32):
        x, tok = rows(T, V, dtype, seed=T + n, pad=1)
        x[0, V // 2:] = 9.0
        x[1, 100:100 + 600] = x[1, 100:100 + 600] * 0.01 + 20.0
        x[T // 2, :V - n // 2] = -math.inf
        check(mem, x, tok, n)


def staged(T, V, seed):
    """Rows whose first elements, which a warp's sums refer to, say little about the others."""
    g = torch.Generator().manual_seed(seed)
    base = 2.0 * torch.randn(T, V, generator=g)
    for split in (V // 3, V - V // 5):
        for low in (-60.0, -95.0, -150.0, -1000.0, -1e30, -math.inf):
            x = base.clone()
            x[:, :split] += low
            yield "rises by %g at %d" % (-low, split), x
            x = base.clone()
            x[:, split:] += low
            yield "falls by %g at %d" % (-low, split), x
    x = base - 400.0
    x[:, ::V // 7] = 3.0
    yield "spikes", x
    x = torch.full((T, V), -math.inf)
    x[:, V - 40:] = base[:, V - 40:] - 300.0
    yield "masked up to a low end", x
    for level in (2.0 ** 19, 2.0 ** 21, -2.0 ** 21, 1e25, -1e25):
        yield "at the level %g" % level, base * max(1.0, abs(level) * 2.0 ** -20) + level


@pytest.mark.parametrize("V,T", [(1500, 2), (5001, 650), (40000, 310), (70001, 3), (151936, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_references_far_from_the_maximum(mem, V, T, dtype):
    """In all kernels' shapes; the rows of a case are the same three, so that the plain form is short."""
    for name, x in staged(min(T, 3), V, V):
        x = x.to(DT[dtype])
        some = x.shape[0]
        tok = torch.tensor([V - 1, 0, V // 2][:some], dtype=torch.int32)
        try:
            lp, H, ids, top = check(mem, x.cuda(), tok.cuda(), 5)
            if T > some:
                again = T // some
                many = mem.memra_token_logprobs(x.cuda().repeat(again, 1), tok.cuda().repeat(again), top_n=5)
                w_lp, w_H, w_ids, w_top, W = reference(x, tok.numpy(), 5)
                E = (V / 256 + 2 * W + 80) * 2.0 ** -24
                for r in (0, again // 2, again - 1):
                    part = slice(r * some, (r + 1) * some)
                    assert np.array_equal(many[2][part].cpu().numpy(), w_ids)
                    near(many[0][part], w_lp, E + 3 * 2.0 ** -24 * np.abs(w_lp), "logprobs")
                    near(many[1][part], w_H, (1 + W) * E + 3 * 2.0 ** -24 * w_H, "entropy")
        except AssertionError as e:
            raise AssertionError("%s: %s" % (name, e))


def test_log_probabilities_near_zero_keep_their_digits(mem):
    """-lp of a token that is almost certain is the others' mass, relative to its own size: each of its terms is off by
    (2 * 25 + 4) 2^-24 and the sum by the additions' share, 2 ^-24 (V / 256 + 40)."""
    V = 50000
    g = torch.Generator().manual_seed(8)
    x = torch.randn(6, V, generator=g)
    at = [0, 1, 777, 25000, 49998, 49999]
    for t, j in enumerate(at):
        x[t, j] = 25.0 + 0.5 * t
    tok = torch.tensor(at, dtype=torch.int32).cuda()
    lp, H, ids, top = mem.memra_token_logprobs(x.cuda(), tok, top_n=1)
    want = reference(x, tok.cpu().numpy(), 1)
    tol = (54 + V / 256 + 40) * 2.0 ** -24
    assert np.abs(lp.double().cpu().numpy() / want[0] - 1).max() < tol and np.abs(H.double().cpu().numpy() / want[1] - 1).max() < 2 * tol
    assert torch.equal(top[:, 0], lp) and ids[:, 0].tolist() == at


def test_tokens_out_of_range(mem):
    x, _ = rows(5, 300, "fp32")
    tok = torch.tensor([0, -1, 300, -2, 299], dtype=torch.int32).cuda()
    lp, *_ = check(mem, x, tok, 2, status=1)
    assert float(lp[1]) == 0.0 and bool(torch.isneginf(lp[2:4]).all())


def test_without_tokens_or_top(mem):
    x, tok = rows(3, 5000, "bf16")
    a = mem.memra_token_logprobs(x, tok, top_n=3)
    b = mem.memra_token_logprobs(x, top_n=3)
    assert b[0] is None and all(torch.equal(p, q) for p, q in zip(a[1:], b[1:]))
    c = mem.memra_token_logprobs(x, tok)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1]) and c[2].shape == (3, 0)
    empty = mem.memra_token_logprobs(x[:0], tok[:0], top_n=3)
    assert empty[0].shape == (0,) and empty[2].shape == (0, 3)


def test_outputs_given_and_nothing_beside_them(mem):
    x, tok = rows(70, 9001, "fp32", pad=1)
    want = mem.memra_token_logprobs(x, tok, top_n=5)
    g = [Guarded((70,), torch.float32), Guarded((70,), torch.float32), Guarded((70, 5), torch.int32), Guarded((70, 5), torch.float32)]
    got = mem.memra_token_logprobs(x, tok, top_n=5, logprobs=g[0].view, entropy=g[1].view, top_ids=g[2].view, top_logprobs=g[3].view)
    assert all(o.intact() for o in g) and all(torch.equal(a, b) for a, b in zip(want, got))


def test_rows_are_independent_and_repeatable(mem):
    """A row's results do not depend on the rows beside it where as many CTAs take it, nor on the run."""
    x, tok = rows(200, 30000, "bf16")
    a = mem.memra_token_logprobs(x, tok, top_n=6)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(a, mem.memra_token_logprobs(x, tok, top_n=6)))
    perm = torch.randperm(200, generator=torch.Generator().manual_seed(1)).cuda()
    b = mem.memra_token_logprobs(x[perm], tok[perm], top_n=6)
    assert all(torch.equal(p[perm], q) for p, q in zip(a, b))


def test_offsets_past_32_bits(mem):
    """Rows whose bytes lie past 2^32: a stride of 2^21 elements (fp32) over 600 rows."""
    T, V, stride = 600, 5000, 1 << 21
    buf = torch.empty(T * stride, dtype=torch.float32, device="cuda")
    x = buf.view(T, stride)[:, :V]
    small, tok = rows(T, V, "fp32")
    x.copy_(small)
    a, b = mem.memra_token_logprobs(x, tok, top_n=4), mem.memra_token_logprobs(small, tok, top_n=4)
    assert torch.equal(a[2], b[2])
    for p, q in zip((a[0], a[1], a[3]), (b[0], b[1], b[3])):
        assert torch.allclose(p, q, rtol=1e-5, atol=1e-5)


def test_streams_and_graphs(mem):
    x, tok = rows(16, 151936, "fp32")
    want = mem.memra_token_logprobs(x, tok, top_n=20)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = mem.memra_token_logprobs(x, tok, top_n=20)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mem.memra_token_logprobs(x, tok, top_n=20)
        twice = mem.memra_token_logprobs(x, tok, top_n=20)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, out, twice))


def test_refusals(mem):
    x, tok = rows(4, 50, "fp32")
    call = mem.memra_token_logprobs
    with pytest.raises(TypeError):
        call(x.half(), tok)
    with pytest.raises(ValueError, match="dense"):
        call(x.t().contiguous().t(), tok)
    with pytest.raises(ValueError, match="top_n"):
        call(x, tok, top_n=51)
    with pytest.raises(ValueError, match="top_n"):
        call(x, tok, top_n=-1)
    with pytest.raises((TypeError, ValueError)):
        call(x, tok.long())
    with pytest.raises((TypeError, ValueError)):
        call(x, tok[:3])
    with pytest.raises(ValueError, match="tokens"):
        call(x, None, logprobs=torch.empty(4, device="cuda"))
    with pytest.raises(mem.MemraError) as e:
        call(x, tok, top_n=33)
    assert e.value.status == 3
    with pytest.raises(mem.MemraError) as e:
        call(torch.zeros(1, 2 ** 20 + 1, device="cuda"), tok[:1])
    assert e.value.status == 3
