"""Token log probabilities at the limits of their values: infinities and what equals them.  The reference and its tolerances are those
of test_gpu_logprobs.py; every case runs with each number of threads to a row."""
import math

import numpy as np
import pytest
import torch

from test_gpu_logprobs import DT, HUGE, check, mem, reference  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
ROWS = (2, 200, 400, 700)   # a cluster or CTAs of 512, 256 and 128 threads to a row


def infinities(V):
    g = torch.Generator().manual_seed(V)
    base = 2.0 * torch.randn(2, V, generator=g)
    yield "all", torch.full((2, V), math.inf)
    some = torch.rand(2, V, generator=g) < 0.5
    yield "half", torch.where(some, math.inf, base)
    yield "half, the others masked", torch.where(some, math.inf, -math.inf)
    yield "beside the largest finite value", torch.where(some, math.inf, HUGE)
    x = base.clone()
    x[:, 0], x[:, 1 % V] = HUGE, math.inf
    yield "one behind the largest finite value", x
    x = base.clone()
    x[:, V - 1], x[:, V // 2] = math.inf, HUGE
    yield "one at the end", x
    x = torch.full((2, V), -math.inf)
    x[:, :256], x[:, 256:768] = HUGE, math.inf
    yield "two blocks behind one of the largest finite value", x
    x = torch.full((2, V), math.nan)
    x[:, V // 3:V // 3 + 600] = math.inf
    x[:, V // 3 + 5:V // 3 + 9] = HUGE
    yield "a range among no numbers", x


@pytest.mark.parametrize("V", [4, 40, 600, 5000, 16385, 70001])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 5, 32])
def test_infinities_tie_with_the_largest_finite_value(mem, V, dtype, n):
    """Ids are the lowest indexes among equals, more than 512 of them or fewer (bf16's own largest is less than fp32's,
    which +inf counts as, and HUGE rounds to +inf there)."""
    for name, x in infinities(V):
        x = x.to(DT[dtype]).cuda()
        tok = torch.tensor([V - 1, V // 2], dtype=torch.int32, device="cuda")
        try:
            _, _, ids, _ = check(mem, x, tok, min(n, V))
            for T in ROWS[1:]:
                many = mem.memra_token_logprobs(x.repeat(T // 2, 1), tok.repeat(T // 2), top_n=min(n, V))
                assert torch.equal(many[2], ids.repeat(T // 2, 1)), "ids of %d rows" % T
        except AssertionError as e:
            raise AssertionError("%s: %s" % (name, e))


def tails(mem, name, x, top, dtype):
    """The log probability and the entropy of rows whose token `top` is almost certain, relative to their own size.  A term 2^u, |u| <= 128
    from what a warp's sums refer to, is off by ln 2 2^-18 = 45 2^-24 from u's rounding, by 27 2^-24 from log2 e's in fp32 (|d| <= 106, 2^-26 |d|),
    4 2^-24 from the exponential, and each addition that it takes part in: V / 128 in a lane, 40 in the joins, 10 in what follows: E.  The
    entropy's terms are these times u, as a difference of two numbers up to 5 times as large: 6 E."""
    x = x.to(DT[dtype])[None]
    V = x.shape[1]
    want = reference(x, np.array([top]), 1)
    E = (126 + V / 128) * 2.0 ** -24
    for T in ROWS:
        tok = torch.full((T,), top, dtype=torch.int32, device="cuda")
        lp, H, ids, _ = mem.memra_token_logprobs(x.cuda().expand(T, V), tok, top_n=1)
        assert bool((ids == top).all())
        for what, got, w, tol in (("log probability", lp, want[0][0], E), ("entropy", H, want[1][0], 6 * E)):
            off = float((got.double() / w - 1).abs().max())
            assert off <= tol, "%s, %d rows: %s off by %g of %g, tolerance %g" % (name, T, what, off, w, tol)


@pytest.mark.parametrize("V,masked", [(60000, 17000), (151936, 76000), (60000, 59960)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_tails_behind_masked_tokens(mem, V, masked, dtype):
    """Every warp's first logits, or all but a few, are masked, and those that are left are far below 0."""
    g = torch.Generator().manual_seed(V)
    for high, low in ((-69.0, -87.6), (-55.0, -80.0), (-69.0, -94.0), (-3.0, -28.0), (40.0, 20.0), (-160.0, -180.0)):
        x = low + 0.2 * torch.randn(V, generator=g)
        x[:masked] = -math.inf
        x[V - 7] = high
        tails(mem, "%g over %g" % (high, low), x, V - 7, dtype)


@pytest.mark.parametrize("V", [60000, 151936])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_tails_far_above_what_their_sums_refer_to(mem, V, dtype):
    """A warp's first logits are up to 150 powers of two below the row's largest, its others less than 90."""
    g = torch.Generator().manual_seed(V)
    for rise, high in ((66.0, 106.0), (60.0, 104.0), (30.0, 60.0), (66.0, 90.0), (39.0, 99.0), (41.0, 95.0), (45.0, 95.0)):
        x = 0.5 * torch.randn(V, generator=g)
        x[V // 2:] += rise
        x[V // 5] = high
        tails(mem, "%g over %g" % (high, rise), x, V // 5, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", ROWS)
@pytest.mark.parametrize("level", [1.2345, -7.77])
def test_sums_of_equal_terms(mem, dtype, T, level):
    """Equal logits, whose sums round the same way throughout.  A term takes part in 16 additions of its batch (64 bytes a lane, two
    halves), one for each further batch of a lane (V / 2048 in fp32, V / 4096 in bf16, with the fewest threads, 128, on a row), and 15 in the
    joins; it is off by 6 2^-24 itself.  The entropy is ln V too; its second sum is 0 but for twice as much."""
    V = 151936
    x = torch.full((1, V), level).to(DT[dtype])
    E = (16 + V / (2048 if dtype == "fp32" else 4096) + 15 + 6) * 2.0 ** -24
    tok = torch.full((T,), V - 1, dtype=torch.int32, device="cuda")
    lp, H, ids, top = mem.memra_token_logprobs(x.cuda().expand(T, V), tok, top_n=2)
    half = 2.0 ** -24 * math.log(V)                      # the result's own rounding
    assert ids.tolist() == [[0, 1]] * T
    for got, want, tol in ((lp, -math.log(V), E + half), (top, -math.log(V), E + half), (H, math.log(V), 3 * E + half)):
        assert float((got.double() - want).abs().max()) <= tol
