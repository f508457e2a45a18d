"""Token log probabilities at the limits of their values: infinities and what equals them.  The reference and its tolerances are those
of test_gpu_logprobs.py; every case runs with each number of threads to a row."""
import math

import pytest
import torch

from test_gpu_logprobs import DT, HUGE, check, mem  # noqa: F401 (a fixture)

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
