"""Norm and rotation at the limits of their values.  The reference and its tolerances are those of test_gpu_rope.py."""
import math

import pytest
import torch

from test_gpu_rope import DT, case, check, mem, reference  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
TOKENS = (1, 700, 2500)     # one, two and four tokens to a CTA


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", TOKENS)
def test_heads_full_of_the_largest_values(mem, D, dtype, T):
    """|x| = 2^60 throughout, the mean of whose squares is 2^120, and 2^-60 with small values beside."""
    _, q, k, pos, f, w = case(T, 3, 2, D, D // 2, dtype, seed=D)
    q, k = q.sign() * 2.0 ** 60, k * 2.0 ** -60 / k.float().abs().max(-1, keepdim=True).values.to(k.dtype)
    for eps in (0.0, 1e-6):
        qo, ko = mem.memra_qk_norm_rope(q, k, pos, f, q_weight=w[0], k_weight=w[1], eps=eps, q_dtype=torch.float32, k_dtype=torch.float32)
        for x, o, wt in ((q, qo, w[0]), (k, ko, w[1])):
            check(o, *reference(x, pos, f, wt, eps, "halves"), "eps %g" % eps)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R", [0, 32])
@pytest.mark.parametrize("T", TOKENS)
def test_what_is_no_number_stays_none(mem, D, dtype, R, T):
    """A NaN makes its head's mean, and so all of the head, no number; an infinity makes itself none and the others 0.
    Other heads and tokens are as without."""
    _, q, k, pos, f, w = case(T, 3, 2, D, R, dtype, seed=D)
    norm = dict(q_weight=w[0], k_weight=w[1], eps=1e-6)
    want = mem.memra_qk_norm_rope(q, k, pos, f, **norm)
    q = q.clone()
    t, u = T // 3, T - 1
    q[t, 0, D - 1] = math.nan
    q[u, 2, D - 2] = -math.inf
    qo, ko = mem.memra_qk_norm_rope(q, k, pos, f, **norm)
    assert bool(torch.isnan(qo[t, 0]).all())
    got = qo[u, 2].float()
    assert bool(torch.isnan(got[D - 2])) and bool((got[:D - 2] == 0).all()) and bool((got[D - 1:] == 0).all())
    qo[t, 0], qo[u, 2] = want[0][t, 0], want[0][u, 2]
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
