"""Norm and rotation at the limits of their values.  The reference and its tolerances are those of test_gpu_rope.py."""

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
