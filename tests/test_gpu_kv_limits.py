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
