"""Token log probabilities: outputs that overlap something are refused (host-side checks, no GPU)."""
import pytest

A = 0x7f0000000000     # never dereferenced: every call below is refused, or has no device to run on
M = 1 << 28            # between arrays, farther than any of them is long


@pytest.fixture(scope="module")
def L():
    import block_quantized_decode_quantize_gb300 as m
    from block_quantized_decode_quantize_gb300 import build
    build.build()
    return m.lib()


def call(L, x=A, dt=1, T=5, V=100, st=128, tok=A + M, n=3, lp=A + 2 * M, h=A + 3 * M, ids=A + 4 * M, top=A + 5 * M, status=None):
    return L.memra_token_logprobs(x, dt, T, V, st, tok, n, lp, h, ids, top, status, None)


def test_outputs_that_overlap_are_refused(L):
    for name in ("lp", "h", "ids", "top", "status"):
        for at in (A, A + 4 * (4 * 128 + 99), A + 4 * 130, A + 4 * 99, A + M, A + M + 16):
            assert call(L, **{name: at}) == 1, (name, at - A)
    assert call(L, h=A + 2 * M) == 1 and call(L, h=A + 2 * M + 16) == 1 and call(L, lp=A + 3 * M + 16) == 1
    assert call(L, top=A + 4 * M) == 1 and call(L, top=A + 4 * M + 56) == 1 and call(L, ids=A + 5 * M + 56) == 1
    assert call(L, status=A + 5 * M + 56) == 1 and call(L, status=A + 2 * M + 16) == 1 and call(L, ids=A + 2 * M - 56) == 1
    assert call(L, x=A + M + 16, tok=A, h=A + M) == 1    # an output that begins before the logits and reaches them
    assert call(L, st=0, h=A + 396) == 1 and call(L, st=100, h=A + 4 * 300) == 1 and call(L, st=100, h=A + 4 * 496) == 1
    assert call(L, dt=0, h=A + 2 * (4 * 128 + 98)) == 1
    assert call(L, h=A + 4 * 124, T=5) == 1              # begins between two rows and reaches the second


def test_outputs_beside_others_pass_the_checks(L):
    """Refusals come before the launch, which has no device here (4)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch")
    assert call(L) == 4
    assert call(L, h=A + 2 * M + 20) == 4 and call(L, top=A + 4 * M + 60) == 4 and call(L, status=A + 2 * M + 20) == 4
    assert call(L, h=A + 4 * (4 * 128 + 100)) == 4 and call(L, h=A - 20) == 4 and call(L, h=A + M + 20) == 4
    assert call(L, h=A + 4 * 100) == 4 and call(L, h=A + 4 * (128 + 123)) == 4   # 20 bytes between two rows
    assert call(L, st=0, h=A + 400) == 4 and call(L, dt=0, h=A + 2 * (4 * 128 + 100)) == 4
    assert call(L, n=0, ids=None, top=None) == 4 and call(L, n=0, ids=A, top=A) == 4 and call(L, tok=None, lp=None, h=A + M) == 4
    assert call(L, st=50) == 4 and call(L, T=1, st=0) == 4           # rows may share memory
