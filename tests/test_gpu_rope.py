"""Norm and rotation of queries and keys against the formula in 64 bits.

Tolerances.  n = x r w: the sum of squares of D values is off by 13 roundings at most (8 in a lane, 5 exchanges), its root by
half of that, the reciprocal root by 2 ulp (2^-22), and three more roundings follow, so n is off by 11 * 2^-24 + 2^-22.  The rotation
rounds three times, and sine and cosine are off by 2 ulp (2^-22) and the angle's 2^-22: together 18 * 2^-24 + 3 * 2^-22 = 30 * 2^-24,
less than 2^-19, of |n_a| + |n_b|.  bf16 output adds half a step, 2^-8 of the
value."""
import math

import numpy as np
import pytest
import torch

from _util import Guarded

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def mem():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_decode_quantize_gb300 as m
    from block_quantized_decode_quantize_gb300 import build
    build.build()
    m.lib()
    return m


def reference(x, pos, freq, weight, eps, layout):
    """(result, |n_a| + |n_b| of each value) in 64 bits."""
    x = x.double().cpu()
    if eps is not None:
        ms = x.square().mean(-1, keepdim=True) + eps
        x = torch.where(ms > 0, x / ms.clamp(min=1e-300).sqrt(), 0.0)
        if weight is not None:
            x = x * weight.double().cpu()
    size = x.abs()
    if freq is not None and freq.numel():
        R = 2 * freq.numel()
        ang = pos.cpu().double()[:, None, None] * freq.cpu()
        c, s = ang.cos(), ang.sin()
        a, b = (x[..., :R // 2], x[..., R // 2:R]) if layout == "halves" else (x[..., 0:R:2], x[..., 1:R:2])
        ra, rb, both = a * c - b * s, b * c + a * s, a.abs() + b.abs()
        x, size = x.clone(), size.clone()
        if layout == "halves":
            x[..., :R // 2], x[..., R // 2:R] = ra, rb
            size[..., :R // 2], size[..., R // 2:R] = both, both
        else:
            x[..., 0:R:2], x[..., 1:R:2] = ra, rb
            size[..., 0:R:2], size[..., 1:R:2] = both, both
    if pos is not None:
        x[pos.cpu() < 0] = 0.0
    return x, size


def check(got, want, size, what):
    tol = size * 2.0 ** -19 + (want.abs() * 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0) + 1e-37
    err = (got.double().cpu() - want).abs()
    assert bool((err <= tol).all()), "%s: %g over" % (what, float((err - tol).max()))


def freqs(R, base=10000.0):
    j = torch.arange(R // 2, dtype=torch.float64)
    return (base ** (-2.0 * j / R)).cuda()


def case(T, Hq, Hkv, D, R, dtype, seed=0, far=5000, norm=True, size=1.0):
    g = torch.Generator().manual_seed(seed)
    rows = (size * torch.randn(T, (Hq + 2 * Hkv) * D, generator=g)).to(DT[dtype]).cuda()
    q = rows[:, :Hq * D].view(T, Hq, D)
    k = rows[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    pos = torch.randint(0, far, (T,), generator=g, dtype=torch.int32).cuda()
    w = [(1 + 0.3 * torch.randn(D, generator=g)).cuda() for _ in range(2)] if norm else [None, None]
    return rows, q, k, pos, freqs(R) if R else None, w


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("layout", ["halves", "pairs"])
@pytest.mark.parametrize("part", [1.0, 0.5, 0.25, 0.0])
@pytest.mark.parametrize("dtype,qd,kd", [("fp32", "bf16", "fp32"), ("bf16", "bf16", "bf16"), ("bf16", "fp32", "fp32")])
def test_layouts_and_types(mem, D, layout, part, dtype, qd, kd):
    R = int(part * D)
    _, q, k, pos, f, w = case(5, 7, 3, D, R, dtype, seed=D + R)
    qo, ko = mem.memra_qk_norm_rope(q, k, pos, f, q_weight=w[0], k_weight=w[1], eps=1e-6, layout=layout, q_dtype=DT[qd],
                                    k_dtype=DT[kd])
    assert qo.dtype == DT[qd] and ko.dtype == DT[kd]
    for x, o, wt in ((q, qo, w[0]), (k, ko, w[1])):
        check(o, *reference(x, pos, f, wt, 1e-6, layout), "D %d R %d" % (D, R))


@pytest.mark.parametrize("T", [1, 2, 3, 16, 303, 304, 305, 700, 1217, 3001])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (40, 8), (33, 1)])
def test_rows_and_heads(mem, T, Hq, Hkv):
    """Both sides of the grid's rule (a CTA to a token's heads or to several tokens), odd numbers of heads."""
    D = 128 if T < 1000 else 64
    _, q, k, pos, f, w = case(T, Hq, Hkv, D, D, "bf16", seed=T)
    pos[T // 2:T // 2 + 2] = -1
    qo, ko = mem.memra_qk_norm_rope(q, k, pos, f, q_weight=w[0], k_weight=w[1], eps=1e-5)
    for x, o, wt in ((q, qo, w[0]), (k, ko, w[1])):
        check(o, *reference(x, pos, f, wt, 1e-5, "halves"), "T %d" % T)
        assert bool((o[pos < 0] == 0).all())


@pytest.mark.parametrize("T", [2431, 2432, 2437, 4863, 4864, 4866, 4881])
@pytest.mark.parametrize("Hq,Hkv,D,layout,dtype", [(1, 1, 128, "halves", "bf16"), (4, 4, 128, "pairs", "fp32"), (16, 1, 64, "halves", "fp32"),
                                                   (8, 1, 128, "halves", "bf16"), (3, 0, 256, "pairs", "bf16")])
def test_few_heads_of_many_tokens(mem, T, Hq, Hkv, D, layout, dtype):
    """Several sets of tokens to a CTA, the last of them cut anywhere; beside what is compared, the rows of
    tokens alone are the same bits."""
    _, q, k, pos, f, w = case(T, Hq, Hkv, D, D // 2, dtype, seed=T + D)
    pos[T - 3] = -1
    norm = dict(q_weight=w[0], k_weight=w[1], eps=1e-5, layout=layout)
    qo, ko = mem.memra_qk_norm_rope(q, k, pos, f, **norm)
    for x, o, wt in ((q, qo, w[0]), (k, ko, w[1])):
        if x.shape[1]:
            check(o, *reference(x, pos, f, wt, 1e-5, layout), "T %d" % T)
    for t0, t1 in ((0, 1), (5, 7), (T - 5, T)):
        a, b = mem.memra_qk_norm_rope(q[t0:t1], k[t0:t1], pos[t0:t1], f, **norm)
        assert torch.equal(a, qo[t0:t1]) and torch.equal(b, ko[t0:t1])


@pytest.mark.parametrize("R", [8, 24, 40, 72, 120, 128])
@pytest.mark.parametrize("layout", ["halves", "pairs"])
def test_any_rotated_part(mem, R, layout):
    _, q, k, pos, f, _ = case(9, 4, 2, 128, R, "fp32", seed=R, norm=False)
    qo, ko = mem.memra_qk_norm_rope(q, k, pos, f, layout=layout)
    for x, o in ((q, qo), (k, ko)):
        check(o, *reference(x, pos, f, None, None, layout), "R %d" % R)
        assert torch.equal(o[..., R:], x[..., R:])


@pytest.mark.parametrize("pos", [0, 1, 131071, 1000003, 2 ** 24 + 1, 2 ** 31 - 1])
def test_far_positions(mem, pos):
    """Angles far out: in fp32 pos * freq would be off by up to 128 radians at the last."""
    _, q, k, _, _, _ = case(3, 2, 2, 64, 64, "fp32", norm=False)
    p = torch.full((3,), pos, dtype=torch.int32, device="cuda")
    f = torch.tensor([1.0, 0.73, 2.5, 1e-4] * 8, dtype=torch.float64, device="cuda")
    qo, _ = mem.memra_qk_norm_rope(q, k, p, f)
    want, size = reference(q, p, f, None, None, "halves")
    err = (qo.double().cpu() - want).abs()
    # the angle in 64 bits is itself off by pos * freq * 2^-53, the kernel's by twice that
    assert bool((err <= size * (2.0 ** -19 + pos * 2.5 * 2.0 ** -51) + 1e-37).all())


def test_frequencies_of_any_sign_and_size(mem):
    _, q, k, pos, _, _ = case(6, 2, 1, 64, 64, "fp32", far=100, norm=False)
    f = torch.tensor([-1.0, 7.5, 0.0, -1e-9, 100.0, 6.283185307179586, 1e-300, -0.0] * 4, dtype=torch.float64, device="cuda")
    qo, ko = mem.memra_qk_norm_rope(q, k, pos, f, layout="pairs")
    for x, o in ((q, qo), (k, ko)):
        check(o, *reference(x, pos, f, None, None, "pairs"), "frequencies")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 4, 401])
def test_in_place_within_the_projection(mem, T, dtype):
    """K stays beside V with its strides, Q too; V and what lies beside are left alone."""
    rows, q, k, pos, f, w = case(T, 6, 2, 128, 64, dtype, seed=3)
    before = rows.clone()
    want = mem.memra_qk_norm_rope(q, k, pos, f, q_weight=w[0], k_weight=w[1], eps=1e-6)
    qo, ko = mem.memra_qk_norm_rope(q, k, pos, f, q_weight=w[0], k_weight=w[1], eps=1e-6, q_out=q, k_out=k)
    assert qo.data_ptr() == q.data_ptr() and ko.data_ptr() == k.data_ptr() and ko.stride() == k.stride()
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1]) and torch.equal(rows[:, 8 * 128:], before[:, 8 * 128:])


def test_outputs_with_strides_of_their_own(mem):
    """Heads first, and rows with room between them, which stays as it was."""
    _, q, k, pos, f, w = case(10, 4, 2, 64, 64, "fp32", seed=9)
    want = mem.memra_qk_norm_rope(q, k, pos, f, eps=1e-6)
    qo = torch.empty(4, 10, 64, device="cuda").transpose(0, 1)
    room = torch.full((10, 2, 96), 7.0, device="cuda", dtype=torch.float32)
    mem.memra_qk_norm_rope(q, k, pos, f, eps=1e-6, q_out=qo, k_out=room[..., :64])
    assert torch.equal(qo, want[0]) and torch.equal(room[..., :64], want[1]) and bool((room[..., 64:] == 7).all())


def test_nothing_is_written_beside_the_outputs(mem):
    for T, Hq, Hkv, D in ((1, 5, 1, 64), (307, 3, 1, 128), (1300, 1, 2, 256)):
        _, q, k, pos, f, _ = case(T, Hq, Hkv, D, D, "bf16", seed=T)
        qo, ko = Guarded((T, Hq, D), torch.bfloat16), Guarded((T, Hkv, D), torch.float32)
        mem.memra_qk_norm_rope(q, k, pos, f, eps=1e-6, q_out=qo.view, k_out=ko.view)
        want = mem.memra_qk_norm_rope(q, k, pos, f, eps=1e-6, k_dtype=torch.float32)
        assert qo.intact() and ko.intact() and torch.equal(qo.view, want[0]) and torch.equal(ko.view, want[1])


def test_queries_alone_and_broadcast_rows(mem):
    _, q, k, pos, f, w = case(7, 4, 2, 64, 64, "bf16", seed=1)
    want, _ = mem.memra_qk_norm_rope(q, k, pos, f, q_weight=w[0], eps=1e-6)
    out, none = mem.memra_qk_norm_rope(q, None, pos, f, q_weight=w[0], eps=1e-6)
    assert none is None and torch.equal(out, want)
    one = q[:1].expand(7, 4, 64)                         # every row the same memory
    got, _ = mem.memra_qk_norm_rope(one, k, pos, f, eps=1e-6)
    full, _ = mem.memra_qk_norm_rope(one.contiguous(), k, pos, f, eps=1e-6)
    assert torch.equal(got, full)
    empty, _ = mem.memra_qk_norm_rope(q[:0], k[:0], pos[:0], f, eps=1e-6)
    assert empty.shape == (0, 4, 64)


def test_zeros_small_and_large_values(mem):
    """A zero row stays zero with and without eps; values to 2^60 keep their norm; padded rows' inputs may be anything."""
    q = torch.zeros(6, 2, 64, device="cuda")
    q[1] = 2.0 ** 60
    q[2] = 2.0 ** -60
    q[3, :, 5] = 1.0
    q[4] = float("nan")
    pos = torch.tensor([3, 3, 3, 0, -1, 9], dtype=torch.int32, device="cuda")
    for eps in (0.0, 1e-6):
        out, _ = mem.memra_qk_norm_rope(q, q.clone(), pos, freqs(64), eps=eps)
        clean = torch.where(torch.isnan(q), 0.0, q)
        check(out, *reference(clean, pos, freqs(64), None, eps, "halves"), "eps %g" % eps)
        assert bool((out[0] == 0).all()) and bool((out[4] == 0).all())


def test_without_positions(mem):
    _, q, k, _, _, w = case(11, 3, 1, 128, 0, "bf16", seed=4)
    qo, ko = mem.memra_qk_norm_rope(q, k, q_weight=w[0], k_weight=w[1], eps=1e-6)
    for x, o, wt in ((q, qo, w[0]), (k, ko, w[1])):
        check(o, *reference(x, None, None, wt, 1e-6, "halves"), "norm alone")


def test_refusals(mem):
    _, q, k, pos, f, w = case(4, 4, 2, 64, 64, "bf16")
    call = mem.memra_qk_norm_rope
    with pytest.raises(TypeError):
        call(q.half(), k.half(), pos, f)
    with pytest.raises(ValueError, match="k must"):
        call(q, k.float(), pos, f)
    with pytest.raises(ValueError, match="k must"):
        call(q, k[:3], pos, f)
    with pytest.raises(ValueError, match="layout"):
        call(q, k, pos, f, layout="both")
    with pytest.raises(ValueError, match="positions"):
        call(q, k, None, f)
    with pytest.raises((TypeError, ValueError)):
        call(q, k, pos.long(), f)
    with pytest.raises((TypeError, ValueError)):
        call(q, k, pos, f.float())
    with pytest.raises(ValueError, match="eps"):
        call(q, k, pos, f, q_weight=w[0])
    with pytest.raises(ValueError, match="eps"):
        call(q, k, pos, f, eps=-1.0)
    with pytest.raises((TypeError, ValueError)):
        call(q, k, pos, f, eps=1e-6, q_weight=w[0].bfloat16())
    with pytest.raises(TypeError):
        call(q, k, pos, f, q_dtype=torch.float16)
    with pytest.raises(TypeError):
        call(q, k, pos, f, q_dtype=torch.float32, q_out=torch.empty_like(q))
    with pytest.raises(ValueError, match="q_out"):
        call(q, k, pos, f, q_out=torch.empty(4, 4, 32, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="dense"):
        call(q.transpose(1, 2).contiguous().transpose(1, 2), k, pos, f)
    for bad, status in ((dict(q_out=k.expand(4, 2, 64)[:, :1].expand(4, 4, 64)), 1), (dict(k_out=q[:, 1:3]), 1)):
        with pytest.raises(mem.MemraError) as e:
            call(q, k, pos, f, **bad)
        assert e.value.status == status
    with pytest.raises(mem.MemraError) as e:
        call(q[..., :48], k[..., :48], pos, f[:16])
    assert e.value.status == 3
    shifted = torch.zeros(4 * 4 * 64 + 8, device="cuda", dtype=torch.bfloat16)[4:4 + 4 * 4 * 64].view(4, 4, 64)
    with pytest.raises(mem.MemraError) as e:
        call(shifted, k, pos, f)
    assert e.value.status == 2


def test_other_streams_and_graphs(mem):
    _, q, k, pos, f, w = case(16, 8, 2, 128, 128, "fp32", seed=2)
    want = mem.memra_qk_norm_rope(q, k, pos, f, q_weight=w[0], k_weight=w[1], eps=1e-6, q_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = mem.memra_qk_norm_rope(q, k, pos, f, q_weight=w[0], k_weight=w[1], eps=1e-6, q_dtype=torch.bfloat16)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mem.memra_qk_norm_rope(q, k, pos, f, q_weight=w[0], k_weight=w[1], eps=1e-6, q_dtype=torch.bfloat16)
    pos += 11
    graph.replay()
    torch.cuda.synchronize()
    again = mem.memra_qk_norm_rope(q, k, pos, f, q_weight=w[0], k_weight=w[1], eps=1e-6, q_dtype=torch.bfloat16)
    assert all(torch.equal(a, b) for a, b in zip(out, again)) and not torch.equal(out[0], want[0])
    assert math.isfinite(float(np.abs(out[1].cpu().numpy()).max()))
