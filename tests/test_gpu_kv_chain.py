"""The cache, attention and routing calls as a server makes them: one after another on a stream and
in a CUDA graph; at the sizes where the attention kernels change; with codes far into a large pool;
and when a wait of the many-row kernel runs out at any point of its work."""
import numpy as np
import pytest
import torch

from test_gpu_kv_route import attention_case, check_attention, dev

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
# A step's calls back to back.
# ---------------------------------------------------------------------------

class Step:
    """Plan, write, attention, read-back, an O product and routing on the attention's output."""

    def __init__(self, mem, new, G, dtype, B=6, Hkv=4, D=64, P=16, S=8, seed=0):
        rs = np.random.RandomState(seed)
        g = torch.Generator().manual_seed(seed)
        self.mem, self.P, self.T, self.D = mem, P, B * new, D
        ctx = rs.randint(1, 200, B)
        have = -(-ctx // P)
        pages = int((-(-(ctx + new) // P)).sum()) + 2
        ids = rs.permutation(pages)
        table = np.full((B, 16), -1, np.int64)
        at = 0
        for b in range(B):
            table[b, :have[b]] = ids[at:at + have[b]]
            at += have[b]
        self.start = dict(lens=dev(ctx, i32), table=dev(table, i32), head=dev([0], i32),
                          kq=torch.randint(-127, 128, (pages, Hkv, P, D), generator=g, dtype=torch.int8).cuda(),
                          vq=torch.randint(-127, 128, (pages, Hkv, P, D), generator=g, dtype=torch.int8).cuda(),
                          kd=torch.rand(pages, Hkv, P // S, generator=g).cuda() * 0.02,
                          vd=torch.rand(pages, Hkv, P // S, generator=g).cuda() * 0.02)
        self.now = {k: v.clone() for k, v in self.start.items()}
        self.new, self.free = torch.full((B,), new, dtype=i32, device="cuda"), dev(ids[at:], i32)
        tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.qkv = torch.randn(self.T, (G + 2) * Hkv, D, generator=g).to(tdt).cuda()
        self.heads, self.kv = G * Hkv, Hkv
        self.o = mem.memra_quantize_q8_0(torch.randn(256, self.heads * D, generator=g).cuda())
        self.ws = torch.zeros(mem.KV_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
        self.status = torch.zeros(1, dtype=i32, device="cuda")

    def run(self, sync=False):
        def step(v):
            if sync:
                torch.cuda.synchronize()
            return v
        mem, n = self.mem, self.now
        for k, v in self.start.items():
            n[k].copy_(v)
        cache = n["kq"], n["kd"], n["vq"], n["vd"]
        lens, cu, slots, pos, head = step(mem.memra_kv_plan(n["lens"], self.new, self.P, self.free, n["table"], self.T,
                                                            free_head=n["head"], free_head_out=n["head"], dev_status=self.status))
        q, k, v = self.qkv.split((self.heads, self.kv, self.kv), 1)
        step(mem.memra_kv_append_q8(k, v, slots, *cache, dev_status=self.status))
        out, lse = step(mem.memra_kv_attention_q8(q, *cache, n["table"], lens, cu, scale=0.125, workspace=self.ws,
                                                  dev_status=self.status))
        y = step(mem.memra_q8_0_quant_gemm(*self.o, out.view(self.T, -1)[:16]))
        ids, w = step(mem.memra_moe_route(y, 8, score="sigmoid", n_groups=8, topk_groups=4, group_top=2))
        rk, rv = step(mem.memra_kv_read_q8(slots, *cache, dtype=torch.float32))
        return [lens, cu, slots, pos, head, n["table"], out, lse, y, ids, w, rk, rv, *cache]


def bits(ts):
    torch.cuda.synchronize()
    return [t.clone().view(torch.uint8) for t in ts]


@pytest.mark.parametrize("new,G,dtype", [(1, 5, "bf16"), (1, 8, "fp32"), (3, 8, "bf16"), (8, 8, "bf16"), (12, 16, "bf16"), (8, 8, "fp32")])
def test_a_step_back_to_back_and_as_a_graph(mem, new, G, dtype):
    s = Step(mem, new, G, dtype)
    want = bits(s.run(sync=True))
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, bits(s.run())))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = s.run()
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, bits(outs)))
    assert int(s.status) == 0 and bool(torch.isfinite(outs[6]).all())


# ---------------------------------------------------------------------------
# Attention where its kernels change, and with codes far into a pool.
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("new,Hkv,G", [([1, 1, 1], 2, 8), ([1, 1, 2], 2, 8), ([2, 2], 2, 8), ([2, 3], 2, 8), ([4] * 4, 8, 8),
                                       ([4, 4, 4, 5], 8, 8), ([5] * 3, 8, 8), ([5] * 3, 9, 8), ([8] * 3, 6, 8), ([8, 8, 9], 6, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_on_both_sides_of_each_rule(mem, new, Hkv, G, dtype):
    """8 and 9 rows to a request, 16 and 17, 32 and 33 (with 1024 in all and more), 1024 in all and
    fewer, 64 and 65."""
    rs = np.random.RandomState(sum(new) + Hkv)
    c = attention_case(rs, rs.randint(20, 400, len(new)), new, G * Hkv, Hkv, 64, 32, 8, dtype)
    check_attention(mem, *c, code_unit=dtype == "bf16" and sum(new) * G <= 8 * len(new))


@pytest.mark.parametrize("n,dtype", [(1, "fp32"), (2, "bf16"), (3, "bf16"), (8, "fp32"), (40, "bf16")])
def test_attention_negative_scales_of_exact_codes(mem, n, dtype):
    """Scales of either sign in the kernels whose codes of V carry no 128, without its allowance."""
    c = list(attention_case(np.random.RandomState(97), [300, 170], [n, n], 32, 4, 64, 32, 8, dtype))
    for change in (lambda d: -d, lambda d: np.where(np.arange(d.shape[2]) % 2, d, -d).astype(np.float32)):
        check_attention(mem, c[0], c[1], change(c[2]), c[3], change(c[4]), *c[5:])


@pytest.mark.parametrize("n", [1, 2, 60])
def test_attention_rows_of_no_request_before_the_first(mem, n):
    c = attention_case(np.random.RandomState(98), [300, 170], [n, n], 32, 4, 64, 32, 8, "bf16")
    q = torch.cat([c[0][:1].expand(5, -1, -1), c[0], c[0][:1].expand(3, -1, -1)])
    out, lse = check_attention(mem, q, *c[1:7], c[7] + 5, scale=0.1)
    for part in (slice(0, 5), slice(2 * n + 5, None)):
        assert bool((out[part] == 0).all()) and bool(torch.isneginf(lse[part]).all())


@pytest.mark.parametrize("n", [8, 16])
def test_attention_wide_long_pool(mem, n):
    """Pages whose byte offsets pass 2^31 and 2^32, in units of 64 and of 128 rows."""
    Hkv, P, D = 4, 64, 128
    c = attention_case(np.random.RandomState(24), [300, 900, 20, 77], [n] * 4, 8 * Hkv, Hkv, D, P, 16, "bf16")
    q, planes, table = c[0], c[1:5], c[5]
    n_pages, small = (1 << 32) // (Hkv * P * D) + 4, planes[0].shape[0]
    big = [torch.zeros((n_pages,) + x.shape[1:], dtype=torch.from_numpy(x).dtype, device="cuda") for x in planes]
    for b, x in zip(big, planes):
        b[n_pages - small:] = dev(x)
        b[n_pages // 2:n_pages // 2 + small] = dev(x)
    at = [dev(x, i32) for x in c[6:]]
    o, l = mem.memra_kv_attention_q8(q, *[dev(x) for x in planes], dev(table, i32), *at)
    for first in (n_pages - small, n_pages // 2):
        o2, l2 = mem.memra_kv_attention_q8(q, *big, dev(np.where(table >= 0, table + first, -1), i32), *at)
        assert torch.equal(o, o2) and torch.equal(l, l2)


# ---------------------------------------------------------------------------
# A wait of the many-row kernel that runs out.
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("tiles", [1, 2, 3, 5])
@pytest.mark.parametrize("n", [8, 16])
def test_attention_wide_gives_up_in_the_middle(mem, tiles, n):
    """The feeding warps stop after some tiles, with products, copies and finished parts of units
    behind them: every value is NaN or what it should be, status bit 2 is set, and with a zeroed
    workspace the next call is as before."""
    rs = np.random.RandomState(80)
    lens = [9000, 700, 64, 3000, 5000, 130]
    c = attention_case(rs, lens, [n] * 6, 64, 8, 64, 32, 16, "bf16")
    t = [c[0]] + [dev(x) for x in c[1:5]] + [dev(x, i32) for x in c[5:]]
    ws = torch.zeros(mem.KV_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=i32, device="cuda")
    want = mem.memra_kv_attention_q8(*t, scale=0.1, workspace=ws, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    out, lse = torch.full_like(want[0], 777.0), torch.full_like(want[1], 777.0)
    try:
        mem.memra_debug_set_wait_test(1 << 16, tiles)
        mem.memra_kv_attention_q8(*t, scale=0.1, out=out, lse=lse, workspace=ws, dev_status=st)
        torch.cuda.synchronize()                         # the kernel returned
    finally:
        mem.memra_debug_set_wait_test()
    assert int(st) == 2
    assert bool(torch.isnan(out).any()) and bool(torch.isnan(lse).any())
    assert bool((torch.isnan(out) | (out == want[0])).all()) and bool((torch.isnan(lse) | (lse == want[1])).all())
    ws.zero_()
    st.zero_()
    again = mem.memra_kv_attention_q8(*t, scale=0.1, workspace=ws, dev_status=st)
    assert int(st) == 0 and torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
