"""The example's steps with normed heads, and with samples that share pages, against plain float32 torch; and the calls of
such a step one after another and as a graph."""
import sys
import types

import numpy as np
import pytest
import torch

from test_gpu_decode_loop import CFG, example, reference  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def normed(example, model, wq, wk):
    """The example's functions with the rotation of normed heads."""
    heads = model.cfg["heads"]

    def rotate(x, positions):
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        x = torch.cat([x[:, :heads] * wq, x[:, heads:] * wk], 1)
        return example.rotate(x, positions)

    return types.SimpleNamespace(rms_norm=example.rms_norm, rotate=rotate)


def near(x, want):
    return (x - want).norm(dim=-1) / want.norm(dim=-1)


def test_samples_of_normed_heads(example):
    """Prompts, a fork of unequal numbers, steps of the samples on their own, a choice among them, steps after it and a
    compaction: every row is compared with its whole history without a cache, as near as 8-bit products and cache come (the
    measures of the plain decode loop's test, whose layers these are)."""
    gen = torch.Generator().manual_seed(7)
    model = example.Decoder(dict(CFG, qk_norm=True), 3, 48, samples=3)
    for layer in model.layers[1:]:
        layer.q_norm, layer.k_norm = model.layers[0].q_norm, model.layers[0].k_norm
    plain = normed(example, model, model.layers[0].q_norm, model.layers[0].k_norm)
    history = [torch.zeros(0, dtype=torch.int64, device="cuda") for _ in range(3)]
    off = []

    def step(new):
        nonlocal history
        rows = [torch.randint(0, CFG["vocab"], (n,), generator=gen).cuda() for n in new]
        history = [torch.cat([h, r]) for h, r in zip(history, rows)]
        x, cu_q = model.step(torch.cat(rows), torch.tensor(new, dtype=torch.int32, device="cuda"))
        want = torch.cat([r[r.shape[0] - n:] for r, n in zip(reference(plain, model, history), new)])
        off.append(near(x, want))
        ids, lp = model.alternatives(x, cu_q, 4)
        logits = model.product(model.head, example.rms_norm(x[(cu_q[1:].long() - 1).clamp(min=0)]))
        top = torch.log_softmax(logits.double(), -1).topk(4)
        assert torch.equal(ids, top.indices) and float((lp - top.values).abs().max()) < 1e-5

    def keep(parents):
        nonlocal history
        model.keep(torch.tensor(parents, dtype=torch.int32, device="cuda"))
        history = [history[p] for p in parents]

    for new in ([5, 0, 3], [5, 4, 5], [2, 5, 9]):
        step(new)
    keep([0, 0, 0, 1, 2, 2, 2])
    for new in ([1] * 7, [1, 2, 0, 3, 1, 1, 2], [1] * 7, [2] * 7):
        step(new)
    keep([1, 4, 4, 6])
    step([1, 1, 1, 1])
    used = int(model.compact())
    P = CFG["page"]
    table = model.table.cpu().numpy()
    held = {int(table[b, i]) for b, h in enumerate(history) for i in range(-(-h.shape[0] // P))}
    assert held == set(range(used)) and int(model.free_head) == used
    for new in ([1] * 4, [3, 1, 9, 2], [1] * 4):
        step(new)
    off = torch.cat(off)
    assert int(model.status) == 0 and model.lens.tolist() == [h.shape[0] for h in history]
    assert float(off.median()) < 0.05 and float((off < 0.1).float().mean()) > 0.8
    keep([])
    assert int(model.free_head) == 0 and not bool(model.refs.any())
    assert sorted(model.free.tolist()) == list(range(model.cfg["pages"]))


def test_the_example_with_samples(example, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["decode_loop.py", "--layers", "1", "--sequences", "2", "--samples", "3", "--steps", "70"])
    example.main()
    assert "3 samples each" in capsys.readouterr().out


class Calls:
    """A step's calls around the products, on inputs that stay: fork, copy on write, plan, norm and rotation, write,
    attention, log probabilities, release."""

    def __init__(self, mem, dtype):
        g = torch.Generator().manual_seed(3)
        rs = np.random.RandomState(4)
        B, P, Hkv, G, D, n = 5, 16, 2, 4, 64, 80
        i32 = dict(dtype=torch.int32, device="cuda")
        self.mem, self.P, self.D, self.dtype = mem, P, D, dtype
        lens = rs.randint(1, 120, B)
        have = -(-lens // P)
        ids = rs.permutation(n)
        table = np.full((B, 9), -1)
        at = 0
        for b in range(B):
            table[b, :have[b]] = ids[at:at + have[b]]
            at += have[b]
        self.start = dict(lens=torch.tensor(lens, **i32), table=torch.tensor(table, **i32), refs=torch.zeros(n, **i32),
                          free=torch.tensor(ids, **i32), head=torch.tensor([at], **i32),
                          kq=torch.randint(-127, 128, (n, Hkv, P, D), generator=g, dtype=torch.int8).cuda(),
                          kd=torch.rand(n, Hkv, P // 8, generator=g).cuda(),
                          vq=torch.randint(-127, 128, (n, Hkv, P, D), generator=g, dtype=torch.int8).cuda(),
                          vd=torch.rand(n, Hkv, P // 8, generator=g).cuda())
        self.now = {k: v.clone() for k, v in self.start.items()}
        self.parents = torch.tensor([0, 0, 1, 3, 3, 3, 4], **i32)
        C = 7
        self.new = torch.ones(C, **i32)
        self.rows = torch.randn(C, (G + 2) * Hkv, D, generator=g).to(dtype).cuda()
        self.heads, self.kv = G * Hkv, Hkv
        self.freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).cuda()
        self.weight = torch.randn(D, generator=g).cuda()
        self.logits = (3 * torch.randn(C, 5003, generator=g)).to(dtype).cuda()
        self.workspace = torch.zeros(mem.KV_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
        self.status = torch.zeros(1, **i32)

    def run(self, sync=False):
        def done(v):
            if sync:
                torch.cuda.synchronize()
            return v
        m, n, st = self.mem, self.now, self.status
        for k, v in self.start.items():
            n[k].copy_(v)
        cache = n["kq"], n["kd"], n["vq"], n["vd"]
        lens, table = done(m.memra_kv_fork(self.parents, n["lens"], n["table"], self.P, n["refs"], dev_status=st))
        new, src, dst, tokens, head = done(m.memra_kv_unshare(lens, self.new, self.P, n["refs"], n["free"], table, free_head=n["head"],
                                                              dev_status=st))
        done(m.memra_kv_copy_pages(src, dst, [cache], tokens=tokens, dev_status=st))
        kv_lens, cu, slots, pos, head = done(m.memra_kv_plan(lens, new, self.P, n["free"], table, 7, free_head=head, free_head_out=head,
                                                             dev_status=st))
        q, k, v = self.rows.clone().split((self.heads, self.kv, self.kv), 1)
        q, k = done(m.memra_qk_norm_rope(q, k, pos, self.freq, q_weight=self.weight, k_weight=self.weight, eps=1e-6, k_out=k))
        done(m.memra_kv_append_q8(k, v, slots, *cache, dev_status=st))
        out, lse = done(m.memra_kv_attention_q8(q, *cache, table, kv_lens, cu, scale=0.125, workspace=self.workspace, dev_status=st))
        lp = done(m.memra_token_logprobs(self.logits, slots, top_n=9, dev_status=st))
        gone, back = done(m.memra_kv_release(kv_lens, self.P, table, n["refs"], n["free"], head, dev_status=st))
        t2, r2, f2, a, b, used = done(m.memra_kv_compact(n["lens"], n["table"], self.P, 80, dev_status=st))
        done(m.memra_kv_copy_pages(a, b, [cache], dev_status=st))
        return [lens, table, new, src, dst, tokens, kv_lens, slots, pos, q, k, out, lse, *lp, gone, back, t2, r2, f2, a, b, used, n["refs"],
                n["free"], head, *cache]


def bits(ts):
    torch.cuda.synchronize()
    return [t.clone().contiguous().view(torch.uint8) for t in ts]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_calls_back_to_back_and_as_a_graph(example, dtype):
    import block_quantized_decode_quantize_gb300 as mem
    c = Calls(mem, dtype)
    want = bits(c.run(sync=True))
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, bits(c.run())))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = c.run()
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, bits(outs)))
    assert int(c.status) == 0


def test_the_long_way_gives_the_same(example, monkeypatch):
    """Without the extension module every call goes through ctypes."""
    import block_quantized_decode_quantize_gb300 as mem
    c = Calls(mem, torch.float32)
    want = bits(c.run())
    monkeypatch.setattr(mem, "_fast", mem._NoBinding)
    assert all(torch.equal(a, b) for a, b in zip(want, bits(c.run())))
