"""A decode loop of a small routed model on the library: every step plans its pages, norms and
rotates queries and keys, writes K and V into the paged 8-bit cache, attends over it, routes and
runs the experts.

    python examples/decode_loop.py [--layers 2] [--sequences 4] [--samples 2] [--steps 32]

The weights are random (Q8_0), so the tokens mean nothing; the sequence of calls is the one a
server makes.  Prompts go in a few tokens a step (a product takes up to 16 rows), then each
sequence is forked into samples that share its pages, begin with different tokens and decode
one token a step; the likeliest sample of each stays, and the pages of the others go back.
Lengths, pages, slots and tokens stay on the GPU: the host only counts how many rows a step has.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_quantized_decode_quantize_gb300 as memra  # noqa: E402

MAX_ROWS = memra.MAX_M


def rms_norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


def rotate(x, positions):
    """Rotary embedding of x [rows, heads, D] at the rows' positions: the plain form of what
    memra_qk_norm_rope does in the steps below, to compare with."""
    half = x.shape[-1] // 2
    freq = 10000.0 ** (-torch.arange(half, device=x.device, dtype=torch.float32) / half)
    angle = positions.clamp(min=0).float()[:, None, None] * freq
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1)


class Layer:
    def __init__(self, cfg, gen, device):
        def weights(rows, cols):
            return torch.randn(rows, cols, generator=gen, device=device) * cols ** -0.5

        H, D, E, F = cfg["hidden"], cfg["head_dim"], cfg["experts"], cfg["ffn"]
        self.qkv = memra.memra_quantize_q8_0(weights((cfg["heads"] + 2 * cfg["kv_heads"]) * D, H))
        self.o = memra.memra_quantize_q8_0(weights(H, cfg["heads"] * D))
        self.router = memra.memra_quantize_q8_0(weights(E, H))
        self.bias = 0.01 * torch.randn(E, generator=gen, device=device)
        self.q_norm = self.k_norm = None
        if cfg.get("qk_norm"):
            self.q_norm = 1 + 0.1 * torch.randn(D, generator=gen, device=device)
            self.k_norm = 1 + 0.1 * torch.randn(D, generator=gen, device=device)
        q, d = memra.memra_quantize_q8_0(weights(E * 2 * F, H))
        self.gate_up = q.view(E, 2 * F, H), d.view(E, 2 * F, H // 32)
        q, d = memra.memra_quantize_q8_0(weights(E * H, F))
        self.down = q.view(E, H, F), d.view(E, H, F // 32)
        pages, P, S = cfg["pages"], cfg["page"], cfg["block"]
        planes = (pages, cfg["kv_heads"], P)
        self.cache = (torch.empty(planes + (D,), dtype=torch.int8, device=device),
                      torch.empty(planes[:2] + (P // S,), device=device),
                      torch.empty(planes + (D,), dtype=torch.int8, device=device),
                      torch.empty(planes[:2] + (P // S,), device=device))


class Decoder:
    """The model and the state of its sequences."""

    def __init__(self, cfg, sequences, max_len, device="cuda", seed=0, samples=1):
        self.cfg, self.device, self.B = cfg, device, sequences
        gen = torch.Generator(device=device).manual_seed(seed)
        cfg["pages"] = sequences * samples * -(-max_len // cfg["page"]) + 2
        self.embedding = torch.randn(cfg["vocab"], cfg["hidden"], generator=gen, device=device)
        head = torch.randn(cfg["vocab"], cfg["hidden"], generator=gen, device=device)
        self.head = memra.memra_quantize_q8_0(head * cfg["hidden"] ** -0.5)
        self.layers = [Layer(cfg, gen, device) for _ in range(cfg["layers"])]
        i32 = dict(dtype=torch.int32, device=device)
        self.lens = torch.zeros(sequences, **i32)
        self.table = torch.full((sequences, -(-max_len // cfg["page"])), -1, **i32)
        self.free = torch.randperm(cfg["pages"], generator=gen, device=device).int()
        self.free_head = torch.zeros(1, **i32)
        self.refs = torch.zeros(cfg["pages"], **i32)     # holders of each page beyond the first
        half = cfg["head_dim"] // 2
        self.inv_freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
        self.workspace = torch.zeros(memra.KV_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device=device)
        self.status = torch.zeros(1, **i32)
        self.forked = False

    def product(self, weights, x):
        return memra.memra_q8_0_quant_gemm(*weights, x)

    def step(self, tokens, new_lens):
        """tokens int [rows], sequence after sequence, new_lens int32 [sequences] on the GPU ->
        the hidden rows after the last layer, and the plan's cu_q."""
        cfg, rows = self.cfg, tokens.shape[0]
        heads, kv, D = cfg["heads"], cfg["kv_heads"], cfg["head_dim"]
        if self.forked:  # sequences about to write into a page that others hold too take one of their own
            new_lens, src, dst, copied, _ = memra.memra_kv_unshare(
                self.lens, new_lens, cfg["page"], self.refs, self.free, self.table, free_head=self.free_head,
                free_head_out=self.free_head, dev_status=self.status)
            memra.memra_kv_copy_pages(src, dst, [layer.cache for layer in self.layers], tokens=copied, dev_status=self.status)
        self.lens, cu_q, slots, positions, _ = memra.memra_kv_plan(
            self.lens, new_lens, cfg["page"], self.free, self.table, rows, free_head=self.free_head,
            free_head_out=self.free_head, dev_status=self.status)
        x = self.embedding[tokens]
        for layer in self.layers:
            qkv = self.product(layer.qkv, rms_norm(x)).view(rows, heads + 2 * kv, D)
            q, k, v = qkv.split((heads, kv, kv), 1)
            # queries in bf16 for attention; keys stay where they are, beside the values
            q, k = memra.memra_qk_norm_rope(q, k, positions, self.inv_freq, q_weight=layer.q_norm, k_weight=layer.k_norm,
                                            eps=None if layer.q_norm is None else 1e-6, q_dtype=torch.bfloat16, k_out=k)
            memra.memra_kv_append_q8(k, v, slots, *layer.cache, dev_status=self.status)
            attended, _ = memra.memra_kv_attention_q8(
                q, *layer.cache, self.table, self.lens, cu_q, scale=D ** -0.5,
                workspace=self.workspace, dev_status=self.status)
            x = x + self.product(layer.o, attended.view(rows, heads * D))
            h = rms_norm(x)
            ids, gate_w = memra.memra_moe_route(self.product(layer.router, h), cfg["top_k"], bias=layer.bias,
                                                score="sigmoid", n_groups=cfg["groups"],
                                                topk_groups=cfg["groups"] // 2, group_top=2)
            x = x + memra.memra_q8_0_moe_ffn_tokens(*layer.gate_up, *layer.down, ids, gate_w, h)
        return x, cu_q

    def alternatives(self, x, cu_q, n):
        """The n likeliest tokens after each sequence's last row and their log probabilities."""
        last = x[(cu_q[1:].long() - 1).clamp(min=0)]
        _, _, ids, logprobs = memra.memra_token_logprobs(self.product(self.head, rms_norm(last)), top_n=n)
        return ids.long(), logprobs

    def next_tokens(self, x, cu_q):
        """The likeliest token after each sequence's last row."""
        return self.alternatives(x, cu_q, 1)[0][:, 0]

    def keep(self, parents):
        """Sequences parents int32 [n] go on, each as often as it is named; the pages that only the
        others held go back to the free list."""
        lens, table = memra.memra_kv_fork(parents, self.lens, self.table, self.cfg["page"], self.refs, dev_status=self.status)
        memra.memra_kv_release(self.lens, self.cfg["page"], self.table, self.refs, self.free, self.free_head,
                               free_head_out=self.free_head, dev_status=self.status)
        self.lens, self.table, self.forked = lens, table, True

    def compact(self):
        """The pages in use come first in the pool; returns their number (on the GPU)."""
        self.table, self.refs, self.free, src, dst, self.free_head = memra.memra_kv_compact(
            self.lens, self.table, self.cfg["page"], self.cfg["pages"], dev_status=self.status)
        memra.memra_kv_copy_pages(src, dst, [layer.cache for layer in self.layers], dev_status=self.status)
        return self.free_head


CONFIG = {"hidden": 2048, "heads": 32, "kv_heads": 4, "head_dim": 128, "experts": 128, "top_k": 8, "groups": 8,
          "ffn": 768, "vocab": 8192, "page": 64, "block": 16, "layers": 2, "qk_norm": True}


def arguments(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=CONFIG["layers"])
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--samples", type=int, help="of each sequence; by default 2, or 1 where %d in all are too few for 2" % MAX_ROWS)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--prompt", type=int, default=21, help="tokens of the longest prompt")
    a = ap.parse_args(argv)
    if a.samples is None:
        a.samples = 2 if 2 * a.sequences <= MAX_ROWS else 1
    if a.sequences < 1 or a.samples < 1 or a.sequences * a.samples > MAX_ROWS:
        ap.error("1 to %d samples in all" % MAX_ROWS)
    if a.samples > memra.MAX_TOP_LOGPROBS:
        ap.error("up to %d samples of a sequence" % memra.MAX_TOP_LOGPROBS)
    return a


def main():
    a = arguments()
    model = Decoder(dict(CONFIG, layers=a.layers), a.sequences, a.prompt + a.steps + 1, samples=a.samples)
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, CONFIG["vocab"], (max(1, a.prompt - 3 * i),), generator=gen) for i in range(a.sequences)]
    given, first, scores = [0] * a.sequences, None, None
    per_step = MAX_ROWS // a.sequences
    while any(g < len(p) for g, p in zip(given, prompts)):  # prompts, a few tokens a step
        new = [min(per_step, len(p) - g) for g, p in zip(given, prompts)]
        rows = torch.cat([p[g:g + n] for p, g, n in zip(prompts, given, new)]).to(model.device)
        x, cu_q = model.step(rows, torch.tensor(new, dtype=torch.int32, device=model.device))
        after, logprobs = model.alternatives(x, cu_q, a.samples)
        took = torch.tensor([n > 0 for n in new], device=model.device)[:, None]
        first = after if first is None else torch.where(took, after, first)
        scores = logprobs if scores is None else torch.where(took, logprobs, scores)
        given = [g + n for g, n in zip(given, new)]
    # sample i of a sequence begins with its i-th likeliest token
    model.keep(torch.arange(a.sequences, dtype=torch.int32, device=model.device).repeat_interleave(a.samples))
    one = torch.ones(a.sequences * a.samples, dtype=torch.int32, device=model.device)
    out, scores = [first.flatten()], scores.flatten()
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(a.steps):
        x, cu_q = model.step(out[-1], one)
        ids, logprobs = model.alternatives(x, cu_q, 1)
        out.append(ids[:, 0])
        scores = scores + logprobs[:, 0]
    torch.cuda.synchronize()
    took = time.perf_counter() - began
    best = scores.view(a.sequences, a.samples).argmax(-1) + a.samples * torch.arange(a.sequences, device=model.device)
    model.keep(best.int())
    used = int(model.compact())
    assert int(model.status) == 0, "a length, slot or page was out of range (status %d)" % int(model.status)
    for i, row in enumerate(torch.stack(out).t()[best].tolist()):
        print("sequence %d (%d tokens, log probability %.2f): %s ..." % (i, int(model.lens[i]), float(scores[best[i]]), row[:8]))
    print("%d steps of %d sequences, %d samples each, %d layers: %.2f ms a step; %d of %d pages in use"
          % (a.steps, a.sequences, a.samples, a.layers, took / a.steps * 1e3, used, model.cfg["pages"]))


if __name__ == "__main__":
    main()
