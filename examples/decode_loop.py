"""A decode loop of a small routed model on the library: every step plans its pages, writes
K and V into the paged 8-bit cache, attends over it, routes and runs the experts.

    python examples/decode_loop.py [--layers 2] [--sequences 4] [--steps 32]

The weights are random (Q8_0), so the tokens mean nothing; the sequence of calls is the one a
server makes.  Prompts go in a few tokens a step (a product takes up to 16 rows), then each
sequence decodes one token a step.  Lengths, pages, slots and tokens stay on the GPU: the
host only counts how many rows a step has.
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
    """Rotary embedding of x [rows, heads, D] at the rows' positions."""
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

    def __init__(self, cfg, sequences, max_len, device="cuda", seed=0):
        self.cfg, self.device, self.B = cfg, device, sequences
        gen = torch.Generator(device=device).manual_seed(seed)
        cfg["pages"] = sequences * -(-max_len // cfg["page"]) + 2
        self.embedding = torch.randn(cfg["vocab"], cfg["hidden"], generator=gen, device=device)
        head = torch.randn(cfg["vocab"], cfg["hidden"], generator=gen, device=device)
        self.head = memra.memra_quantize_q8_0(head * cfg["hidden"] ** -0.5)
        self.layers = [Layer(cfg, gen, device) for _ in range(cfg["layers"])]
        i32 = dict(dtype=torch.int32, device=device)
        self.lens = torch.zeros(sequences, **i32)
        self.table = torch.full((sequences, -(-max_len // cfg["page"])), -1, **i32)
        self.free = torch.randperm(cfg["pages"], generator=gen, device=device).int()
        self.free_head = torch.zeros(1, **i32)
        self.workspace = torch.zeros(memra.KV_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device=device)
        self.status = torch.zeros(1, **i32)

    def product(self, weights, x):
        return memra.memra_q8_0_quant_gemm(*weights, x)

    def step(self, tokens, new_lens):
        """tokens int [rows], sequence after sequence, new_lens int32 [sequences] on the GPU ->
        the hidden rows after the last layer, and the plan's cu_q."""
        cfg, rows = self.cfg, tokens.shape[0]
        heads, kv, D = cfg["heads"], cfg["kv_heads"], cfg["head_dim"]
        self.lens, cu_q, slots, positions, _ = memra.memra_kv_plan(
            self.lens, new_lens, cfg["page"], self.free, self.table, rows, free_head=self.free_head,
            free_head_out=self.free_head, dev_status=self.status)
        x = self.embedding[tokens]
        for layer in self.layers:
            qkv = self.product(layer.qkv, rms_norm(x)).view(rows, heads + 2 * kv, D)
            qk = rotate(qkv[:, :heads + kv], positions)
            memra.memra_kv_append_q8(qk[:, heads:].contiguous(), qkv[:, heads + kv:].contiguous(), slots, *layer.cache,
                                     dev_status=self.status)
            attended, _ = memra.memra_kv_attention_q8(
                qk[:, :heads].bfloat16(), *layer.cache, self.table, self.lens, cu_q, scale=D ** -0.5,
                workspace=self.workspace, dev_status=self.status)
            x = x + self.product(layer.o, attended.view(rows, heads * D))
            h = rms_norm(x)
            ids, gate_w = memra.memra_moe_route(self.product(layer.router, h), cfg["top_k"], bias=layer.bias,
                                                score="sigmoid", n_groups=cfg["groups"],
                                                topk_groups=cfg["groups"] // 2, group_top=2)
            x = x + memra.memra_q8_0_moe_ffn_tokens(*layer.gate_up, *layer.down, ids, gate_w, h)
        return x, cu_q

    def next_tokens(self, x, cu_q):
        """The likeliest token after each sequence's last row."""
        last = x[(cu_q[1:].long() - 1).clamp(min=0)]
        return self.product(self.head, rms_norm(last)).argmax(-1)


CONFIG = {"hidden": 2048, "heads": 32, "kv_heads": 4, "head_dim": 128, "experts": 128, "top_k": 8, "groups": 8,
          "ffn": 768, "vocab": 8192, "page": 64, "block": 16, "layers": 2}


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=CONFIG["layers"])
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--prompt", type=int, default=21, help="tokens of the longest prompt")
    a = ap.parse_args()
    if not 1 <= a.sequences <= MAX_ROWS:
        ap.error("1 to %d sequences" % MAX_ROWS)
    model = Decoder(dict(CONFIG, layers=a.layers), a.sequences, a.prompt + a.steps + 1)
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, CONFIG["vocab"], (max(1, a.prompt - 3 * i),), generator=gen) for i in range(a.sequences)]
    given, tokens = [0] * a.sequences, None
    per_step = MAX_ROWS // a.sequences
    while any(g < len(p) for g, p in zip(given, prompts)):  # prompts, a few tokens a step
        new = [min(per_step, len(p) - g) for g, p in zip(given, prompts)]
        rows = torch.cat([p[g:g + n] for p, g, n in zip(prompts, given, new)]).to(model.device)
        x, cu_q = model.step(rows, torch.tensor(new, dtype=torch.int32, device=model.device))
        after = model.next_tokens(x, cu_q)
        took = torch.tensor([n > 0 for n in new], device=model.device)
        tokens = after if tokens is None else torch.where(took, after, tokens)
        given = [g + n for g, n in zip(given, new)]
    one = torch.ones(a.sequences, dtype=torch.int32, device=model.device)
    out = [tokens]
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(a.steps):
        x, cu_q = model.step(out[-1], one)
        out.append(model.next_tokens(x, cu_q))
    torch.cuda.synchronize()
    took = time.perf_counter() - began
    assert int(model.status) == 0, "a length, slot or page was out of range (status %d)" % int(model.status)
    for i, row in enumerate(torch.stack(out).t().tolist()):
        print("sequence %d (%d tokens): %s ..." % (i, int(model.lens[i]), row[:8]))
    print("%d steps of %d sequences, %d layers: %.2f ms a step" % (a.steps, a.sequences, a.layers, took / a.steps * 1e3))


if __name__ == "__main__":
    main()
