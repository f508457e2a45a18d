"""The example's decode step against the same step in plain float32 torch."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_decode_quantize_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decode_loop
    return decode_loop


CFG = {"hidden": 256, "heads": 8, "kv_heads": 2, "head_dim": 64, "experts": 16, "top_k": 4, "groups": 4, "ffn": 64,
       "vocab": 512, "page": 16, "block": 16, "layers": 2}


def dense(q, d):
    return (q.float().unflatten(-1, (-1, 32)) * d.float()[..., None]).flatten(-2)


def reference(example, model, history):
    """The last layer's rows of each sequence from its whole history, without a cache."""
    cfg = model.cfg
    heads, kv, D = cfg["heads"], cfg["kv_heads"], cfg["head_dim"]
    rows = []
    for tokens in history:
        n = tokens.shape[0]
        x = model.embedding[tokens]
        pos = torch.arange(n, device=x.device)
        for layer in model.layers:
            qkv = (example.rms_norm(x) @ dense(*layer.qkv).t()).view(n, heads + 2 * kv, D)
            qk = example.rotate(qkv[:, :heads + kv], pos)
            q = qk[:, :heads].view(n, kv, heads // kv, D)
            s = torch.einsum("ikgd,jkd->kgij", q, qk[:, heads:]) * D ** -0.5
            s = s.masked_fill(pos[None, :] > pos[:, None], float("-inf")).softmax(-1)
            a = torch.einsum("kgij,jkd->ikgd", s, qkv[:, heads + kv:]).reshape(n, heads * D)
            x = x + a @ dense(*layer.o).t()
            h = example.rms_norm(x)
            score = torch.sigmoid(h @ dense(*layer.router).t())
            ranks = (score + layer.bias).view(n, cfg["groups"], cfg["experts"] // cfg["groups"])
            best = ranks.topk(2, -1).values.sum(-1).topk(cfg["groups"] // 2, -1).indices
            keep = torch.zeros(n, cfg["groups"], dtype=torch.bool, device=x.device).scatter(1, best, True)
            ids = ranks.masked_fill(~keep[..., None], float("-inf")).flatten(1).topk(cfg["top_k"], -1).indices
            w = score.gather(1, ids)
            w = w / w.sum(-1, keepdim=True)
            gu, dn = dense(*layer.gate_up), dense(*layer.down)
            y = torch.zeros_like(x)
            for k in range(cfg["top_k"]):
                g, u = torch.einsum("nfh,nh->nf", gu[ids[:, k]], h).chunk(2, -1)
                y += w[:, k:k + 1] * torch.einsum("nhf,nf->nh", dn[ids[:, k]], torch.nn.functional.silu(g) * u)
            x = x + y
        rows.append(x)
    return rows


def test_decode_steps(example):
    """Ragged prompts over several steps and decode steps after them.  Activations are rounded
    to 8 bits before every product and K, V to 8 bits in the cache: about 1 % of a row for each
    of the six products and two layers.  A near tie may choose another expert, so most rows,
    not every one, have to come as near as that."""
    gen = torch.Generator().manual_seed(5)
    model = example.Decoder(dict(CFG), 3, 40)
    history = [torch.zeros(0, dtype=torch.int64, device="cuda") for _ in range(3)]
    near = []
    for new in ([5, 0, 3], [5, 4, 1], [2, 5, 9], [1, 1, 1], [1, 1, 1], [0, 1, 1], [1, 16 - 2, 1]):
        rows = [torch.randint(0, CFG["vocab"], (n,), generator=gen).cuda() for n in new]
        history = [torch.cat([h, r]) for h, r in zip(history, rows)]
        x, cu_q = model.step(torch.cat(rows), torch.tensor(new, dtype=torch.int32, device="cuda"))
        assert cu_q.tolist() == [0, new[0], new[0] + new[1], sum(new)]
        want = torch.cat([r[r.shape[0] - n:] for r, n in zip(reference(example, model, history), new)])
        near.append((x - want).norm(dim=-1) / want.norm(dim=-1))
        assert model.next_tokens(x, cu_q).shape == (3,)
    near = torch.cat(near)
    assert int(model.status) == 0
    assert model.lens.tolist() == [h.shape[0] for h in history]
    assert float(near.median()) < 0.05 and float((near < 0.1).float().mean()) > 0.8


def test_the_example_runs(example, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["decode_loop.py", "--layers", "1", "--sequences", "3", "--steps", "4"])
    example.main()
    assert "4 steps of 3 sequences" in capsys.readouterr().out
