"""A small language model trained privately end to end: token embedding,
projected linear layers (or gated feed-forward blocks), and a loss that mixes cross
entropy with distillation from a teacher's top logits, against a frozen [V, d] head.

    python examples/private_lm.py [steps] [--gated]

Synthetic data: sequences from a random bigram table, some of them padded. The
teacher is the table itself: for every position, the k most likely next tokens
and their logits. The embedding table and the linear layers are updated with
one clip per sample across all of them; the head stays as it is, as do the
places where the data only enters through public values (norm, activation).
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dp_grape_projection_amd as dpg  # noqa: E402


class PrivateLM(torch.nn.Module):
    """Embedding, two residual layers of ProjectedLinear pairs (or of gated blocks, which
    keep their activations in 8 bits), final norm."""

    def __init__(self, V, d, head, dtype, gated=False):
        super().__init__()
        self.embed = dpg.TokenEmbedding(V, d, layer_id=0, scale=math.sqrt(d), dtype=dtype)
        self.register_buffer("head", head.to(dtype).contiguous())
        self.blocks = None
        if gated:
            self.blocks = torch.nn.ModuleList(
                [dpg.GatedFeedForward(d, 2 * d, (1 + 2 * i, 2 + 2 * i), checkpoint="int8")
                 for i in range(2)])
            return
        self.up = torch.nn.ModuleList(
            [dpg.ProjectedLinear(d, 2 * d, layer_id=1 + 2 * i) for i in range(2)])
        self.down = torch.nn.ModuleList(
            [dpg.ProjectedLinear(2 * d, d, layer_id=2 + 2 * i) for i in range(2)])

    def linears(self):
        if self.blocks is not None:
            return [l for block in self.blocks for l in block.linears()]
        return [*self.up, *self.down]

    def forward(self, ids):
        x = self.embed(ids)
        if self.blocks is not None:
            for block in self.blocks:
                x = x + block(torch.nn.functional.layer_norm(x, x.shape[-1:]))
            return torch.nn.functional.layer_norm(x, x.shape[-1:])
        for up, down in zip(self.up, self.down):
            h = torch.nn.functional.layer_norm(x, x.shape[-1:])
            x = x + down(torch.nn.functional.gelu(up(h)))
        return torch.nn.functional.layer_norm(x, x.shape[-1:])


def bigram_batch(table, B, T, generator):
    """Ids [B, T] and next-token targets [B, T] from the bigram logits; the
    last quarter of every other sample is padding (-1)."""
    V = table.shape[0]
    probs = torch.softmax(table, 1)
    ids = [torch.randint(0, V, (B,), generator=generator, device=table.device)]
    for _ in range(T):
        ids.append(torch.multinomial(probs[ids[-1]], 1, generator=generator)[:, 0])
    seq = torch.stack(ids, 1)
    x, y = seq[:, :-1].contiguous(), seq[:, 1:].contiguous()
    x[::2, 3 * T // 4:] = -1
    y[::2, 3 * T // 4:] = -1
    return x, y


def train(steps=40, V=512, d=64, B=64, T=32, k=8, sigma=0.2, clip_C=1.0, mix=0.5,
          dtype=torch.bfloat16, seed=0, keep=None, gated=False):
    """Runs `steps` private steps; returns the mean loss per token before each.
    keep: a list that receives the optimizer and model (for checks). gated: gated
    feed-forward blocks instead of pairs of linear layers."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    bigram = 3.0 * torch.randn(V, V, generator=g, device="cuda")
    head = torch.randn(V, d, generator=g, device="cuda") / math.sqrt(d)
    torch.manual_seed(seed)
    model = PrivateLM(V, d, head, dtype, gated)
    opt = dpg.GrapeOptimizer(model.linears(), r=16, clip_C=clip_C, sigma=sigma, seed=seed,
                             lr=3e-3, embeddings=[model.embed], table_lr=4.0)
    if keep is not None:
        keep += [opt, model]
    losses = []
    for _ in range(steps):
        ids, targets = bigram_batch(bigram, B, T, g)
        top = torch.topk(bigram[ids.clamp(min=0)], k, dim=-1)
        top_ids = top.indices.masked_fill((targets < 0)[..., None], -1)
        opt.zero_grad()
        x = model(ids)
        ce = dpg.vocab_cross_entropy(x, model.head, targets)
        kd = dpg.distill_cross_entropy(x, model.head, top_ids, top.values, temperature=2.0)
        n = (targets >= 0).sum(1, keepdim=True)
        # every sample's mean loss; their sum, so that a sample's gradient is its own
        ((1.0 - mix) * ce + mix * kd).div(n).sum().backward()
        opt.step()
        losses.append(float((ce.detach() / n).sum() / B))
    return losses


if __name__ == "__main__":
    gated = "--gated" in sys.argv[1:]
    steps = [int(a) for a in sys.argv[1:] if a != "--gated"] or [40]
    for i, loss in enumerate(train(steps[0], gated=gated)):
        print(f"step {i + 1}: cross entropy {loss:.4f}", flush=True)
