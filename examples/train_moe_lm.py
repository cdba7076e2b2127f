"""A small mixture-of-experts language model trained with the library's
operators and optimizers: every matrix product, the embedding, the loss, all
gradients and both optimizer steps run in its kernels; torch holds memory,
sorts the tokens by expert and applies the activation.

    python examples/train_moe_lm.py [--steps 30] [--vocab 8192] ...

The model is one residual block, logits = head (h + down(relu(up h)^2)) with
h an embedding row and the block's weights an expert chosen by the token's
id.  Its task is a fixed random successor for every token, so the loss falls
from ln(vocab) towards 0.

Masters are fp32: the experts' matrices under Muon (their gradients bf16), the
embedding and the head under AdamW (fp32 gradients); the products read bf16
copies.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import optimizer_muon_step_gb300 as m  # noqa: E402

BF16 = torch.bfloat16


class MoeLm:
    def __init__(self, vocab, dim, hidden, experts, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        new = lambda *shape: torch.randn(shape, generator=gen, device=device)  # noqa: E731
        self.table = new(vocab, dim) * 0.02
        self.head = new(vocab, dim) * 0.02
        self.up = new(experts, hidden, dim) / math.sqrt(dim)
        self.down = new(experts, dim, hidden) / math.sqrt(hidden) * 0.1
        self.scale = math.sqrt(dim)
        self.experts = experts

        # optimizer state, and the gradients' buffers, which stay where they are
        self.d_up = torch.empty_like(self.up, dtype=BF16)
        self.d_down = torch.empty_like(self.down, dtype=BF16)
        self.d_table = torch.empty_like(self.table)
        self.d_head = torch.empty_like(self.head)
        w = [*self.up.unbind(), *self.down.unbind()]
        g = [*self.d_up.unbind(), *self.d_down.unbind()]
        self.muon = m.MuonBatch(w, g, [torch.zeros_like(x) for x in w])
        self.adamw = [(p, d, torch.zeros_like(p), torch.zeros_like(p))
                      for p, d in ((self.table, self.d_table), (self.head, self.d_head))]
        self.t = 0

    def gradients(self, ids, targets):
        """The mean loss; every gradient into its buffer."""
        up, down, head = self.up.to(BF16), self.down.to(BF16), self.head.to(BF16)
        # tokens in the order of their experts
        expert = ids * 2654435761 % 4294967291 % self.experts
        order = torch.sort(expert, stable=True).indices
        edges = torch.bincount(expert, minlength=self.experts).cumsum(0)
        offsets = torch.cat([edges.new_zeros(1), edges])
        ids, targets = ids[order], targets[order]

        h = m.muon_embedding_lookup(self.table, ids, scale=self.scale, out_dtype=BF16)
        u = m.muon_expert_matmul(h, up, offsets)
        a = torch.relu(u).square()
        x = h + m.muon_expert_matmul(a, down, offsets)

        row_scale = torch.full((ids.numel(),), 1.0 / ids.numel(), device=ids.device)
        loss, _, dx, _ = m.muon_linear_ce_grad(x, head, targets, row_scale=row_scale, d_weight=self.d_head)

        da = m.muon_expert_matmul(dx, down, offsets, transpose=True)
        m.muon_expert_wgrad(dx, a, offsets, out=self.d_down)
        du = da * (2.0 * torch.relu(u))
        m.muon_expert_wgrad(du, h, offsets, out=self.d_up)
        dh = dx + m.muon_expert_matmul(du, up, offsets, transpose=True)
        m.muon_embedding_grad(dh, ids, self.table.shape[0], scale=self.scale, out=self.d_table)
        return loss.mean()

    def step(self, ids, targets, muon_hp, adamw_hp):
        loss = self.gradients(ids, targets)
        self.t += 1
        self.muon.step(muon_hp)
        m.adamw_step_batched(self.adamw, adamw_hp, step=self.t)
        return loss


def train(steps=30, vocab=8192, dim=256, hidden=512, experts=8, tokens=4096, seed=0, log=print):
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    successor = torch.randperm(vocab, generator=gen, device="cuda")
    model = MoeLm(vocab, dim, hidden, experts, seed)
    muon_hp, adamw_hp = m.MuonHparams(lr=0.01, weight_decay=0.0), m.AdamwHparams(lr=5e-3, weight_decay=0.0)
    losses = []
    for step in range(steps):
        ids = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
        losses.append(model.step(ids, successor[ids], muon_hp, adamw_hp))
        if step % 10 == 0 or step + 1 == steps:
            log(f"step {step:4d}  loss {losses[-1].item():.4f}")
    return [x.item() for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    for name, value in (("steps", 30), ("vocab", 8192), ("dim", 256), ("hidden", 512), ("experts", 8), ("tokens", 4096),
                        ("seed", 0)):
        ap.add_argument(f"--{name}", type=int, default=value)
    train(**vars(ap.parse_args()))
