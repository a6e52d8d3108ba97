"""One feed-forward block trained to match a teacher's top logits, every product in NVFP4.

    python examples/distill_block.py

Embedding lookup, the gated block with its down projection and a residual, the output head, the
distillation loss, and back: the loss's gradient, the block's, the embedding table's.  Weights are
kept in float32 and quantized once a step; activations are quantized along both axes, gradients with
stochastic rounding and the random Hadamard transform on the transposed copies.  Synthetic data: the
teacher's entries are a fixed random function of the token.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import bit_block_scaled_quant_amd as nv  # noqa: E402


class Block:
    def __init__(self, vocab=2048, width=256, hidden=512, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(rows, cols, std):
            return std * torch.randn(rows, cols, generator=g, device=device)

        self.table = normal(vocab, width, 1.0 / math.sqrt(width))  # scaled by sqrt(width) at the lookup
        self.gate_up = normal(2 * hidden, width, 1.0 / math.sqrt(width))
        self.down = normal(width, hidden, 1.0 / math.sqrt(hidden))
        self.head = normal(vocab, width, 0.5 / math.sqrt(width))
        self.width, self.act = width, nv.SILU

    def step(self, tokens, idx, top, weight, seed, rate):
        """The mean loss of a batch (tokens [T], the teacher's idx and top [T][K], weight [T]), after which
        every weight has taken a step of size rate against its gradient."""
        scale = math.sqrt(self.width)
        rht = dict(rht_t=True, rht_seed=7)
        gate_up, down, head = (nv.quantize_2d(w) for w in (self.gate_up, self.down, self.head))

        x = nv.embed(tokens, self.table, scale=scale).bfloat16()
        qx, qx_t = nv.quantize_cast_transpose(x, **rht)
        h = nv.gated_ffn(qx, gate_up, self.act)
        qh, qh_t = nv.quantize_cast_transpose(h, **rht)
        y = (x + nv.gemm(qh, down)).bfloat16()
        qy, qy_t = nv.quantize_cast_transpose(y, **rht)
        logits = nv.gemm_ex(qy, head, dtype=torch.bfloat16)
        loss, _, dlogits = nv.distill_topk_loss_and_grad(logits, idx, top, weight=weight)

        def gradients(grad, w, x_t, n):
            q, q_t = nv.quantize_cast_transpose(grad, rounding=nv.SR, seed=seed + n, seed_t=seed + n + 1, **rht)
            return nv.gemm_ex(q, w.transposed(), dtype=torch.bfloat16), nv.gemm(q_t, x_t)

        dy, dhead = gradients(dlogits, head, qy_t, 0)
        dh, ddown = gradients(dy, down, qh_t, 2)
        dx, dgate_up = nv.gated_ffn_backward(dh, qx, qx_t, gate_up, self.act, rounding=nv.SR, seed=seed + 4,
                                             seed_t=seed + 5, **rht)
        dtable = nv.embed_grad(tokens, (dx + dy).bfloat16(), self.table.shape[0], scale=scale)
        for w, grad in ((self.table, dtable), (self.gate_up, dgate_up), (self.down, ddown), (self.head, dhead)):
            w.sub_(rate * grad)
        return loss.sum()


def train(steps=40, tokens=512, vocab=2048, entries=8, rate=0.25, device="cuda", report=None):
    """The loss of every step."""
    g = torch.Generator(device=device).manual_seed(1)
    idx = torch.stack([torch.randperm(vocab, generator=g, device=device)[:entries] for _ in range(vocab)]).int()
    top = 2.0 * torch.randn(vocab, entries, generator=g, device=device)
    block, losses = Block(vocab, device=device), []
    for i in range(steps):
        tok = torch.pow(float(vocab), torch.rand(tokens, generator=g, device=device)).int() - 1
        tok[:: 64] = -1  # padding
        at = tok.clamp(min=0).long()
        weight = (tok >= 0).float() / (tok >= 0).sum()
        losses.append(block.step(tok, idx[at], top[at], weight, seed=6 * i, rate=rate).item())
        if report:
            report(i, losses[-1])
    return losses


if __name__ == "__main__":
    train(report=lambda i, loss: print(f"step {i:3d}  loss {loss:.4f}", flush=True))
