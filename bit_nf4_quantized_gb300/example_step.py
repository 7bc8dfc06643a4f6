"""A training step over NF4 weights, from token ids to adapter gradients, in the library's calls.

    python -m bit_nf4_quantized_gb300.example_step [--steps 20]

A stack of pre-norm MLP blocks (a transformer without its attention, which this library does not
have) with LoRA adapters on gate, up and down, an NF4 embedding table, and the table's own head:

    h = embedding rows
    block:  n = RMS norm of (h + previous block's output), kept in 8 bits
            gate, up = QLoRA linears of n * weight;  a = silu(gate) * up, kept in 8 bits
            output = QLoRA linear (down) of a
    loss = cross entropy of the last norm's output against the next token, over the whole table

Between forward and backward a block keeps its norm's checkpoint and 1 / rms, the gated
activation's checkpoint, the adapters' T, and gate and up in 16 bits; the residual stream is
not kept.  The elementwise silu and its gradient are plain torch.
"""

import argparse

import torch

from . import binding as b
from . import workloads as wl


class Linear:
    """A frozen NF4 weight [N, K] with a LoRA adapter (A float32 [r, K], B float32 [N, r])."""

    def __init__(self, N, K, r, alpha, tensor_id, device):
        w = wl.device_normal((N, K), 0.5 * K ** -0.5, wl.seed_for(8, tensor_id), device, torch.float32)
        self.W = b.nf4_quantize(w)
        self.A = wl.device_normal((r, K), 1.0 / r, wl.seed_for(8, tensor_id + 1), device, torch.float32)
        self.B = torch.zeros(N, r, device=device)
        self.alpha = alpha

    def item(self, x):
        return dict(x=x, W=self.W, A=self.A, B=self.B, alpha=self.alpha)


class Model:
    def __init__(self, vocab=1000, hidden=256, inner=640, blocks=3, rank=8, alpha=16.0, dtype=torch.bfloat16,
                 device="cuda"):
        self.dtype, self.hidden = dtype, hidden
        self.table = b.nf4_quantize(wl.device_normal((vocab, hidden), 0.05, wl.seed_for(8, 1), device, torch.float32))
        self.blocks = []
        for i in range(blocks):
            t = 10 * (i + 1)
            self.blocks.append(dict(norm=torch.ones(hidden, device=device),
                                    gate=Linear(inner, hidden, rank, alpha, t, device),
                                    up=Linear(inner, hidden, rank, alpha, t + 2, device),
                                    down=Linear(hidden, inner, rank, alpha, t + 4, device)))
        self.last_norm = torch.ones(hidden, device=device)

    def parameters(self):
        """(name, A or B) of every adapter."""
        return [(f"{i}.{k}.{p}", getattr(blk[k], p)) for i, blk in enumerate(self.blocks)
                for k in ("gate", "up", "down") for p in ("A", "B")]

    def loss_and_gradients(self, ids, targets):
        """(mean loss, {name: gradient}) of one batch of token ids [M] and targets [M] (int64; -100 for a
        token that does not count)."""
        h = b.nf4_embedding_rows(self.table, ids, torch.float32).to(self.dtype)
        saved, out = [], None
        for blk in self.blocks:
            y, h, rstd, ckpt = b.qlora_rms_norm_fwd(h, blk["norm"], residual=out, checkpoint=True)
            (gate, Tg), (up, Tu) = b.qlora_linear_fwd_batch([blk["gate"].item(y), blk["up"].item(y)])
            act = torch.nn.functional.silu(gate) * up
            down = blk["down"]
            out, Td = b.qlora_linear_fwd(act, down.W, down.A, down.B, down.alpha)
            saved.append((rstd, ckpt, gate, up, Tg, Tu, b.qlora_act8_quantize(act), Td))
        y, h, rstd, ckpt = b.qlora_rms_norm_fwd(h, self.last_norm, residual=out, checkpoint=True)

        counts = (targets != -100).sum().clamp(min=1)
        loss, _, dy = b.qlora_lm_loss(y, self.table, targets, grad_scale=counts.reciprocal().float())

        grads = {}
        dh, _ = b.qlora_rms_norm_bwd(dy, ckpt, rstd, self.last_norm)
        for i in reversed(range(len(self.blocks))):
            blk = self.blocks[i]
            rstd, ckpt, gate, up, Tg, Tu, act, Td = saved[i]
            d = blk["down"]
            dact, grads[f"{i}.down.A"], grads[f"{i}.down.B"] = b.qlora_linear_bwd_act8(dh, act, Td, d.W, d.A, d.B, d.alpha)
            sig = torch.sigmoid(gate)
            dgate = dact * up * sig * (1 + gate * (1 - sig))
            dup = dact * gate * sig
            dy = None
            for k, g, T in (("gate", dgate, Tg), ("up", dup, Tu)):
                p = blk[k]
                dx, grads[f"{i}.{k}.A"], grads[f"{i}.{k}.B"] = b.qlora_linear_bwd_act8(
                    g, ckpt, T, p.W, p.A, p.B, p.alpha, weight=blk["norm"])
                dy = dx if dy is None else dy + dx
            dh, _ = b.qlora_rms_norm_bwd(dy, ckpt, rstd, blk["norm"], dresidual=dh)
        return loss.sum() / counts, grads


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=512)
    a = ap.parse_args()
    model = Model()
    vocab = model.table.shape[0]
    ids = torch.from_numpy(wl.token_ids(a.tokens, vocab, 8, 2)).cuda()
    targets = (ids * 7 + 3) % vocab            # a rule that the adapters can learn
    targets[::16] = -100
    optimizer = torch.optim.Adam([p for _, p in model.parameters()], lr=2e-3)
    for step in range(a.steps):
        loss, grads = model.loss_and_gradients(ids, targets)
        for name, p in model.parameters():
            p.grad = grads[name]
        optimizer.step()
        print(f"step {step}: loss {loss.item():.4f}")
    if b.device_status() != b.NF4_OK:
        raise RuntimeError("device status word set")


if __name__ == "__main__":
    main()
