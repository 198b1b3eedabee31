#!/usr/bin/env python3
"""Tokenize, train and generate on one GPU: the token operators around a model's layers.

    python examples/next_token.py [--steps 60] [--chars 200000] [--tokens 2000] [--dim 256] [--new 48]

The model is the smallest that uses them all: h = f(E[id]), logits = h E^T, with one tied table E for the
lookup and the logits and f(e) = e + e M.  A step encodes nothing anew: the IDs stay on the device from the
tokenizer on.

    toktier_embed            float32 master table -> bfloat16 activations
    toktier_cross_entropy    loss, and the gradient of the logits in their place
    toktier_embed_backward   adds the lookup's part of the tied table's gradient to the logits' part
    toktier_sample           next IDs of several sequences, each with its own settings
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import exact_bpe_tokenization_amd as tt  # noqa: E402
from workloads import textgen  # noqa: E402


class Model:
    """Parameters, and the buffers of one step of `n` tokens."""

    def __init__(self, n_vocab, dim, n, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.table = 0.02 * torch.randn(n_vocab, dim, generator=g, device="cuda")
        self.mix = torch.zeros(dim, dim, device="cuda")
        self.squares = [torch.zeros_like(self.table), torch.zeros_like(self.mix)]   # Adagrad's sums
        self.scale = dim ** 0.5
        f32, bf16 = dict(device="cuda"), dict(device="cuda", dtype=torch.bfloat16)
        self.e, self.logits = torch.empty(n, dim, **bf16), torch.empty(n, n_vocab, **bf16)
        self.loss, self.lse, self.weight = torch.empty(n, **f32), torch.empty(n, **f32), torch.empty(n, **f32)
        self.grad_table = torch.empty(n_vocab, dim, **f32)
        size = max(tt.toktier_cross_entropy_workspace_bytes(n, n_vocab), tt.toktier_embed_backward_workspace_bytes(n, n_vocab, dim),
                   tt.toktier_sample_workspace_bytes(n, n_vocab))
        self.workspace = torch.empty(size, dtype=torch.uint8, device="cuda")

    def hidden(self, ids, e):
        tt.toktier_embed(self.table, ids, e, scale=self.scale)
        return e + e @ self.mix.bfloat16()

    def gradients(self, ids, targets):
        """(mean loss of the targets that are IDs, gradient of the table, gradient of the mix), on the device."""
        h = self.hidden(ids, self.e)
        tied = self.table.bfloat16()
        torch.mm(h, tied.t(), out=self.logits)
        kept = (targets >= 0).sum()
        self.weight.copy_(1.0 / kept)
        tt.toktier_cross_entropy(self.logits, targets, self.loss, self.lse, self.workspace, grad_logits=self.logits,
                                 grad_loss=self.weight)
        grad_h = self.logits @ tied
        self.grad_table.copy_(self.logits.t() @ h)
        grad_mix = self.e.t() @ grad_h
        grad_e = grad_h + grad_h @ self.mix.bfloat16().t()
        tt.toktier_embed_backward(grad_e, ids, self.grad_table, self.workspace, scale=self.scale, accumulate=True)
        return self.loss.sum() / kept, self.grad_table, grad_mix.float()

    def step(self, ids, targets, rate):
        """One step of Adagrad; returns the mean loss."""
        loss, *grads = self.gradients(ids, targets)
        for p, g, s in zip((self.table, self.mix), grads, self.squares):
            p.addcdiv_(g, s.addcmul_(g, g).sqrt().add_(1e-8), value=-rate)
        return loss

    def generate(self, start, n_new, uniform, temperature, top_k, top_p):
        """IDs [n_new, sequences] after the IDs `start`; uniform: [n_new, sequences].  Nothing leaves the device."""
        n = start.numel()
        ids = torch.empty(n_new, n, dtype=torch.int32, device="cuda")
        logprobs, e = torch.empty(n_new, n, device="cuda"), self.e[:n]
        last = start
        for i in range(n_new):
            logits = self.hidden(last, e) @ self.table.bfloat16().t()
            tt.toktier_sample(logits, uniform[i], ids[i], logprobs[i], self.workspace, temperature=temperature, top_k=top_k,
                              top_p=top_p)
            last = ids[i]
        return ids, logprobs


def token_bytes(merges):
    """The bytes of every ID: 256 single bytes, then the merges in order."""
    out = [bytes([b]) for b in range(256)]
    for a, b in merges:
        out.append(out[int(a)] + out[int(b)])
    return out


def run(steps=60, chars=200_000, tokens=2000, dim=256, n_new=48, rate=0.02, seed=0):
    """Returns (losses, IDs [n_new, 4] on the host, their texts)."""
    merges, family = textgen.load_vocab("v1")
    tok = tt.Tokenizer(merges, family)
    data, offsets = textgen.to_batch([textgen.english_code(seed + i, chars // 4) for i in range(4)])
    ids, _, n_ids = tok.encode_device(torch.from_numpy(data).cuda(), torch.from_numpy(offsets.astype("int64")).cuda())
    n_vocab = 256 + len(merges)
    n = min(tokens, n_ids - 1)
    model = Model(n_vocab, dim, max(n, 4), seed)
    losses = []
    for i in range(steps):
        at = i * n % (n_ids - n)
        losses.append(model.step(ids[at:at + n], ids[at + 1:at + 1 + n], rate))
    losses = torch.stack(losses).tolist()
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, _ = model.generate(ids[:4].clone(), n_new, torch.rand(n_new, 4, generator=g, device="cuda"),
                            temperature=torch.tensor([0.0, 0.7, 0.9, 1.0], device="cuda"),
                            top_k=torch.tensor([0, 50, 0, 0], dtype=torch.int32, device="cuda"),
                            top_p=torch.tensor([1.0, 0.95, 0.9, 1.0], device="cuda"))
    new = new.cpu()
    table = token_bytes(merges)
    texts = [b"".join(table[j] for j in new[:, s].tolist()).decode("utf-8", "replace") for s in range(4)]
    return losses, new, texts


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--chars", type=int, default=200_000)
    ap.add_argument("--tokens", type=int, default=2000)
    ap.add_argument("--dim", type=int, default=256)
    ap.add_argument("--new", type=int, default=48)
    a = ap.parse_args()
    losses, _, texts = run(a.steps, a.chars, a.tokens, a.dim, a.new)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i:4d}  loss {losses[i]:.3f}")
    print(f"step {len(losses) - 1:4d}  loss {losses[-1]:.3f}")
    for name, t in zip(("greedy", "top-k 50, top-p 0.95", "top-p 0.9", "all"), texts):
        print(f"[{name}] {t!r}")


if __name__ == "__main__":
    main()
