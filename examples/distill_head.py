"""Trains a 4-bit output head from a 16-bit teacher's best logits, then answers
tokens with the packed weights.

    python examples/distill_head.py [--steps 60] [--features 512] [--vocab 4096]

The teacher is a fixed norm and bf16 projection; its best logits of every
token are all that the student sees.  The student is an NVFP4Head: layer norm,
NVFP4 linear layer, distillation loss, and their gradients.  At the end its
weights are packed once, and single tokens are answered with the
matrix-vector product; how often the best answer is the teacher's is printed.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gemm_amax_reduce_amd.head import NVFP4Head  # noqa: E402


def teacher_lists(x, weight, top):
    """Indices and logits of the teacher's `top` best entries per token."""
    h = torch.nn.functional.layer_norm(x.float(), (x.shape[-1],))
    best = torch.topk(h @ weight.float().t(), top, dim=1)
    return best.indices, best.values


def train(steps=60, features=512, vocab=4096, tokens=1024, top=32, lr=1e-2, seed=0, log=print):
    """Runs the example; returns (first loss, last loss, agreement before and
    after, of answers with the teacher's)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    torch.manual_seed(seed + 1)                  # a student of other weights than the teacher
    teacher = 0.15 * torch.randn((vocab, features), device="cuda", generator=gen)
    head = NVFP4Head(features, vocab, device="cuda", dtype=torch.float32)
    opt = torch.optim.Adam(head.parameters(), lr=lr)
    held_out = torch.randn((64, features), device="cuda", generator=gen)
    wanted = teacher_lists(held_out, teacher, 1)[0][:, 0]

    def agreement():
        packed = head.pack()
        answers = [head.answer(held_out[i:i + 1], packed).argmax(-1) for i in range(held_out.shape[0])]
        return (torch.cat(answers) == wanted).float().mean().item()

    before = agreement()
    first = last = None
    for step in range(steps):
        x = torch.randn((tokens, features), device="cuda", generator=gen)
        indices, logits = teacher_lists(x, teacher, top)
        loss = head.loss(x, indices, logits)
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        if step % 10 == 0 or step == steps - 1:
            last = loss.item()
            first = last if first is None else first
            log(f"step {step:4d}  loss {last:.4f}")
    after = agreement()
    log(f"best answer as the teacher's: {before:.2f} before, {after:.2f} after")
    return first, last, before, after


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--features", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=4096)
    a = ap.parse_args()
    train(a.steps, a.features, a.vocab)
