"""Trains a language model's output matrix with the vocabulary losses.

The hidden states of a batch of tokens are given (random here, leaning
towards their own next token as a trained model's do); a teacher's output
matrix exists.  Each step takes the cross entropy against the next tokens
and the distillation from the teacher's best logits, adds their gradients and
moves the matrix.  The logits of the student are never stored; the teacher's
come once from the library's 16-bit product.

    python examples/train_head.py [--steps 20] [--tokens 2048] [--vocab 8000]
"""

from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from dense_fp32_matrix_02_gb300 import gemm, loss  # noqa: E402


def train(steps=20, tokens=2048, vocab=8000, width=512, top=16,
          temperature=2.0, rate=5.0, seed=0, device="cuda:0"):
    """The (cross entropy, distillation) means before each step and after
    the last."""
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=device)

    teacher = normal(vocab, width) * 2 / width ** 0.5
    targets = torch.randint(0, vocab, (tokens,), generator=gen, device=device)
    x = gemm.round16(normal(tokens, width) + 2 * teacher[targets])
    targets[: tokens // 8] = -100  # a prompt: not learnt from
    learnt = tokens - tokens // 8

    # the teacher's best logits, once
    logits = gemm.gemm_f32_mixed(x.float(), teacher.t().contiguous())
    top_logits, top_ids = logits.topk(top)
    del logits
    top_ids[targets < 0] = -1

    master = torch.zeros(vocab, width, device=device)  # the student, in fp32
    mean = torch.tensor(1.0 / learnt, device=device).expand(tokens)
    history = []
    for step in range(steps + 1):
        w = gemm.round16(master)
        ce, ce_lse = loss.cross_entropy(x, w, targets)
        kd, kd_lse = loss.distill(x, w, top_logits, top_ids, temperature)
        history.append((float(ce.sum() / learnt), float(kd.sum() / learnt)))
        if step == steps:
            return history
        _, dw = loss.cross_entropy_grad(x, w, targets, ce_lse, mean)
        _, dw2 = loss.distill_grad(x, w, top_logits, top_ids, kd_lse, mean,
                                   temperature)
        master -= rate * (dw.float() + dw2.float())


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("steps", 20), ("tokens", 2048), ("vocab", 8000),
                        ("width", 512), ("top", 16)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    for step, (ce, kd) in enumerate(train(a.steps, a.tokens, a.vocab, a.width,
                                          a.top)):
        print(f"step {step:3d}  cross entropy {ce:8.4f}  distillation "
              f"{kd:8.4f}")


if __name__ == "__main__":
    main()
