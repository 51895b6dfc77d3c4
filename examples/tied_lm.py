"""A small language model with a tied table, trained by W data-parallel replicas on one GPU.

Each step runs the two ends of the model and the bucket reduction together, the way a
training loop uses them:

    x = scale * table[ids]            TokenEmbedding.forward
    h = tanh(x @ mix)                 (torch)
    loss = cross entropy of h against the same table    VocabLoss.forward
    dh, dtable = VocabLoss.backward   the projection's gradient,
    dtable += TokenEmbedding.backward  and the lookup's added to it: one gradient of the tied table
    BucketReducer.step                the replicas' gradients, averaged in ring order
    GradClipper.clip                  the reduced gradients, clipped by their global norm
    SGD on fp32 weights, bf16 copies for the next step

The task: the next token is a fixed function of the last one, and a third of the targets
carry no loss.

    python examples/tied_lm.py [steps]
"""
from __future__ import annotations

import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import allreduce_ddp_assign_gb300 as D
from allreduce_ddp_assign_gb300 import lm
from allreduce_ddp_assign_gb300.session import BucketReducer

VOCAB, DIM, TOKENS, W = 1009, 128, 512, 2
IGNORE = -100


def train(steps=60, lr=2.0, max_norm=0.5, seed=0, report=None):
    """(mean loss of each step, norms before clipping, the replicas' weights)"""
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    scale = math.sqrt(DIM)
    embed = lm.TokenEmbedding(VOCAB, DIM, torch.bfloat16, scale=scale)
    loss_of = lm.VocabLoss(VOCAB, DIM, torch.bfloat16, ignore_index=IGNORE)

    shapes = [(VOCAB, DIM), (DIM, DIM)]
    start = [torch.randn(s, generator=gen, device=dev) / math.sqrt(DIM) for s in shapes]
    master = [[p.clone() for p in start] for _ in range(W)]          # fp32, one set a replica
    grads = [[torch.zeros(s, dtype=torch.bfloat16, device=dev) for s in shapes] for _ in range(W)]
    numels = [p.numel() for p in start]
    reducer = BucketReducer(numels, [D.DDP_BF16] * len(numels), W, D.DDP_ALLREDUCE, D.DDP_ORDER_REVERSE, 25 << 20,
                            1 << 20, 1, grads, coalesce=True)
    clippers = [lm.GradClipper.of_reducer(reducer, w) for w in range(W)]

    losses, norms = [], []
    for step in range(steps):
        total = count = 0.0
        for w in range(W):
            table, mix = (p.to(torch.bfloat16) for p in master[w])
            ids = torch.randint(0, VOCAB, (TOKENS,), generator=gen, device=dev)
            targets = (ids * 7 + 3) % VOCAB
            targets[torch.rand(TOKENS, generator=gen, device=dev) < 1 / 3] = IGNORE
            valid = (targets != IGNORE).float()

            x = embed.forward(table, ids)
            hidden = torch.tanh(x.float() @ mix.float())
            h = hidden.to(torch.bfloat16)
            loss, lse = loss_of.forward(h, table, targets)
            dh, dtable = loss_of.backward(h, table, targets, lse, valid / valid.sum(), grad_weight=grads[w][0])
            dpre = dh.float() * (1 - hidden * hidden)
            grads[w][1].copy_(x.float().t() @ dpre)
            dx = (dpre @ mix.float().t()).to(torch.bfloat16)
            embed.backward(dx, ids, grad_weight=dtable, accumulate=True)
            total, count = total + loss.sum(), count + valid.sum()
        reducer.step()
        for w in range(W):
            norm = clippers[w].clip(max_norm)
            for p, weight in enumerate(master[w]):
                weight.sub_(reducer.view(p, w).view_as(weight), alpha=lr)
        losses.append(float(total / count))
        norms.append(float(norm))
        if report:
            report(step, losses[-1], norms[-1])
    reducer.close()
    return losses, norms, master


def main():
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 60

    def report(step, loss, norm):
        if step % 10 == 0 or step == steps - 1:
            print(f"step {step:4d}  loss {loss:.4f}  gradient norm {norm:.4f}")

    train(steps, report=report)


if __name__ == "__main__":
    main()
