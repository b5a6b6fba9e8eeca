"""Distil a toy teacher into a toy student, with and without the student's logits in memory.

    python examples/distill_step.py [--steps 60]

One offline pass keeps the teacher's top-K logits and the logsumexp of its whole rows.  Then
  dense   a student that hands out its logits: KL with the teacher's remaining mass as one
          class, plus the hard-label term, on [N, V] logits
  fused   the same hard-label term and the KL straight from hidden states: no [N, V] logits
and at the end the trained student scores a few tokens, with its alternatives.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_teacher_kl_gb300 as kd  # noqa: E402

N, V, D, K, CHUNK = 512, 4096, 128, 32, 256
ALPHA = 0.5  # weight of the KL; 1 - ALPHA goes to the hard labels


def teacher_cache(g):
    """Hidden states, labels and the offline cache of a random teacher."""
    Ht = torch.randn((N, 256), generator=g, device="cuda").to(torch.bfloat16)
    Wt = (torch.randn((V, 256), generator=g, device="cuda") * 0.2).to(torch.bfloat16)
    ids, vals, lse = kd.teacher_topk(Ht, Wt, K, chunk=CHUNK, with_lse=True)
    labels = ids[:, 0].contiguous()  # the teacher's own choice as the hard label
    x = Ht[:, :D].float()            # what the student sees of the input
    return x, labels, ids, vals, lse


class Student(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.body = torch.nn.Linear(D, D)
        self.head = torch.nn.Parameter(torch.randn((V, D)) * D ** -0.5)

    def hidden(self, x):
        return torch.tanh(self.body(x)).to(torch.bfloat16)

    def weight(self):
        return self.head.to(torch.bfloat16)


def dense_loss(student, x, labels, ids, vals, lse):
    logits = student.hidden(x) @ student.weight().T
    logp, _ = kd.token_logprobs(logits, labels)
    return ALPHA * kd.logits_kl(logits, ids, vals, t_lse=lse) - (1 - ALPHA) * logp.mean()


def fused_loss(student, x, labels, ids, vals, lse):
    H, W = student.hidden(x).contiguous(), student.weight().contiguous()
    hard = kd.fused_cross_entropy(H, W, labels, chunk=CHUNK)
    return ALPHA * kd.fused_kl(H, W, ids, vals, chunk=CHUNK) + (1 - ALPHA) * hard


def train(loss_of, data, steps):
    torch.manual_seed(0)
    student = Student().cuda()
    opt = torch.optim.Adam(student.parameters(), lr=1e-2)
    first = last = 0.0
    for step in range(steps):
        opt.zero_grad()
        loss = loss_of(student, *data)
        loss.backward()
        opt.step()
        last = float(loss)
        first = last if step == 0 else first
    return student, first, last


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=60)
    steps = p.parse_args().steps
    g = torch.Generator(device="cuda").manual_seed(1)
    data = teacher_cache(g)
    for name, loss_of in (("dense", dense_loss), ("fused", fused_loss)):
        student, first, last = train(loss_of, data, steps)
        print(f"{name}: loss {first:.3f} -> {last:.3f} in {steps} steps")
        assert last < first
    x, labels = data[:2]
    with torch.no_grad():
        H, W = student.hidden(x[:4]).contiguous(), student.weight().contiguous()
        logp, _, entropy, _ = kd.fused_logprobs_forward(H, W, labels[:4].contiguous(), entropy=True)
        scores = kd.token_logprobs_forward(H @ W.T, labels[:4].contiguous(), top=3, entropy=True)
    for i in range(4):
        top = ", ".join(f"{int(t)} ({float(q):.2f})" for t, q in zip(scores.top_ids[i], scores.top_logp[i]))
        print(f"token {int(labels[i])}: log p {float(logp[i]):.2f} (from logits {float(scores.logp[i]):.2f}), "
              f"entropy {float(entropy[i]):.2f}; top 3: {top}")


if __name__ == "__main__":
    main()
