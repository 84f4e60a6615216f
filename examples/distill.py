"""A student taught by a teacher's top logits, then by a reward.

    python examples/distill.py [--rows 256] [--vocab 32000] [--steps 30]

The student is a table of logits, a row per context, so that the vocabulary rows are
all there is to train. Its life runs through the library's operators as a
language model's would:

1. the teacher's pass: its 64 likeliest tokens and their log probabilities
   (token_logprobs);
2. distillation: the loss against them, what they leave of 1 as one more
   outcome, and its gradient in one call (distill_topk_step);
3. a policy gradient with an entropy bonus, for a reward on tokens drawn from the
   student (token_logprobs in automatic differentiation);
4. the greedy answer (argmax).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import row_wise_arg_gb300 as A  # noqa: E402


def main(rows=256, vocab=32000, steps=30, seed=0, say=print):
    gen = torch.Generator("cuda").manual_seed(seed)
    teacher_logits = (torch.randn(rows, vocab, device="cuda", generator=gen) * 3).bfloat16()
    student = torch.zeros(rows, vocab, device="cuda")

    # 1. what the teacher says
    taught = A.token_logprobs(teacher_logits, top_k=64)

    # 2. distillation: plain gradient steps on the mean loss
    weight = torch.full((rows,), 1.0 / rows, device="cuda")
    losses = []
    for _ in range(steps):
        loss, grad = A.distill_topk_step(student, taught.top_ids, taught.top_logprobs, weight, tail=True)
        student.sub_(grad, alpha=8.0 * rows)
        losses.append(loss.mean().item())
    greedy = A.argmax(student)
    agree = (greedy == taught.top_ids[:, 0]).float().mean().item()
    say(f"distillation: loss {losses[0]:.3f} -> {losses[-1]:.3f}, greedy answers as the teacher's: {agree:.0%}")

    # 3. the same student, rewarded for even tokens
    policy = student.clone().requires_grad_()
    rewards = []
    for _ in range(steps):
        with torch.no_grad():
            noise = torch.rand(rows, vocab, device="cuda", generator=gen).clamp_(1e-9, 1 - 1e-7)
            tokens = A.argmax(policy - torch.log(-torch.log(noise)))  # a draw from the softmax
        reward = (tokens % 2 == 0).float()
        r = A.token_logprobs(policy, tokens)
        objective = ((reward - 0.5) * r.logprob + 0.01 * r.entropy).mean()
        (grad,) = torch.autograd.grad(-objective, policy)
        with torch.no_grad():
            policy.sub_(grad, alpha=8.0 * rows)
        rewards.append(reward.mean().item())
    say(f"policy gradient: reward {sum(rewards[:5]) / 5:.2f} -> {sum(rewards[-5:]) / 5:.2f}")

    # 4. what it answers, and how sure it is
    after = A.token_logprobs(policy.detach(), A.argmax(policy.detach()), top_k=3)
    say(f"greedy log probability {after.logprob.mean().item():.3f}, entropy {after.entropy.mean().item():.3f} nats")
    return losses, agree, rewards


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--rows", type=int, default=256)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    main(a.rows, a.vocab, a.steps)
