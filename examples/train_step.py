"""A GRPO training loop on a policy small enough to read: the log-prob entry
points, the loss and the gradient clipping together, as a trainer calls them.

    python examples/train_step.py [--steps N]

The policy is a bigram model, logits[t] = embedding[token[t]] @ head.  Each
step samples completions at a temperature, scores them (grpo_token_logps: the
behaviour log-probs, with the alternatives a log would show), rewards a
completion for the tokens it takes from a target set, and takes a few updates:

    logits -> grpo_token_logps -> grpo_loss_from_logps (dL/dlogp)
           -> grpo_token_logps_grad (+ entropy bonus) -> the model's gradients
           -> grpo_clip_grad_norm -> SGD
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import grad_row_online_gb300 as g  # noqa: E402


class Policy:
    def __init__(self, V: int, D: int, seed: int):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.embedding = torch.randn((V, D), generator=gen, device="cuda") * 0.3
        self.head = torch.randn((D, V), generator=gen, device="cuda") * 0.3

    def parameters(self):
        return [self.embedding, self.head]

    def logits(self, tokens):
        return self.embedding[tokens] @ self.head

    def gradients(self, tokens, dlogits):
        """[dL/dembedding, dL/dhead] from dL/dlogits."""
        d, t = dlogits.flatten(0, 1), tokens.flatten()
        hidden = self.embedding[t]
        demb = torch.zeros_like(self.embedding).index_add_(0, t, d @ self.head.t())
        return [demb, hidden.t() @ d]


def train(steps=30, prompts=8, samples=8, T=24, V=601, D=32, lr=300.0, updates=2, temperature=1.0,
          entropy_bonus=1e-3, max_norm=0.05, seed=0):
    """Returns the mean reward of every step."""
    policy = Policy(V, D, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    B = prompts * samples
    good = torch.arange(V, device="cuda") % 4 == 0
    status = g.status_buffer()
    history = []
    for _ in range(steps):
        # rollout: one token at a time, scored as it is drawn (the serving form)
        first = torch.randint(0, V, (prompts,), generator=gen, device="cuda").repeat_interleave(samples)
        inputs = torch.empty((B, T), dtype=torch.int64, device="cuda")
        actions, old = torch.empty_like(inputs), torch.empty((B, T), device="cuda")
        token = first
        for t in range(T):
            inputs[:, t] = token
            z = policy.logits(token)
            token = torch.multinomial(torch.softmax(z / temperature, -1), 1, generator=gen)[:, 0]
            scored = g.grpo_token_logps(z, token, temperature=temperature, top_k=4)
            actions[:, t], old[:, t] = token, scored["logps"]
        lengths = torch.randint(T // 2, T + 1, (B,), generator=gen, device="cuda")
        mask = torch.arange(T, device="cuda") < lengths[:, None]
        rewards = (good[actions] & mask).sum(1).float() / lengths
        history.append(float(rewards.mean()))
        for _ in range(updates):
            z = policy.logits(inputs)
            new = g.grpo_token_logps(z, actions, mask, temperature=temperature, want_entropy=True,
                                     want_stats=True, status=status)
            loss = g.grpo_loss_from_logps(new["logps"], old, None, mask, rewards,
                                          samples_per_prompt=samples, beta=0.0, clip_eps=0.2,
                                          clip_eps_hi=0.28)
            dentropy = mask * (-entropy_bonus / mask.sum())
            dlogits = g.grpo_token_logps_grad(z, actions, mask, new["stats"],
                                              grad_logps=loss["grad"], entropy=new["entropy"],
                                              grad_entropy=dentropy, temperature=temperature,
                                              grad=z)  # in place: z is not needed again
            grads = policy.gradients(inputs, dlogits)
            g.grpo_clip_grad_norm(grads, max_norm)
            for p, d in zip(policy.parameters(), grads):
                p.sub_(d, alpha=lr)
    if g.grpo_read_device_status(status) != 0:
        raise RuntimeError("an action id outside the vocabulary")
    return history


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    for i, r in enumerate(train(a.steps)):
        print(f"step {i:3d}  mean reward {r:.3f}")


if __name__ == "__main__":
    main()
