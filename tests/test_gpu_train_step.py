"""The log-prob entry points, the loss and the clipping together: the example
learns, and its gradients are those of the whole chain in 64 bits."""
import os
import sys

import pytest
import torch

import grad_row_online_gb300 as g

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    if not os.path.exists(g.library_path()):
        __graft_entry__.build()


def test_the_example_learns():
    import train_step
    history = train_step.train(steps=25)
    # a quarter of the tokens earns a reward: chance is 0.25
    assert sum(history[:3]) / 3 < 0.35 and sum(history[-3:]) / 3 > 0.6, history


def test_chain_against_autograd():
    """Loss and gradients of one step against PyTorch's autograd in 64 bits."""
    import train_step
    B, T, V = 8, 5, 611
    pol = train_step.Policy(V, 16, 3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    inputs = torch.randint(0, V, (B, T), generator=gen, device="cuda")
    actions = torch.randint(0, V, (B, T), generator=gen, device="cuda")
    mask = torch.arange(T, device="cuda") < torch.randint(1, T + 1, (B, 1), generator=gen, device="cuda")
    rewards = torch.rand(B, generator=gen, device="cuda")
    temp, bonus = 0.9, 0.01

    z = pol.logits(inputs)
    new = g.grpo_token_logps(z, actions, mask, temperature=temp, want_entropy=True, want_stats=True)
    old = new["logps"] + 0.1 * torch.randn((B, T), generator=gen, device="cuda")
    loss = g.grpo_loss_from_logps(new["logps"], old, None, mask, rewards, samples_per_prompt=4,
                                  beta=0.0)
    N = mask.sum()
    d = g.grpo_token_logps_grad(z, actions, mask, new["stats"], grad_logps=loss["grad"],
                                entropy=new["entropy"], grad_entropy=mask * (-bonus / N),
                                temperature=temp)
    grads = pol.gradients(inputs, d)
    clipped = [x.clone() for x in grads]
    res = g.grpo_clip_grad_norm(clipped, 1e-3)

    emb, head = (p.double().requires_grad_() for p in pol.parameters())
    lsm = torch.log_softmax(emb[inputs] @ head / temp, -1)
    lp = lsm.gather(-1, actions[..., None])[..., 0]
    H = -(lsm.exp() * lsm).sum(-1)
    R = rewards.double().reshape(2, 4)
    A = ((R - R.mean(1, keepdim=True)) / R.std(1, unbiased=False, keepdim=True)).reshape(-1, 1)
    r = (lp - old.double()).exp()
    p = -torch.minimum(r * A, r.clamp(0.8, 1.2) * A)
    total = ((p - bonus * H) * mask).sum() / N
    total.backward()
    assert abs(float(loss["loss"]) - float((p.detach() * mask).sum() / N)) < 1e-5
    ref = [emb.grad, head.grad]
    # fp32 products with 16 or 40 terms, logits and log-probs of fp32: 300 roundings of the largest
    for a, b in zip(grads, ref):
        assert float((a.double() - b).abs().max()) <= 300 * 2.0 ** -24 * float(b.abs().max())
    norm = sum(float(b.square().sum()) for b in ref) ** 0.5
    assert abs(float(res["norm"]) - norm) <= 1e-4 * norm
    for a, b in zip(clipped, ref):
        want = b * (1e-3 / (norm + 1e-6))
        assert float((a.double() - want).abs().max()) <= 1e-4 * float(want.abs().max())
