"""Embedding, head log-probs, loss, both gradients and the clipping together, as
a step calls them, against PyTorch's autograd in 64 bits: an untied and a tied
weight (whose two gradients meet in one buffer)."""
import os
import sys

import pytest
import torch

import grad_row_online_gb300 as g
from linear_reference import gradient
from token_reference import U

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


def step_inputs(B, T, V, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    tokens = torch.randint(0, V, (B, T), generator=gen, device="cuda")
    actions = torch.randint(0, V, (B, T), generator=gen, device="cuda")
    mask = torch.arange(T, device="cuda") < torch.randint(1, T + 1, (B, 1), generator=gen, device="cuda")
    return gen, tokens, actions, mask, torch.rand(B, generator=gen, device="cuda")


def reference(emb, weight, tokens, actions, mask, old, rewards, scale, temp, bonus):
    """The loss and the gradients of emb and weight by autograd."""
    lsm = torch.log_softmax(scale * emb[tokens] @ weight.t() / temp, -1)
    lp = lsm.gather(-1, actions[..., None])[..., 0]
    H = -(lsm.exp() * lsm).sum(-1)
    R = rewards.double().reshape(-1, 4)
    A = ((R - R.mean(1, keepdim=True)) / R.std(1, unbiased=False, keepdim=True)).reshape(-1, 1)
    r = (lp - old.double()).exp()
    p = -torch.minimum(r * A, r.clamp(0.8, 1.2) * A)
    ((p - bonus * H) * mask).sum().div(mask.sum()).backward()
    return float((p.detach() * mask).sum() / mask.sum())


@pytest.mark.parametrize("B,T,D,V", [(8, 5, 16, 611), (16, 33, 72, 3001)])
def test_example_step_against_autograd(B, T, D, V):
    import train_step
    pol = train_step.Policy(V, D, 3)
    gen, tokens, actions, mask, rewards = step_inputs(B, T, V, 4)
    temp, bonus = 0.9, 0.01
    h = pol.hidden(tokens)
    assert torch.equal(h, pol.embedding[tokens])
    new = g.grpo_linear_logps(h, pol.weight, actions, mask, temperature=temp, want_entropy=True, want_stats=True)
    old = new["logps"] + 0.1 * torch.randn((B, T), generator=gen, device="cuda")
    loss = g.grpo_loss_from_logps(new["logps"], old, None, mask, rewards, samples_per_prompt=4, beta=0.0)
    grads = pol.backward(tokens, h, actions, mask, new, loss["grad"], mask * (-bonus / mask.sum()), temp)
    emb, head = (p.double().requires_grad_() for p in pol.parameters())
    want = reference(emb, head.t(), tokens, actions, mask, old, rewards, 1.0, temp, bonus)
    assert abs(float(loss["loss"]) - want) < 1e-5
    # fp32 sums of up to D, V or B T terms, formed 16 at a time, logits and log-probs of fp32
    for a, b in zip(grads, (emb.grad, head.grad)):
        assert float((a.double() - b).abs().max()) <= 600 * U * float(b.abs().max())
    # the logits path of the same policy gives the same gradients
    z = pol.logits(tokens)
    other = g.grpo_token_logps(z, actions, mask, temperature=temp, want_entropy=True, want_stats=True)
    d = g.grpo_token_logps_grad(z, actions, mask, other["stats"], grad_logps=loss["grad"],
                                entropy=other["entropy"], grad_entropy=mask * (-bonus / mask.sum()), temperature=temp)
    for a, b in zip(grads, pol.gradients(tokens, d)):
        assert float((a - b).abs().max()) <= 1200 * U * float(b.abs().max())
    norm = sum(float(x.double().square().sum()) for x in (emb.grad, head.grad)) ** 0.5
    res = g.grpo_clip_grad_norm(grads, 1e-3)
    assert abs(float(res["norm"]) - norm) <= 1e-4 * norm


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tied_weight(dtype):
    """One matrix at both ends; the embedding's gradient is added to the head's
    in single precision, in place."""
    B, T, K, V, scale, temp, bonus = 12, 40, 64, 1500, 8.0, 1.0, 0.02
    gen, tokens, actions, mask, rewards = step_inputs(B, T, V, 7)
    W = (torch.randn((V, K), generator=gen, device="cuda") * 0.05).to(dtype)
    status = g.status_buffer()
    h = g.grpo_embed_tokens(W, tokens, scale=scale, status=status)
    new = g.grpo_linear_logps(h, W, actions, mask, temperature=temp, want_entropy=True, want_stats=True, status=status)
    old = new["logps"] + 0.1 * torch.randn((B, T), generator=gen, device="cuda")
    loss = g.grpo_loss_from_logps(new["logps"], old, None, mask, rewards, samples_per_prompt=4, beta=0.0)
    dentropy = mask * (-bonus / mask.sum())
    total = torch.zeros((V, K), device="cuda")
    d = g.grpo_linear_logps_grad(h, W, actions, mask, new["stats"], grad_logps=loss["grad"], entropy=new["entropy"],
                                 grad_entropy=dentropy, temperature=temp, grad_weight=total, add_weight=total,
                                 status=status)
    g.grpo_embed_tokens_grad(d["grad_hidden"], tokens, V, mask, scale=scale, add=total, out=total, status=status)
    assert g.grpo_read_device_status(status) == 0
    # autograd of h (as it was rounded) and of W at the head, then the embedding's sum
    hd, Wd = h.double().requires_grad_(), W.double().requires_grad_()
    lsm = torch.log_softmax(hd @ Wd.t() / temp, -1)
    lp = lsm.gather(-1, actions[..., None])[..., 0]
    H = -(lsm.exp() * lsm).sum(-1)
    ((lp * loss["grad"].double() + H * dentropy.double()) * mask).sum().backward()
    on = mask.reshape(-1)
    want = Wd.grad.index_add(0, tokens.reshape(-1)[on], scale * hd.grad.reshape(-1, K)[on])
    flat = lambda x: x.reshape(-1, *x.shape[2:])  # noqa: E731
    _, gh_tol, _, gw_tol = gradient(flat(h), W, flat(actions), on, flat(loss["grad"]), flat(dentropy), temp,
                                    wdtype=torch.float32)
    tol = gw_tol.index_add(0, flat(tokens)[on], scale * gh_tol[on])
    tol = tol + 64 * U * (want.abs() + Wd.grad.abs())  # (sums of a few tokens, in fp32)
    assert float(((total.double() - want).abs() - tol).max()) <= 0


def test_the_example_runs():
    import train_step
    history = train_step.train(steps=3, V=203, D=24, T=9)
    assert len(history) == 3 and all(0 <= x <= 1 for x in history)


def test_a_captured_step_beside_an_eager_one():
    """The whole step captured and replayed, with eager calls on the same tensors between."""
    B, T, K, V = 8, 24, 64, 900
    gen, tokens, actions, mask, rewards = step_inputs(B, T, V, 5)
    W = torch.randn((V, K), generator=gen, device="cuda").bfloat16()

    def step():
        h = g.grpo_embed_tokens(W, tokens)
        new = g.grpo_linear_logps(h, W, actions, mask, want_stats=True)
        dlogp = new["logps"] * 0.01
        d = g.grpo_linear_logps_grad(h, W, actions, mask, new["stats"], grad_logps=dlogp)
        return g.grpo_embed_tokens_grad(d["grad_hidden"], tokens, V, mask, add=d["grad_weight"])

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        graph.replay()
        eager = step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(eager, want)
