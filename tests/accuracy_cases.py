"""Sharp rows for tests of accuracy: temperature 0.6, logits of deviation 3,
tokens drawn from the policy itself, so that an error of the logits shows in
full in log-probs and gradients."""
import math

import torch

TEMPERATURE, SIGMA = 0.6, 3.0


def make(N, K, V, dtype, device, seed):
    gen = torch.Generator(device=device).manual_seed(seed)
    h = torch.randn((N, K), generator=gen, device=device).to(dtype)
    W = (torch.randn((V, K), generator=gen, device=device) * (SIGMA / math.sqrt(K))).to(dtype)
    x = h.double() @ W.double().t()
    noise = torch.rand(x.shape, generator=gen, device=device, dtype=torch.float64).clamp_(1e-12, 1 - 1e-12)
    ids = (x / TEMPERATURE - (-noise.log()).log()).argmax(-1)
    w = torch.randn((N,), generator=gen, device=device)
    b = torch.randn((N,), generator=gen, device=device) * 0.1
    return h, W, ids, w, b


def exact(x, ids, s=1.0 / TEMPERATURE):
    """(log-probs, entropies) of logits x in 64 bits."""
    lp = torch.log_softmax(x * s, -1)
    return lp.gather(-1, ids[:, None])[:, 0], -(lp.exp() * lp).sum(-1)


def exact_d(x, ids, w, b, s=1.0 / TEMPERATURE):
    """The gradient of the logits x from those of log-probs and entropies, in 64 bits."""
    lp = torch.log_softmax(x * s, -1)
    p = lp.exp()
    H = -(p * lp).sum(-1, keepdim=True)
    d = -p * (w.double()[:, None] + b.double()[:, None] * (lp + H))
    return d.scatter_add_(-1, ids[:, None], w.double()[:, None]) * s


def off(got, want):
    """The difference's norm over the result's."""
    return float((got.double() - want).norm() / want.norm())


# Bounds of it, each about twice what the kernels' design gives, and below what
# they would give with less:
# - fp32 operands in three bf16 planes, six products: what is left out is of third
#   order, (1.7e-3)^3 = 5e-9, where one product more left out is of second, 3e-6 of
#   the logits' deviation; sums of 512 products, 1e-6 at most (5e-5 in one sum).
F32 = 3e-6
# - 16-bit operands: a logit is off by 2e-8 of its size for each block of 64 in one
#   sum, and sharp log-probs, in norm over many tokens, by some six times that.
#   Sums of up to 32 blocks: 4e-6 (twice that at a width of 4,096 in one sum).
WIDE = 6e-6
# - up to 128 tokens: sums of half that length.
SHORT = WIDE / 2


def logp_bound(x, blocks, s=1.0 / TEMPERATURE):
    """Of one token's log-prob and entropy, whatever their size: the token's own
    logit and those that make Z are each off by 2e-8 of the largest's size a block
    of one sum, and by as much as ten blocks for the fp32 arithmetic behind them.
    That is a figure in norm; the largest of 500 normal deviates is 3.1 of them."""
    return 3.1 * 2 * s * (2e-8 * blocks + 2e-7) * x.abs().amax(-1)


def rounded(dtype):
    """Gradients in 16 bits: the rounding of d to that type for its products, and
    the result's own, each eps / 2 times 0.43 in norm (uniform over a step, the
    steps' sizes over a binade); together 0.61."""
    return torch.finfo(dtype).eps / 2 * 0.77


# - fp32 grad_weight of 16-bit operands: d in two parts, off by 2^-17 of it, beside
#   the logits' error above.
TWO_PARTS = 1e-5
