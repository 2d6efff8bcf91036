"""How far log-probs, entropies and gradients are from 64 bits, in norm: bounds
that less exact products, shorter parts or single sums would not keep."""
import pytest
import torch

import grad_row_online_gb300 as g
from accuracy_cases import F32, SHORT, TEMPERATURE, TWO_PARTS, WIDE, exact, exact_d, logp_bound, make, off, rounded

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import os
    import __graft_entry__
    if not os.path.exists(g.library_path()):
        __graft_entry__.build()


def scores(h, W, ids):
    return g.grpo_linear_logps(h, W, ids, temperature=TEMPERATURE, want_entropy=True, want_stats=True)


def gradient(h, W, ids, s, w, b, **more):
    return g.grpo_linear_logps_grad(h, W, ids, None, s["stats"], grad_logps=w, entropy=s["entropy"], grad_entropy=b,
                                    temperature=TEMPERATURE, **more)


@pytest.mark.parametrize("N,K,V", [(1, 2048, 9000), (12, 4096, 5000), (17, 512, 9000), (64, 2048, 9000),
                                   (100, 4096, 3000), (128, 512, 9000), (300, 512, 9000), (300, 4096, 3000), (1000, 1021, 5000)])
def test_fp32(N, K, V):
    h, W, ids, w, b = make(N, K, V, torch.float32, "cuda", N + K)
    s = scores(h, W, ids)
    x = h.double() @ W.double().t()
    logps, entropy = exact(x, ids)
    d = exact_d(x, ids, w, b)
    r = gradient(h, W, ids, s, w, b)
    found = {"logps": off(s["logps"], logps), "entropy": off(s["entropy"], entropy),
             "grad_hidden": off(r["grad_hidden"], d @ W.double()), "grad_weight": off(r["grad_weight"], d.t() @ h.double())}
    print(N, K, V, found)
    assert max(found.values()) <= F32, found


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N,K,V", [(1, 2048, 9000), (64, 2048, 9000), (100, 4096, 3000), (128, 8320, 3000), (300, 1024, 9000),
                                   (300, 2048, 9000), (500, 4096, 5000), (200, 8320, 3000)])
def test_scores_of_16_bits(dtype, N, K, V):
    h, W, ids, _, _ = make(N, K, V, DT[dtype], "cuda", N + K)
    s = scores(h, W, ids)
    x = h.double() @ W.double().t()
    logps, entropy = exact(x, ids)
    found = {"logps": off(s["logps"], logps), "entropy": off(s["entropy"], entropy)}
    print(dtype, N, K, V, found)
    if N > 1:
        assert max(found.values()) <= (SHORT if N <= 128 and K <= 4096 else WIDE), found
    blocks = min(32, -(-K // 64) / (4 if K > 2048 else 2)) if N <= 128 else min(32, -(-K // 64))
    for n, want in (("logps", logps), ("entropy", entropy)):
        far = (s[n].double() - want).abs() / logp_bound(x, blocks)
        print(n, float(far.max()))
        assert float(far.max()) <= 1


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N,K,V", [(20, 512, 9000), (128, 2048, 5000), (700, 1024, 9000), (5000, 256, 3000), (14000, 128, 2000),
                                   (1, 64, 700), (100, 4096, 3000), (60, 8320, 1500), (300, 4096, 3000)])
def test_gradients_of_16_bits(dtype, N, K, V):
    """grad_weight of the operands' type and, more exactly, in fp32; added to what is there."""
    h, W, ids, w, b = make(N, K, V, DT[dtype], "cuda", N + K)
    s = scores(h, W, ids)
    d = exact_d(h.double() @ W.double().t(), ids, w, b)
    gh, gw = d @ W.double(), d.t() @ h.double()
    r = gradient(h, W, ids, s, w, b)
    wide = gradient(h, W, ids, s, w, b, grad_weight=torch.empty(W.shape, device="cuda"))
    found = {"grad_hidden": off(r["grad_hidden"], gh), "grad_weight": off(r["grad_weight"], gw),
             "grad_hidden beside fp32": off(wide["grad_hidden"], gh)}
    exactly = off(wide["grad_weight"], gw)
    print(dtype, N, K, V, found, exactly)
    assert max(found.values()) <= rounded(DT[dtype]), found
    assert exactly <= TWO_PARTS
    add = torch.randn(W.shape, device="cuda")
    more = gradient(h, W, ids, s, w, b, add_weight=add, grad_hidden=None)
    assert off(more["grad_weight"], gw + add.double()) <= TWO_PARTS


@pytest.mark.parametrize("N,K", [(17, 512), (64, 256), (128, 512), (128, 100), (128, 2048), (300, 512)])
def test_the_gradient_forms_the_logits_of_its_statistics(N, K):
    """Each row's p sums up to 1: a word's logit is the same number in the forward
    pass and the gradient, and so is its exponential, but for some eight roundings
    of 2^-24: Z's sum and its scalings to a larger maximum, 1 / Z and its products."""
    h, W, ids, w, _ = make(N, K, 9000, torch.float32, "cuda", N + K)
    h[:, :16] = 0.0
    h[:16, :16] = torch.eye(16, device="cuda")  # (column t of grad_weight: d of token t)
    s = scores(h, W, ids)
    d = g.grpo_linear_logps_grad(h, W, ids, None, s["stats"], grad_logps=torch.ones_like(w), temperature=TEMPERATURE,
                                 grad_hidden=None)["grad_weight"][:, :16]
    far = d.double().sum(0).abs() * TEMPERATURE
    print(N, K, float(far.max()))
    assert float(far.max()) <= 8 * 2.0 ** -24
