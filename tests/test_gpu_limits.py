"""The head's and the embedding's entry points at their largest sizes."""
import pytest
import torch

import grad_row_online_gb300 as g

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import os
    import __graft_entry__
    if not os.path.exists(g.library_path()):
        __graft_entry__.build()


def room(gb):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"{gb} GB are not free")


def test_embedding_gradient_of_two_billion_tokens():
    """The sort's last chunk ends at 2^31: every token is counted once.  (The
    sums are whole numbers below 2^24, exact in fp32 in any order.)"""
    room(80)
    B, T, V = 65536, 32767, 1000
    N = B * T
    ids = torch.arange(N, device="cuda").remainder_(V).view(B, T)
    out = g.grpo_embed_tokens_grad(torch.ones((1,), device="cuda").expand(B, T, 1), ids, V)
    v = torch.arange(V, device="cuda")
    assert torch.equal(out[:, 0].long(), N // V + (v < N % V).long())
    del ids
    torch.cuda.empty_cache()


def test_head_of_a_billion_words():
    """More tiles of words than 2^31 holds of the rows' 32 MB: each token's own
    logit comes from its tile, Z from all.  A warp of the join adds 65,536
    records in groups of four, a rounding of 2^-24 each at most."""
    room(60)
    N, K, V = 129, 8, 1 << 30
    gen = torch.Generator(device="cuda").manual_seed(0)
    W = torch.empty((V, K), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    h = torch.randn((N, K), generator=gen, device="cuda").bfloat16()
    ids = torch.randint(0, V, (N,), generator=gen, device="cuda")
    ids[:4] = torch.tensor([0, V - 1, V - 256, 255], device="cuda")
    got = g.grpo_linear_logps(h, W, ids, want_stats=True)
    torch.cuda.empty_cache()
    parts = [h.float() @ w.float().t() for w in (W[:1 << 22],)]  # (the first part's maxima are good references)
    ref = parts.pop().amax(-1, keepdim=True)
    top, Z = ref.clone(), torch.zeros((N,), dtype=torch.float64, device="cuda")
    for w in W.split(1 << 22):
        z = h.float() @ w.float().t()
        top = torch.maximum(top, z.amax(-1, keepdim=True))
        Z += z.sub_(ref).exp_().sum(-1).double()
    x = (h.double() * W[ids].double()).sum(-1)
    want = x - ref[:, 0].double() - Z.log()
    tol = 65536 * 2.0 ** -24 + 2.0 ** -18 * top[:, 0].double().abs()
    assert bool(((got["logps"].double() - want).abs() <= tol).all())
    assert bool(((got["stats"][0] - top[:, 0]).abs() <= 2.0 ** -18 * top[:, 0].abs()).all())
    del W, z
    torch.cuda.empty_cache()
