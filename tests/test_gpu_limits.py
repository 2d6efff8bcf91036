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
