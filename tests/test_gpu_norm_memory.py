"""The results of the clipping call hold no more memory than they show."""
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


def test_a_norm_holds_its_own_bytes():
    res = g.grpo_clip_grad_norm([torch.ones(10, device="cuda") for _ in range(3)], 1.0)
    for v in (res["norm"], res["factor"]):
        assert v.untyped_storage().nbytes() <= 64


def test_kept_norms_do_not_grow():
    """A trainer's list of a thousand norms: a block of the allocator each
    (512 bytes) at most, not a workspace."""
    t = [torch.ones(10, device="cuda")]
    g.grpo_clip_grad_norm(t, 1.0)
    before = torch.cuda.memory_allocated()
    kept = [g.grpo_clip_grad_norm(t, 1.0)["norm"] for _ in range(1000)]
    assert torch.cuda.memory_allocated() - before <= 512 * len(kept)
    assert all(float(n) <= 3.2 for n in kept[::100])
