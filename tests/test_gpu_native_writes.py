"""What the native calls write is seen by autograd."""
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


def _scored(x):
    ids = torch.zeros(x.shape[:-1], dtype=torch.int64, device="cuda")
    f = g.grpo_token_logps(x, ids, want_stats=True)
    return ids, f["stats"], torch.ones_like(f["logps"])


def test_an_overwritten_saved_tensor_is_an_error():
    """sin saves its input; the gradient written over it must not be taken for it."""
    leaf = torch.randn((4, 100), device="cuda", requires_grad=True)
    z = leaf * 1.0
    y = z.sin()
    ids, stats, w = _scored(z)
    g.grpo_token_logps_grad(z, ids, None, stats, grad_logps=w, grad=z)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()
    z = leaf * 1.0
    y = z.sin()
    g.grpo_clip_grad_norm([z], 1e-3)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()


def test_versions():
    x = torch.randn((4, 100), device="cuda")
    ids, stats, w = _scored(x)
    base = torch.zeros((8, 100), device="cuda")
    versions = lambda *ts: [t._version for t in ts]
    before = versions(x, stats, w, base)
    d = g.grpo_token_logps_grad(x, ids, None, stats, grad_logps=w)
    assert versions(x, stats, w, base) == before and d._version == 0
    g.grpo_token_logps_grad(x, ids, None, stats, grad_logps=w, grad=base[:4])  # a view shares its base's
    assert base._version == before[3] + 1
    a, b = torch.ones(10, device="cuda"), torch.ones(5, device="cuda").bfloat16()
    out = [torch.zeros_like(a), torch.zeros_like(b)]
    before = versions(a, b, *out)
    g.grpo_clip_grad_norm([a, b], 1.0, norm_only=True)
    with pytest.raises(g.GrpoError):
        g.grpo_clip_grad_norm([a, b], -1.0)
    assert versions(a, b, *out) == before
    g.grpo_clip_grad_norm([a, b], 1.0, out=out)
    assert versions(a, b) == before[:2] and versions(*out) == [v + 1 for v in before[2:]]
    g.grpo_clip_grad_norm([a, b], 1.0)
    assert versions(a, b) == [v + 1 for v in before[:2]]


def test_inference_tensors():
    """(they have no version counter)"""
    with torch.inference_mode():
        x = torch.randn((4, 100), device="cuda")
        ids, stats, w = _scored(x)
        want = g.grpo_token_logps_grad(x, ids, None, stats, grad_logps=w)
        g.grpo_token_logps_grad(x, ids, None, stats, grad_logps=w, grad=x)
        assert torch.equal(x, want)
        g.grpo_clip_grad_norm([x], 1e-3)
    g.grpo_clip_grad_norm([x], 1e-4)
    assert abs(float(x.norm()) - 1e-4) < 1e-6
