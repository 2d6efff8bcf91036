"""A truth value that cannot be formed is its own error in the native calls."""
import pytest
import torch

import grad_row_online_gb300 as g
from test_abi import lib  # noqa: F401  (the built library)

NEITHER = torch.zeros(2)


def test_norm_only(lib):  # noqa: F811
    for tensors in ([torch.zeros(3)], [None]):
        with pytest.raises(RuntimeError, match="ambiguous"):
            g.grpo_clip_grad_norm(tensors, 1.0, norm_only=NEITHER)


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="no CUDA device")
def test_flags_of_the_token_calls():
    x = torch.randn((2, 3, 50), device="cuda")
    ids = torch.zeros((2, 3), dtype=torch.int64, device="cuda")
    f = g.grpo_token_logps(x, ids, want_stats=True)
    for name in ("want_entropy", "want_stats"):
        with pytest.raises(RuntimeError, match="ambiguous"):
            g.grpo_token_logps(x, ids, **{name: NEITHER})
    with pytest.raises(RuntimeError, match="ambiguous"):
        g.grpo_token_logps_grad(x, ids, None, f["stats"], grad_logps=f["logps"],
                                skip_masked_grad_rows=NEITHER)
    assert g.grpo_token_logps(x, ids, want_entropy=torch.ones(1))["entropy"] is not None
