"""Logits of fp32 operands that leave the range of fp32."""
import pytest
import torch

import grad_row_online_gb300 as g
from linear_reference import forward
from test_gpu_linear import _built, make, scores  # noqa: F401  (builds the library)
from token_reference import assert_close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("big", [1e30, 1.003e30, 3e19])
def test_few_tokens_have_infinite_logits(big):
    """Multiplied as they are: -inf has p = 0; +inf, or nothing but -inf, has no distribution."""
    h, W, ids, _, w, b = make(6, 64, 300, "f32", seed=2)
    h[0] = big
    W[10:20] = -big
    ids[0] = 5
    s = scores(h, W, ids, None)
    ref = forward(h[:1], torch.cat([W[:10], W[20:]]), ids[:1], None)
    assert_close(s["logps"][:1], ref["logps"], ref["logps_tol"], "logps beside -inf")
    d = g.grpo_linear_logps_grad(h, W, ids, None, s["stats"], grad_logps=w.abs() + 1, grad_entropy=b,
                                 entropy=s["entropy"], grad_weight=None)
    assert not torch.isnan(d["grad_hidden"][0]).any()
    h[1], h[2] = -big, big
    W[:] = -big
    W[3] = 0
    h[3:] = 0
    s = scores(h, W, ids, None)
    assert bool(torch.isnan(s["logps"][1])) and bool(torch.isnan(s["stats"][1, 1]))
    assert bool(torch.isfinite(s["logps"][3:]).all()) and bool(torch.isfinite(s["stats"][1, 2]))
    W[3] = -big
    s = scores(h, W, ids, None)
    assert bool(torch.isnan(s["entropy"][:3]).all()) and bool(torch.isfinite(s["entropy"][3:]).all())


@pytest.mark.parametrize("N", [40, 300])
def test_parts_of_finite_operands_may_overflow(N):
    """Beyond 16 tokens the products of an operand's parts overflow on their own:
    such a logit is infinite or NaN, for its token alone."""
    h, W, ids, _, _, _ = make(N, 64, 300, "f32", seed=2)
    W[10:20] = -1.003e30
    ids[ids // 10 == 1] = 5
    h[:, 0], h[:, 1:] = h[:, 0].abs() + 1, h[:, 1:] * 1e-3  # (words 10 to 19 are far below the others)
    good = scores(h, W, ids, None)
    assert bool(torch.isfinite(good["logps"]).all()) and bool(torch.isfinite(good["entropy"]).all())
    row = N // 2
    h[row] = 1.003e30
    s = scores(h, W, ids, None)
    rest = torch.arange(N, device="cuda") != row
    for n in ("logps", "entropy"):
        assert torch.equal(s[n][rest], good[n][rest])
    assert bool(torch.isnan(s["logps"][row])) and bool(torch.isnan(s["entropy"][row]))
