"""Gradient norms at and beyond the end of the fp32 range.

A norm that is infinite as an fp32 number leaves every output as it was and
makes the factor NaN, even where every gradient is finite and the sum of the
squares is held in 64 bits."""
import math

import pytest
import torch

import grad_row_online_gb300 as g
from token_reference import U, half_step

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import os
    import __graft_entry__
    if not os.path.exists(g.library_path()):
        __graft_entry__.build()


def full(n, value, dtype):
    return torch.full((n,), value, device="cuda", dtype=dtype)


# finite gradients whose norm is 2^128 or more
BEYOND = {
    "four": lambda: [full(4, 2.0 ** 127, torch.float32)],
    "many": lambda: [full(50_000, 3e38, torch.float32), full(100, 0.0, torch.float32)],
    "bf16": lambda: [full(999, 2.0 ** 126, torch.bfloat16), full(7, 1.0, torch.float16)],
}


@pytest.mark.parametrize("name", BEYOND)
@pytest.mark.parametrize("max_norm", [0.0, 1.0, 1e38, math.inf])
def test_an_infinite_norm_leaves_everything(name, max_norm):
    ts = BEYOND[name]()
    keep = [t.clone() for t in ts]
    res = g.grpo_clip_grad_norm(ts, max_norm)
    assert float(res["norm"]) == math.inf and math.isnan(float(res["factor"]))
    assert all(torch.equal(a, b) for a, b in zip(ts, keep))
    out = [torch.full_like(t, 2.0) for t in ts]
    res = g.grpo_clip_grad_norm(ts, max_norm, out=out)
    assert float(res["norm"]) == math.inf and math.isnan(float(res["factor"]))
    assert all((o == 2).all() for o in out)


@pytest.mark.parametrize("scale", [1.0, 0.5])
def test_the_largest_norms_are_clipped(scale):
    """norm = 1.5 2^127 scale, exactly: within the range, so it is clipped."""
    ts = [full(4, 0.75 * 2.0 ** 127, torch.float32)]
    out = [torch.zeros_like(ts[0])]
    res = g.grpo_clip_grad_norm(ts, 2.0 ** 100, eps=0.0, scale=scale, out=out)
    assert float(res["norm"]) == 1.5 * 2.0 ** 127 * scale
    want = 0.5 * 2.0 ** 100  # each of four
    # the factor's rounding and the product's
    assert abs(float(out[0][0]) - want) <= (U + half_step(torch.float32)) * 1.01 * want
    assert torch.equal(out[0], out[0][:1].expand(4))


def test_a_scale_brings_the_norm_into_the_range():
    ts = [full(4, 2.0 ** 127, torch.float32)]
    res = g.grpo_clip_grad_norm(ts, math.inf, scale=2.0 ** -10)
    assert float(res["norm"]) == 2.0 ** 118 and float(res["factor"]) == 2.0 ** -10
    assert (ts[0] == 2.0 ** 117).all()


def test_norm_only_gives_the_factor_of_the_64_bit_norm():
    ts = [full(4, 2.0 ** 127, torch.float32)]
    res = g.grpo_clip_grad_norm(ts, 2.0 ** 100, norm_only=True)
    assert float(res["norm"]) == math.inf and float(res["factor"]) == 2.0 ** -28
    assert (ts[0] == 2.0 ** 127).all()
