"""The embedding of tokens and its gradient by sorted tokens against 64-bit
statements of the formulas."""
import math

import pytest
import torch

import grad_row_online_gb300 as g
from token_reference import U, assert_close, half_step, smallest

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


def make(N, K, V, dtype, seed=0, frequent=0.3, pad=0):
    """Ids with a few frequent ones among them; rows padded beyond K."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    W = torch.randn((V, K + pad), generator=gen, device="cuda").to(DT[dtype])[:, :K]
    ids = torch.randint(0, V, (N,), generator=gen, device="cuda")
    often = torch.rand((N,), generator=gen, device="cuda") < frequent
    ids = torch.where(often, ids % max(1, V // 50), ids)
    mask = torch.rand((N,), generator=gen, device="cuda") >= 0.2
    grad = torch.randn((N, K + pad), generator=gen, device="cuda").to(DT[dtype])[:, :K]
    return W, ids, mask, grad


def check_gradient(got, grad, ids, mask, V, scale, add=None):
    rows = grad.double()
    on = torch.ones_like(ids, dtype=torch.bool) if mask is None else mask.bool()
    zero = torch.zeros((V, grad.shape[1]), dtype=torch.float64, device="cuda")
    want = zero.index_add(0, ids[on], rows[on]) * scale
    mag = zero.index_add(0, ids[on], rows[on].abs()) * abs(scale)
    # one rounding a token, three behind the sum
    counts = torch.bincount(ids[on], minlength=V)[:, None].double()
    tol = U * (counts + 3) * mag
    if add is not None:
        want = want + add.double()
        tol = tol + U * want.abs()
    tol = tol + half_step(got.dtype) * 1.01 * (want.abs() + tol) + smallest(got.dtype)
    assert_close(got, want, torch.where(want == 0, torch.where(mag > 0, tol, torch.zeros_like(tol)), tol), "gradient")


SIZES = [(1, 1, 1, 0), (1, 64, 100, 0), (5, 3, 2, 0), (33, 129, 50, 0), (64, 4096, 3000, 0),
         (31, 8, 1 << 20, 0), (1000, 65, 700, 7), (4099, 256, 513, 0), (2048, 1021, 40000, 3),
         (9000, 40, 3, 0), (70001, 24, 151936, 8)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,K,V,pad", SIZES)
def test_lookup_and_gradient(dtype, N, K, V, pad):
    W, ids, mask, grad = make(N, K, V, dtype, seed=N, pad=pad)
    for m, scale in ((None, 1.0), (mask, math.sqrt(K))):
        out = g.grpo_embed_tokens(W, ids, m, scale=scale)
        s32 = torch.tensor(scale, dtype=torch.float32, device="cuda")
        want = (W[ids].float() * s32).to(W.dtype)
        if m is not None:
            want[~m] = 0
        assert torch.equal(out, want)
        s = float(s32)
        check_gradient(g.grpo_embed_tokens_grad(grad, ids, V, m, scale=scale), grad, ids, m, V, s)
        if V * K > 1 << 24:
            continue
        for t in {DT[dtype], torch.float32}:
            add = torch.randn((V, K), device="cuda").to(t)
            keep = add.clone()
            d = g.grpo_embed_tokens_grad(grad, ids, V, m, scale=scale, add=add)
            assert d.dtype == t and torch.equal(add, keep)
            check_gradient(d, grad, ids, m, V, s, add)
            r = g.grpo_embed_tokens_grad(grad, ids, V, m, scale=scale, add=add, out=add)
            assert r.data_ptr() == add.data_ptr() and torch.equal(r, d)
