"""Alternatives of rows of ties, in every number of threads that a row gets: a
row of equal logits holds more keys at its bound than a CTA's or warp's list.

The log-probs' bound counts roundings (2^-24 each): a thread adds V / threads
terms, 16 bytes at a time, then a tree; three roundings of the log-prob's own
size, and the logarithm's."""
import math

import pytest
import torch

import grad_row_online_gb300 as g
from token_reference import U, assert_close, forward

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


def fill(rows, V, dtype):
    """Rows of ties of ten kinds in turn, the last one ordinary."""
    gen = torch.Generator(device="cuda").manual_seed(V)
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    x = (torch.randn((rows, V), generator=gen, device="cuda") * 2).to(dtype)
    i = torch.arange(V, device="cuda")
    x[0::10] = 0.0
    x[1::10] = (i % 2).to(dtype)
    x[2::10] = -math.inf
    x[2::10, V // 2:V // 2 + 3] = 1.5                       # three allowed, fewer than the alternatives
    x[3::10] = low
    x[4::10] = torch.where(i >= V - V // 3, 3.0, x[4::10].float()).to(dtype)  # ties at the end
    x[5::10] = x[5::10].round()
    x[6::10] = torch.where(i % 256 < 8, 2.0, -1.0).to(dtype)  # ties in a few threads' slices
    x[7::10] = (i // 64).to(dtype) / V                      # rising steps: every bound is passed later
    x[8::10] = high
    x[8::10, ::3] = low
    return x


SIZES = [  # rows, threads a row at most 4 bytes x V and 2 bytes x V get, V
    (50, 32, 1001), (50, 32, 577), (77, 32, 33), (2100, 32, 2050), (2300, 32, 6143),
    (400, 128, 3001), (400, 128, 15000), (2100, 128, 16383), (20, 256, 16384), (20, 256, 50021),
    (330, 256, 40001),
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,threads,V", SIZES)
@pytest.mark.parametrize("k", [5, 32])
def test_rows_of_ties(dtype, rows, threads, V, k):
    x = fill(rows, V, DT[dtype])
    ids = torch.arange(rows, device="cuda") % V
    got = g.grpo_token_logps(x, ids, top_k=k, want_entropy=True)
    ref = forward(x, ids, None, 1.0, k)
    assert not bool(ref["bad"].any())
    assert torch.equal(got["top_ids"], ref["top_ids"])
    lnV = max(1.0, math.log(V))
    z_err = U * (V / threads / (16 // x.element_size()) + 20 + 4 * lnV + 16)
    for name in ("logps", "top_logps"):
        want = ref[name]
        tol = U * (6 * want.abs().nan_to_num(0, 0, 0) + 4 * lnV + 4) + z_err
        assert_close(got[name], want, tol, name)
    assert_close(got["entropy"], ref["entropy"], U * (6 * lnV + 8) + z_err * (1 + 2 * lnV), "entropy")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_of_ties_off_alignment(dtype):
    """The same rows three elements further on, and masked in part."""
    for rows, V in ((2100, 2049), (60, 999)):
        x = fill(rows, V, DT[dtype])
        y = torch.zeros((rows, V + 7), device="cuda", dtype=DT[dtype])[:, 3:V + 3]
        y.copy_(x)
        mask = torch.arange(rows, device="cuda") % 7 != 0
        got = g.grpo_token_logps(y, None, mask, top_k=32)["top_ids"]
        want = forward(x, torch.zeros(rows, dtype=torch.int64, device="cuda"), mask, 1.0, 32)["top_ids"]
        assert torch.equal(got, want)
