"""Log-probs of given tokens from hidden states and the head's weight, and
their gradient, against 64-bit statements of the formulas."""
import math

import pytest
import torch

import grad_row_online_gb300 as g
from linear_reference import forward, gradient
from token_reference import assert_close

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


def make(N, K, V, dtype, seed=0, sigma=2.0, p_mask=0.3, pad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.randn((N, K + pad), generator=gen, device="cuda").to(DT[dtype])[:, :K]
    W = (torch.randn((V, K + pad), generator=gen, device="cuda") * (sigma / math.sqrt(K))).to(DT[dtype])[:, :K]
    ids = torch.randint(0, V, (N,), generator=gen, device="cuda")
    mask = torch.rand((N,), generator=gen, device="cuda") >= p_mask
    w = torch.randn((N,), generator=gen, device="cuda") / N
    w[torch.rand((N,), generator=gen, device="cuda") < 0.2] = 0.0
    b = torch.randn((N,), generator=gen, device="cuda") / N
    return h, W, ids, mask, w, b


def scores(h, W, ids, mask, temperature=1.0):
    return g.grpo_linear_logps(h, W, ids, mask, temperature=temperature, want_entropy=True,
                               want_stats=True)


def check_scores(got, ref):
    assert_close(got["logps"], ref["logps"], ref["logps_tol"], "logps")
    assert_close(got["entropy"], ref["entropy"], ref["entropy_tol"], "entropy")
    assert_close(got["stats"][0], ref["m"], ref["m_tol"], "m")
    assert_close(got["stats"][1], ref["Z"], ref["Z_tol"], "Z")


def check_gradient(got, ref):
    gh, gh_tol, gw, gw_tol = ref
    if got["grad_hidden"] is not None:
        assert_close(got["grad_hidden"], gh, gh_tol, "grad_hidden")
    if got["grad_weight"] is not None:
        assert_close(got["grad_weight"], gw, gw_tol, "grad_weight")


SIZES = [  # N, K, V, padding of the rows, temperature
    (1, 64, 128, 0, 1.0), (128, 64, 256, 0, 1.0), (1, 1, 1, 0, 1.0), (3, 5, 7, 0, 0.5),
    (1, 128, 1000, 0, 1.0), (64, 256, 777, 0, 0.8), (65, 72, 64, 8, 1.3), (127, 100, 513, 4, 1.0),
    (129, 64, 256, 0, 1.0), (200, 130, 65, 0, 1.0), (256, 512, 2048, 0, 1.0), (300, 65, 5003, 7, 0.7),
    (513, 256, 300, 0, 1.0), (700, 1021, 4999, 0, 1.0), (1030, 320, 6001, 0, 1.0), (40, 2048, 9001, 0, 1.0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,K,V,pad,temperature", SIZES)
def test_scores_and_gradient(dtype, N, K, V, pad, temperature):
    h, W, ids, mask, w, b = make(N, K, V, dtype, seed=N + V, pad=pad)
    got = scores(h, W, ids, mask, temperature)
    check_scores(got, forward(h, W, ids, mask, temperature))
    for dl, dh in ((w, None), (None, b), (w, b)):
        d = g.grpo_linear_logps_grad(h, W, ids, mask, got["stats"], grad_logps=dl, grad_entropy=dh,
                                     entropy=got["entropy"] if dh is not None else None,
                                     temperature=temperature)
        assert d["grad_hidden"].shape == h.shape and d["grad_hidden"].dtype == h.dtype
        assert d["grad_weight"].shape == W.shape and d["grad_weight"].dtype == W.dtype
        check_gradient(d, gradient(h, W, ids, mask, dl, dh, temperature))
