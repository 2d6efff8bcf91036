"""What the bounds of the tests of accuracy tell apart: products of planes stated
in 64 bits, with and without a mistake planted in the statement (no GPU)."""
import pytest
import torch

from accuracy_cases import F32, TWO_PARTS, exact, exact_d, make, off, rounded

PAIRS = [(0, 2), (2, 0), (1, 1), (0, 1), (1, 0), (0, 0)]


def planes(x, n, dtype=torch.bfloat16):
    out, rest = [], x.float()
    for _ in range(n):
        out.append(rest.to(dtype).double())
        rest = rest - out[-1].float()
    return out


@pytest.mark.parametrize("N,K,V", [(17, 512, 3000), (40, 2048, 1500)])
def test_fp32_needs_all_six_products(N, K, V):
    h, W, ids, w, b = make(N, K, V, torch.float32, "cpu", N)
    x = h.double() @ W.double().t()
    right = exact(x, ids)
    hp, wp = planes(h, 3), planes(W, 3)

    def far(pairs):
        """scores and gradients of logits of these products, the gradients' products in 64 bits"""
        y = sum(hp[i] @ wp[j].t() for i, j in pairs)
        d, e = exact_d(y, ids, w, b), exact_d(x, ids, w, b)
        return max([off(a, c) for a, c in zip(exact(y, ids), right)]
                   + [off(d @ W.double(), e @ W.double()), off(d.t() @ h.double(), e.t() @ h.double())])

    assert far(PAIRS) <= F32 / 10
    for left_out in PAIRS:
        assert far([p for p in PAIRS if p != left_out]) > F32, left_out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_fp32_results_need_two_parts_of_d(dtype):
    h, W, ids, w, b = make(200, 256, 1500, dtype, "cpu", 3)
    d = exact_d(h.double() @ W.double().t(), ids, w, b)
    want = d.t() @ h.double()
    scale = 2.0 ** 13 if dtype == torch.float16 else 1.0  # (f16: into its range)
    one, two = planes(d * scale, 2, dtype)
    assert off((one + two).t() @ h.double() / scale, want) <= TWO_PARTS / 2
    single = one.t() @ h.double() / scale
    assert off(single, want) > 10 * TWO_PARTS
    # a 16-bit result has room for both roundings
    assert off(single.to(dtype) if dtype == torch.bfloat16 else (single * 64).half() / 64, want) <= rounded(dtype)
