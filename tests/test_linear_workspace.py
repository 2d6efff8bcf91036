"""What the workspace of the head's gradient holds, as the header states it (no GPU)."""
import pytest

from test_abi import FAKE, lib  # noqa: F401  (the built library)

MB = 1 << 20


def up(a, b):
    return -(-a // b) * b


@pytest.mark.parametrize("dt,N,K,V", [(0, 65536, 64, 151936), (0, 200000, 64, 151936), (1, 300000, 64, 151936),
                                      (2, 131072, 64, 151936), (1, 65536, 64, 151936), (1, 4608, 2048, 151936),
                                      (0, 43000, 64, 151936), (1, 1000, 64, 300)])
def test_gradient(lib, dt, N, K, V):  # noqa: F811
    rows, planes = up(N, 256), 3 if dt == 0 else 1
    # the logits' gradient: 512 MB, or 2,048 words; two parts of it in 16 bits, where grad_weight is fp32
    d = max(512 * MB, 2 * max(planes, 2) * 2048 * rows)
    operands = 2 * planes * (rows + (up(V, 256) if dt == 0 else 0)) * K
    sums = 4 * 4 * rows * up(K, 256)  # (four parts of grad_hidden at most where tokens are many)
    size = lib.grpo_linear_workspace_size(FAKE, dt, 1, N, K, V, K, 1)
    assert 0 < size <= d + operands + sums + 24 * rows + 4096
    assert size >= min(d, 2 * planes * rows * V) * 0.9
