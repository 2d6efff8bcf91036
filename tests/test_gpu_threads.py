"""Calls from two host threads at once, on streams of their own: each kernel
takes as much shared memory as its call's sizes need, whatever the other's."""
import threading

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


def head(N, K, V, dtype):
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    h = torch.randn((N, K), generator=gen, device="cuda").to(dtype)
    W = (torch.randn((V, K), generator=gen, device="cuda") * K ** -0.5).to(dtype)
    ids = torch.randint(0, V, (N,), generator=gen, device="cuda")
    w = torch.ones((N,), device="cuda")

    def call():
        s = g.grpo_linear_logps(h, W, ids, want_stats=True)
        d = g.grpo_linear_logps_grad(h, W, ids, None, s["stats"], grad_logps=w)
        return s["logps"], d["grad_hidden"], d["grad_weight"]
    return call


def embedding(N, K, V):
    gen = torch.Generator(device="cuda").manual_seed(N + V)
    grad = torch.randn((N, K), generator=gen, device="cuda")
    ids = torch.randint(0, V, (N,), generator=gen, device="cuda")
    return lambda: (g.grpo_embed_tokens_grad(grad, ids, V),)


PAIRS = {
    "head of few tokens": lambda: (head(128, 256, 2000, torch.bfloat16), head(1, 64, 100, torch.bfloat16)),
    "head of many tokens": lambda: (head(300, 256, 2000, torch.bfloat16), head(300, 64, 100, torch.bfloat16)),
    "head in parts": lambda: (head(100, 1024, 2000, torch.float32), head(17, 1024, 70, torch.float32)),
    "head of single tokens in fp32": lambda: (head(8, 4096, 300, torch.float32), head(8, 64, 300, torch.float32)),
    "embedding's gradient": lambda: (embedding(4096, 8, 151936), embedding(4096, 8, 100)),
}


@pytest.mark.parametrize("name", PAIRS)
def test_two_threads(name):
    calls = PAIRS[name]()
    want = [[x.clone() for x in c()] for c in calls]
    torch.cuda.synchronize()
    start, failed = threading.Barrier(2), []

    def loop(call, right):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                start.wait(30)
                for i in range(1000):
                    got = call()
                    if i % 100 == 0:
                        stream.synchronize()
                        assert all(torch.equal(a, b) for a, b in zip(got, right))
                stream.synchronize()
        except Exception as e:  # noqa: BLE001  (told by the main thread)
            failed.append(repr(e))

    threads = [threading.Thread(target=loop, args=x) for x in zip(calls, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
