"""The global gradient norm and clipping against 64-bit sums.

Bounds: a thread's fp32 sum of 64 squares is off by at most 64 roundings
(2^-24 each, all terms positive), so the norm by 32 and its own rounding; the
factor by those and three more; a product adds its type's half step."""
import math

import pytest
import torch

import grad_row_online_gb300 as g
from token_reference import U, half_step, smallest

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
NORM = 34 * U


@pytest.fixture(scope="module", autouse=True)
def _built():
    import os
    import __graft_entry__
    if not os.path.exists(g.library_path()):
        __graft_entry__.build()


def norm64(ts, scale=1.0):
    if not ts:
        return 0.0
    return scale * math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def check(ts, max_norm, got, res, eps=1e-6, scale=1.0):
    n = norm64(ts, scale)
    assert abs(float(res["norm"]) - n) <= NORM * n, (float(res["norm"]), n)
    c = scale * min(1.0, max_norm / (n + eps)) if n + eps > 0 else scale
    assert abs(float(res["factor"]) - c) <= (NORM + 4 * U) * c
    for t, o in zip(ts, got):
        want = t.double() * c
        tol = (half_step(t.dtype) + NORM + 5 * U) * want.abs() + smallest(t.dtype)
        assert o.dtype == t.dtype and bool(((o.double() - want).abs() <= tol).all())


SETS = {
    "one": [(1,)], "scalar": [()], "odd": [(7,), (1023,), (3, 5, 7)], "chunk": [(16384,)],
    "past": [(16385,)], "before": [(16383,), (0,), (32769,)], "zero-size": [(0,), (0, 4)],
    "matrix": [(300, 401), (401,), (1000, 33)], "large": [(3000, 2900), (2900,)],
}


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("name", SETS)
@pytest.mark.parametrize("max_norm", [0.05, 1e6])
def test_norm_and_clip(dtype, name, max_norm):
    gen = torch.Generator(device="cuda").manual_seed(len(name))
    ts = [torch.randn(s, generator=gen, device="cuda").to(DT[dtype]) for s in SETS[name]]
    out = [torch.full_like(t, 9.0) for t in ts]
    res = g.grpo_clip_grad_norm(ts, max_norm, out=out)
    check(ts, max_norm, out, res)
    own = [t.clone() for t in ts]
    res2 = g.grpo_clip_grad_norm(own, max_norm)
    assert torch.equal(res2["norm"], res["norm"]) and torch.equal(res2["factor"], res["factor"])
    assert all(torch.equal(a, b) for a, b in zip(own, out))
    if max_norm == 1e6:
        assert float(res["factor"]) == 1.0 and all(torch.equal(a, b) for a, b in zip(own, ts))
    keep = [t.clone() for t in ts]
    res3 = g.grpo_clip_grad_norm(keep, max_norm, norm_only=True)
    assert torch.equal(res3["norm"], res["norm"])
    assert all(torch.equal(a, b) for a, b in zip(keep, ts))


def _mixed(count, seed=0, sigma=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kinds = list(DT.values())
    return [(torch.randn(1 + (i * 37) % 5000, generator=gen, device="cuda") * sigma).to(kinds[i % 3])
            for i in range(count)]


@pytest.mark.parametrize("count", [0, 1, 63, 64, 65, 200, 1000, 1001, 2500])
def test_many_tensors(count):
    ts = _mixed(count)
    out = [torch.zeros_like(t) for t in ts]
    res = g.grpo_clip_grad_norm(ts, 1.0, out=out)
    check(ts, 1.0, out, res)


def test_views_without_alignment():
    flat = torch.randn(200_003, device="cuda")
    half = torch.randn(200_003, device="cuda").bfloat16()
    ts = [flat[1:50_000], flat[50_001:50_004], half[3:70_002], half[70_003:200_003], flat[60_002:]]
    res = g.grpo_clip_grad_norm(ts, 3.0, norm_only=True)
    n = norm64(ts)
    assert abs(float(res["norm"]) - n) <= NORM * n
    # outputs aligned otherwise than the inputs, and nothing beside them written
    spare = [torch.full((t.numel() + 16,), 5.0, device="cuda", dtype=t.dtype) for t in ts]
    out = [s[i:i + t.numel()] for i, (s, t) in enumerate(zip(spare, ts))]
    check(ts, 3.0, out, g.grpo_clip_grad_norm(ts, 3.0, out=out))
    for i, (s, t) in enumerate(zip(spare, ts)):
        assert (s[:i] == 5).all() and (s[i + t.numel():] == 5).all()


def test_other_orders():
    a = torch.randn((300, 200), device="cuda").t()
    b = torch.randn((2, 3, 8, 9), device="cuda").to(memory_format=torch.channels_last)
    want = [t.clone(memory_format=torch.preserve_format) for t in (a, b)]
    res = g.grpo_clip_grad_norm([a, b], 1.0)
    check(want, 1.0, [a, b], res)


@pytest.mark.parametrize("size", [1e-30, 1e-22, 1e-10, 1e18, 1e30, 3e38])
def test_range(size):
    """Squares that overflow or vanish in fp32."""
    ts = [torch.randn(50_000, device="cuda").clamp(-1, 1) * size, torch.zeros(100, device="cuda"),
          (torch.randn(999, device="cuda").clamp(-1, 1) * size).bfloat16()]
    n = norm64(ts)
    res = g.grpo_clip_grad_norm(ts, math.inf, norm_only=True)
    if n > 3.4e38:
        assert float(res["norm"]) == math.inf and math.isfinite(float(res["factor"]))
    else:
        # subnormal bf16 inputs and results are exact here; the norm is an fp32 number
        assert abs(float(res["norm"]) - n) <= NORM * n
    out = [torch.zeros_like(t) for t in ts]
    if n < 3.4e38:
        check(ts, n / 8, out, g.grpo_clip_grad_norm(ts, n / 8, eps=0.0, out=out), eps=0.0)


def test_mixed_sizes_in_one_thread():
    t = torch.full((100_000,), 1e-25, device="cuda")
    t[::1000] = 1.0
    res = g.grpo_clip_grad_norm([t], 1.0, norm_only=True)
    assert abs(float(res["norm"]) - 10.0) <= NORM * 10


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_non_finite_norm_leaves_everything(bad, dtype):
    ts = [torch.randn(40_000, device="cuda").to(DT[dtype]) for _ in range(3)]
    ts[1][12_345] = bad
    keep = [t.clone() for t in ts]
    res = g.grpo_clip_grad_norm(ts, 1.0)
    assert not math.isfinite(float(res["norm"])) and math.isnan(float(res["factor"]))
    assert math.isnan(float(res["norm"])) == math.isnan(bad)
    assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(ts, keep))
    out = [torch.full_like(t, 2.0) for t in ts]
    g.grpo_clip_grad_norm(ts, 1.0, out=out)
    assert all((o == 2).all() for o in out)


def test_limits():
    ts = [torch.randn(5000, device="cuda"), torch.zeros(10, device="cuda")]
    keep = [t.clone() for t in ts]
    res = g.grpo_clip_grad_norm(ts, 0.0)
    assert float(res["factor"]) == 0 and all((t == 0).all() for t in ts)
    res = g.grpo_clip_grad_norm(ts, 1.0)  # all zero: the norm is 0, nothing changes
    assert float(res["norm"]) == 0 and float(res["factor"]) == 1
    ts = [t.clone() for t in keep]
    res = g.grpo_clip_grad_norm(ts, math.inf, scale=0.25)
    assert float(res["factor"]) == 0.25 and all(torch.equal(a, b * 0.25) for a, b in zip(ts, keep))
    ts = [t.clone() for t in keep]
    out = [torch.empty_like(t) for t in ts]
    check(ts, 2.0, out, g.grpo_clip_grad_norm(ts, 2.0, scale=1.0 / 16, out=out), scale=1.0 / 16)


def test_beyond_32_bits():
    n = (1 << 32) + 12_345
    t = torch.full((n,), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    t[-1] = 1024.0
    want = math.sqrt((n - 1) * 2.0 ** -20 + 2.0 ** 20)
    res = g.grpo_clip_grad_norm([t], want / 2, eps=0.0)
    assert abs(float(res["norm"]) - want) <= NORM * want
    assert float(t[-1]) == 512.0 and float(t[-2]) == 2.0 ** -11 and float(t[0]) == 2.0 ** -11
    assert bool((t[:-1] == 2.0 ** -11).all())


def test_repeatable_streams_and_graph():
    ts = _mixed(150, seed=4)
    want = [torch.zeros_like(t) for t in ts]
    r = g.grpo_clip_grad_norm(ts, 1.0, out=want)
    ws = torch.empty(g.grpo_clip_workspace_size(150), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = [torch.zeros_like(t) for t in ts]
    s.wait_stream(torch.cuda.current_stream())
    r2 = g.grpo_clip_grad_norm(ts, 1.0, out=out, stream=s)
    s.synchronize()
    assert torch.equal(r["norm"], r2["norm"])
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    src = [torch.zeros_like(t) for t in ts]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r3 = g.grpo_clip_grad_norm(src, 1.0, out=out, workspace=ws)
    for a, b in zip(src, ts):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(r["norm"], r3["norm"])
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_python_refusals():
    a, b = torch.zeros(10, device="cuda"), torch.zeros((4, 6), device="cuda")
    for bad in ([a, a], [b[:, ::2]], [b[:, :3]], [a.double()], [a, a.cpu()], [a.cpu()]):
        with pytest.raises(ValueError):
            g.grpo_clip_grad_norm(bad, 1.0)
    for out in ([a.clone()], [a.clone(), b.t()], [a.clone(), b.bfloat16()], [a.clone(), b.cpu()]):
        with pytest.raises(ValueError):
            g.grpo_clip_grad_norm([a, b], 1.0, out=out)
    with pytest.raises(ValueError):
        g.grpo_clip_grad_norm([a], 1.0, out=[a.clone()], norm_only=True)
    with pytest.raises(g.GrpoError):
        g.grpo_clip_grad_norm([a], -1.0)
    with pytest.raises(g.GrpoError):
        g.grpo_clip_grad_norm([a], 1.0, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
