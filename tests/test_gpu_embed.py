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


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("K", [64, 131])
def test_layouts(dtype, K):
    """[B, T] shapes, slices and orders of either side, padded and shifted weights."""
    B, T, V = 6, 37, 500
    W, ids, mask, grad = make(B * T, K, V, dtype, seed=K)
    W, grad = W.contiguous(), grad.contiguous()
    out = g.grpo_embed_tokens(W, ids, mask, scale=3.0)
    d = g.grpo_embed_tokens_grad(grad, ids, V, mask, scale=3.0)
    i2, m2 = ids.view(B, T), mask.view(B, T)
    wide = torch.randn((V, K + 9), device="cuda").to(W.dtype)
    for shift in (0, 3):
        wide[:, shift:K + shift] = W
        assert torch.equal(g.grpo_embed_tokens(wide[:, shift:K + shift], i2, m2, scale=3.0), out.view(B, T, K))
    room = torch.full((B, T + 4, K + 5), 7.0, device="cuda", dtype=W.dtype)
    for view in (room[:, 2:T + 2, 1:K + 1], torch.full((T, B, K), 7.0, device="cuda", dtype=W.dtype).transpose(0, 1)):
        r = g.grpo_embed_tokens(W, i2, m2, scale=3.0, out=view)
        assert r.data_ptr() == view.data_ptr() and torch.equal(view, out.view(B, T, K))
    room[:, 2:T + 2, 1:K + 1] = 7.0
    assert bool((room == 7).all())
    long = torch.randn((B, T + 5, K + 3), device="cuda").to(W.dtype)
    sliced, turned = long[:, 3:T + 3, 1:K + 1], grad.view(B, T, K).transpose(0, 1).contiguous().transpose(0, 1)
    sliced.copy_(grad.view(B, T, K))
    for x in (sliced, turned, grad.view(B, T, K)):
        assert torch.equal(g.grpo_embed_tokens_grad(x, i2, V, m2, scale=3.0), d)
    gw = torch.full((V, K + 6), 7.0, device="cuda", dtype=W.dtype)
    g.grpo_embed_tokens_grad(grad, ids, V, mask, scale=3.0, out=gw[:, 5:K + 5])
    assert torch.equal(gw[:, 5:K + 5], d)
    gw[:, 5:K + 5] = 7.0
    assert bool((gw == 7).all())
    # one row for every token: a bias, say
    row = grad[:1].expand(B * T, K)
    assert torch.equal(g.grpo_embed_tokens_grad(row, ids, V, mask), g.grpo_embed_tokens_grad(row.contiguous(), ids, V, mask))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [40, 1021, 264])
@pytest.mark.parametrize("first", [0, 1, 31])
def test_ids_over_many_chunks(dtype, K, first):
    """Runs of an id around 16, 17 and 18 chunks of 32 sorted tokens, and long
    ones side by side, from each place in a chunk."""
    runs = [first, 512, 544, 513, 545, 576, 577, 543, 31, 33, 64, 3, 1, 70, 2100, 608, 4500, 640, 5, 1500]
    V = len(runs) + 1
    ids = torch.repeat_interleave(torch.arange(len(runs)), torch.tensor(runs))
    gen = torch.Generator().manual_seed(K)
    ids = ids[torch.randperm(len(ids), generator=gen)].cuda()
    grad = torch.randn((len(ids), K), generator=gen).to(DT[dtype]).cuda()
    d = g.grpo_embed_tokens_grad(grad, ids, V)
    check_gradient(d, grad, ids, None, V, 1.0)
    assert torch.equal(g.grpo_embed_tokens_grad(grad, ids, V), d)
    add = torch.randn((V, K), device="cuda").to(DT[dtype])
    r = g.grpo_embed_tokens_grad(grad, ids, V, add=add)
    check_gradient(r, grad, ids, None, V, 1.0, add)
    assert torch.equal(g.grpo_embed_tokens_grad(grad, ids, V, add=add, out=add), r)


@pytest.mark.parametrize("N", [1, 40, 5000, 9000])
def test_one_id_and_no_id(N):
    """Every token the same word: its rows in every chunk; nothing taking part."""
    K, V = 72, 300
    _, _, _, grad = make(N, K, V, "bf16", seed=N)
    ids = torch.full((N,), V - 1, device="cuda")
    check_gradient(g.grpo_embed_tokens_grad(grad, ids, V), grad, ids, None, V, 1.0)
    none = torch.zeros(N, dtype=torch.bool, device="cuda")
    poison = torch.full_like(grad, float("nan"))
    add = torch.randn((V, K), device="cuda")
    assert not g.grpo_embed_tokens_grad(poison, ids, V, none).any()
    assert torch.equal(g.grpo_embed_tokens_grad(poison, ids, V, none, add=add), add)
    assert not g.grpo_embed_tokens(poison[:1], ids * 0, none).any()


def test_no_tokens():
    W = torch.randn((30, 17), device="cuda")
    none = torch.empty((0,), dtype=torch.int64, device="cuda")
    assert g.grpo_embed_tokens(W, none).shape == (0, 17)
    assert g.grpo_embed_tokens(W, none.view(0, 5)).shape == (0, 5, 17)
    assert not g.grpo_embed_tokens_grad(W[:0], none, 30).any()
    assert torch.equal(g.grpo_embed_tokens_grad(W[:0], none, 30, add=W), W)


@pytest.mark.parametrize("N", [7, 6000])
def test_ids_outside_the_vocabulary(N):
    W, ids, mask, grad = make(N, 40, 100, "bf16", seed=3)
    ids[mask.logical_not()] = -7  # (masked: not used)
    for bad in (100, -1, 1 << 40, -(1 << 62)):
        where = int(mask.nonzero()[N // 20])
        broken = ids.clone()
        broken[where] = bad
        status = g.status_buffer()
        out = g.grpo_embed_tokens(W, broken, mask, scale=2.0, status=status)
        assert bool(torch.isnan(out[where]).all()) and int(torch.isnan(out).any(1).sum()) == 1
        assert g.grpo_read_device_status(status) == g.GRPO_ERR_ACTION_RANGE
        status = g.status_buffer()
        d = g.grpo_embed_tokens_grad(grad, broken, 100, mask, status=status)
        left = mask.clone()
        left[where] = False
        check_gradient(d, grad, broken.clamp(0, 99), left, 100, 1.0)
        assert g.grpo_read_device_status(status) == g.GRPO_ERR_ACTION_RANGE
    status = g.status_buffer()
    g.grpo_embed_tokens(W, ids, mask, status=status)
    g.grpo_embed_tokens_grad(grad, ids, 100, mask, status=status)
    assert g.grpo_read_device_status(status) == 0


def test_values_pass():
    """Copies at scale 1 keep every bit; infinities and NaN reach their word alone."""
    W = torch.arange(1 << 16, dtype=torch.int32, device="cuda").to(torch.int16).view(1024, 64).view(torch.bfloat16)
    ids = torch.randint(0, 1024, (500,), device="cuda")
    assert torch.equal(g.grpo_embed_tokens(W, ids).view(torch.int16), W[ids].view(torch.int16))
    grad = torch.ones((64, 16), device="cuda")
    ids = torch.arange(64, device="cuda") % 16
    grad[5], grad[6], grad[22] = float("nan"), float("inf"), 3.0
    d = g.grpo_embed_tokens_grad(grad, ids, 16)
    rest = torch.tensor([i not in (5, 6) for i in range(16)], device="cuda")
    assert bool(torch.isnan(d[5]).all()) and bool((d[6] == float("inf")).all()) and bool((d[rest] == 4).all())


def test_the_same_bits_whatever_the_workspace_holds():
    N, K, V = 7000, 48, 900
    _, ids, mask, grad = make(N, K, V, "bf16", seed=1)
    want = g.grpo_embed_tokens_grad(grad, ids, V, mask)
    for fill in (0, 255, 127):
        ws = torch.full((g.grpo_embed_workspace_size(N, K, V),), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(g.grpo_embed_tokens_grad(grad, ids, V, mask, workspace=ws), want)
    with pytest.raises(g.GrpoError):
        g.grpo_embed_tokens_grad(grad, ids, V, mask, workspace=ws[:-256])


def test_streams_and_graphs():
    N, K, V = 5000, 64, 700
    sets = [make(N, K, V, "bf16", seed=s) for s in (1, 2, 3)]
    run = lambda W, i, m, d: (g.grpo_embed_tokens(W, i, m), g.grpo_embed_tokens_grad(d, i, V, m))  # noqa: E731
    want = [run(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [(g.grpo_embed_tokens(W, i, m, stream=s), g.grpo_embed_tokens_grad(d, i, V, m, stream=s))
           for _ in range(3) for s, (W, i, m, d) in zip(streams, sets)]
    torch.cuda.synchronize()
    for a, b in zip(got, want * 3):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    held = [x.clone() for x in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(*held)
    for inputs, result in zip(sets[1:], want[1:]):
        for x, y in zip(held, inputs):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], result[0]) and torch.equal(out[1], result[1])


def test_refusals():
    W, ids, mask, grad = make(20, 32, 50, "bf16")
    for kw in (dict(token_ids=ids.int()), dict(token_ids=ids.view(2, 2, 5)), dict(token_ids=ids[::2]),
               dict(token_mask=mask[:19]), dict(token_mask=mask.float()), dict(out=torch.empty((20, 31), device="cuda")),
               dict(out=torch.empty((20, 32), device="cuda")), dict(weight=W.cpu()), dict(weight=W.double()),
               dict(weight=W.t()), dict(token_ids=ids.cpu())):
        a = dict(weight=W, token_ids=ids) | kw
        with pytest.raises(ValueError):
            g.grpo_embed_tokens(**a)
    for kw in (dict(grad=grad[:19]), dict(grad=grad[:, ::2]), dict(V=0), dict(V=-1), dict(add=W.half()),
               dict(add=W[:49]), dict(out=torch.empty((50, 31), device="cuda", dtype=W.dtype)),
               dict(out=W.half()), dict(add=W, out=W.float()), dict(token_mask=mask[:3])):
        a = dict(grad=grad, token_ids=ids, V=50) | kw
        with pytest.raises(ValueError):
            g.grpo_embed_tokens_grad(**a)
    with pytest.raises(g.GrpoError):
        g.grpo_embed_tokens(W, ids, scale=math.inf)
    with pytest.raises(g.GrpoError):
        g.grpo_embed_tokens(W, ids, out=W[:1].clone().expand(20, 32))
