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
    (24, 4100, 1111, 0, 0.9), (7, 8320, 333, 0, 1.0),
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


def test_pieces_of_the_vocabulary():
    """More tokens than one piece of the logits' gradient holds for all words."""
    for dtype, N, V in (("bf16", 40000, 9000), ("f32", 16000, 8000)):
        h, W, ids, mask, w, b = make(N, 40, V, dtype, seed=5)
        got = scores(h, W, ids, mask)
        check_scores(got, forward(h, W, ids, mask))
        d = g.grpo_linear_logps_grad(h, W, ids, mask, got["stats"], grad_logps=w, grad_entropy=b,
                                     entropy=got["entropy"])
        check_gradient(d, gradient(h, W, ids, mask, w, b))


def all_of(h, W, ids, mask, w, b, **kw):
    """(scores, gradients) of one set of tensors."""
    s = scores(h, W, ids, mask)
    return s, g.grpo_linear_logps_grad(h, W, ids, mask, s["stats"], grad_logps=w, grad_entropy=b,
                                       entropy=s["entropy"], **kw)


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8))
               for s, t in zip(a, b) for x, y in zip(s.values(), t.values()) if x is not None)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,T", [(4, 16), (6, 50)])
@pytest.mark.parametrize("K", [64, 131])
def test_layouts(dtype, B, T, K):
    """Slices of longer sequences, [T, B, K] orders, padded and shifted weights,
    broadcast rows: the bits of the same numbers side by side."""
    V = 777
    h, W, ids, mask, w, b = make(B * T, K, V, dtype, seed=K)
    h, ids, mask, w, b = (x.reshape(B, T, *x.shape[1:]).contiguous() for x in (h, ids, mask, w, b))
    want = all_of(h, W, ids, mask, w, b)
    long = torch.randn((B, T + 3, K + 5), device="cuda").to(h.dtype)
    sliced = long[:, 2:T + 2, 1:K + 1]
    sliced.copy_(h)
    turned = h.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.randn((V, K + 11), device="cuda").to(W.dtype)
    padded, shifted = wide[:, :K], wide[:, 3:K + 3]
    flat = torch.randn(V * K + 1, device="cuda").to(W.dtype)[1:].view(V, K)
    flat.copy_(W)
    for x, y in ((sliced, W), (turned, W), (h, flat)):
        assert same(all_of(x, y, ids, mask, w, b), want)
    for y in (padded, shifted):
        y.copy_(W)
        assert same(all_of(h, y, ids, mask, w, b), want)
    # [N, K]: the same rows
    two = all_of(h.reshape(B * T, K), W, *(x.reshape(-1) for x in (ids, mask, w, b)))
    assert torch.equal(two[0]["logps"], want[0]["logps"].reshape(-1))
    assert torch.equal(two[1]["grad_weight"], want[1]["grad_weight"])
    # outputs into views, and nothing beside them
    room = torch.full((B, T + 2, K + 3), 7.0, device="cuda", dtype=h.dtype)
    gw_room = torch.full((V, K + 9), 7.0, device="cuda", dtype=W.dtype)
    out = all_of(h, W, ids, mask, w, b, grad_hidden=room[:, 1:T + 1, 2:K + 2], grad_weight=gw_room[:, 4:K + 4])
    assert same(out, want)
    room[:, 1:T + 1, 2:K + 2] = 7.0
    gw_room[:, 4:K + 4] = 7.0
    assert bool((room == 7).all()) and bool((gw_room == 7).all())
    # one row for every token
    row = h[:1, :1].expand(B, T, K)
    again = all_of(row.contiguous(), W, ids, mask, w, b)
    assert same(all_of(row, W, ids, mask, w, b), again)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N", [50, 300])
def test_weight_gradient_forms(dtype, N):
    """Single precision, added to what is there, in place, alone."""
    K, V = 72, 601
    h, W, ids, mask, w, b = make(N, K, V, dtype, seed=N)
    s = scores(h, W, ids, mask)
    kw = dict(grad_logps=w, grad_entropy=b, entropy=s["entropy"])
    call = lambda **more: g.grpo_linear_logps_grad(h, W, ids, mask, s["stats"], **kw, **more)  # noqa: E731
    gen = torch.Generator(device="cuda").manual_seed(3)
    for t in {h.dtype, torch.float32}:
        add = torch.randn((V, K), generator=gen, device="cuda").to(t)
        keep = add.clone()
        d = call(add_weight=add)
        assert d["grad_weight"].dtype == t and torch.equal(add, keep)
        check_gradient(d, gradient(h, W, ids, mask, w, b, add=add, wdtype=t))
        r = call(add_weight=add, grad_weight=add)["grad_weight"]
        assert r.data_ptr() == add.data_ptr() and torch.equal(r, d["grad_weight"])
        out = torch.empty((V, K), device="cuda", dtype=t)
        check_gradient(call(grad_weight=out), gradient(h, W, ids, mask, w, b, wdtype=t))
    full = call()
    a, c = call(grad_weight=None), call(grad_hidden=False)
    assert a["grad_weight"] is None and torch.equal(a["grad_hidden"], full["grad_hidden"])
    assert c["grad_hidden"] is None and torch.equal(c["grad_weight"], full["grad_weight"])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N", [1, 30, 140, 1500])
def test_masks(dtype, N):
    """No token, one token; what masked tokens hold does not matter."""
    K, V = 96, 500
    h, W, ids, mask, w, b = make(N, K, V, dtype, seed=9)
    for m in (torch.zeros_like(mask), torch.arange(N, device="cuda") == N // 2, mask):
        want = forward(h, W, ids, m)
        x, j, u, c = h.clone(), ids.clone(), w.clone(), b.clone()
        x[~m] = float("nan")
        j[~m] = -5
        u[~m] = float("nan")
        c[~m] = float("inf")
        status = g.status_buffer()
        s = g.grpo_linear_logps(x, W, j, m, want_entropy=True, want_stats=True, status=status)
        check_scores(s, want)
        d = g.grpo_linear_logps_grad(x, W, j, m, s["stats"], grad_logps=u, grad_entropy=c,
                                     entropy=s["entropy"], status=status)
        check_gradient(d, gradient(h, W, ids, m, w, b))
        assert bool((d["grad_hidden"][~m] == 0).all())
        assert g.grpo_read_device_status(status) == 0
        kept = torch.full_like(h, 3.0)
        g.grpo_linear_logps_grad(x, W, j, m, s["stats"], grad_logps=u, grad_entropy=c, entropy=s["entropy"],
                                 grad_hidden=kept, grad_weight=None, skip_masked_grad_rows=True)
        assert bool((kept[~m] == 3).all()) and torch.equal(kept[m], d["grad_hidden"][m])
    # no mask, bytes for a mask
    assert same([scores(h, W, ids, None)], [scores(h, W, ids, torch.ones_like(mask))])
    assert same([scores(h, W, ids, mask)], [scores(h, W, ids, mask.to(torch.uint8) * 7)])
    # tokens without a gradient: as if masked
    s = scores(h, W, ids, mask)
    z = torch.zeros_like(w)
    d = g.grpo_linear_logps_grad(h, W, ids, None, s["stats"], grad_logps=z)
    assert not d["grad_hidden"].any() and not d["grad_weight"].any()


def test_no_tokens():
    W = torch.randn((70, 33), device="cuda")
    h, ids = torch.empty((0, 33), device="cuda"), torch.empty((0,), dtype=torch.int64, device="cuda")
    s = scores(h, W, ids, None)
    assert s["logps"].shape == (0,) and s["stats"].shape == (2, 0)
    add = torch.randn_like(W)
    e = torch.empty((0,), device="cuda")
    d = g.grpo_linear_logps_grad(h, W, ids, None, s["stats"], grad_logps=e, add_weight=add)
    assert d["grad_hidden"].shape == (0, 33) and torch.equal(d["grad_weight"], add)
    d = g.grpo_linear_logps_grad(h.reshape(0, 4, 33), W, ids.reshape(0, 4), None, s["stats"].reshape(2, 0, 4),
                                 grad_logps=e.reshape(0, 4))
    assert not d["grad_weight"].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [6, 300])
def test_logits_without_a_finite_value(dtype, N):
    K, V = 64, 300
    h, W, ids, _, w, b = make(N, K, V, dtype, seed=2)
    big = 3e19
    if dtype == "bf16":
        # logits of -inf: words that the first token cannot take
        h[0] = big
        W[10:20] = -big
        ids[0] = 5
        s = scores(h, W, ids, None)
        ref = forward(h[:1], torch.cat([W[:10], W[20:]]), ids[:1], None)
        assert_close(s["logps"][:1], ref["logps"], ref["logps_tol"], "logps beside -inf")
        assert_close(s["entropy"][:1], ref["entropy"], ref["entropy_tol"] + 1e-30, "entropy beside -inf")
        d = g.grpo_linear_logps_grad(h, W, ids, None, s["stats"], grad_logps=w.abs() + 1, grad_entropy=b,
                                     entropy=s["entropy"], grad_hidden=True, grad_weight=None)
        assert bool(torch.isfinite(s["logps"][0])) and not torch.isnan(d["grad_hidden"][0]).any()
        # +inf, and nothing but -inf: no distribution, for that token alone
        h[1] = -big
        h[2] = big
        W[:] = -big
        W[3] = 0
        h[3:] = 0
        s = scores(h, W, ids, None)
        assert bool(torch.isnan(s["logps"][1])) and bool(torch.isnan(s["stats"][1, 1]))
        assert bool(torch.isfinite(s["logps"][3:]).all()) and bool(torch.isfinite(s["stats"][1, 2]))
        W[3] = -big
        s = scores(h, W, ids, None)
        assert bool(torch.isnan(s["entropy"][[0, 1, 2]]).all()) and bool(torch.isfinite(s["entropy"][3:]).all())
    h, W, ids, _, w, b = make(N, K, V, dtype, seed=2)
    good = scores(h, W, ids, None)
    h[N // 2, 5] = float("nan")
    s = scores(h, W, ids, None)
    rest = torch.arange(N, device="cuda") != N // 2
    assert bool(torch.isnan(s["logps"][N // 2])) and torch.equal(s["logps"][rest], good["logps"][rest])
    w = w.abs() + 1
    d = g.grpo_linear_logps_grad(h, W, ids, None, s["stats"], grad_logps=w)
    assert bool(torch.isnan(d["grad_hidden"][N // 2]).all()) and bool(torch.isfinite(d["grad_hidden"][rest]).all())
    assert bool(torch.isnan(d["grad_weight"]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [5, 200])
def test_ids_outside_the_vocabulary(dtype, N):
    K, V = 64, 300
    h, W, ids, _, w, _ = make(N, K, V, dtype, seed=6)
    w = w.abs() + 0.1
    good = scores(h, W, ids, None)
    for bad in (-1, V, 1 << 40, -(1 << 62)):
        ids[3] = bad
        status = g.status_buffer()
        s = g.grpo_linear_logps(h, W, ids, None, want_entropy=True, status=status)
        rest = torch.arange(N, device="cuda") != 3
        assert bool(torch.isnan(s["logps"][3])) and torch.equal(s["logps"][rest], good["logps"][rest])
        assert torch.equal(s["entropy"], good["entropy"])
        assert g.grpo_read_device_status(status) == g.GRPO_ERR_ACTION_RANGE
        status = g.status_buffer()
        d = g.grpo_linear_logps_grad(h, W, ids, None, good["stats"], grad_logps=w, status=status)
        assert bool(torch.isnan(d["grad_hidden"][3]).all()) and bool(torch.isfinite(d["grad_hidden"][rest]).all())
        assert bool(torch.isnan(d["grad_weight"]).all())
        assert g.grpo_read_device_status(status) == g.GRPO_ERR_ACTION_RANGE
        # an id is not used where its log-prob has no gradient
        status = g.status_buffer()
        d = g.grpo_linear_logps_grad(h, W, ids, None, good["stats"], grad_logps=w * rest,
                                     grad_entropy=w, entropy=good["entropy"], status=status)
        assert bool(torch.isfinite(d["grad_weight"]).all()) and g.grpo_read_device_status(status) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_values_at_the_ends_of_the_types(dtype):
    """f32 values beyond bf16's largest, small gradients, sharp and flat softmaxes."""
    K, V, N = 64, 1000, 150
    h, W, ids, mask, w, b = make(N, K, V, dtype, seed=8)
    if dtype == "f32":
        x, y = h * 0, W * 0
        x[:, 0], y[:, 0] = 3.4e38, W[:, 0] * 1e-32
        s = scores(x, y, ids, mask, 1e6)
        check_scores(s, forward(x, y, ids, mask, 1e6))
    for scale, temperature in ((1e-6, 1.0), (1e3, 1.0), (1.0, 0.05), (1.0, 30.0)):
        s = scores(h, W, ids, mask, temperature)
        d = g.grpo_linear_logps_grad(h, W, ids, mask, s["stats"], grad_logps=w * scale, grad_entropy=b * scale,
                                     entropy=s["entropy"], temperature=temperature)
        check_scores(s, forward(h, W, ids, mask, temperature))
        check_gradient(d, gradient(h, W, ids, mask, w * scale, b * scale, temperature))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N", [100, 600])
def test_the_same_bits_whatever_the_workspace_holds(dtype, N):
    K, V = 136, 1500
    h, W, ids, mask, w, b = make(N, K, V, dtype, seed=1)
    want = all_of(h, W, ids, mask, w, b)
    for fill in (0, 255, 127):
        ws = torch.full((g.grpo_linear_workspace_size(h, W),), fill, dtype=torch.uint8, device="cuda")
        wb = torch.full((g.grpo_linear_workspace_size(h, W, True),), fill, dtype=torch.uint8, device="cuda")
        s = g.grpo_linear_logps(h, W, ids, mask, want_entropy=True, want_stats=True, workspace=ws)
        d = g.grpo_linear_logps_grad(h, W, ids, mask, s["stats"], grad_logps=w, grad_entropy=b,
                                     entropy=s["entropy"], workspace=wb)
        assert same((s, d), want)
    with pytest.raises(g.GrpoError):
        g.grpo_linear_logps(h, W, ids, mask, workspace=ws[:-256])
    with pytest.raises(g.GrpoError):
        g.grpo_linear_logps_grad(h, W, ids, mask, s["stats"], grad_logps=w, workspace=wb[:-256])


@pytest.mark.parametrize("N,K,V", [(2, 4096, 300), (16, 4100, 515), (9, 33, 1000), (16, 1024, 4097),
                                   (17, 64, 100), (1, 60000, 65), (4, 1, 7), (8, 129, 2051)])
def test_few_tokens_in_single_precision(N, K, V):
    """One to sixteen tokens, and just beyond: every form of the gradient."""
    h, W, ids, mask, w, b = make(N, K, V, "f32", seed=K, pad=K % 3)
    mask[0], w[0] = True, 0.5
    s = scores(h, W, ids, mask)
    check_scores(s, forward(h, W, ids, mask))
    kw = dict(grad_logps=w, grad_entropy=b, entropy=s["entropy"])
    call = lambda **more: g.grpo_linear_logps_grad(h, W, ids, mask, s["stats"], **kw, **more)  # noqa: E731
    full = call()
    check_gradient(full, gradient(h, W, ids, mask, w, b))
    assert torch.equal(call(grad_weight=None)["grad_hidden"], full["grad_hidden"])
    assert torch.equal(call(grad_hidden=False)["grad_weight"], full["grad_weight"])
    add = torch.randn((V, K), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    r = call(add_weight=add)
    check_gradient(r, gradient(h, W, ids, mask, w, b, add=add))
    room = torch.full((V, K + 3), 7.0, device="cuda")
    room[:, 1:K + 1] = add
    call(add_weight=room[:, 1:K + 1], grad_weight=room[:, 1:K + 1])
    assert torch.equal(room[:, 1:K + 1], r["grad_weight"])
    assert bool((room[:, 0] == 7).all()) and bool((room[:, K + 1:] == 7).all())
    for fill in (255, 127):
        ws = torch.full((g.grpo_linear_workspace_size(h, W),), fill, dtype=torch.uint8, device="cuda")
        wb = torch.full((g.grpo_linear_workspace_size(h, W, True),), fill, dtype=torch.uint8, device="cuda")
        again = g.grpo_linear_logps(h, W, ids, mask, want_entropy=True, want_stats=True, workspace=ws)
        assert same((again, call(workspace=wb)), (s, full))


def test_outputs_asked_for_alone():
    h, W, ids, mask, _, _ = make(300, 64, 400, "bf16")
    full = scores(h, W, ids, mask)
    lp = g.grpo_linear_logps(h, W, ids, mask)
    assert torch.equal(lp["logps"], full["logps"]) and lp["entropy"] is None and lp["stats"] is None
    ent = g.grpo_linear_logps(h, W, None, mask, want_entropy=True)
    assert ent["logps"] is None and torch.equal(ent["entropy"], full["entropy"])


@pytest.mark.parametrize("N", [3, 400])
def test_streams_and_graphs(N):
    """A stream argument, two calls at once, a captured call replayed on other inputs."""
    K, V = 128, 3000
    sets = [make(N, K, V, "bf16", seed=s) for s in (1, 2, 3)]
    want = [all_of(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(3):
        got.clear()
        for s, (h, W, ids, mask, w, b) in zip(streams, sets):
            f = g.grpo_linear_logps(h, W, ids, mask, want_entropy=True, want_stats=True, stream=s)
            with torch.cuda.stream(s):
                d = g.grpo_linear_logps_grad(h, W, ids, mask, f["stats"], grad_logps=w, grad_entropy=b,
                                             entropy=f["entropy"])
            got.append((f, d))
    torch.cuda.synchronize()
    assert all(same(a, c) for a, c in zip(got, want))
    held = [x.clone() for x in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_of(*held)
    for inputs, result in zip(sets[1:] + sets[:1], want[1:] + want[:1]):
        for x, y in zip(held, inputs):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, result)


def test_against_the_token_entry_points():
    """The same numbers as grpo_token_logps gives for logits formed beforehand."""
    h, W, ids, mask, w, b = make(200, 256, 5000, "f32", seed=4)
    z = (h.double() @ W.double().t()).float()
    a, c = scores(h, W, ids, mask), g.grpo_token_logps(z, ids, mask, want_entropy=True, want_stats=True)
    ref = forward(h, W, ids, mask)
    for n in ("logps", "entropy"):
        assert_close(a[n], c[n].double(), 2 * ref[n + "_tol"], n)
    dz = g.grpo_token_logps_grad(z, ids, mask, c["stats"], grad_logps=w, grad_entropy=b, entropy=c["entropy"])
    d = g.grpo_linear_logps_grad(h, W, ids, mask, a["stats"], grad_logps=w, grad_entropy=b, entropy=a["entropy"])
    _, gh_tol, _, gw_tol = gradient(h, W, ids, mask, w, b)
    assert_close(d["grad_hidden"], dz.double() @ W.double(), 2 * gh_tol, "grad_hidden")
    assert_close(d["grad_weight"], dz.double().t() @ h.double(), 2 * gw_tol, "grad_weight")


def test_gradient_against_differences():
    """Central differences of the sum that the incoming gradients weigh, along
    random directions: the second-order error of a step e is below e^2 / 6
    times the third derivative, which for steps of 2^-6 along unit directions
    stays below 1e-4 of the slope's scale here; fp32 log-probs are good to
    1e-6 each, over 2 e = 2^-5."""
    N, K, V = 40, 32, 200
    h, W, ids, mask, w, b = make(N, K, V, "f32", seed=11, sigma=1.0)
    s = scores(h, W, ids, mask)
    d = g.grpo_linear_logps_grad(h, W, ids, mask, s["stats"], grad_logps=w, grad_entropy=b, entropy=s["entropy"])

    def total(x, y):
        r = scores(x, y, ids, mask)
        return float((r["logps"].double() * w.double() + r["entropy"].double() * b.double())[mask].sum())

    gen = torch.Generator(device="cuda").manual_seed(0)
    e = 2.0 ** -6
    size = float((w.abs() + b.abs() * 6).sum())
    for _ in range(5):
        u = torch.randn(h.shape, generator=gen, device="cuda")
        u /= u.norm()
        v = torch.randn(W.shape, generator=gen, device="cuda")
        v /= v.norm()
        slope = (total(h + e * u, W) - total(h - e * u, W)) / (2 * e)
        assert abs(slope - float((d["grad_hidden"].double() * u).sum())) <= size * (1e-4 + 2e-6 * 6 / (2 * e))
        slope = (total(h, W + e * v) - total(h, W - e * v)) / (2 * e)
        assert abs(slope - float((d["grad_weight"].double() * v).sum())) <= size * (1e-4 + 2e-6 * 6 / (2 * e))


def test_what_is_written_counts_as_modified():
    h, W, ids, mask, w, _ = make(20, 32, 50, "f32")
    s = scores(h, W, ids, mask)
    gh, gw = torch.empty_like(h), torch.empty_like(W)
    before = gh._version, gw._version
    g.grpo_linear_logps_grad(h, W, ids, mask, s["stats"], grad_logps=w, grad_hidden=gh, grad_weight=gw)
    assert gh._version > before[0] and gw._version > before[1]


def test_refusals():
    h, W, ids, mask, w, b = make(20, 32, 50, "bf16")
    s = scores(h, W, ids, mask)
    bad = [dict(weight=W.float()), dict(weight=W[:, :31]), dict(weight=W.cpu()), dict(weight=W[0]),
           dict(weight=W.t().contiguous().t()), dict(hidden=h.double()), dict(ids=ids.int()),
           dict(ids=ids[:19]), dict(mask=mask[:19]), dict(mask=mask.float())]
    for kw in bad:
        a = dict(hidden=h, weight=W, ids=ids, mask=mask) | kw
        with pytest.raises(ValueError):
            g.grpo_linear_logps(a["hidden"], a["weight"], a["ids"], a["mask"])
        with pytest.raises(ValueError):
            g.grpo_linear_logps_grad(a["hidden"], a["weight"], a["ids"], a["mask"], s["stats"], grad_logps=w)
    for kw in (dict(grad_hidden=torch.empty_like(h).float()), dict(grad_hidden=torch.empty_like(h)[:19]),
               dict(grad_weight=torch.empty_like(W)[:49]), dict(grad_weight=torch.empty_like(W).half()),
               dict(add_weight=torch.empty_like(W).half()), dict(grad_weight=None, add_weight=W),
               dict(grad_weight=torch.empty_like(W), add_weight=torch.empty_like(W).float()),
               dict(grad_hidden=torch.empty_like(W)[:20, ::2])):
        with pytest.raises(ValueError):
            g.grpo_linear_logps_grad(h, W, ids, mask, s["stats"], grad_logps=w, **kw)
    with pytest.raises(ValueError):
        g.grpo_linear_logps_grad(h, W, ids, mask, None, grad_logps=w)
    for kw in (dict(), dict(grad_logps=w, grad_hidden=None, grad_weight=None), dict(grad_entropy=b),
               dict(grad_logps=w, temperature=0.0)):
        with pytest.raises(g.GrpoError):
            g.grpo_linear_logps_grad(h, W, ids, mask, s["stats"], **kw)
    with pytest.raises(g.GrpoError):  # rows that overlap
        g.grpo_linear_logps_grad(h, W, ids, mask, s["stats"], grad_logps=w, grad_hidden=h[:1].clone().expand(20, 32))
    with pytest.raises(g.GrpoError):
        g.grpo_linear_logps(h, W, ids, mask, temperature=-1.0)
