"""Log-probs of given tokens, entropy, top alternatives and their gradient
against 64-bit statements of the formulas, at the sizes, layouts and values
where they can go wrong."""
import math

import pytest
import torch

import grad_row_online_gb300 as g
from token_reference import assert_close, check_forward, check_gradient, forward, gradient

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


def make(B, T, V, dtype, pad=0, seed=0, sigma=2.0, p_mask=0.3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((B, T, V + pad), generator=gen, device="cuda") * sigma).to(DT[dtype])[..., :V]
    ids = torch.randint(0, V, (B, T), generator=gen, device="cuda")
    mask = torch.rand((B, T), generator=gen, device="cuda") >= p_mask
    return x, ids, mask


def scores(x, ids, mask, k=0, temperature=1.0):
    return g.grpo_token_logps(x, ids, mask, temperature=temperature, top_k=k, want_entropy=True,
                              want_stats=True)


SIZES = [  # B, T, V, pad, k, temperature
    (1, 1, 1, 0, 1, 1.0), (2, 3, 2, 0, 2, 1.0), (3, 5, 7, 0, 7, 0.5), (4, 2, 33, 1, 32, 1.0),
    (8, 16, 64, 0, 5, 1.0), (5, 7, 1000, 3, 20, 1.3), (3, 4, 2047, 0, 32, 1.0),
    (3, 4, 2049, 0, 32, 1.0), (2, 3, 5003, 5, 8, 0.7), (1, 1, 32768, 0, 5, 1.0),
    (7, 1, 49999, 49, 32, 0.8), (2, 9, 32768, 0, 0, 1.0), (1, 5, 151936, 0, 20, 1.0),
    (3, 1, 151935, 0, 1, 1.0), (40, 17, 4099, 0, 4, 1.0),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,T,V,pad,k,temperature", SIZES)
def test_forward_and_gradient(dtype, B, T, V, pad, k, temperature):
    x, ids, mask = make(B, T, V, dtype, pad, seed=V + B)
    got = scores(x, ids, mask, k, temperature)
    ref = forward(x, ids, mask, temperature, k)
    check_forward(got, ref, x, temperature)
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn((B, T), generator=gen, device="cuda")
    w[torch.rand((B, T), generator=gen, device="cuda") < 0.2] = 0.0
    h = torch.randn((B, T), generator=gen, device="cuda")
    for dl, dh in ((w, None), (None, h), (w, h)):
        d = g.grpo_token_logps_grad(x, ids, mask, got["stats"], grad_logps=dl, grad_entropy=dh,
                                    entropy=got["entropy"] if dh is not None else None,
                                    temperature=temperature)
        assert d.shape == x.shape and d.dtype == x.dtype and d.is_contiguous()
        check_gradient(d, *gradient(x, ids, mask, dl, dh, temperature), x)


@pytest.mark.parametrize("rows", [1, 2, 5, 19, 76, 152, 305])
@pytest.mark.parametrize("V", [8191, 65536, 100003])
def test_few_rows(rows, V):
    """Every way a row is divided when there are few of them."""
    x, ids, _ = make(rows, 1, V, "bf16", seed=rows)
    x, ids = x[:, 0], ids[:, 0]
    got = g.grpo_token_logps(x, ids, top_k=20, want_entropy=True, want_stats=True)
    check_forward(got, forward(x, ids, None, 1.0, 20), x)


def test_outputs_asked_for_alone():
    x, ids, mask = make(3, 4, 6000, "bf16")
    full = scores(x, ids, mask, 6)
    lp = g.grpo_token_logps(x, ids, mask)
    assert torch.equal(lp["logps"], full["logps"]) and lp["entropy"] is None and lp["stats"] is None
    top = g.grpo_token_logps(x, None, mask, top_k=6)
    assert top["logps"] is None and torch.equal(top["top_ids"], full["top_ids"])
    assert torch.equal(top["top_logps"], full["top_logps"])
    uint = g.grpo_token_logps(x, ids, mask.to(torch.uint8), want_entropy=True)
    assert torch.equal(uint["entropy"], full["entropy"])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [64, 3001, 40000])
def test_special_values(dtype, V):
    """Rows of ties, of -inf, of the type's lowest value, NaN and +inf."""
    x, ids, _ = make(1, 14, V, dtype, seed=3)
    x = x.clone()
    low = torch.finfo(DT[dtype]).min
    ids[0, :8] = torch.arange(8, device="cuda")
    x[0, 0] = 0.0                                  # all equal
    x[0, 1] = low                                  # all at the lowest value
    x[0, 2] = -math.inf                            # nothing
    x[0, 3, 3:] = -math.inf                        # three tokens allowed
    x[0, 3, :3] = torch.tensor([0.5, -0.0, 0.0])
    x[0, 4, 10:] = low                             # masked by the lowest value
    x[0, 5, V // 2] = math.nan
    x[0, 6, V - 1] = math.inf
    x[0, 7, :] = -math.inf
    x[0, 7, V - 1] = 2.0                           # certain of the last token, not the given one
    x[0, 8] = x[0, 8].round()                      # many ties
    x[0, 9] = torch.arange(V, device="cuda").to(DT[dtype]) / V  # rising, ties by rounding
    x[0, 10] = (torch.arange(V, device="cuda") % 2).to(DT[dtype])
    x[0, 11] = torch.finfo(DT[dtype]).max          # all at the largest value
    x[0, 12, 1:] = low
    x[0, 12, 0] = torch.finfo(DT[dtype]).max
    k = 32
    got = scores(x, ids, None, k)
    ref = forward(x, ids, None, 1.0, k)
    # 64-bit sort sees -0 == 0, as the kernel does; rows 2, 5 and 6 have no distribution
    assert ref["bad"][0].nonzero().flatten().tolist() == [2, 5, 6]
    check_forward({n: got[n] for n in ("logps", "entropy", "top_ids", "top_logps")}, ref, x)
    # gradients of the rows that have one
    rows = [0, 1, 3, 4, 8, 9, 10, 11]
    sub, i = x[:, rows].contiguous(), ids[:, rows].contiguous()
    f = scores(sub, i, None)
    w = torch.linspace(-1, 1, len(rows), device="cuda").reshape(1, -1).contiguous()
    h = torch.full_like(w, 0.25)
    d = g.grpo_token_logps_grad(sub, i, None, f["stats"], grad_logps=w, entropy=f["entropy"],
                                grad_entropy=h)
    check_gradient(d, *gradient(sub, i, None, w, h), sub)
    # a row without a distribution has a NaN gradient, unless nothing flows into it
    f = scores(x[:, 5:7].contiguous(), ids[:, 5:7].contiguous(), None)
    d = g.grpo_token_logps_grad(x[:, 5:7].contiguous(), ids[:, 5:7].contiguous(), None, f["stats"],
                                grad_logps=torch.tensor([[1.0, 0.0]], device="cuda"))
    assert torch.isnan(d[0, 0]).all() and (d[0, 1] == 0).all()


@pytest.mark.parametrize("k", [1, 7, 32])
def test_alternatives_in_one_place(k):
    """The largest logits side by side, at the row's ends, or all in one
    thread's slice."""
    V = 50021
    gen = torch.Generator(device="cuda").manual_seed(9)
    base = torch.randn((6, V), generator=gen, device="cuda")
    base[0, 1000:1100] += 50
    base[1, :40] += 50
    base[2, V - 40:] += 50
    base[3, ::2048] += 50   # vectors of one slice (8 elements x 256 threads)
    base[4] = torch.sort(base[4]).values
    base[5] = torch.sort(base[5], descending=True).values
    ids = torch.zeros(6, dtype=torch.int64, device="cuda")
    for dt in (torch.bfloat16, torch.float32):
        x = base.to(dt)
        got = g.grpo_token_logps(x, ids, top_k=k, want_entropy=True)
        check_forward(got, forward(x, ids, None, 1.0, k), x)


def test_masked_rows_are_not_read_and_zero():
    x, ids, mask = make(4, 6, 5000, "bf16", p_mask=0.5)
    x = x.clone()
    x[~mask] = math.nan
    ids[~mask] = -7
    got = scores(x, ids, mask, 3)
    off = ~mask
    assert (got["logps"][off] == 0).all() and (got["entropy"][off] == 0).all()
    assert (got["top_ids"][off] == -1).all() and (got["top_logps"][off] == 0).all()
    assert (got["stats"][0][off] == 0).all() and (got["stats"][1][off] == 1).all()
    w = torch.ones((4, 6), device="cuda")
    d = g.grpo_token_logps_grad(x, ids, mask, got["stats"], grad_logps=w)
    assert (d[off] == 0).all() and torch.isfinite(d[mask].float()).all()
    keep = torch.full_like(d, 3.0)
    g.grpo_token_logps_grad(x, ids, mask, got["stats"], grad_logps=w, grad=keep,
                            skip_masked_grad_rows=True)
    assert (keep[off] == 3).all() and torch.equal(keep[mask], d[mask])
    none = torch.zeros_like(mask)
    got = scores(x, ids, none, 2)
    assert (got["logps"] == 0).all() and (got["top_ids"] == -1).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [4000, 4097])
def test_row_strides(dtype, V):
    """[T,B,V] order, padded rows, a shifted slice, one row for all, and
    gradients with strides of their own: the bits of the contiguous call."""
    x, ids, mask = make(5, 6, V, dtype)
    w = torch.randn((5, 6), device="cuda")
    want = scores(x, ids, mask, 4)
    wantd = g.grpo_token_logps_grad(x, ids, mask, want["stats"], grad_logps=w)
    views = {
        "order": x.transpose(0, 1).contiguous().transpose(0, 1),
        "padded": torch.nn.functional.pad(x, (0, 13))[..., :V],
        "slice": torch.cat([x, x], 1)[:, :6],
        "offset": torch.nn.functional.pad(x, (3, 0))[..., 3:],
    }
    for name, v in views.items():
        assert torch.equal(v, x)
        got = scores(v, ids, mask, 4)
        ref = forward(x, ids, mask, 1.0, 4)
        check_forward(got, ref, x)
        assert torch.equal(got["top_ids"], want["top_ids"]), name
        # alignment decides which thread sums what: values agree, not bits
        d = g.grpo_token_logps_grad(v, ids, mask, want["stats"], grad_logps=w)
        assert torch.equal(d, wantd), name
        into = torch.empty_strided(v.shape, v.stride(), dtype=v.dtype, device="cuda")
        assert g.grpo_token_logps_grad(v, ids, mask, want["stats"], grad_logps=w, grad=into) is into
        assert torch.equal(into, wantd), name
        same = v.clone(memory_format=torch.preserve_format) if name == "order" else v
        g.grpo_token_logps_grad(same, ids, mask, want["stats"], grad_logps=w, grad=same)
        assert torch.equal(same, wantd), name
        x = x.clone()  # (views of x itself are not used above)
    one = x[:1, :1].expand(5, 6, V)
    got = scores(one, ids, None, 4)
    check_forward(got, forward(one, ids, None, 1.0, 4), one)


def test_in_place_gradient():
    for dtype in DT:
        x, ids, mask = make(4, 5, 10007, dtype)
        f = scores(x, ids, mask)
        w = torch.randn((4, 5), device="cuda")
        want = g.grpo_token_logps_grad(x, ids, mask, f["stats"], grad_logps=w)
        y = x.clone()
        g.grpo_token_logps_grad(y, ids, mask, f["stats"], grad_logps=w, grad=y)
        assert torch.equal(y, want)


def test_gradient_against_differences():
    """Central differences of sum(w logp + h H), the function in 64 bits."""
    x, ids, mask = make(2, 3, 70, "f32", seed=5, sigma=1.0)
    T = 0.8
    gen = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randn((2, 3), generator=gen, device="cuda")
    h = torch.randn((2, 3), generator=gen, device="cuda")
    f = scores(x, ids, mask, 0, T)
    d = g.grpo_token_logps_grad(x, ids, mask, f["stats"], grad_logps=w, entropy=f["entropy"],
                                grad_entropy=h, temperature=T)

    def loss(z):
        r = forward(z, ids, mask, T)
        return (w.double() * r["logps"] + h.double() * r["entropy"]).sum()

    step = 1e-5
    z = x.double()
    num = torch.zeros_like(z)
    for b in range(2):
        for t in range(3):
            for v in range(70):
                up, dn = z.clone(), z.clone()
                up[b, t, v] += step
                dn[b, t, v] -= step
                num[b, t, v] = (loss(up) - loss(dn)) / (2 * step)
    # differences: step^2 x third derivative (|w| + |h| (ln V + 1) <~ 20) + 2^-53 x loss / step;
    # fp32 kernel: 100 roundings of terms of that size
    assert_close(d, num, 20 * step * step + 2.0 ** -50 * 20 / step + 100 * 2.0 ** -24 * 4, "grad")


def test_action_out_of_range():
    x, ids, mask = make(3, 4, 5000, "bf16", p_mask=0)
    ids[1, 2], ids[2, 0], ids[0, 0] = 5000, -1, 1 << 40
    mask[0, 0] = False
    st = g.status_buffer()
    got = g.grpo_token_logps(x, ids, mask, want_stats=True, status=st)
    assert g.grpo_read_device_status(st) == g.GRPO_ERR_ACTION_RANGE
    bad = torch.zeros_like(mask)
    bad[1, 2] = bad[2, 0] = True
    assert torch.equal(torch.isnan(got["logps"]), bad)
    assert torch.equal(torch.isnan(g.grpo_token_logps(x, ids, mask)["logps"]), bad)
    st.zero_()
    w = torch.ones((3, 4), device="cuda")
    d = g.grpo_token_logps_grad(x, ids, mask, got["stats"], grad_logps=w, status=st)
    assert g.grpo_read_device_status(st) == g.GRPO_ERR_ACTION_RANGE
    assert torch.equal(torch.isnan(d).all(-1), bad) and torch.equal(torch.isnan(d).any(-1), bad)
    st.zero_()
    w[1, 2] = w[2, 0] = 0
    d = g.grpo_token_logps_grad(x, ids, mask, got["stats"], grad_logps=w, status=st)
    assert g.grpo_read_device_status(st) == 0 and not torch.isnan(d).any()


def test_empty():
    for B, T in ((0, 4), (3, 0), (0, 0)):
        x = torch.empty((B, T, 100), device="cuda")
        ids = torch.empty((B, T), dtype=torch.int64, device="cuda")
        got = scores(x, ids, None, 3)
        assert got["logps"].shape == (B, T) and got["top_ids"].shape == (B, T, 3)
        w = torch.empty((B, T), device="cuda")
        assert g.grpo_token_logps_grad(x, ids, None, got["stats"], grad_logps=w).shape == x.shape


def test_rows_beyond_32_bits():
    """Rows whose element offset passes 2^31 and 2^32."""
    V, stride = 1000, 1 << 30
    flat = torch.empty(5 * stride, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((5, V), (stride, 1))
    x.copy_(torch.randn((5, V), device="cuda"))
    ids = torch.arange(5, device="cuda")
    got = g.grpo_token_logps(x, ids, top_k=3, want_entropy=True, want_stats=True)
    check_forward(got, forward(x, ids, None, 1.0, 3), x)
    w = torch.ones(5, device="cuda")
    want = g.grpo_token_logps_grad(x.contiguous(), ids, None, got["stats"], grad_logps=w)
    g.grpo_token_logps_grad(x, ids, None, got["stats"], grad_logps=w, grad=x)
    assert torch.equal(x, want)


def test_side_stream_and_graph():
    x, ids, mask = make(3, 4, 20000, "bf16")
    want = scores(x, ids, mask, 5)
    w = torch.randn((3, 4), device="cuda")
    wantd = g.grpo_token_logps_grad(x, ids, mask, want["stats"], grad_logps=w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = g.grpo_token_logps(x, ids, mask, top_k=5, want_entropy=True, want_stats=True,
                                 stream=stream)
        d = g.grpo_token_logps_grad(x, ids, mask, got["stats"], grad_logps=w, stream=stream)
        s.synchronize()
        assert all(torch.equal(got[n], want[n]) for n in want) and torch.equal(d, wantd)
    y = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = scores(y, ids, mask, 5)
        d = g.grpo_token_logps_grad(y, ids, mask, got["stats"], grad_logps=w)
    y.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want) and torch.equal(d, wantd)


def test_repeatable():
    x, ids, mask = make(30, 11, 32768, "bf16", seed=8)
    a, b = scores(x, ids, mask, 9), scores(x, ids, mask, 9)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_python_refusals():
    x, ids, mask = make(2, 3, 50, "f32")
    with pytest.raises(ValueError):
        g.grpo_token_logps(x[..., ::2], ids, mask)
    with pytest.raises(ValueError):
        g.grpo_token_logps(x, ids[:, :2], mask)
    with pytest.raises(ValueError):
        g.grpo_token_logps(x, ids.int(), mask)
    with pytest.raises(ValueError):
        g.grpo_token_logps(x, ids, mask.float())
    with pytest.raises(ValueError):
        g.grpo_token_logps(x.double(), ids, mask)
    with pytest.raises(ValueError):
        g.grpo_token_logps(x.cpu(), ids, mask)
    with pytest.raises(g.GrpoError):
        g.grpo_token_logps(x, ids, mask, top_k=33)
    with pytest.raises(g.GrpoError):
        g.grpo_token_logps(x, ids, mask, temperature=0.0)
    f = scores(x, ids, mask)
    w = torch.ones((2, 3), device="cuda")
    with pytest.raises(g.GrpoError):
        g.grpo_token_logps_grad(x, ids, mask, f["stats"])
    with pytest.raises(ValueError):
        g.grpo_token_logps_grad(x, ids, mask, f["stats"][0], grad_logps=w)
    with pytest.raises(ValueError):
        g.grpo_token_logps_grad(x, ids, mask, f["stats"], grad_logps=w[:1].expand(2, 3))
    with pytest.raises(ValueError):
        g.grpo_token_logps_grad(x, ids, mask, f["stats"], grad_logps=w, grad=x.bfloat16())
    with pytest.raises(ValueError):
        g.grpo_token_logps_grad(x, ids, mask, None, grad_logps=w)
    with pytest.raises(ValueError):
        g.grpo_token_logps(x, ids, mask, status=torch.zeros(8, device="cuda"))
    with pytest.raises(TypeError):
        g.grpo_token_logps(x, ids, mask, temperature="hot")
    with pytest.raises(g.GrpoError):
        g.grpo_token_logps(x, ids, mask, top_k=-1)
    with pytest.raises(g.GrpoError):  # rows of the gradient overlap
        g.grpo_token_logps_grad(x, ids, mask, f["stats"], grad_logps=w,
                                grad=torch.empty((1, 1, 50), device="cuda").expand(2, 3, 50))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,T,V,pad,k", [(40, 30, 8192, 0, 0), (31, 37, 8219, 0, 7),
                                         (25, 40, 16411, 5, 32), (1100, 1, 50001, 0, 3)])
def test_many_rows(dtype, B, T, V, pad, k):
    """Enough rows for CTAs to take several: ragged masks, rows of special
    values between ordinary ones, ids out of range."""
    x, ids, mask = make(B, T, V, dtype, pad, seed=V, p_mask=0.4)
    if T > 1:
        mask &= torch.arange(T, device="cuda")[None] < torch.randint(0, T + 1, (B, 1), device="cuda")
    low = torch.finfo(DT[dtype]).min
    rows = x.reshape(B * T, -1)[:, :V] if pad == 0 else x.flatten(0, 1)
    for i, v in enumerate((-math.inf, low, math.nan, math.inf, 0.0)):
        rows[5 + 7 * i] = v
        rows[300 + 11 * i, 3:] = v
    x = rows.reshape(B, T, V)
    flat = ids.flatten()
    flat[600:640:5] = V
    st = g.status_buffer()
    got = g.grpo_token_logps(x, ids, mask, top_k=k, want_entropy=True, want_stats=True, status=st)
    ref = forward(x, ids, mask, 1.0, k)
    del got["stats"]
    check_forward(got, ref, x)
    seen = bool((mask.flatten() & (flat == V)).any())
    assert g.grpo_read_device_status(st) == (g.GRPO_ERR_ACTION_RANGE if seen else 0)
    again = g.grpo_token_logps(x, ids, mask, top_k=k, want_entropy=True)
    for n in ("logps", "entropy", "top_ids", "top_logps"):
        if got[n] is not None:
            assert torch.equal(got[n].nan_to_num(), again[n].nan_to_num())
    alone = g.grpo_token_logps(x, ids, mask)
    assert torch.equal(alone["logps"].nan_to_num(), got["logps"].nan_to_num())


@pytest.mark.parametrize("rows", [3, 400])
@pytest.mark.parametrize("offset", [3e3, 1e5, -1e5, 1e20, -1e20])
def test_offsets(rows, offset):
    """Logits far from zero: rows that the fast arithmetic does not take."""
    V, k = 20000, 6
    x, ids, _ = make(rows, 1, V, "f32", seed=7)
    x = x + offset
    x[rows // 2] -= offset  # one row that it does take
    got = scores(x, ids, None, k)
    check_forward(got, forward(x, ids, None, 1.0, k), x)
    w = torch.linspace(-1, 1, rows, device="cuda")[:, None].contiguous()
    h = torch.full_like(w, 0.5)
    d = g.grpo_token_logps_grad(x, ids, None, got["stats"], grad_logps=w, entropy=got["entropy"],
                                grad_entropy=h)
    check_gradient(d, *gradient(x, ids, None, w, h), x)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("temperature", [1e-35, 1e-4, 0.02, 40.0, 1e4, 1e36])
def test_temperatures(dtype, temperature):
    x, ids, mask = make(3, 5, 5001, dtype, seed=11)
    ids[0] = x[0].argmax(-1)
    k = 5
    got = scores(x, ids, mask, k, temperature)
    s = torch.tensor(1.0 / temperature, dtype=torch.float64).to(torch.float32).double().item()
    ref = forward(x, ids, mask, 1.0 / s, k)  # the fp32 scale itself
    V, n = 5001, 5001 / 256 / 4 + 20
    top = ref["top_logps"].abs()
    # a log-prob of |s t| carries three roundings of its own size; sums as in check_forward
    lnV = math.log(V)
    z_err = 2.0 ** -24 * (n + 4 * lnV + 16)
    tol = lambda v: 2.0 ** -24 * (6 * v.abs().nan_to_num(0, 0, 0) + 4 * lnV + 4) + z_err
    assert_close(got["logps"], ref["logps"], tol(ref["logps"]), "logps")
    assert torch.equal(got["top_ids"], ref["top_ids"])
    assert_close(got["top_logps"], ref["top_logps"], tol(ref["top_logps"]), "top_logps")
    assert_close(got["entropy"], ref["entropy"], 2.0 ** -24 * (6 * lnV + 8) + z_err * (1 + 2 * lnV),
                 "entropy")


def test_null_stream():
    x, ids, mask = make(2, 3, 9000, "bf16")
    want = scores(x, ids, mask, 2)
    torch.cuda.synchronize()
    got = g.grpo_token_logps(x, ids, mask, top_k=2, want_entropy=True, want_stats=True, stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,T,V,k", [(1, 2003, 5003, 9), (67, 61, 2500, 4), (3000, 1, 1025, 32),
                                     (1, 20001, 64, 3)])
def test_many_short_rows(dtype, B, T, V, k):
    """Rows that share a CTA, in a number that does not fill the last one."""
    x, ids, mask = make(B, T, V, dtype, seed=B + T)
    got = scores(x, ids, mask, k)
    check_forward(got, forward(x, ids, mask, 1.0, k), x)
    w = torch.randn((B, T), device="cuda")
    h = torch.randn((B, T), device="cuda")
    w[:, ::3] = 0.0
    for dl, dh in ((w, None), (w, h)):
        d = g.grpo_token_logps_grad(x, ids, mask, got["stats"], grad_logps=dl, grad_entropy=dh,
                                    entropy=got["entropy"] if dh is not None else None)
        check_gradient(d, *gradient(x, ids, mask, dl, dh), x)
    y = x.clone()
    assert torch.equal(g.grpo_token_logps_grad(y, ids, mask, got["stats"], grad_logps=w, grad=y),
                       g.grpo_token_logps_grad(x, ids, mask, got["stats"], grad_logps=w))
