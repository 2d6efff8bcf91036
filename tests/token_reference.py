"""64-bit statements of the token log-probs, their gradient and the gradient
clipping, and the bounds the tests hold the kernels to.

The bounds count roundings, u = 2^-24 each in fp32.  A sum of n logits' worth
of exponentials is formed by at least 32 threads (256 for rows above 4 KB), so
a thread adds at most n / 32 terms in sequence, then a tree of a few levels;
an exponential has an argument of size |s (x - m)| with three roundings and
2^u itself good to four.
"""
import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    """Half the spacing of the subnormals, or the fp32 flush bound 2^-126."""
    f = torch.finfo(dtype)
    return max(f.smallest_normal * f.eps / 2, 2.0 ** -126)


def sum_roundings(V, es):
    threads = 32 if V * es <= 4096 else 256
    return V / threads / (16 // es) + 20


def forward(x, ids, mask, temperature=1.0, k=0):
    """(logp, H, m, Z, top_ids, top_logps) in 64 bits on the tensors' device."""
    s = 1.0 / temperature
    z = x.double()
    m = z.amax(-1)
    t = (z - m[..., None]) * s
    e = t.exp()
    Z = e.sum(-1)
    lp = t - Z.log()[..., None]
    p = e / Z[..., None]
    H = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(-1)
    bad = ~torch.isfinite(Z)
    H = torch.where(bad, torch.full_like(H, float("nan")), H)
    safe = ids.clamp(0, x.shape[-1] - 1)
    logp = lp.gather(-1, safe[..., None])[..., 0]
    logp = torch.where((ids == safe) & ~bad, logp, torch.full_like(logp, float("nan")))
    out = {"logps": logp, "entropy": H, "m": m, "Z": Z, "bad": bad}
    if k:
        # NaN rows are replaced below: sort something orderly
        order = torch.sort(torch.where(bad[..., None], torch.zeros_like(z), z), dim=-1,
                           descending=True, stable=True).indices[..., :k]
        out["top_ids"] = torch.where(bad[..., None], -1, order)
        top = lp.gather(-1, order)
        out["top_logps"] = torch.where(bad[..., None], torch.full_like(top, float("nan")), top)
    if mask is not None:
        on = mask.bool()
        for n, v in (("logps", 0.0), ("entropy", 0.0), ("m", 0.0), ("Z", 1.0)):
            out[n] = torch.where(on, out[n], torch.full_like(out[n], v))
        if k:
            out["top_ids"] = torch.where(on[..., None], out["top_ids"], -1)
            out["top_logps"] = torch.where(on[..., None], out["top_logps"], 0.0)
    return out


def gradient(x, ids, mask, dlogp, dH, temperature=1.0):
    """(grad, magnitude of its terms, |log2 p|) in 64 bits."""
    s = 1.0 / temperature
    z = x.double()
    t = (z - z.amax(-1, keepdim=True)) * s
    logZ = t.exp().sum(-1, keepdim=True).log()
    lp = t - logZ
    p = lp.exp()
    zero = torch.zeros(ids.shape, dtype=torch.float64, device=x.device)
    w = zero if dlogp is None else dlogp.double()
    h = zero if dH is None else dH.double()
    if mask is not None:
        w, h = torch.where(mask.bool(), w, zero), torch.where(mask.bool(), h, zero)
    plp = torch.where(p > 0, p * lp, torch.zeros_like(p))
    H = -plp.sum(-1, keepdim=True)
    hot = torch.zeros_like(p).scatter_(-1, ids[..., None], 1.0)
    grad = s * (w[..., None] * (hot - p) - h[..., None] * (plp + p * H))
    mag = s * (w[..., None].abs() * (hot + p) + h[..., None].abs() * (plp.abs() + p * (H + logZ + 1)))
    off = ((w == 0) & (h == 0))[..., None]
    grad, mag = (torch.where(off, torch.zeros_like(v), v) for v in (grad, mag))
    return grad, mag, (lp / 0.6931471805599453).abs().clamp(max=200)


def assert_close(got, want, tol, what):
    """|got - want| <= tol where want is finite; the same NaN and infinities."""
    got = got.double()
    want = torch.where(want.abs() > torch.finfo(torch.float32).max, want.sign() * float("inf"), want)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), what
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what
    fine = ~(nan | inf)
    tol = tol if isinstance(tol, torch.Tensor) else torch.full_like(want, tol)
    over = (got - want).abs()[fine] - tol[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, (what, float(over.max()))


def check_forward(got, ref, x, temperature=1.0):
    V, es = x.shape[-1], x.element_size()
    n = sum_roundings(V, es)
    lnV = max(1.0, torch.log(torch.tensor(float(V))).item())
    # sum p |u| <= ln V / ln 2 + 1: the arguments' roundings inside Z
    z_err = U * (n + 4 * lnV + 16)
    lp_tol = U * (6 * ref["logps"].abs().nan_to_num(0, 0, 0) + 4 * lnV + 4) + z_err
    assert_close(got["logps"], ref["logps"], lp_tol, "logps")
    if got.get("entropy") is not None:
        assert_close(got["entropy"], ref["entropy"],
                     U * (6 * lnV + 8) + z_err * (1 + 2 * lnV), "entropy")
    if got.get("stats") is not None:
        assert_close(got["stats"][0], ref["m"], 0.0, "m")
        Z = torch.where(ref["bad"], torch.full_like(ref["Z"], float("nan")), ref["Z"])
        assert_close(got["stats"][1], Z, Z.nan_to_num(0) * z_err, "Z")
    if got.get("top_ids") is not None:
        assert torch.equal(got["top_ids"], ref["top_ids"])
        tol = U * (6 * ref["top_logps"].abs().nan_to_num(0, 0, 0) + 4 * lnV + 4) + z_err
        assert_close(got["top_logps"], ref["top_logps"], tol, "top_logps")


def check_gradient(got, grad, mag, ulog, x):
    V, es = x.shape[-1], x.element_size()
    lnV = max(1.0, torch.log(torch.tensor(float(V))).item())
    rel = U * (sum_roundings(V, es) + 8 * lnV + 40 + 4 * ulog)
    tol = half_step(got.dtype) * 1.01 * grad.abs() + rel * mag + smallest(got.dtype) * (1 + mag.amax(-1, keepdim=True))
    assert_close(got, grad, tol, "grad")
