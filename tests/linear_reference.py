"""64-bit statements of the head's log-probs from hidden states and of their
gradient, and the bounds the tests hold the kernels to.

A logit is a sum of K products formed 16 at a time into an fp32 accumulator:
K / 16 additions (times six for the planes of f32 operands), each off by at
most one unit in the last place (2^-23) of sum |h_k W_k|, and as much again for
the alignment of the 16 products to their largest.  Everything behind the
logits is in fp32, a rounding of 2^-24 each.
"""
import torch

from token_reference import U, half_step, smallest


def logits_error(h, W):
    """(logits, bound of the kernel's distance from them), in 64 bits."""
    K, planes = h.shape[-1], 6 if h.dtype == torch.float32 else 1
    x = h.double() @ W.double().t()
    mag = h.double().abs() @ W.double().abs().t()
    return x, 4 * U * (planes * (-(-K // 64) * 4) + 4) * mag


def forward(h, W, ids, mask, temperature=1.0):
    """logps, entropy, m, Z with the bounds of each ("logps_tol", ...)."""
    s = 1.0 / temperature
    V = W.shape[0]
    x, ex = logits_error(h, W)
    ex = ex.amax(-1)
    m = x.amax(-1)
    t = (x - m[..., None]) * s
    Z = t.exp().sum(-1)
    lp = t - Z.log()[..., None]
    p = lp.exp()
    H = -(p * torch.where(p > 0, lp, torch.zeros_like(lp))).sum(-1)
    safe = ids.clamp(0, V - 1)
    logp = lp.gather(-1, safe[..., None])[..., 0]
    logp = torch.where(ids == safe, logp, torch.full_like(logp, float("nan")))
    lnV = max(1.0, torch.log(torch.tensor(float(V))).item())
    # a thread adds 32 terms, 8 such sums, every eighth tile of at least 64, eight of those
    n = 32 + 8 + V / 64 / 8 + 8
    z = U * (n + 4 * lnV + 16)
    out = {"logps": logp, "entropy": H, "m": m, "Z": Z}
    out["logps_tol"] = U * (6 * logp.abs().nan_to_num(0, 0, 0) + 4 * lnV + 4) + z + 2 * s * ex
    # dH = -sum p (log p + H) dx: sum p |log p + H| is at most 2 H
    out["entropy_tol"] = U * (6 * lnV + 8) + z * (1 + 2 * lnV) + 2 * s * ex * H
    out["m_tol"] = ex
    out["Z_tol"] = Z * (z + 2 * s * ex)
    if mask is not None:
        on = mask.bool()
        for n, v in (("logps", 0.0), ("entropy", 0.0), ("m", 0.0), ("Z", 1.0)):
            out[n] = torch.where(on, out[n], torch.full_like(out[n], v))
            out[n + "_tol"] = torch.where(on, out[n + "_tol"], torch.zeros_like(out[n]))
    return out


def gradient(h, W, ids, mask, dlogp, dH, temperature=1.0, add=None, wdtype=None):
    """(grad_hidden, its bound, grad_weight, its bound) in 64 bits; h [N, K]."""
    s = 1.0 / temperature
    V, N = W.shape[0], h.shape[0]
    x, ex = logits_error(h, W)
    t = (x - x.amax(-1, keepdim=True)) * s
    lp = t - t.exp().sum(-1, keepdim=True).log()
    p = lp.exp()
    zero = torch.zeros(N, dtype=torch.float64, device=h.device)
    w = zero if dlogp is None else dlogp.double()
    b = zero if dH is None else dH.double()
    if mask is not None:
        w, b = torch.where(mask.bool(), w, zero), torch.where(mask.bool(), b, zero)
    on = (w != 0) | (b != 0)
    plp = torch.where(p > 0, p * lp, torch.zeros_like(p))
    H = -plp.sum(-1, keepdim=True)
    hot = torch.zeros_like(p).scatter_(-1, ids.clamp(0, V - 1)[:, None], 1.0)
    d = s * (w[:, None] * (hot - p) - b[:, None] * (plp + p * H))
    lnV = max(1.0, torch.log(torch.tensor(float(V))).item())
    mag = s * (w.abs()[:, None] * (hot + p) + b.abs()[:, None] * (plp.abs() + p * (H + lnV + 1)))
    # d: errors of the logits, some 40 roundings, one to the products' type
    rows = U * (40 + 8 * lnV + 4 * lp.abs().clamp(max=140)) + 2 * s * (ex.amax(-1, keepdim=True) + ex)
    low = half_step(h.dtype) * 1.01 if h.dtype != torch.float32 else U
    ed = low * d.abs() + rows * mag * (1 + (b.abs() > 0)[:, None] * 2)
    if h.dtype == torch.float16:  # fp16 spacing below 2^-14 of what scales into [2^13, 2^15)
        ed = ed + float((s * (w.abs() + b.abs() * (0.37 + lnV))).max()) * 2.0 ** -37
    d, mag, ed = (torch.where(on[:, None], v, torch.zeros_like(v)) for v in (d, mag, ed))
    planes = 6 if h.dtype == torch.float32 else 1
    gh = d @ W.double()
    sums = lambda n: 4 * U * (planes * (-(-n // 64) * 4 + 4) + 8)  # noqa: E731
    gh_tol = ed @ W.double().abs() + sums(V) * (d.abs() @ W.double().abs())
    gh_tol = gh_tol + half_step(h.dtype) * 1.01 * (gh.abs() + gh_tol) + smallest(h.dtype)
    gw = d.t() @ h.double()
    gw_tol = ed.t() @ h.double().abs() + sums(N) * (d.abs().t() @ h.double().abs())
    if add is not None:
        gw = gw + add.double()
        gw_tol = gw_tol + U * (gw.abs() + gw_tol)
    wdtype = wdtype or W.dtype
    gw_tol = gw_tol + half_step(wdtype) * 1.01 * (gw.abs() + gw_tol) + smallest(wdtype)
    return gh, gh_tol, gw, gw_tol
