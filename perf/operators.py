"""Cases of the training-step operators around the GRPO loss: the log-probs of
given tokens with entropy and top alternatives, their gradient, and the global
gradient norm with clipping.

``run`` computes a case in its plain form (elementary torch operations) or,
with ``own`` true, by the library's entry points; ``exact`` gives the results
in 64 bits.

The formulas, for a row x of V logits, s = 1 / temperature, z = s x:

    m = max_v x_v,  Z = sum_v exp(s (x_v - m)),  log p_v = s (x_v - m) - log Z
    logp = log p_a,  H = -sum_v p_v log p_v
    top alternatives: the k largest x_v, equal ones by lowest index first
    dL/dx_v = s (dlogp (1[v = a] - p_v) - dH p_v (log p_v + H))

and for gradient tensors g_i: norm = scale sqrt(sum |g_i|^2),
c = min(1, max_norm / (norm + eps)), out_i = scale c g_i.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _logps(name, B, T, V, dtype, *, pad=0, low=None, k=0, entropy=True, temperature=1.0, sigma=2.0, spikes=False):
    return {"name": name, "op": "logps", "B": B, "T": T, "V": V, "dtype": dtype, "pad": pad, "low": T if low is None else low,
            "k": k, "entropy": entropy, "temperature": temperature, "sigma": sigma, "spikes": spikes}


def _grad(name, B, T, V, dtype, *, pad=0, low=None, entropy=True, temperature=1.0, sigma=2.0):
    return {"name": name, "op": "grad", "B": B, "T": T, "V": V, "dtype": dtype, "pad": pad, "low": T if low is None else low,
            "entropy": entropy, "temperature": temperature, "sigma": sigma, "spikes": False}


def _clip(name, layers, width, inner, vocab, dtype, *, packed=False, norm=3.0, scale=1.0):
    return {"name": name, "op": "clip", "layers": layers, "width": width, "inner": inner, "vocab": vocab, "dtype": dtype,
            "packed": packed, "norm": norm, "scale": scale}


def listed():
    return [
        # one sequence that generates: its next token with the alternatives that a client shows; latency is all
        _logps("one token", 1, 1, 32768, "bf16", k=5),
        # a serving step of a batch: behaviour log-probs at the sampling temperature, with 20 alternatives
        _logps("decode step", 64, 1, 151936, "bf16", k=20, temperature=0.8, sigma=3.0, spikes=True),
        # a whole rollout scored at once for the loss: ragged completions, entropy as a training signal
        _logps("rollout", 64, 1024, 32768, "bf16", low=128),
        # a large vocabulary with the alternatives logged for each token
        _logps("rollout alternatives", 16, 512, 151936, "bf16", low=64, k=8, sigma=3.0, spikes=True),
        # an odd vocabulary inside rows padded to a multiple of 64, odd lengths, many alternatives
        _logps("padded odd", 12, 333, 49999, "f16", pad=49, low=9, k=32, temperature=0.7),
        # single-precision logits, log-probs alone
        _logps("rollout f32", 32, 256, 128256, "f32", low=16, entropy=False),
        # the smallest training batch
        _grad("grad tiny", 8, 16, 64, "f32", low=4, sigma=1.0),
        # the training step on the rollout, with an entropy bonus
        _grad("grad rollout", 64, 512, 32768, "bf16", low=64),
        # single-precision logits, no entropy term
        _grad("grad f32", 16, 256, 128256, "f32", low=16, entropy=False),
        # a small policy's gradients, below the limit: nothing is scaled
        _clip("clip small", 2, 256, 704, 512, "f32", norm=0.5),
        # a policy of 1.8 G parameters in bf16
        _clip("clip layers", 32, 2048, 5632, 32768, "bf16"),
        # odd widths packed without gaps: rows that start anywhere, single and half precision mixed, a loss scale
        _clip("clip packed", 12, 1021, 2731, 9973, "mixed", packed=True, scale=1.0 / 1024),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["logps", "logps", "grad", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "clip":
        layers, width = _spread(rng, 1, 24), _spread(rng, 64, 1800)
        c = _clip("", layers, width, _spread(rng, width, 3 * width), _spread(rng, 256, 30000), rng.choice(["bf16", "f16", "f32", "mixed"]),
                  packed=rng.random() < 0.5, norm=rng.choice([0.3, 2.0, 40.0]), scale=rng.choice([1.0, 1.0, 1.0 / 256]))
    else:
        V = rng.choice([_spread(rng, 50, 4000), _spread(rng, 4000, 160000), 32768, 128256, 151936])
        most = 400_000_000 // V
        B = 1 if rng.random() < 0.2 else _spread(rng, 1, 96)
        T = 1 if rng.random() < 0.3 else _spread(rng, 1, max(1, min(2000, most // B)))
        low = T if T == 1 or rng.random() < 0.3 else rng.randint(0, T)
        t, pad = rng.choice([1.0, 1.0, 0.6, 1.3]), rng.choice([0, 0, rng.randint(1, 130)])
        if op == "logps":
            c = _logps("", B, T, V, dtype, pad=pad, low=low, k=min(V, rng.choice([0, 0, 1, 5, rng.randint(1, 32)])), entropy=rng.random() < 0.7,
                       temperature=t, sigma=rng.choice([1.0, 2.0, 3.0]), spikes=rng.random() < 0.3)
        else:
            c = _grad("", B, T, V, dtype, pad=pad, low=low, entropy=rng.random() < 0.6, temperature=t, sigma=rng.choice([1.0, 2.0]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lengths(case):
    """Completion lengths, evenly from low to T."""
    B, T, low = case["B"], case["T"], case["low"]
    return [T if B == 1 else low + (T - low) * b // (B - 1) for b in range(B)]


def _shapes(case):
    """The parameter shapes of a decoder of this size, one list entry a tensor."""
    w, f, v = case["width"], case["inner"], case["vocab"]
    layer = [(w,), (w, w), (w, w), (w, w), (w, w), (w,), (f, w), (f, w), (w, f)]
    return [(v, w)] + layer * case["layers"] + [(w,), (v, w)]


def _kinds(case):
    """Each tensor's type: in "mixed", the vectors and every third matrix are in single precision."""
    if case["dtype"] != "mixed":
        return [DTYPES[case["dtype"]]] * len(_shapes(case))
    return [torch.float32 if len(s) == 1 or i % 3 == 0 else torch.bfloat16 for i, s in enumerate(_shapes(case))]


def _flat(case, fill):
    """One buffer for each type and the tensors as views of it, packed or at multiples of 16 bytes."""
    size, at = {}, []
    for s, t in zip(_shapes(case), _kinds(case)):
        n = math.prod(s)
        at.append((t, size.get(t, 0), n, s))
        size[t] = size.get(t, 0) + (n if case["packed"] else (n + 7) // 8 * 8)
    flat = {t: fill(n, t) for t, n in size.items()}
    return list(flat.values()), [flat[t][o:o + n].view(s) for t, o, n, s in at]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "clip":
        total = sum(math.prod(s) for s in _shapes(case))
        sigma = case["norm"] / math.sqrt(total) / case["scale"]
        _, grads = _flat(case, lambda n, t: torch.randn(n, generator=g, device="cuda", dtype=t).mul_(sigma))
        flat_out, outs = _flat(case, lambda n, t: torch.zeros(n, device="cuda", dtype=t))
        return {"case": case, "grads": grads, "outs": outs, "flat_out": flat_out, "max_norm": 1.0}
    B, T, V = case["B"], case["T"], case["V"]
    dt = DTYPES[case["dtype"]]
    wide = torch.randn((B, T, V + case["pad"]), generator=g, device="cuda", dtype=dt).mul_(case["sigma"])
    if case["spikes"]:
        wide.add_(torch.empty_like(wide).bernoulli_(0.01, generator=g), alpha=8.0)
    x = wide[..., :V]
    # the tokens are drawn from the policy itself (the largest of x s plus Gumbel noise)
    u = torch.rand(x.shape, generator=g, device="cuda").clamp_(1e-12, 1 - 1e-7).log_().neg_().log_().neg_()
    ids = u.add_(x, alpha=1.0 / case["temperature"]).argmax(-1)
    del u
    order = torch.tensor(random.Random(seed).sample(_lengths(case), B), device="cuda")
    mask = torch.arange(T, device="cuda")[None, :] < order[:, None]
    state = {"case": case, "logits": x, "ids": ids, "mask": mask}
    if case["op"] == "grad":
        # what the forward pass left, and the loss' gradients: a fifth of the tokens is clipped
        z = x.float()
        m = z.amax(-1)
        e = (z - m[..., None]).mul_(1.0 / case["temperature"])
        p = e.exp()
        Z = p.sum(-1)
        state["stats"] = torch.stack([m, Z])
        state["entropy"] = Z.log() - p.mul_(e).sum(-1) / Z
        del z, e, p
        keep = torch.rand((B, T), generator=g, device="cuda") < 0.8
        keep[0, 0] = True
        state["dlogp"] = torch.randn((B, T), generator=g, device="cuda") * keep
        state["dH"] = torch.full((B, T), -0.01, device="cuda")
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    case = state["case"]
    return {"logps": _run_logps, "grad": _run_grad, "clip": _run_clip}[case["op"]](state, case)


def _run_logps(state, case):
    x, ids, mask, k = state["logits"], state["ids"], state["mask"], case["k"]
    if own:
        import grad_row_online_gb300 as lib
        r = lib.grpo_token_logps(x, ids, mask, temperature=case["temperature"], top_k=k, want_entropy=case["entropy"])
        out = {"logps": r["logps"]}
        if case["entropy"]:
            out["entropy"] = r["entropy"]
        if k:
            out["top_ids"], out["top_logps"] = r["top_ids"], r["top_logps"]
        return out
    s = 1.0 / case["temperature"]
    z = x.float()
    t = (z - z.amax(-1, keepdim=True)) * s
    e = t.exp()
    Z = e.sum(-1)
    logZ = Z.log()
    zero = torch.zeros((), device=x.device)
    out = {"logps": torch.where(mask, t.gather(-1, ids[..., None])[..., 0] - logZ, zero)}
    if case["entropy"]:
        out["entropy"] = torch.where(mask, logZ - (e * t).sum(-1) / Z, zero)
    del e
    if k:
        # one whole number for each logit that orders by value, then by lowest index
        bits = (z + 0.0).view(torch.int32)
        bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
        key = bits.to(torch.int64) * (1 << 32) + (0xFFFFFFFF - torch.arange(case["V"], device=x.device))
        del bits
        top = 0xFFFFFFFF - (key.topk(k, dim=-1).values & 0xFFFFFFFF)
        out["top_ids"] = torch.where(mask[..., None], top, torch.full((), -1, dtype=torch.int64, device=x.device))
        out["top_logps"] = torch.where(mask[..., None], t.gather(-1, top) - logZ[..., None], zero)
    return out


def _run_grad(state, case):
    x, ids, mask, stats, H = (state[n] for n in ("logits", "ids", "mask", "stats", "entropy"))
    if own:
        import grad_row_online_gb300 as lib
        more = {"entropy": H, "grad_entropy": state["dH"]} if case["entropy"] else {}
        return lib.grpo_token_logps_grad(x, ids, mask, stats, grad_logps=state["dlogp"], temperature=case["temperature"], **more)
    s = 1.0 / case["temperature"]
    dlogp, dH = (torch.where(mask, state[n], torch.zeros((), device=x.device)) for n in ("dlogp", "dH"))
    t = (x.float() - stats[0][..., None]) * s
    p = t.exp() / stats[1][..., None]
    grad = -dlogp[..., None] * p
    if case["entropy"]:
        grad -= dH[..., None] * p * (t + (H - stats[1].log())[..., None])
    grad.scatter_add_(-1, ids[..., None], dlogp[..., None])
    return (grad * s).to(x.dtype)


def _run_clip(state, case):
    grads, outs, limit, scale = state["grads"], state["outs"], state["max_norm"], case["scale"]
    if own:
        import grad_row_online_gb300 as lib
        r = lib.grpo_clip_grad_norm(grads, limit, eps=EPS, scale=scale, out=outs)
        return {"norm": r["norm"], "grads": state["flat_out"]}
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads]).sum().sqrt() * scale
    c = (limit / (norm + EPS)).clamp(max=1.0) * scale
    _ = [o.copy_(g.float() * c.float()) for o, g in zip(outs, grads)]
    return {"norm": norm.float(), "grads": state["flat_out"]}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "clip":
        n = [(math.prod(s), t.itemsize) for s, t in zip(_shapes(case), _kinds(case))]
        return {"bytes": 2 * sum(a * b for a, b in n), "flops": 3 * sum(a for a, _ in n)}
    B, T, V, size = case["B"], case["T"], case["V"], DTYPES[case["dtype"]].itemsize
    active = sum(_lengths(case))
    if case["op"] == "logps":
        row = 4 + 8 + 4 * case["entropy"] + 12 * case["k"]
        return {"bytes": active * V * size + B * T * (row + 1), "flops": active * V * (6 if case["entropy"] else 4)}
    # without an entropy term, the clipped tokens' rows (a fifth) are zero and need no logits
    read = active if case["entropy"] else 0.8 * active
    return {"bytes": read * V * size + active * 24 + B * T * (V * size + 1), "flops": read * V * (7 if case["entropy"] else 4)}


# ---------------------------------------------------------------------------
# the same in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "clip":
        grads = [g.double() * case["scale"] for g in state["grads"]]
        norm = torch.linalg.vector_norm(torch.cat([torch.linalg.vector_norm(g).reshape(1) for g in grads]))
        c = min(1.0, state["max_norm"] / (float(norm) + EPS))
        flat, views = _flat(case, lambda n, t: torch.zeros(n, device="cuda", dtype=torch.float64))
        for v, g in zip(views, grads):
            v.copy_(g * c)
        return {"norm": norm, "grads": flat}
    B, T, V, k = case["B"], case["T"], case["V"], case.get("k", 0)
    x, ids, mask = state["logits"].reshape(B * T, V), state["ids"].reshape(-1), state["mask"].reshape(-1)
    step = max(1, (1 << 28) // V)
    got = {}
    for i in range(0, B * T, step):
        rows, a, on = x[i:i + step].double() / case["temperature"], ids[i:i + step], mask[i:i + step]
        lp = torch.log_softmax(rows, -1)
        n = torch.arange(len(a), device="cuda")
        if case["op"] == "logps":
            part = {"logps": lp[n, a]}
            if case["entropy"]:
                part["entropy"] = -(lp.exp() * lp).sum(-1)
            if k:
                top = torch.sort(rows, dim=-1, descending=True, stable=True).indices[:, :k]
                part["top_ids"], part["top_logps"] = top, lp.gather(-1, top)
            for name, v in part.items():
                on_v = on.reshape([-1] + [1] * (v.dim() - 1))
                got.setdefault(name, []).append(torch.where(on_v, v, torch.full((), -1 if name == "top_ids" else 0, device="cuda", dtype=v.dtype)))
            continue
        w = state["dlogp"].reshape(-1)[i:i + step].double()
        p = lp.exp()
        d = -p * w[:, None]
        if case["entropy"]:
            h = -(p * lp).sum(-1, keepdim=True)
            d -= state["dH"].reshape(-1)[i:i + step].double()[:, None] * p * (lp + h)
        d[n, a] += w
        got.setdefault("grad", []).append(d.mul_(on[:, None] / case["temperature"]))
    if case["op"] == "grad":
        return torch.cat(got["grad"]).reshape(B, T, V)
    return {name: torch.cat(v).reshape(B, T, *v[0].shape[1:]) for name, v in got.items()}
