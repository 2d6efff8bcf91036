"""Cases of the two ends of a policy around the GRPO loss: the log-probs of given
tokens straight from hidden states and the head's weight, without the logits in
memory, their gradient to both, the embedding of tokens, and its gradient by
sorted tokens (the same weight, where head and embedding are tied).

``run`` computes a case in its plain form (elementary torch operations) or,
with ``own`` true, by the library's entry points; ``exact`` gives the results
in 64 bits.

The formulas, for hidden states h [N, K], the weight W [V, K], s = 1 / temperature:

    x_v = sum_k h_k W_vk,  m = max_v x_v,  Z = sum_v exp(s (x_v - m))
    log p_v = s (x_v - m) - log Z,  logp = log p_a,  H = -sum_v p_v log p_v
    d_v = s (dlogp (1[v = a] - p_v) - dH p_v (log p_v + H))
    dL/dh_k = sum_v d_v W_vk,  dL/dW_vk = sum over tokens of d_v h_k

    embedding: e_t = scale W[id_t],  dL/dW_v = scale sum over tokens with id_t = v of g_t
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CLIPPED = 0.2  # share of the tokens whose log-prob gets no gradient


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _head(name, B, T, K, V, dtype, *, lead=0, low=None, entropy=True, temperature=1.0, sigma=2.0):
    return {"name": name, "op": "head", "B": B, "T": T, "K": K, "V": V, "dtype": dtype, "lead": lead, "low": T if low is None else low,
            "entropy": entropy, "temperature": temperature, "sigma": sigma}


def _head_grad(name, B, T, K, V, dtype, *, lead=0, low=None, entropy=True, temperature=1.0, sigma=2.0):
    return {**_head(name, B, T, K, V, dtype, lead=lead, low=low, entropy=entropy, temperature=temperature, sigma=sigma), "op": "head_grad"}


def _embed(name, B, T, K, V, dtype, *, scale=1.0):
    return {"name": name, "op": "embed", "B": B, "T": T, "K": K, "V": V, "dtype": dtype, "low": T, "scale": scale}


def _embed_grad(name, B, T, K, V, dtype, *, low=None, scale=1.0, tied=False):
    return {"name": name, "op": "embed_grad", "B": B, "T": T, "K": K, "V": V, "dtype": dtype, "low": T if low is None else low,
            "scale": scale, "tied": tied}


def listed():
    return [
        # one sequence that generates with a small model: the next token's log-prob; the weight is read once
        _head("head one token", 1, 1, 2048, 32768, "bf16"),
        # a serving step of a batch at the sampling temperature
        _head("head decode step", 64, 1, 4096, 151936, "bf16", temperature=0.8, sigma=3.0),
        # a rollout scored at once behind its prompts, ragged completions, entropy as a training signal
        _head("head rollout", 16, 1024, 2048, 151936, "bf16", lead=64, low=128),
        # odd everything: vocabulary, width (rows of the weight start anywhere), lengths
        _head("head odd", 12, 333, 1021, 49999, "f16", lead=5, low=9, temperature=0.7),
        # single precision, log-probs alone
        _head("head f32", 8, 256, 1024, 32768, "f32", low=16, entropy=False),
        # the smallest training batch
        _head_grad("head grad tiny", 8, 16, 64, 512, "f32", low=4, sigma=1.0),
        # the training step on a rollout, with an entropy bonus
        _head_grad("head grad rollout", 8, 1024, 2048, 151936, "bf16", lead=64, low=128),
        # odd sizes in half precision, no entropy term
        _head_grad("head grad odd", 6, 333, 1021, 49999, "f16", lead=5, low=9, entropy=False),
        # a serving step's tokens into a wide model, scaled by the root of its width
        _embed("embed decode step", 64, 1, 4096, 151936, "bf16", scale=64.0),
        # a training batch of prompts and completions
        _embed("embed rollout", 64, 1024, 2048, 151936, "bf16"),
        # its gradient: padding left out, frequent tokens by the thousand, absent ones zero
        _embed_grad("embed grad rollout", 64, 1024, 2048, 151936, "bf16", low=192),
        # a tied weight's gradient, added to what the head left there; odd width
        _embed_grad("embed grad tied", 8, 257, 1021, 9973, "f32", low=31, scale=32.0, tied=True),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["head", "head", "head_grad", "head_grad", "embed", "embed_grad"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    V = rng.choice([_spread(rng, 50, 4000), _spread(rng, 4000, 152000), 32768, 128256, 151936])
    K = rng.choice([_spread(rng, 16, 1200), 8 * _spread(rng, 16, 512), 1024, 2048, 4096])
    if op in ("embed", "embed_grad"):
        most = min(65536, 130_000_000 // K)
        V = min(V, 300_000_000 // K)
    else:
        # single precision costs several times the products of the others
        most = {"head": 1500, "head_grad": 600}[op] * 10 ** 9 // (K * V * (4 if dtype == "f32" else 1))
        most = max(1, min(16384, most))
    B = 1 if rng.random() < 0.2 else _spread(rng, 1, min(64, most))
    T = 1 if rng.random() < 0.3 else _spread(rng, 1, max(1, min(1200, most // B)))
    low = T if T == 1 or rng.random() < 0.3 else rng.randint(0, T)
    t, lead, sigma = rng.choice([1.0, 1.0, 0.6, 1.3]), rng.choice([0, 0, rng.randint(1, 70)]), rng.choice([1.0, 2.0, 3.0])
    if op == "embed":
        c = _embed("", B, T, K, V, dtype, scale=rng.choice([1.0, 0.5, math.sqrt(K)]))
    elif op == "embed_grad":
        c = _embed_grad("", B, T, K, V, dtype, low=low, scale=rng.choice([1.0, 0.5, math.sqrt(K)]), tied=rng.random() < 0.4)
    else:
        make = _head if op == "head" else _head_grad
        c = make("", B, T, K, V, dtype, lead=lead, low=low, entropy=rng.random() < 0.6, temperature=t, sigma=sigma)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lengths(case):
    """Completion lengths, evenly from low to T."""
    B, T, low = case["B"], case["T"], case["low"]
    return [T if B == 1 else low + (T - low) * b // (B - 1) for b in range(B)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, T, K, V, dt = case["B"], case["T"], case["K"], case["V"], DTYPES[case["dtype"]]
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=dt)  # noqa: E731
    order = torch.tensor(random.Random(seed).sample(_lengths(case), B), device="cuda")
    mask = torch.arange(T, device="cuda")[None, :] < order[:, None]
    state = {"case": case, "mask": mask}
    if case["op"] in ("embed", "embed_grad"):
        # token n of the vocabulary's order by frequency has a share of about 1 / n; the order is not that of the ids
        u = torch.rand((B, T), generator=g, device="cuda", dtype=torch.float64)
        rank = (float(V + 1) ** u).long().sub_(1).clamp_(0, V - 1)
        state["ids"] = torch.randperm(V, generator=g, device="cuda")[rank]
        if case["op"] == "embed":
            state["weight"] = normal(V, K).mul_(0.02)
            return state
        state["grad"] = normal(B, T, K).mul_(1e-3)
        # a tied weight's gradient: the head's part is there already, in single precision
        state["head_grad"] = normal(V, K).float().mul_(1e-4) if case["tied"] else None
        return state
    # hidden states behind a norm, of whole sequences: the completion's come behind `lead` others
    state["hidden"] = normal(B, case["lead"] + T, K)[:, case["lead"]:]
    state["weight"] = normal(V, K).mul_(case["sigma"] / math.sqrt(K))
    # the tokens are drawn from the policy itself (the largest of x s plus Gumbel noise), a part of the rows at a time
    rows, ids, stats, entropy = state["hidden"].reshape(B * T, K), [], [], []
    s = 1.0 / case["temperature"]
    weight = state["weight"].float() if case["op"] == "head_grad" else state["weight"]
    for part in rows.to(weight.dtype).split(max(1, (1 << 29) // V)):
        z = (part @ weight.t()).float()
        u = torch.rand(z.shape, generator=g, device="cuda").clamp_(1e-12, 1 - 1e-7).log_().neg_().log_().neg_()
        ids.append(u.add_(z, alpha=s).argmax(-1))
        del u
        if case["op"] == "head_grad":  # what the forward pass left
            m = z.amax(-1)
            e = z.sub_(m[:, None]).mul_(s)
            p = e.exp()
            Z = p.sum(-1)
            stats.append(torch.stack([m, Z]))
            entropy.append(Z.log() - p.mul_(e).sum(-1) / Z)
            del p, e
        del z
    state["ids"] = torch.cat(ids).reshape(B, T)
    if case["op"] == "head_grad":
        state["stats"] = torch.cat(stats, 1).reshape(2, B, T)
        state["entropy"] = torch.cat(entropy).reshape(B, T)
        # the loss' gradients, means over the tokens: some tokens are clipped
        keep = torch.rand((B, T), generator=g, device="cuda") >= CLIPPED
        keep[0, 0] = True
        state["dlogp"] = torch.randn((B, T), generator=g, device="cuda") * keep / (B * T)
        state["dH"] = torch.full((B, T), -0.01 / (B * T), device="cuda")
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    case = state["case"]
    return {"head": _run_head, "head_grad": _run_head_grad, "embed": _run_embed, "embed_grad": _run_embed_grad}[case["op"]](state, case)


def _run_head(state, case):
    h, W, ids, mask = (state[n] for n in ("hidden", "weight", "ids", "mask"))
    if own:
        import grad_row_online_gb300 as lib
        r = lib.grpo_linear_logps(h, W, ids, mask, temperature=case["temperature"], want_entropy=case["entropy"])
        return {n: r[n] for n in (("logps", "entropy") if case["entropy"] else ("logps",))}
    s = 1.0 / case["temperature"]
    z = h[mask].float() @ W.float().t()
    t = (z - z.amax(-1, keepdim=True)).mul_(s)
    del z
    e = t.exp()
    Z = e.sum(-1)
    out = {"logps": torch.zeros(ids.shape, device=h.device)}
    out["logps"][mask] = t.gather(-1, ids[mask][:, None])[:, 0] - Z.log()
    if case["entropy"]:
        out["entropy"] = torch.zeros(ids.shape, device=h.device)
        out["entropy"][mask] = Z.log() - e.mul_(t).sum(-1) / Z
    return out


def _run_head_grad(state, case):
    h, W, ids, mask, stats, H = (state[n] for n in ("hidden", "weight", "ids", "mask", "stats", "entropy"))
    if own:
        import grad_row_online_gb300 as lib
        more = {"entropy": H, "grad_entropy": state["dH"]} if case["entropy"] else {}
        return lib.grpo_linear_logps_grad(h, W, ids, mask, stats, grad_logps=state["dlogp"], temperature=case["temperature"], **more)
    s = 1.0 / case["temperature"]
    # a token without a gradient adds nothing
    on = mask if case["entropy"] else mask & (state["dlogp"] != 0)
    rows, w, dlogp, dH, (m, Z) = h[on].float(), W.float(), state["dlogp"][on], state["dH"][on], stats[:, on]
    t = (rows @ w.t()).sub_(m[:, None]).mul_(s)
    p = t.exp() / Z[:, None]
    d = -dlogp[:, None] * p
    if case["entropy"]:
        d -= p.mul_(t.add_((H[on] - Z.log())[:, None])).mul_(dH[:, None])
    del t, p
    d.scatter_add_(-1, ids[on][:, None], dlogp[:, None]).mul_(s)
    grad = torch.zeros(h.shape, device=h.device)
    grad[on] = d @ w
    return {"grad_hidden": grad.to(h.dtype), "grad_weight": (d.t() @ rows).to(W.dtype)}


def _run_embed(state, case):
    W, ids = state["weight"], state["ids"]
    if own:
        import grad_row_online_gb300 as lib
        return lib.grpo_embed_tokens(W, ids, scale=case["scale"])
    return (W[ids].float() * case["scale"]).to(W.dtype)


def _run_embed_grad(state, case):
    grad, ids, mask, head = (state[n] for n in ("grad", "ids", "mask", "head_grad"))
    if own:
        import grad_row_online_gb300 as lib
        return lib.grpo_embed_tokens_grad(grad, ids, case["V"], mask, scale=case["scale"], add=head)
    sums = torch.zeros((case["V"], case["K"]), device=grad.device).index_add_(0, ids[mask], grad[mask].float()).mul_(case["scale"])
    return sums.add_(head) if case["tied"] else sums.to(grad.dtype)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    B, T, K, V, size = case["B"], case["T"], case["K"], case["V"], DTYPES[case["dtype"]].itemsize
    n = sum(_lengths(case))
    if case["op"] == "head":
        return {"bytes": (V + n) * K * size + B * T * (1 + 8 + 4 + 4 * case["entropy"]), "flops": n * V * (2 * K + 5)}
    if case["op"] == "head_grad":
        # the logits are not kept: three products
        on = n if case["entropy"] else (1 - CLIPPED) * n
        return {"bytes": (2 * V + on + B * T) * K * size + B * T * (1 + 8 + 12 + 8 * case["entropy"]), "flops": on * V * (6 * K + 7)}
    # rows of the weight that some token takes, by the share of each in the draw
    q = [math.log1p(1 / i) / math.log(V + 1) for i in range(1, V + 1)]
    taken = sum(-math.expm1(n * math.log1p(-p)) if p < 1 else 1.0 for p in q)
    if case["op"] == "embed":
        return {"bytes": (taken + B * T) * K * size + 8 * B * T, "flops": B * T * K}
    rows = 2 * V * 4 if case["tied"] else V * size
    return {"bytes": (n * size + rows) * K + 9 * B * T, "flops": (n + taken) * K}


# ---------------------------------------------------------------------------
# the same in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] in ("head", "head_grad") and work(case)["flops"] > 1.2e13:
        return None  # (64-bit products run at about 1 TFLOP/s)
    state = prepare(case, seed)
    ids, on = state["ids"].reshape(-1), state["mask"].reshape(-1).double()
    if case["op"] == "embed":
        return state["weight"].double().index_select(0, ids).mul_(case["scale"]).reshape(*state["ids"].shape, case["K"])
    if case["op"] == "embed_grad":
        order = torch.sort(ids, stable=True).indices
        rows = state["grad"].reshape(-1, case["K"])[order].double() * (on[order] * case["scale"])[:, None]
        counts = torch.bincount(ids, minlength=case["V"])
        sums = torch.segment_reduce(rows, "sum", lengths=counts, initial=0.0)
        return sums if state["head_grad"] is None else sums + state["head_grad"].double()
    B, T, K, V = case["B"], case["T"], case["K"], case["V"]
    rows, W = state["hidden"].reshape(B * T, K), state["weight"].double()
    if case["op"] == "head":
        live = on.nonzero()[:, 0]
        logps, entropy = torch.zeros(B * T, device="cuda", dtype=torch.float64), torch.zeros(B * T, device="cuda", dtype=torch.float64)
        for part in live.split(max(1, (1 << 28) // V)):
            lp = torch.log_softmax(torch.matmul(rows[part].double(), W.T) / case["temperature"], -1)
            logps[part] = lp[torch.arange(len(part), device="cuda"), ids[part]]
            entropy[part] = -(lp.exp() * lp).sum(-1)
        return {"logps": logps.reshape(B, T), "entropy": entropy.reshape(B, T)} if case["entropy"] else {"logps": logps.reshape(B, T)}
    a = on * state["dlogp"].reshape(-1).double()
    b = on * state["dH"].reshape(-1).double() if case["entropy"] else torch.zeros_like(a)
    dh, dW = torch.zeros((B * T, K), device="cuda", dtype=torch.float64), torch.zeros((V, K), device="cuda", dtype=torch.float64)
    for part in ((a != 0) | (b != 0)).nonzero()[:, 0].split(max(1, (1 << 28) // V)):
        x = rows[part].double()
        lp = torch.log_softmax(torch.matmul(x, W.T) / case["temperature"], -1)
        p = lp.exp()
        H = -(p * lp).sum(-1, keepdim=True)
        d = -p * (a[part][:, None] + b[part][:, None] * (lp + H))
        d[torch.arange(len(part), device="cuda"), ids[part]] += a[part]
        d /= case["temperature"]
        dh[part] = d @ W
        dW += d.T @ x
    return {"grad_hidden": dh.reshape(B, T, K), "grad_weight": dW}
