"""Measured cases of the training operators: the gated feed-forward block (``layers``) and the
two vocabulary losses (``losses``).

A case is a dict of plain values. ``run`` computes it in plain torch operations in 32 bits,
rounded once at the end, or, with ``own`` true, through the framework's kernels. ``exact``
computes it in 64 bits with torch's automatic differentiation.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token through the 7B shape set's feed-forward block: the weights' HBM traffic
        ffn("ffn_7b_one_token", "ffn", 1, 3584, 18944),
        # a ragged prompt through the single-matrix workload's 2560 x 9728 shape
        ffn("ffn_2560x9728_333_tokens", "ffn", 333, 2560, 9728, act="gelu_tanh"),
        # a long prompt through the 7B block: bound by the matrix cores
        ffn("ffn_7b_4096_tokens", "ffn", 4096, 3584, 18944),
        # the smallest training step: fp32, the 256 x 1024 workload's shape
        ffn("ffn_train_f32_256x1024", "ffn_train", 100, 256, 1024, dtype="f32"),
        # odd sizes in every direction: nothing is 16-byte aligned from row to row
        ffn("ffn_train_odd_sizes", "ffn_train", 1537, 413, 1111, act="gelu_tanh"),
        # a training step of the 24-layer decoder's block
        ffn("ffn_train_2048x8192", "ffn_train", 2048, 2048, 8192),
        # a training step of the 7B block: the largest case
        ffn("ffn_train_7b_4096_tokens", "ffn_train", 4096, 3584, 18944),
        # a few sampled tokens over the 7B vocabulary: latency
        policy("policy_16_tokens", 16, 152064),
        # a batch of responses with padding rows, logits a slice of a wider buffer
        policy("policy_4096_tokens_padded", 4096, 151936, pad=128, masked=0.2),
        # fp32 logits of an odd vocabulary, no reference model
        policy("policy_f32_odd_vocabulary", 1000, 32003, dtype="f32", kl=0.0, masked=0.1),
        # distillation from 64 kept logits a token over the 7B vocabulary
        distill("distill_2048_tokens_top64", 2048, 152064, 64, masked=0.1),
        # few tokens, fp32, few and partly absent entries, teacher normaliser given
        distill("distill_f32_77_tokens_top7", 77, 32003, 7, dtype="f32", absent=0.2, given_lse=True),
    ]


def ffn(name, op, tokens, dim, hidden, dtype="bf16", act="silu"):
    return {"name": name, "op": op, "tokens": tokens, "dim": dim, "hidden": hidden, "dtype": dtype, "act": act}


def policy(name, rows, vocab, dtype="bf16", pad=0, masked=0.0, kl=0.05, temperature=1.0):
    return {"name": name, "op": "policy", "rows": rows, "vocab": vocab, "dtype": dtype, "pad": pad,
            "masked": masked, "kl": kl, "temperature": temperature}


def distill(name, rows, vocab, top, dtype="bf16", masked=0.0, absent=0.0, given_lse=False, temperature=2.0):
    return {"name": name, "op": "distill", "rows": rows, "vocab": vocab, "top": top, "dtype": dtype,
            "masked": masked, "absent": absent, "given_lse": given_lse, "temperature": temperature}


def draw(rng):
    def size(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return n if rng.random() < 0.5 else max(lo, n // 64 * 64)   # ragged and whole sizes

    dtype = "bf16" if rng.random() < 0.7 else "f32"
    op = rng.choice(["ffn", "ffn_train", "policy", "distill"])
    if op in ("ffn", "ffn_train"):
        dim, hidden = size(64, 3584), size(128, 18944)
        # fp32 costs more a product than bf16
        most = (1 << 38) // (1 if dtype == "bf16" else 8) // (dim * hidden)
        tokens = min(size(1, 4096), max(1, most))
        c = ffn("", op, tokens, dim, hidden, dtype, rng.choice(["silu", "gelu_tanh"]))
    else:
        vocab = size(1000, 152064)
        rows = min(size(1, 4096), (1 << 29) // vocab)
        masked = rng.choice([0.0, 0.1, 0.5])
        temperature = rng.choice([1.0, 0.7, 2.0])
        if op == "policy":
            c = policy("", rows, vocab, dtype, rng.choice([0, 5, 64]), masked, rng.choice([0.0, 0.05]), temperature)
        else:
            c = distill("", rows, vocab, min(size(1, 256), vocab), dtype, masked, rng.choice([0.0, 0.3]),
                        rng.random() < 0.5, temperature)
    del c["name"]
    return c


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("ffn", "ffn_train"):
        t, d, f = case["tokens"], case["dim"], case["hidden"]
        if case["op"] == "ffn":
            return {"bytes": es * (2 * t * d + 3 * d * f), "flops": 6 * t * d * f}
        return {"bytes": es * (4 * t * d + 6 * d * f), "flops": 18 * t * d * f}
    n, v = case["rows"], case["vocab"]
    live = n - int(n * case["masked"])
    small = 24 * n if case["op"] == "policy" else n * (8 + 12 * case["top"])
    return {"bytes": es * v * (live + n) + small, "flops": 6 * live * v}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * scale

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    dt = DTYPES[case["dtype"]]
    state = dict(case)
    if case["op"] in ("ffn", "ffn_train"):
        t, d, f = case["tokens"], case["dim"], case["hidden"]
        # activations of a normalised stream, weights that keep its scale, so that the
        # gate's curved range is met
        state["x"] = normal(t, d).to(dt)
        state["w_gate"] = normal(f, d, scale=1.5 / math.sqrt(d)).to(dt)
        state["w_up"] = normal(f, d, scale=1.0 / math.sqrt(d)).to(dt)
        state["w_down"] = normal(d, f, scale=1.0 / math.sqrt(f)).to(dt)
        if case["op"] == "ffn_train":
            state["dy"] = normal(t, d, scale=1e-3).to(dt)
        return state

    n, v = case["rows"], case["vocab"]
    pad = case.get("pad", 0)
    wide = torch.empty(n, v + pad, dtype=dt, device="cuda")
    for r in range(0, n, 512):   # a language model's logits: most of the mass on few entries
        wide[r:r + 512] = (normal(min(512, n - r), v + pad, scale=2.5)).to(dt)
    logits = wide[:, :v]
    weights = torch.full((n,), 1.0 / n, device="cuda")
    masked = int(n * case["masked"])
    if masked:   # padding rows hold whatever the buffer held before
        rows = torch.randperm(n, generator=gen, device="cuda")[:masked]
        weights[rows] = 0.0
        logits[rows] = float("nan")
    state["logits"], state["weights"] = logits, weights
    if case["op"] == "policy":
        # sampled tokens: raise each one's logit, as a model that sampled it gave it some mass
        targets = torch.randint(0, v, (n,), generator=gen, device="cuda")
        at = torch.arange(n, device="cuda")
        logits[at, targets] += (6.0 + 4.0 * uniform(n)).to(dt)
        lp = torch.empty(n, device="cuda")
        for r in range(0, n, 512):
            z = logits[r:r + 512].double() / case["temperature"]
            lp[r:r + 512] = (z.gather(1, targets[r:r + 512, None])[:, 0] - z.logsumexp(1)).float()
        # log ratios of an older policy, clipped on both sides for some, none within 1e-3 of a border
        ratio = torch.exp(0.2 * normal(n))
        for border in (0.8, 1.28):
            ratio = torch.where((ratio - border).abs() < 1e-3, torch.full_like(ratio, border + 2e-3), ratio)
        live = weights > 0
        state["targets"] = targets
        state["old_logp"] = torch.where(live, lp - ratio.log(), 0.0)
        state["advantages"] = normal(n)
        state["ref_logp"] = torch.where(live, lp + 0.3 * normal(n), 0.0) if case["kl"] else None
    else:
        k = case["top"]
        # distinct ids in each row: a random start and an odd stride through the vocabulary
        stride = 2 * torch.randint(0, max(1, v // (2 * k)), (n, 1), generator=gen, device="cuda") + 1
        start = torch.randint(0, v, (n, 1), generator=gen, device="cuda")
        span = torch.arange(k, device="cuda")[None, :]
        ids = (start + stride * span) % v
        top = normal(n, k, scale=2.0).sort(dim=1, descending=True).values + 8.0
        if case["absent"]:
            gone = uniform(n, k) < case["absent"]
            ids = torch.where(gone, torch.full_like(ids, -1), ids)
        state["top_ids"], state["top_logits"] = ids, top
        if case["given_lse"]:
            # the kept entries hold part of the teacher's mass
            kept = torch.logsumexp(top / case["temperature"], dim=1)
            state["top_lse"] = kept + 0.3 * uniform(n)
        else:
            state["top_lse"] = None
    return state


# ---------------------------------------------------------------- one pass

CLIP_LOW, CLIP_HIGH = 0.2, 0.28


def run(state):
    if own:
        return run_own(state)
    return {"ffn": plain_ffn, "ffn_train": plain_ffn_train, "policy": plain_policy, "distill": plain_distill}[state["op"]](state)


def run_own(state):
    from matrix_orthogonalising_optimizer_muon_amd import layers, losses

    if state["op"] == "ffn":
        return layers.ffn_forward(state["x"], state["w_gate"], state["w_up"], state["w_down"],
                                  activation=state["act"])[0]
    if state["op"] == "ffn_train":
        x, wg, wu, wd = state["x"], state["w_gate"], state["w_up"], state["w_down"]
        y, saved = layers.ffn_forward(x, wg, wu, wd, activation=state["act"], save=True)
        return (y, *layers.ffn_backward(state["dy"], x, wg, wu, wd, saved, activation=state["act"]))
    if state["op"] == "policy":
        return losses.policy_loss(state["logits"], state["targets"], state["old_logp"], state["advantages"],
                                  ref_logp=state["ref_logp"], weights=state["weights"], clip_low=CLIP_LOW,
                                  clip_high=CLIP_HIGH, kl_coef=state["kl"], temperature=state["temperature"])
    return losses.distill_loss(state["logits"], state["top_logits"], state["top_ids"], top_lse=state["top_lse"],
                               weights=state["weights"], temperature=state["temperature"])


def act_and_slope(g, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    th = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * c * (1.0 + 3 * 0.044715 * g * g)


def plain_ffn(state):
    x, wg, wu, wd = (state[k].float() for k in ("x", "w_gate", "w_up", "w_down"))
    a, _ = act_and_slope(x @ wg.T, state["act"])
    return ((a * (x @ wu.T)) @ wd.T).to(state["x"].dtype)


def plain_ffn_train(state):
    dt = state["x"].dtype
    x, wg, wu, wd, dy = (state[k].float() for k in ("x", "w_gate", "w_up", "w_down", "dy"))
    g, u = x @ wg.T, x @ wu.T
    a, slope = act_and_slope(g, state["act"])
    h = a * u
    y = h @ wd.T
    dh = dy @ wd
    dg, du = dh * u * slope, dh * a
    return (y.to(dt), (dg @ wg + du @ wu).to(dt), (dg.T @ x).to(dt), (du.T @ x).to(dt), (dy.T @ h).to(dt))


def log_softmax_rows(state):
    """(live rows, their scaled logits' log-probabilities, 32 bits)."""
    live = state["weights"] > 0
    z = state["logits"].float() / state["temperature"]
    z = torch.where(live[:, None], z, torch.zeros_like(z))
    z = z - z.amax(dim=1, keepdim=True)
    return live, z - torch.exp(z).sum(dim=1, keepdim=True).log()


def plain_policy(state):
    dt, w, t = state["logits"].dtype, state["weights"], state["targets"][:, None]
    live, lq = log_softmax_rows(state)
    lp = lq.gather(1, t)[:, 0]
    adv = state["advantages"]
    ratio = torch.exp(lp - state["old_logp"])
    kept, cut = ratio * adv, ratio.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH) * adv
    loss = -torch.minimum(kept, cut)
    slope = torch.where(kept <= cut, -kept, torch.zeros_like(kept))
    if state["ref_logp"] is not None:
        d = state["ref_logp"] - lp
        loss = loss + state["kl"] * (torch.expm1(d) - d)
        slope = slope - state["kl"] * torch.expm1(d)
    slope = torch.where(live, slope * w, torch.zeros_like(w)) / state["temperature"]
    grad = torch.exp(lq) * -slope[:, None]
    grad.scatter_add_(1, t, slope[:, None])
    zero = torch.zeros_like(w)
    return torch.where(live, loss * w, zero), torch.where(live, lp, zero), grad.to(dt)


def plain_distill(state):
    dt, w, tau = state["logits"].dtype, state["weights"], state["temperature"]
    live, lq = log_softmax_rows(state)
    ids = state["top_ids"]
    there = ids >= 0
    ids = ids.clamp(min=0)
    t = torch.where(there, state["top_logits"] / tau, torch.full_like(state["top_logits"], -torch.inf))
    if state["top_lse"] is not None:
        norm = state["top_lse"][:, None]
    else:
        most = t.amax(dim=1, keepdim=True).clamp(min=-1e30)
        norm = most + torch.exp(t - most).sum(dim=1, keepdim=True).log()
    lp = torch.where(there, t - norm, torch.zeros_like(t))
    p = torch.where(there, torch.exp(lp), torch.zeros_like(t))
    loss = (p * (lp - lq.gather(1, ids))).sum(dim=1) * w
    coef = torch.where(live, w / tau, torch.zeros_like(w))[:, None]
    grad = torch.exp(lq) * (coef * p.sum(dim=1, keepdim=True))
    grad.scatter_add_(1, ids, -coef * p)
    return torch.where(live, loss, torch.zeros_like(w)), grad.to(dt)


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("ffn", "ffn_train"):
        leaves = [s[k].double().requires_grad_(case["op"] == "ffn_train") for k in ("x", "w_gate", "w_up", "w_down")]
        x, wg, wu, wd = leaves
        gate = torch.nn.functional.linear(x, wg)
        if case["act"] == "silu":
            gate = gate * torch.sigmoid(gate)
        else:
            gate = torch.nn.functional.gelu(gate, approximate="tanh")
        y = torch.nn.functional.linear(gate * torch.nn.functional.linear(x, wu), wd)
        if case["op"] == "ffn":
            return y
        grads = torch.autograd.grad(y, leaves, s["dy"].double())
        return (y.detach(), *grads)

    n, w = case["rows"], s["weights"].double()
    rows, second, grads = [], [], []
    for r in range(0, n, 256):   # rows are independent
        part = slice(r, min(n, r + 256))
        wr = w[part]
        live = wr > 0
        z = torch.where(live[:, None], s["logits"][part].double(), 0.0).requires_grad_(True)
        q = torch.log_softmax(z / case["temperature"], dim=1)
        if case["op"] == "policy":
            lp = q.gather(1, s["targets"][part, None])[:, 0]
            ratio, adv = torch.exp(lp - s["old_logp"][part].double()), s["advantages"][part].double()
            each = torch.maximum(-adv * ratio, -adv * ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH))
            if s["ref_logp"] is not None:
                d = s["ref_logp"][part].double() - lp
                each = each + case["kl"] * (torch.exp(d) - d - 1)
            second.append(torch.where(live, lp, 0.0).detach())
        else:
            ids, t = s["top_ids"][part], s["top_logits"][part].double() / case["temperature"]
            t = t.masked_fill(ids < 0, -torch.inf)
            norm = (torch.logsumexp(t, 1) if s["top_lse"] is None else s["top_lse"][part].double())[:, None]
            p = torch.where(ids < 0, 0.0, torch.exp(t - norm))
            each = (torch.special.xlogy(p, p) - p * q.gather(1, ids.clamp(min=0))).sum(1)
        loss = torch.where(live, wr * each, 0.0)
        grads.append(torch.autograd.grad(loss.sum(), z)[0])
        rows.append(loss.detach())
    out = [torch.cat(rows)] + ([torch.cat(second)] if second else []) + [torch.cat(grads)]
    return tuple(out)
