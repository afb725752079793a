"""Measured cases of what a decoder layer's training pass runs beside its feed-forward block:
linear attention with a decay for each head (``mixers``), tokens sorted by expert and back
(``experts``) and dropout from a counter (``dropout``).

A case is a dict of plain values. ``run`` computes it in plain torch operations in 32 bits,
rounded once at the end, or, with ``own`` true, through the framework's kernels. ``exact``
computes it in 64 bits: the attention token by token, from its recurrence.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one request generating: the state of 16 heads, latency
        step("mix_step_one_request", 1, 16, 16, 128, 128),
        # a batch generating with the 7B shape set's heads (28, of 4 for k and v): the states' HBM traffic
        step("mix_step_128_requests", 128, 28, 4, 128, 128),
        # prompts of several lengths padded to one, continued from a state each
        mix("mix_prompts_padded", "mix", 5, 1000, 16, 16, 64, 64, lengths=True, state=True),
        # one long prompt through the 2048-wide decoder's 16 heads: few heads, a long axis
        mix("mix_long_prompt", "mix", 1, 65536, 16, 16, 128, 128),
        # a training pass of the decoder's layer: forward and the gradients of q, k and v
        mix("mix_train_2048_wide", "mix_train", 8, 2048, 16, 16, 128, 128),
        # training in fp32 at odd sizes, k and v shared by three heads, a state carried in and out
        mix("mix_train_f32_odd_sizes", "mix_train", 2, 777, 6, 2, 40, 72, dtype="f32", state=True),
        # a few tokens through 2 of 8 experts: latency
        route("experts_16_tokens", "experts", 16, 2, 8, 2048),
        # a training step's tokens to 8 of 64 experts, their results back, and all gradients
        route("experts_train_8192_tokens", "experts_train", 8192, 8, 64, 2048),
        # odd sizes in fp32, a tenth of the choices dropped
        route("experts_train_f32_odd_sizes", "experts_train", 3001, 3, 37, 413, dtype="f32", dropped=0.1),
        # a few tokens' residual stream: latency
        drop("dropout_16_tokens", "dropout", 16, 2048, residual=True),
        # a training step over the 7B width: added to the residual stream, and the gradient
        drop("dropout_train_16384_tokens", "dropout_train", 16384, 3584, residual=True),
        # fp32, odd sizes, no residual
        drop("dropout_train_f32_odd_sizes", "dropout_train", 1000, 1111, dtype="f32", p=0.37),
    ]


def step(name, batch, heads, kv_heads, dim, dim_v, dtype="bf16"):
    return {"name": name, "op": "mix_step", "batch": batch, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "dim_v": dim_v, "dtype": dtype}


def mix(name, op, batch, tokens, heads, kv_heads, dim, dim_v, dtype="bf16", lengths=False, state=False):
    return {"name": name, "op": op, "batch": batch, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "dim_v": dim_v, "dtype": dtype, "lengths": lengths, "state": state}


def route(name, op, tokens, top, experts, dim, dtype="bf16", dropped=0.0):
    return {"name": name, "op": op, "tokens": tokens, "top": top, "experts": experts, "dim": dim, "dtype": dtype,
            "dropped": dropped}


def drop(name, op, tokens, dim, dtype="bf16", p=0.1, residual=False):
    return {"name": name, "op": op, "tokens": tokens, "dim": dim, "dtype": dtype, "p": p, "residual": residual}


def draw(rng):
    def size(lo, hi, whole=64):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return n if rng.random() < 0.5 else max(lo, n // whole * whole)   # ragged and whole sizes

    dtype = "bf16" if rng.random() < 0.7 else "f32"
    op = rng.choice(["mix_step", "mix", "mix_train", "experts", "experts_train", "dropout", "dropout_train"])
    if op.startswith("mix"):
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 1, 3, 4])
        dim, dim_v = size(16, 256, 16), size(16, 256, 16)
        if op == "mix_step":
            c = step("", min(size(1, 128), max(1, (1 << 25) // (heads * dim * dim_v))), heads, kv_heads, dim, dim_v, dtype)
        else:
            batch = size(1, 8, 2)
            # an eighth of the longest prompt's products at most for a training pass in 32 bits
            most = (1 << 27) // {"mix": 1, "mix_train": 4}[op] // (heads * max(dim, dim_v)) // batch
            if dtype == "f32":
                most //= 2
            c = mix("", op, batch, min(size(1, 32768), max(1, most)), heads, kv_heads, dim, dim_v, dtype,
                    rng.random() < 0.4, rng.random() < 0.5)
    elif op.startswith("experts"):
        experts = size(2, 256, 8)
        top, dim = rng.randint(1, min(8, experts)), size(64, 4096)
        most = (1 << (27 if dtype == "bf16" else 26)) // (top * dim)
        c = route("", op, min(size(1, 16384), max(1, most)), top, experts, dim, dtype, rng.choice([0.0, 0.0, 0.1, 0.5]))
    else:
        dim = size(64, 4096)
        c = drop("", op, min(size(1, 16384), (1 << (25 if dtype == "bf16" else 24)) // dim), dim, dtype, rng.choice([0.0, 0.05, 0.1, 0.37, 0.5]),
                 rng.random() < 0.5)
    del c["name"]
    return c


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("mix"):
        b, h, hk, d, e = (case[k] for k in ("batch", "heads", "kv_heads", "dim", "dim_v"))
        t = case.get("tokens", 1)
        q, k, v, o, s = b * t * h * d, b * t * hk * d, b * t * hk * e, b * t * h * e, 4 * b * h * d * e
        if op == "mix_step":
            return {"bytes": es * (q + k + v + o) + 2 * s, "flops": 5 * b * h * d * e}
        states = s * (2 if case["state"] else 1)
        flops = 4 * b * t * h * d * e       # the recurrence's own: the state's update and its product with q
        if op == "mix":
            return {"bytes": es * (q + k + v + o) + states, "flops": flops}
        # q, k, v, do read, o and three gradients written; the state and its gradient in and out
        return {"bytes": es * (2 * q + 2 * k + 2 * v + 2 * o) + 2 * states, "flops": 4 * flops}
    if op.startswith("experts"):
        t, j, d = case["tokens"], case["top"], case["dim"]
        there = t * j - int(t * j * case["dropped"])
        if op == "experts":                 # x in, the sorted rows out; the experts' rows in, y out
            return {"bytes": es * d * (2 * t + 2 * there) + 12 * t * j, "flops": 2 * there * d}
        return {"bytes": es * d * (4 * t + 5 * there) + 24 * t * j, "flops": 6 * there * d}
    n = case["tokens"] * case["dim"]
    arrays = 2 + case["residual"]
    if op == "dropout_train":
        arrays += 2
    return {"bytes": es * arrays * n, "flops": 2 * n}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * scale

    dt = DTYPES[case["dtype"]]
    state = dict(case)
    if case["op"].startswith("mix"):
        b, h, hk, d, e = (case[k] for k in ("batch", "heads", "kv_heads", "dim", "dim_v"))
        at = (b,) if case["op"] == "mix_step" else (b, case["tokens"])
        state["q"], state["k"] = normal(*at, h, d).to(dt), normal(*at, hk, d).to(dt)
        state["v"] = normal(*at, hk, e).to(dt)
        # half-lives from 22 tokens for the first head to some thousands for the last
        state["log_decay"] = torch.log1p(-torch.exp2(-5.0 - 7.0 * torch.arange(h, device="cuda") / max(h - 1, 1)))
        state["factor"] = 1.0 / math.sqrt(d)
        # a state as a long past leaves it: the variance of a decayed sum of products
        past = torch.rsqrt(-torch.expm1(2.0 * state["log_decay"])).clamp(max=32.0)[:, None, None]
        if case["op"] == "mix_step":
            state["past"] = normal(b, h, d, e) * past
            state["next"] = torch.empty_like(state["past"])
            return state
        state["past"] = normal(b, h, d, e) * past if case["state"] else None
        state["lens"] = None
        if case["lengths"]:   # one is whole, one is a single token, the padding holds anything
            lens = torch.randint(0, case["tokens"] + 1, (b,), generator=gen, device="cuda", dtype=torch.int32)
            lens[0] = case["tokens"]
            if b > 1:
                lens[1] = 1
            state["lens"] = lens
            gone = torch.arange(case["tokens"], device="cuda")[None, :] >= lens[:, None]
            for name in ("q", "k", "v"):
                state[name][gone] = float("nan")
        if case["op"] == "mix_train":
            state["do"] = normal(*at, h, e, scale=1e-3).to(dt)
            state["d_final"] = normal(b, h, d, e, scale=1e-3) if case["state"] else None
            if case["lengths"]:
                state["do"][gone] = float("nan")
        return state
    t, d = case["tokens"], case["dim"]
    if case["op"].startswith("experts"):
        j, n = case["top"], case["experts"]
        # a router's choice: some experts are liked more than others, each token takes different ones
        liking = normal(n)
        score = liking[None, :] + normal(t, n)
        chosen = score.topk(j, dim=1)
        state["ids"] = chosen.indices
        state["weights"] = torch.softmax(chosen.values, dim=1)
        if case["dropped"]:
            gone = torch.randperm(t * j, generator=gen, device="cuda")[:int(t * j * case["dropped"])]
            state["ids"].view(-1)[gone] = -1
        state["x"] = normal(t, d).to(dt)
        state["ys"] = normal(t * j, d).to(dt)       # what the experts made of the sorted rows
        if case["op"] == "experts_train":
            state["dy"] = normal(t, d, scale=1e-3).to(dt)
            state["dxs"] = normal(t * j, d, scale=1e-3).to(dt)
        return state
    state["x"] = normal(t, d).to(dt)
    state["r"] = normal(t, d, scale=4.0).to(dt) if case["residual"] else None
    state["seed"] = int(torch.randint(0, 1 << 62, (1,), generator=gen, device="cuda"))
    state["offset"] = seed % 1000
    if case["op"] == "dropout_train":
        state["dy"] = normal(t, d, scale=1e-3).to(dt)
    return state


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        return run_own(state)
    return {"mix_step": plain_step, "mix": plain_mix, "mix_train": plain_mix_train, "experts": plain_experts,
            "experts_train": plain_experts, "dropout": plain_dropout, "dropout_train": plain_dropout}[state["op"]](state)


def run_own(state):
    from matrix_orthogonalising_optimizer_muon_amd import dropout, experts, mixers

    op = state["op"]
    if op == "mix_step":
        return mixers.linear_attention_step(state["q"], state["k"], state["v"], state["log_decay"], state["past"],
                                            scale=state["factor"], out_state=state["next"])
    if op.startswith("mix"):
        args = (state["q"], state["k"], state["v"], state["log_decay"])
        kw = dict(scale=state["factor"], state=state["past"], lengths=state["lens"])
        o, final = mixers.linear_attention_forward(*args, **kw, final=True)
        if op == "mix":
            return o, final
        grads = mixers.linear_attention_backward(state["do"], *args, **kw, d_final=state["d_final"],
                                                 need_dstate=state["past"] is not None)
        return (o, final, *grads) if state["past"] is not None else (o, final, *grads[:3])
    if op.startswith("experts"):
        plan = experts.expert_plan(state["ids"], state["experts"])
        xs = experts.dispatch_forward(state["x"], plan)
        y = experts.combine_forward(state["ys"], state["weights"], plan)
        out = (plan.order, plan.slots, plan.offsets, xs, y)
        if op == "experts":
            return out
        dys, dw = experts.combine_backward(state["dy"], state["ys"], state["weights"], plan)
        return (*out, dys, dw, experts.dispatch_backward(state["dxs"], plan))
    out = dropout.dropout_forward(state["x"], state["p"], state["seed"], state["offset"], residual=state["r"])
    if op == "dropout":
        return out
    return out, dropout.dropout_backward(state["dy"], state["p"], state["seed"], state["offset"])


def plain_step(state):
    h = state["heads"]
    q, k, v = state["q"].float(), *(by_head(state[n].float(), h) for n in ("k", "v"))
    decay = torch.exp(state["log_decay"])[:, None, None]
    s = decay * state["past"] + k[..., :, None] * v[..., None, :]
    return ((q[..., :, None] * s).sum(-2) * state["factor"]).to(state["q"].dtype), s


def by_head(t, heads):
    """k or v for every head of q."""
    return t.repeat_interleave(heads // t.shape[-2], dim=-2)


CHUNK = 64


def decayed(a, b, c, g, s0, off, lens):
    """out_i = sum_{j <= i} e^{g (i - j)} (a_i . b_j) c_j + e^{g (i + off)} a_i S_0, in chunks, and
    the state after the last token, S_n = e^{g n} S_0 + sum_j e^{g (n - off - j)} b_j^T c_j.
    a, b, c: batch x heads x tokens x dim in 32 bits; lens: each sequence's tokens."""
    B, H, T, D = a.shape
    E = c.shape[-1]
    n = -(-T // CHUNK)
    pad = n * CHUNK - T
    a, b, c = (torch.nn.functional.pad(t, (0, 0, 0, pad)).reshape(B, H, n, CHUNK, -1) for t in (a, b, c))
    i = torch.arange(CHUNK, device=a.device)
    dist = (i[:, None] - i[None, :]).clamp(min=0)
    within = torch.where(i[:, None] >= i[None, :], torch.exp(g[:, None, None] * dist), 0.0)
    out = ((a @ b.transpose(-1, -2).contiguous()) * within[None, :, None]) @ c
    # tokens of each chunk in each sequence
    full = (lens[:, None] - torch.arange(n, device=a.device)[None, :] * CHUNK).clamp(0, CHUNK)
    left = full[:, None, :, None] - off - i[None, None, None, :]
    w = torch.where(i[None, None, None, :] < full[:, None, :, None], torch.exp(g[None, :, None, None] * left.clamp(min=0)), 0.0)
    added = (b * w[..., None]).transpose(-1, -2).contiguous() @ c
    over = torch.exp(g[None, :, None] * full[:, None, :])
    s = s0 if s0 is not None else torch.zeros(B, H, D, E, device=a.device)
    before = []
    for m in range(n):
        before.append(s)
        s = over[:, :, m, None, None] * s + added[:, :, m]
    if n:
        reach = torch.exp(g[:, None] * (i[None, :] + off))
        out = out + (a * reach[None, :, None, :, None]) @ torch.stack(before, 2)
    return out.reshape(B, H, n * CHUNK, E)[:, :, :T], s


def heads_first(state, *names):
    """The operands as batch x heads x tokens x dim in 32 bits, zero in the padding, and the lengths."""
    h, t = state["heads"], state["tokens"]
    lens = state["lens"]
    if lens is None:
        lens = torch.full((state["batch"],), t, device="cuda", dtype=torch.int32)
    there = torch.arange(t, device="cuda")[None, :] < lens[:, None]
    out = []
    for name in names:
        x = state[name].float()
        x = torch.where(there[:, :, None, None], x, 0.0)
        out.append(by_head(x, h).transpose(1, 2).contiguous())
    return out, lens, there[:, None, :, None]


def plain_mix(state):
    (q, k, v), lens, _ = heads_first(state, "q", "k", "v")
    o, final = decayed(q, k, v, state["log_decay"], state["past"], 1, lens)
    return (o * state["factor"]).transpose(1, 2).contiguous().to(state["q"].dtype), final


def plain_mix_train(state):
    dt, f, g, past = state["q"].dtype, state["factor"], state["log_decay"], state["past"]
    (q, k, v, do), lens, there = heads_first(state, "q", "k", "v", "do")
    o, final = decayed(q, k, v, g, past, 1, lens)
    dq, _ = decayed(do, v, k, g, None if past is None else past.transpose(-1, -2).contiguous(), 1, lens)
    # the other two run from each sequence's last token to its first
    t = torch.arange(state["tokens"], device="cuda")[None, :]
    turned = torch.where(t < lens[:, None], lens[:, None] - 1 - t, t)[:, None, :, None]
    turn = lambda x: x.gather(2, turned.expand_as(x))  # noqa: E731
    qr, kr, vr, dor = turn(q), turn(k), turn(v), turn(do * f)
    d_final = state["d_final"]
    dk, _ = decayed(vr, dor, qr, g, None if d_final is None else d_final.transpose(-1, -2).contiguous(), 0, lens)
    dv, ds = decayed(kr, qr, dor, g, d_final, 0, lens)
    dk, dv = turn(torch.where(there, dk, 0.0)), turn(torch.where(there, dv, 0.0))

    def shared(x):      # the sum over the heads that share one
        return x.reshape(x.shape[0], state["kv_heads"], -1, *x.shape[2:]).sum(2)

    back = lambda x: x.transpose(1, 2).contiguous().to(dt)  # noqa: E731
    out = (back(o * f), final, back(dq * f), back(shared(dk)), back(shared(dv)))
    return (*out, ds) if past is not None else out


def plain_experts(state):
    ids, w, n, top = state["ids"], state["weights"], state["experts"], state["top"]
    dt = state["x"].dtype
    flat = ids.reshape(-1)
    there = (flat >= 0) & (flat < n)
    key = torch.where(there, flat, n)
    order = torch.argsort(key, stable=True)
    slots = torch.empty_like(order)
    slots[order] = torch.arange(order.numel(), device=order.device)
    counts = (key[:, None] == torch.arange(n, device=key.device)[None, :]).sum(0)
    offsets = torch.cat([torch.zeros_like(counts[:1]), counts.cumsum(0)])
    kept = torch.arange(order.numel(), device=order.device) < offsets[-1]
    xs = torch.where(kept[:, None], state["x"][order // top], 0)
    rows = torch.where(there[:, None], state["ys"][slots].float(), 0.0).reshape(*ids.shape, -1)
    y = (rows * w[:, :, None]).sum(1).to(dt)
    order32 = torch.where(kept, order, -1).int()
    slots32 = torch.where(there, slots, -1).int().reshape(ids.shape)
    out = (order32, slots32, offsets.int(), xs, y)
    if state["op"] == "experts":
        return out
    dy = state["dy"].float()
    dw = (rows * dy[:, None, :]).sum(2)
    dys = dy[order // top] * w.reshape(-1)[order][:, None]
    dys = torch.where(kept[:, None], dys, 0.0).to(dt)
    dx = torch.where(there[:, None], state["dxs"][slots].float(), 0.0).reshape(*ids.shape, -1).sum(1).to(dt)
    return (*out, dys, dw, dx)


MASK32 = 0xFFFFFFFF


def random_words(seed, offset, blocks):
    """Philox4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as
    1, 2, 3", SC 2011): four 32-bit words for each counter (block, offset), keyed by seed."""
    i = torch.arange(blocks, device="cuda")
    c = [i & MASK32, i >> 32, torch.full_like(i, offset & MASK32), torch.full_like(i, (offset >> 32) & MASK32)]
    k0, k1 = seed & MASK32, (seed >> 32) & MASK32

    def product(m, x):      # high and low word of a 32 x 32 bit product, 64 bits being signed here
        low, high = (x & 0xFFFF) * m, (x >> 16) * m
        mid = high + (low >> 16)
        return (mid >> 16) & MASK32, ((mid & 0xFFFF) << 16) | (low & 0xFFFF)

    for _ in range(10):
        h0, l0 = product(0xD2511F53, c[0])
        h1, l1 = product(0xCD9E8D57, c[2])
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & MASK32, (k1 + 0xBB67AE85) & MASK32
    return torch.stack(c, 1)


def kept_elements(state):
    """The mask and the factor of what is kept: 16 bits of a word decide one element."""
    n = state["tokens"] * state["dim"]
    threshold = int(math.floor(state["p"] * 65536.0 + 0.5))
    words = random_words(state["seed"], state["offset"], -(-n // 8))
    halves = torch.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)[:n]
    return (halves >= threshold).reshape(state["tokens"], state["dim"]), 65536.0 / (65536 - threshold)


def plain_dropout(state):
    dt = state["x"].dtype
    keep, factor = kept_elements(state)
    out = torch.where(keep, state["x"].float() * factor, 0.0)
    if state["r"] is not None:
        out = out + state["r"].float()
    if state["op"] == "dropout":
        return out.to(dt)
    return out.to(dt), torch.where(keep, state["dy"].float() * factor, 0.0).to(dt)


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("mix"):
        return exact_mix(case, s)
    if case["op"].startswith("experts"):
        return exact_experts(case, s)
    keep, _ = kept_elements(s)
    threshold = round(s["p"] * 65536)
    x = s["x"].double().masked_fill(~keep, 0.0) / (1.0 - threshold / 65536)
    if s["r"] is not None:
        x = x + s["r"].double()
    if case["op"] == "dropout":
        return x
    return x, s["dy"].double().masked_fill(~keep, 0.0) / (1.0 - threshold / 65536)


def exact_mix(case, s):
    h, f = case["heads"], s["factor"]
    group = h // case["kv_heads"]
    wide = lambda x: x.double().repeat_interleave(group, dim=-2)  # noqa: E731
    gamma = torch.exp(s["log_decay"].double())[None, :, None, None]
    if case["op"] == "mix_step":
        new = gamma * s["past"].double() + torch.einsum("bhd,bhe->bhde", wide(s["k"]), wide(s["v"]))
        return torch.einsum("bhd,bhde->bhe", s["q"].double(), new) * f, new
    b, t = case["batch"], case["tokens"]
    tensors = {"q": s["q"].double(), "k": wide(s["k"]), "v": wide(s["v"])}
    if case["op"] == "mix_train":
        tensors["do"] = s["do"].double()
    alive = torch.ones(b, t, dtype=torch.bool, device="cuda")
    if s["lens"] is not None:
        alive = torch.arange(t, device="cuda")[None, :] < s["lens"][:, None]
        tensors = {n: x.masked_fill(~alive[:, :, None, None], 0.0) for n, x in tensors.items()}
    # time first; a token that is not there leaves the state as it is
    q, k, v = (tensors[n].transpose(0, 1).contiguous() for n in ("q", "k", "v"))
    gammas = torch.where(alive.T[:, :, None, None, None], gamma, 1.0)
    one = bool(alive.all())
    S = s["past"].double() if s["past"] is not None else torch.zeros(b, h, case["dim"], case["dim_v"], device="cuda",
                                                                     dtype=torch.float64)
    train = case["op"] == "mix_train"
    o = torch.empty(t, b, h, case["dim_v"], device="cuda", dtype=torch.float64)
    if train:
        do = tensors["do"].transpose(0, 1).contiguous()
        dq, dk, dv = (torch.empty_like(x) for x in (q, k, v))
    for i in range(t):
        S = torch.addcmul((gamma if one else gammas[i]) * S, k[i][..., :, None], v[i][..., None, :])
        torch.matmul(q[i][..., None, :], S, out=o[i].unsqueeze(-2))
        if train:
            torch.sum(S * do[i][..., None, :], -1, out=dq[i])
    o = torch.where(alive.T[:, :, None, None], o * f, 0.0).transpose(0, 1)
    if not train:
        return o, S
    final = S
    dS = s["d_final"].double() if s["d_final"] is not None else torch.zeros_like(S)
    for i in range(t - 1, -1, -1):
        dS = torch.addcmul(dS, q[i][..., :, None], do[i][..., None, :], value=f)
        torch.sum(dS * v[i][..., None, :], -1, out=dk[i])
        torch.sum(dS * k[i][..., :, None], -2, out=dv[i])
        dS = (gamma if one else gammas[i]) * dS
    mask = alive[:, :, None, None]
    dq, dk, dv = (torch.where(mask, x.transpose(0, 1), 0.0) for x in (dq * f, dk, dv))
    dk, dv = (x.unflatten(2, (case["kv_heads"], group)).sum(3) for x in (dk, dv))
    return (o, final, dq, dk, dv, dS) if s["past"] is not None else (o, final, dq, dk, dv)


def exact_experts(case, s):
    n, top, dim = case["experts"], case["top"], case["dim"]
    lists = [(e, p) for p, e in enumerate(s["ids"].reshape(-1).tolist()) if 0 <= e < n]
    lists.sort()                                     # by expert, then by place
    places = torch.tensor([p for _, p in lists], dtype=torch.long, device="cuda")
    m, total = len(lists), case["tokens"] * top
    token = places // top

    def whole(rows):     # rows behind the last expert's are zero
        return torch.cat([rows, rows.new_zeros(total - m, dim)])

    xs = whole(s["x"].double()[token])
    w = s["weights"].double().reshape(-1)[places]
    ys = s["ys"][:m].double()
    y = torch.zeros(case["tokens"], dim, dtype=torch.float64, device="cuda").index_add_(0, token, ys * w[:, None])
    out = (None, None, None, xs, y)
    if case["op"] == "experts":
        return out
    dy = s["dy"].double()[token]
    dw = torch.zeros(total, dtype=torch.float64, device="cuda")
    dw[places] = (dy * ys).sum(1)
    dx = torch.zeros_like(y).index_add_(0, token, s["dxs"][:m].double())
    return (*out, whole(dy * w[:, None]), dw.reshape(case["tokens"], top), dx)
