"""The training and evaluation operators around the linear layers of a
GPT-2-type transformer: what is timed, their plain forms and their values in
64 bits.

  attention     attention's backward pass: dqkv from qkv, the forward's output
                and log-sum-exp, and the output's gradient
  distill       distillation of the logits towards a teacher's top logits: the
                loss ("forward"), its gradient ("backward"), and both in one
                pass over the logits ("both")
  logprobs      log probabilities of given tokens, with the entropy of the
                distribution and its top alternatives
"""
import math

import torch

own = False

HEAD = 64  # width of an attention head
BF16, FP32 = "bf16", "fp32"


def _dtype(name):
    return torch.bfloat16 if name == BF16 else torch.float32


def listed():
    return [
        # GPT-2's batched training step: 64 sequences of 128 tokens
        {"name": "attention_b64_t128_h12", "op": "attention", "B": 64, "T": 128, "H": 12, "causal": True},
        # long-context training, few sequences
        {"name": "attention_b2_t4096_h12", "op": "attention", "B": 2, "T": 4096, "H": 12, "causal": True},
        # an encoder over sequences whose length fills no tile
        {"name": "attention_b3_t777_h5_full", "op": "attention", "B": 3, "T": 777, "H": 5, "causal": False},
        # one short prompt: latency
        {"name": "attention_b1_t19_h12", "op": "attention", "B": 1, "T": 19, "H": 12, "causal": True},
        # the batched LM head's logits, trained against 32 teacher entries a token
        {"name": "distill_both_r8192_v50257", "op": "distill", "form": "both", "R": 8192, "V": 50257, "ld": 50257,
         "K": 32, "dtype": BF16, "teacher": FP32, "ids64": False, "tau": 2.0},
        # the same head with its rows padded for the backward products, gradient given from outside
        {"name": "distill_backward_r2048_v50257_padded", "op": "distill", "form": "backward", "R": 2048, "V": 50257,
         "ld": 50304, "K": 64, "dtype": BF16, "teacher": BF16, "ids64": True, "tau": 1.0},
        # validation loss on fp32 logits of another vocabulary
        {"name": "distill_forward_r777_v32003_fp32", "op": "distill", "form": "forward", "R": 777, "V": 32003,
         "ld": 32003, "K": 100, "dtype": FP32, "teacher": FP32, "ids64": True, "tau": 1.5},
        # one short sequence: latency
        {"name": "distill_both_r9_v50257", "op": "distill", "form": "both", "R": 9, "V": 50257, "ld": 50257, "K": 16,
         "dtype": BF16, "teacher": FP32, "ids64": False, "tau": 1.0},
        # serving: the token just sampled and its alternatives
        {"name": "logprobs_r1_v50257", "op": "logprobs", "R": 1, "V": 50257, "ld": 50257, "top": 20, "dtype": BF16,
         "ids64": True, "tau": 1.0},
        # scoring a batch of sequences
        {"name": "logprobs_r8192_v50257", "op": "logprobs", "R": 8192, "V": 50257, "ld": 50257, "top": 8,
         "dtype": BF16, "ids64": True, "tau": 1.0},
        # fp32 logits of a large vocabulary, at a sampling temperature
        {"name": "logprobs_r301_v128001_fp32", "op": "logprobs", "R": 301, "V": 128001, "ld": 128001, "top": 32,
         "dtype": FP32, "ids64": False, "tau": 0.7},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "distill", "logprobs"])
    if op == "attention":
        T = _log_int(rng, 1, 4096)
        H = rng.randint(1, 16)
        causal = rng.random() < 0.7
        # the largest listed case: 24 heads of 4096 causal tokens, 98304 head rows
        heads = min(128 * H, 64 * 128 * 12 // T, 24 * 4096 * 4097 // (T * (T + 1) * (1 if causal else 2)))
        H = min(H, heads)
        return {"op": op, "B": _log_int(rng, 1, heads // H), "T": T, "H": H, "causal": causal}
    dtype = rng.choice([BF16, BF16, FP32])
    V = _log_int(rng, 300, 131072)
    pad = rng.choice([0, 0, 7, 47, -V % 64])
    # the largest listed case holds 8192 * 50257 bf16 logits
    most = 8192 * 50257 * (2 if dtype == BF16 else 1) // (2 * (V + pad))
    R = _log_int(rng, 1, min(8192, most))
    case = {"op": op, "R": R, "V": V, "ld": V + pad, "dtype": dtype, "ids64": rng.random() < 0.5,
            "tau": rng.choice([1.0, 1.0, 0.7, 2.0, 3.5])}
    if op == "logprobs":
        case["top"] = rng.randint(1, 32)
    else:
        case.update(form=rng.choice(["both", "both", "forward", "backward"]), K=_log_int(rng, 1, 128),
                    teacher=rng.choice([BF16, FP32]))
    return case


# ------------------------------------------------------------------ inputs

def _heads(x, case):
    """(B*T) x C to B x H x T x 64."""
    return x.reshape(case["B"], case["T"], case["H"], HEAD).transpose(1, 2)


def _prepare_attention(case, g):
    B, T, H = case["B"], case["T"], case["H"]
    C = H * HEAD
    # scaled scores with a spread of about 2: some rows flat, some peaked
    qkv = torch.randn(B * T, 3 * C, device="cuda", generator=g)
    qkv[:, :2 * C] *= 1.4
    qkv = qkv.bfloat16()
    out = torch.empty(B * T, C, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(B, H, T, device="cuda")
    q, k, v = (_heads(qkv[:, i * C:(i + 1) * C], case) for i in range(3))
    o = _heads(out, case)
    for b in range(B):  # the forward pass, one sequence at a time
        s = q[b].float() @ k[b].float().transpose(-1, -2) * HEAD ** -0.5
        if case["causal"]:
            s.masked_fill_(torch.ones(T, T, dtype=torch.bool, device="cuda").triu_(1), -math.inf)
        lse[b] = torch.logsumexp(s, -1)
        o[b] = (torch.exp(s - lse[b][..., None]) @ v[b].float()).bfloat16()
    dout = (torch.randn(B * T, C, device="cuda", generator=g) * 0.01).bfloat16()
    return {"qkv": qkv, "out": out, "lse": lse, "dout": dout}


def _logits(case, g):
    """R x V logits (rows ld apart) with the spread of a language model's."""
    R, V = case["R"], case["V"]
    buf = torch.randn(R, case["ld"], device="cuda", generator=g, dtype=_dtype(case["dtype"]))
    buf *= 2.5
    z = buf[:, :V]
    peak = torch.randint(0, V, (R, 4), device="cuda", generator=g)
    z.scatter_add_(1, peak, torch.full((R, 4), 9.0, device="cuda", dtype=z.dtype))
    return z, peak


def _prepare_distill(case, g):
    R, V = case["R"], case["V"]
    K = min(case["K"], V)
    z, _ = _logits(case, g)
    # K distinct tokens a row, most likely first; padded entries have id -1
    base = torch.randint(0, V, (R, 1), device="cuda", generator=g)
    step = torch.randint(1, V // K + 1, (R, 1), device="cuda", generator=g)
    ids = (base + step * torch.arange(K, device="cuda")) % V
    t = 12.0 + 2.0 * torch.randn(R, K, device="cuda", generator=g)
    t = t.sort(dim=1, descending=True).values
    z.scatter_add_(1, ids, (t - 8.0).to(z.dtype))
    held = torch.randint(1, K + 1, (R, 1), device="cuda", generator=g)
    held = torch.where(torch.rand(R, 1, device="cuda", generator=g) < 0.8, K, held)
    if R > 4:
        held[R // 2] = 0  # a padding position: no entry at all
    ids = torch.where(torch.arange(K, device="cuda") < held, ids, -1)
    state = {"logits": z, "ids": ids if case["ids64"] else ids.int(), "teacher": t.to(_dtype(case["teacher"]))}
    weight = torch.rand(R, device="cuda", generator=g) / R
    if R > 4:
        weight[R // 3] = 0.0  # a token that the loss leaves out
    if case["form"] == "backward":
        state["lse"] = torch.cat([torch.logsumexp(c.float() / case["tau"], -1) for c in z.split(1024)])
    state["weight"] = weight
    return state


def _prepare_logprobs(case, g):
    R, V = case["R"], case["V"]
    z, peak = _logits(case, g)
    z[::7, V // 3:V // 2] = -math.inf  # constrained decoding: part of the vocabulary is banned
    tokens = torch.where(torch.rand(R, device="cuda", generator=g) < 0.7, peak[:, 0],
                         torch.randint(0, V, (R,), device="cuda", generator=g))
    if R > 4:
        tokens[R // 2] = -1  # no token here
    return {"logits": z, "tokens": tokens if case["ids64"] else tokens.int()}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    make = {"attention": _prepare_attention, "distill": _prepare_distill, "logprobs": _prepare_logprobs}[case["op"]]
    state = make(case, g)
    state["case"] = case
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return {"attention": _plain_attention, "distill": _plain_distill, "logprobs": _plain_logprobs}[case["op"]](case, state)


def _own(case, s):
    import transformer_linear_layer_gb300 as tll

    if case["op"] == "attention":
        return tll.attention_backward(s["qkv"], s["out"], s["lse"], s["dout"], case["B"], case["T"], case["H"],
                                      causal=case["causal"])
    if case["op"] == "logprobs":
        r = tll.token_logprobs(s["logits"], s["tokens"], top=min(case["top"], case["V"]), temperature=case["tau"])
        return r.logprob, r.entropy, r.top_logprob, r.top_ids
    if case["form"] == "forward":
        return tll.distill_forward(s["logits"], s["ids"], s["teacher"], temperature=case["tau"])
    if case["form"] == "backward":
        return tll.distill_backward(s["logits"], s["ids"], s["teacher"], s["lse"], s["weight"],
                                    temperature=case["tau"])
    return tll.distill_forward_backward(s["logits"], s["ids"], s["teacher"], weight=s["weight"],
                                        temperature=case["tau"])


def _plain_attention(case, s):
    T, C = case["T"], case["H"] * HEAD
    scale = HEAD ** -0.5
    x = s["qkv"].float()
    q, k, v = (_heads(x[:, i * C:(i + 1) * C], case) for i in range(3))
    do = _heads(s["dout"].float(), case)
    delta = (do * _heads(s["out"].float(), case)).sum(-1, keepdim=True)
    p = torch.exp(q @ k.transpose(-1, -2) * scale - s["lse"][..., None])
    if case["causal"]:
        pos = torch.arange(T, device=p.device)
        p = torch.where(pos[None, :] <= pos[:, None], p, 0.0)
    dv = p.transpose(-1, -2) @ do
    ds = p * (do @ v.transpose(-1, -2) - delta) * scale
    grads = [ds @ k, ds.transpose(-1, -2) @ q, dv]
    return torch.cat([d.transpose(1, 2).reshape(-1, C) for d in grads], 1).bfloat16()


def _plain_softmax(z, tau):
    z = z.float() / tau
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m)
    return z, m, e, e.sum(-1, keepdim=True)


def _plain_teacher(ids, t, tau):
    """Probabilities and log probabilities over a row's entries, 0 at padding."""
    held = ids >= 0
    t = torch.where(held, t.float() / tau, -math.inf)
    m = torch.where(held.any(-1, keepdim=True), t.amax(-1, keepdim=True), 0.0)
    e = torch.exp(t - m)
    total = e.sum(-1, keepdim=True).clamp_min(1e-30)
    return held, e / total, torch.where(held, t - m - torch.log(total), 0.0)


def _plain_distill(case, s):
    tau = case["tau"]
    z, ids = s["logits"], s["ids"].long()
    held, q, logq = _plain_teacher(ids, s["teacher"], tau)
    at = ids.clamp_min(0)
    if case["form"] == "backward":
        p = torch.exp(z.float() / tau - s["lse"][:, None])
    else:
        zt, m, e, total = _plain_softmax(z, tau)
        lse = m + torch.log(total)
        logp = zt.gather(1, at) - lse
        loss = tau * tau * torch.where(held, q * (logq - logp), 0.0).sum(-1)
        if case["form"] == "forward":
            return loss, lse[:, 0]
        p = e / total
    # a row without teacher entries has no loss and no gradient
    g = s["weight"][:, None] * tau * held.any(-1, keepdim=True)
    d = (g * p).scatter_add_(1, at, -g * q).to(z.dtype)
    return d if case["form"] == "backward" else (loss, d)


def _plain_logprobs(case, s):
    z, tokens = s["logits"], s["tokens"].long()
    zt, m, e, total = _plain_softmax(z, case["tau"])
    lse = m + torch.log(total)
    logprob = torch.where(tokens >= 0, (zt.gather(1, tokens.clamp_min(0)[:, None]) - lse)[:, 0], 0.0)
    x = zt - m
    entropy = torch.log(total[:, 0]) - torch.where(e > 0, e * x, 0.0).sum(-1) / total[:, 0]
    # unique whole-number keys: the value's order, then the lowest index
    top = []
    V = z.shape[1]
    back = torch.arange(V - 1, -1, -1, device=z.device)
    for rows in z.split(1024):
        bits = (rows.float() + 0.0).view(torch.int32)
        key = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF).long() * (1 << 20) + back
        top.append(V - 1 - torch.topk(key, min(case["top"], V), dim=-1).values % (1 << 20))
    ids = torch.cat(top)
    return logprob, entropy, zt.gather(1, ids) - lse, ids.int()


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "distill": _exact_distill, "logprobs": _exact_logprobs}[case["op"]](case, s)


def _exact_attention(case, s):
    B, T, H = case["B"], case["T"], case["H"]
    C = H * HEAD
    dqkv = torch.zeros(B * T, 3 * C, dtype=torch.float64, device="cuda")
    for b in range(B):
        rows = slice(b * T, (b + 1) * T)
        for h in range(H):
            col = h * HEAD
            q, k, v = (s["qkv"][rows, i * C + col:i * C + col + HEAD].double() for i in range(3))
            o, do = s["out"][rows, col:col + HEAD].double(), s["dout"][rows, col:col + HEAD].double()
            prob = (torch.mm(q, k.T) / math.sqrt(HEAD)).sub_(s["lse"][b, h].double().unsqueeze(1)).exp_()
            if case["causal"]:
                prob.tril_()
            dscore = torch.mm(do, v.T).sub_((o * do).sum(1, keepdim=True)).mul_(prob).div_(math.sqrt(HEAD))
            dqkv[rows, col:col + HEAD] = torch.mm(dscore, k)
            dqkv[rows, C + col:C + col + HEAD] = torch.mm(dscore.T, q)
            dqkv[rows, 2 * C + col:2 * C + col + HEAD] = torch.mm(prob.T, do)
    return dqkv


def _exact_distill(case, s):
    tau, form = case["tau"], case["form"]
    losses, lses, grads = [], [], []
    for r0 in range(0, case["R"], 512):
        rows = slice(r0, r0 + 512)
        z = s["logits"][rows].double() / tau
        ids = s["ids"][rows].long()
        lse = s["lse"][rows].double() if form == "backward" else torch.logsumexp(z, 1)
        teacher = torch.zeros_like(z)
        loss = torch.zeros(z.shape[0], dtype=torch.float64, device="cuda")
        some = torch.zeros(z.shape[0], dtype=torch.float64, device="cuda")
        weights = torch.full(ids.shape, -math.inf, dtype=torch.float64, device="cuda")
        weights[ids >= 0] = s["teacher"][rows][ids >= 0].double() / tau
        norm = torch.logsumexp(weights, 1)
        for j in range(ids.shape[1]):
            n = torch.nonzero(ids[:, j] >= 0)[:, 0]
            logq = weights[n, j] - norm[n]
            teacher[n, ids[n, j]] += logq.exp()
            loss[n] += logq.exp() * (logq - z[n, ids[n, j]] + lse[n])
            some[n] = 1.0
        losses.append(tau ** 2 * loss)
        lses.append(lse)
        if form != "forward":
            scale = some * s["weight"][rows].double() * tau
            grads.append(z.sub_(lse[:, None]).exp_().sub_(teacher).mul_(scale[:, None]))
    if form == "forward":
        return torch.cat(losses), torch.cat(lses)
    return torch.cat(grads) if form == "backward" else (torch.cat(losses), torch.cat(grads))


def _exact_logprobs(case, s):
    k = min(case["top"], case["V"])
    outs = []
    for r0 in range(0, case["R"], 512):
        z = s["logits"][r0:r0 + 512].double()
        t = s["tokens"][r0:r0 + 512].long()
        order = torch.sort(z, dim=1, descending=True, stable=True)
        logp = torch.log_softmax(z / case["tau"], 1)
        token = torch.zeros(t.shape, dtype=torch.float64, device="cuda")
        n = torch.nonzero(t >= 0)[:, 0]
        token[n] = logp[n, t[n]]
        entropy = -torch.nan_to_num(logp.exp() * logp, nan=0.0).sum(1)
        ids = order.indices[:, :k]
        outs.append((token, entropy, logp.gather(1, ids), ids.int()))
    return tuple(torch.cat(x) for x in zip(*outs))


# ------------------------------------------------------------------ work

def work(case):
    if case["op"] == "attention":
        B, T, H = case["B"], case["T"], case["H"]
        pairs = T * (T + 1) // 2 if case["causal"] else T * T
        # qkv, out, dout and lse in, dqkv out; five products over the visible pairs
        return {"bytes": B * T * H * HEAD * 2 * (3 + 1 + 1 + 3) + 4 * B * H * T, "flops": 10 * HEAD * pairs * B * H}
    R, V = case["R"], case["V"]
    e = 2 if case["dtype"] == BF16 else 4
    i = 8 if case["ids64"] else 4
    if case["op"] == "logprobs":
        return {"bytes": R * V * e + R * (i + 8 + 8 * min(case["top"], V)), "flops": 5 * R * V}
    K = min(case["K"], V)
    entries = R * K * (i + (2 if case["teacher"] == BF16 else 4))
    passes = 1 if case["form"] == "forward" else 2
    return {"bytes": passes * R * V * e + entries + 8 * R, "flops": (4 if passes == 1 else 7) * R * V}
