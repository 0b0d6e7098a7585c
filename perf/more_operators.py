"""The operators that serve a transformer block token by token, next to the
rotary positions that it is trained with: what is timed, their plain forms and
their values in 64 bits.

  rotary        rotary positions of query and key heads ("forward") and the
                gradient through them ("backward")
  append        new keys and values into a paged cache, keys and queries
                rotated on the way
  attention     attention of new tokens (single ones, chunks, whole prompts, or
                the queries of a cross attention) over a paged cache
"""
import math

import torch

own = False

BF16, FP32 = "bf16", "fp32"


def _dtype(name):
    return torch.bfloat16 if name == BF16 else torch.float32


def listed():
    return [
        # GPT-2's batched training step, q and k heads of the qkv projection's output
        {"name": "rotary_b64_t128_h24", "op": "rotary", "form": "forward", "B": 64, "T": 128, "heads": 24, "D": 64,
         "rot": 64, "ld": 2304, "interleaved": False, "dtype": BF16, "wide": True, "far": 0, "base": 10000.0,
         "scaling": "none", "factor": 1.0, "length": 0},
        # fine-tuning for a longer context: half of each head rotates, neighbours paired, scaled frequencies
        {"name": "rotary_gradient_b3_t777_far_fp32", "op": "rotary", "form": "backward", "B": 3, "T": 777, "heads": 10,
         "D": 128, "rot": 64, "ld": 1280, "interleaved": True, "dtype": FP32, "wide": False, "far": 100000,
         "base": 500000.0, "scaling": "yarn", "factor": 16.0, "length": 8192},
        # one token of one sequence: latency
        {"name": "rotary_b1_t1_h24", "op": "rotary", "form": "forward", "B": 1, "T": 1, "heads": 24, "D": 64, "rot": 64,
         "ld": 2304, "interleaved": False, "dtype": BF16, "wide": True, "far": 500, "base": 10000.0,
         "scaling": "none", "factor": 1.0, "length": 0},
        # serving, one new token for each of 64 sequences
        {"name": "append_b64_single_h12", "op": "append", "B": 64, "H": 12, "Hkv": 12, "D": 64, "page": 16, "new_lo": 1,
         "new_hi": 1, "mixed": False, "old_lo": 100, "old_hi": 4000, "order": "heads", "rot": 64,
         "interleaved": False, "base": 10000.0, "scaling": "none", "factor": 1.0, "length": 0},
        # a batch of prompts, shared key heads
        {"name": "append_b8_prompts_h32_kv8", "op": "append", "B": 8, "H": 32, "Hkv": 8, "D": 128, "page": 64,
         "new_lo": 400, "new_hi": 1024, "mixed": False, "old_lo": 0, "old_hi": 2000, "order": "tokens", "rot": 128,
         "interleaved": True, "base": 500000.0, "scaling": "linear", "factor": 4.0, "length": 0},
        # one user, one token: latency
        {"name": "attention_b1_single_kv1000_h12", "op": "attention", "B": 1, "H": 12, "Hkv": 12, "D": 64, "page": 16,
         "new_lo": 1, "new_hi": 1, "mixed": False, "old_lo": 999, "old_hi": 999, "order": "heads", "causal": True,
         "lse": False},
        # a served batch of single tokens, ragged contexts, shared key heads
        {"name": "attention_b64_single_h32_kv8", "op": "attention", "B": 64, "H": 32, "Hkv": 8, "D": 128, "page": 16,
         "new_lo": 1, "new_hi": 1, "mixed": False, "old_lo": 100, "old_hi": 8000, "order": "heads", "causal": True,
         "lse": False},
        # two very long contexts, few key heads: the keys have to be split
        {"name": "attention_b2_single_kv131072_h16_kv2", "op": "attention", "B": 2, "H": 16, "Hkv": 2, "D": 128,
         "page": 64, "new_lo": 1, "new_hi": 1, "mixed": False, "old_lo": 131071, "old_hi": 131071, "order": "tokens",
         "causal": True, "lse": True},
        # prompts taken in chunks, GPT-2's heads
        {"name": "attention_b4_chunk512_kv8704_h12", "op": "attention", "B": 4, "H": 12, "Hkv": 12, "D": 64, "page": 16,
         "new_lo": 512, "new_hi": 512, "mixed": False, "old_lo": 8192, "old_hi": 8192, "order": "heads",
         "causal": True, "lse": False},
        # whole prompts into an empty cache
        {"name": "attention_b2_prompt4096_h16_kv2", "op": "attention", "B": 2, "H": 16, "Hkv": 2, "D": 128, "page": 128,
         "new_lo": 4096, "new_hi": 4096, "mixed": False, "old_lo": 0, "old_hi": 0, "order": "heads", "causal": True,
         "lse": False},
        # a decoder's queries over an encoder's states of another length
        {"name": "attention_b8_cross_kv1500_h12", "op": "attention", "B": 8, "H": 12, "Hkv": 12, "D": 64, "page": 32,
         "new_lo": 77, "new_hi": 101, "mixed": False, "old_lo": 1500, "old_hi": 1500, "order": "heads",
         "causal": False, "lse": False},
        # prompts that join a batch of running sequences
        {"name": "attention_b33_mixed_h20_kv4", "op": "attention", "B": 33, "H": 20, "Hkv": 4, "D": 64, "page": 8,
         "new_lo": 200, "new_hi": 301, "mixed": True, "old_lo": 0, "old_hi": 3001, "order": "tokens", "causal": True,
         "lse": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_rotation(rng, D):
    scaling = rng.choice(["none", "none", "linear", "ntk", "yarn"])
    rot = rng.choice([D, D, D // 2, D // 4, 2 * rng.randint(2, D // 2)])
    return {"rot": rot, "interleaved": rng.random() < 0.5, "base": rng.choice([10000.0, 500000.0]), "scaling": scaling,
            "factor": 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 16.0]), "length": rng.choice([2048, 8192])}


def draw(rng):
    op = rng.choice(["rotary", "append", "attention", "attention"])
    if op == "rotary":
        dtype = rng.choice([BF16, FP32])
        D = rng.choice([32, 64, 64, 80, 128, 128, 256])
        heads = rng.randint(1, 48)
        # the largest listed case rotates 8192 x 24 heads of 64 in bf16
        most = 8192 * 24 * 64 * 2 // (heads * D * (2 if dtype == BF16 else 4))
        N = _log_int(rng, 1, min(8192, max(1, most)))
        B = max(1, min(N, rng.choice([1, 2, 8, 64])))
        return {"op": op, "form": rng.choice(["forward", "backward"]), "B": B, "T": max(1, N // B), "heads": heads, "D": D,
                "ld": heads * D + rng.choice([0, 0, 8, D]), "dtype": dtype, "wide": rng.random() < 0.5,
                "far": rng.choice([0, 0, 5000, 1000000]), **_draw_rotation(rng, D)}
    D = rng.choice([64, 64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8, 12])
    G = rng.choice([1, 1, 2, 3, 4, 5, 8])
    B = _log_int(rng, 1, 64)
    case = {"op": op, "B": B, "H": G * Hkv, "Hkv": Hkv, "D": D, "page": rng.choice([8, 16, 16, 32, 64, 128, 256]),
            "mixed": False, "order": rng.choice(["heads", "tokens"])}
    if op == "append":
        # the largest listed case holds about 5700 rows of 48 heads of 128
        rows = min(4096, 5000 * 48 * 128 // ((G + 2) * Hkv * D))
        hi = _log_int(rng, 1, max(1, rows // B))
        case.update(new_lo=max(1, hi // 2), new_hi=hi, old_lo=0, old_hi=_log_int(rng, 1, 60000 // B),
                    **_draw_rotation(rng, D))
        return case
    kind = rng.choice(["single", "single", "chunk", "prompt", "cross", "mixed"])
    # the largest listed cases: 260000 cached tokens of 8 heads of 128; 17 million visible pairs of 16 heads of 128
    cached = min(200000, 250000 * 8 * 128 // (Hkv * D))
    pairs = 16000000 * 16 * 128 // (G * Hkv * D)
    old = _log_int(rng, 1, cached // B)
    case.update(causal=kind != "cross", lse=rng.random() < 0.5, old_lo=rng.choice([old, old // 2, 0]), old_hi=old,
                new_lo=1, new_hi=1)
    if kind == "cross":
        case["old_lo"] = max(1, case["old_lo"])
    if kind == "single":
        case["new_lo"] = case["new_hi"] = 1 if rng.random() < 0.8 else rng.randint(1, 4)
    else:
        hi = _log_int(rng, 2, 4096)
        if kind == "prompt":
            case["old_lo"] = case["old_hi"] = 0
            hi = min(hi, int(math.sqrt(2.0 * pairs / B)) or 1)
        else:
            hi = min(hi, pairs // (B * (old + hi)) or 1)
        hi = max(1, min(hi, cached // B))
        case.update(new_lo=max(1, hi * 2 // 3), new_hi=hi, mixed=kind == "mixed")
    return case


# ------------------------------------------------------------------ inputs

def _spread(lo, hi, step, i):
    return lo + int((i * step + 0.37) % 1.0 * (hi - lo + 1))


def _lengths(case):
    """New tokens and tokens held (the new ones included, where they attend to
    themselves) of each sequence: spread over the case's ranges."""
    new, held = [], []
    for b in range(case["B"]):
        n = _spread(case["new_lo"], case["new_hi"], 0.7548776662466927, b)
        if case["mixed"] and b % 4:
            n = 1
        old = _spread(case["old_lo"], case["old_hi"], 0.6180339887498949, b)
        new.append(n)
        held.append(old + n if case.get("causal", True) else old)
    return new, held


def _frequencies(case):
    """Radians per position of each pair, and the factor on the rotated part."""
    rot, base, s = case["rot"], case["base"], case["factor"]
    if case["scaling"] == "ntk" and rot > 2:
        base *= s ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        f = [x / s for x in f]
    if case["scaling"] == "yarn":
        # pairs that turn at most once in the trained length are stretched, those
        # that turn 32 times or more are kept, a ramp between
        turns = [case["length"] * x / (2 * math.pi) for x in f]
        keep = [min(1.0, max(0.0, (t - 1.0) / 31.0)) for t in turns]
        return [x * k + x / s * (1 - k) for x, k in zip(f, keep)], 0.1 * math.log(s) + 1.0
    return f, 1.0


def _rotary(case):
    import transformer_linear_layer_gb300 as tll

    scaling = None if case["scaling"] == "none" else case["scaling"]
    return tll.Rotary(case["rot"], base=case["base"], interleaved=case["interleaved"], scaling=scaling,
                      factor=case["factor"], original_length=case["length"] or None, device="cuda")


def _prepare_rotary(case, g):
    B, T = case["B"], case["T"]
    N = B * T
    dt = _dtype(case["dtype"])
    x = torch.randn(N, case["ld"], device="cuda", generator=g).to(dt)
    heads = x[:, :case["heads"] * case["D"]].unflatten(1, (case["heads"], case["D"]))
    start = torch.randint(0, case["far"] + 1, (B, 1), device="cuda", generator=g)
    positions = (start + torch.arange(T, device="cuda")).reshape(-1)
    return {"x": heads, "positions": positions if case["wide"] else positions.int()}


def _pages(case, g):
    """A cache of scattered pages, the sequences' page tables and lengths."""
    new, held = _lengths(case)
    B, page, Hkv, D = case["B"], case["page"], case["Hkv"], case["D"]
    need = [-(-h // page) for h in held]
    total = sum(need) + 3
    shape = (total, Hkv, page, D) if case["order"] == "heads" else (total, page, Hkv, D)
    k, v = (torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16) for _ in range(2))
    if case["order"] == "tokens":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    ids = torch.randperm(total, device="cuda", generator=g).int()
    table = torch.full((B, max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    return {"k": k, "v": v, "table": table, "new": new, "held": held, "N": starts[-1], "rows": starts,
            "q_start": torch.tensor(starts, dtype=torch.int32, device="cuda"),
            "kv_len": torch.tensor(held, dtype=torch.int32, device="cuda")}


def _serving(s):
    """The framework's handles of the cache and of the batch."""
    import transformer_linear_layer_gb300 as tll

    s["cache"] = tll.KVCache(s["k"], s["v"])
    s["batch"] = tll.KVBatch(s["q_start"], s["kv_len"], s["table"])


def _prepare_append(case, g):
    s = _pages(case, g)
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    qkv = torch.randn(s["N"], (H + 2 * Hkv) * D, device="cuda", generator=g).bfloat16().unflatten(1, (-1, D))
    s["q"], s["new_k"], s["new_v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    if own:
        _serving(s)
    return s


def _prepare_attention(case, g):
    s = _pages(case, g)
    # scaled scores with a spread of about 2: some rows flat, some peaked
    s["q"] = (2.0 * torch.randn(s["N"], case["H"], case["D"], device="cuda", generator=g)).bfloat16()
    s["max_new"] = max(s["new"])
    if own:
        _serving(s)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    make = {"rotary": _prepare_rotary, "append": _prepare_append, "attention": _prepare_attention}[case["op"]]
    state = make(case, g)
    state["case"] = case
    if case["op"] != "attention":
        f, state["factor"] = _frequencies(case)
        state["frequencies"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        if own:
            state["rotary"] = _rotary(case)
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return {"rotary": _plain_rotary, "append": _plain_append, "attention": _plain_attention}[case["op"]](case, state)


def _own(case, s):
    import transformer_linear_layer_gb300 as tll

    if case["op"] == "rotary":
        call = tll.rotary_forward if case["form"] == "forward" else tll.rotary_backward
        return call(s["x"], s["positions"], s["rotary"])
    if case["op"] == "append":
        q = tll.cache_append(s["q"], s["new_k"], s["new_v"], s["cache"], s["batch"], rotary=s["rotary"])
        return q, s["k"], s["v"]
    return tll.paged_attention(s["q"], s["cache"], s["batch"], causal=case["causal"], max_new=s["max_new"],
                               with_lse=case["lse"])


def _turned(x, positions, s, back=False):
    """x (rows x heads x D) rotated, in fp32; angles in 64 bits."""
    case = s["case"]
    rot = case["rot"]
    angle = positions.double()[:, None] * s["frequencies"]
    cos = (torch.cos(angle) * s["factor"]).float()[:, None]
    sin = (torch.sin(angle) * s["factor"]).float()[:, None]
    if back:
        sin = -sin
    y = x.float()
    if case["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, y[..., rot:]], -1)


def _plain_rotary(case, s):
    return _turned(s["x"], s["positions"], s, case["form"] == "backward").to(s["x"].dtype)


def _plain_slots(case, s):
    """Sequence and position of each row, and the page and slot that take it."""
    n = torch.arange(s["N"], device="cuda")
    b = torch.searchsorted(s["q_start"][1:].contiguous().long(), n, right=True)
    position = (s["kv_len"][b] - s["q_start"][b + 1]).long() + n
    page = s["table"][b, position // case["page"]].long()
    return position, page, position % case["page"]


def _plain_append(case, s):
    position, page, slot = _plain_slots(case, s)
    s["k"][page, :, slot] = _turned(s["new_k"], position, s).bfloat16()
    s["v"][page, :, slot] = s["new_v"]
    return _turned(s["q"], position, s).bfloat16(), s["k"], s["v"]


def _plain_attention(case, s):
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    G = H // Hkv
    outs, lses = [], []
    for b in range(case["B"]):
        n, held = s["new"][b], s["held"][b]
        pages = s["table"][b, :-(-held // case["page"])].long()
        k, v = (c[pages].transpose(0, 1).flatten(1, 2)[:, :held].float() for c in (s["k"], s["v"]))
        q = s["q"][s["rows"][b]:s["rows"][b + 1]].float().unflatten(1, (Hkv, G)).permute(1, 2, 0, 3).flatten(1, 2)
        x = q @ k.transpose(-1, -2) * D ** -0.5
        if case["causal"]:
            position = torch.arange(held - n, held, device=x.device).repeat(G)
            x = torch.where(torch.arange(held, device=x.device) <= position[:, None], x, -math.inf)
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - m)
        total = e.sum(-1, keepdim=True)
        o = e @ v / total
        outs.append(o.unflatten(1, (G, n)).permute(2, 0, 1, 3).flatten(1, 2).bfloat16())
        if case["lse"]:
            lses.append((m + torch.log(total)).unflatten(1, (G, n)).squeeze(-1).permute(2, 0, 1).flatten(1, 2))
    return (torch.cat(outs), torch.cat(lses)) if case["lse"] else torch.cat(outs)


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "append": _exact_append, "attention": _exact_attention}[case["op"]](case, s)


def _exact_turn(x, positions, s, sign=1.0):
    """Each pair as a complex number times factor * e^(i theta)."""
    case = s["case"]
    rot = case["rot"]
    y = x.double().clone()
    theta = torch.outer(positions.double(), s["frequencies"]) * sign
    turn = torch.polar(torch.full_like(theta, s["factor"]), theta).unsqueeze(1)
    if case["interleaved"]:
        first, second = slice(0, rot, 2), slice(1, rot, 2)
    else:
        first, second = slice(0, rot // 2), slice(rot // 2, rot)
    z = torch.complex(y[:, :, first].contiguous(), y[:, :, second].contiguous()) * turn
    y[:, :, first], y[:, :, second] = z.real, z.imag
    return y


def _exact_rotary(case, s):
    return _exact_turn(s["x"], s["positions"], s, 1.0 if case["form"] == "forward" else -1.0)


def _exact_append(case, s):
    k, v = s["k"].double(), s["v"].double()
    q = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    table = s["table"].tolist()
    for b, (n, held) in enumerate(zip(s["new"], s["held"])):
        rows = slice(s["rows"][b], s["rows"][b + 1])
        places = range(held - n, held)
        position = torch.tensor(list(places), device="cuda")
        page = torch.tensor([table[b][p // case["page"]] for p in places], device="cuda")
        slot = torch.tensor([p % case["page"] for p in places], device="cuda")
        q[rows] = _exact_turn(s["q"][rows], position, s)
        k[page, :, slot] = _exact_turn(s["new_k"][rows], position, s)
        v[page, :, slot] = s["new_v"][rows].double()
    return q, k, v


def _exact_attention(case, s):
    G = case["H"] // case["Hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, held) in enumerate(zip(s["new"], s["held"])):
        place = torch.arange(held, device="cuda")
        page, slot = s["table"][b].long()[place // case["page"]], place % case["page"]
        hidden = place[None, :] > (place.new_tensor(range(held - n, held))[:, None] if case["causal"] else held)
        for g in range(case["Hkv"]):
            k, v = s["k"][page, g, slot].double(), s["v"][page, g, slot].double()
            for h in range(g * G, g * G + G):
                score = torch.mm(s["q"][at:at + n, h].double(), k.T).div_(math.sqrt(case["D"]))
                score.masked_fill_(hidden, -math.inf)
                total = torch.logsumexp(score, 1)
                lse[at:at + n, h] = total
                out[at:at + n, h] = torch.mm(score.sub_(total[:, None]).exp_(), v)
        at += n
    return (out, lse) if case["lse"] else out


# ------------------------------------------------------------------ work

def work(case):
    if case["op"] == "rotary":
        N = case["B"] * case["T"]
        e = 2 if case["dtype"] == BF16 else 4
        return {"bytes": 2 * N * case["heads"] * case["D"] * e + N * (8 if case["wide"] else 4),
                "flops": 3 * N * case["heads"] * case["rot"]}
    new, held = _lengths(case)
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    if case["op"] == "append":
        # q, k and v in; q, and k and v in their pages, out
        return {"bytes": 4 * sum(new) * (H + 2 * Hkv) * D, "flops": 3 * sum(new) * (H + Hkv) * case["rot"]}
    pairs = sum(n * h - (n * (n - 1) // 2 if case["causal"] else 0) for n, h in zip(new, held))
    # each held key and value and q in, the output out; two products over the visible pairs
    return {"bytes": 4 * sum(held) * Hkv * D + 4 * sum(new) * H * D + (4 * sum(new) * H if case["lse"] else 0),
            "flops": 4 * D * H * pairs}
