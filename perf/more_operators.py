"""Workloads of a decoder's two ends in a learner's inner step: rotary positions and token
log probabilities.

Before attention every layer turns its queries and keys by their tokens' positions; after
the output layer the loss needs the log probability of each next token, an evaluation also
the entropy and the most probable alternatives. The cases below are these operators,
forward and backward, at the sizes of the repository's own decoder sets, and ``draw``
spreads further ones over the same ranges. With ``own`` false ``run`` computes them with
elementary torch operations; with ``own`` true through the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
LARGEST_ROTARY = 4 * 8192 * 40 * 128      # elements of the largest listed rotation
LARGEST_LOGITS = 8192 * 128256            # of the largest listed log probabilities
INF = float("inf")


# ----------------------------------------------------------------------------
# cases


def listed():
    return [
        # evaluation token by token: one new token of five sequences, the 1.1B set's heads
        {"name": "rotary_token", "op": "rotary", "inverse": False, "batch": 5, "seq": 1,
         "q_heads": 32, "k_heads": 4, "head": 64, "rotated": 64, "interleaved": False,
         "order": "fused", "scaling": "none", "type": "bf16", "far": 8192},
        # odd sizes in fp32: part of the head, neighbouring pairs, heads before tokens
        {"name": "rotary_odd", "op": "rotary", "inverse": False, "batch": 3, "seq": 1023,
         "q_heads": 7, "k_heads": 1, "head": 75, "rotated": 50, "interleaved": True,
         "order": "heads", "scaling": "linear", "type": "f32", "far": 100000},
        # a training microbatch of the 10B set, queries and keys inside fused rows, long context
        {"name": "rotary_10b", "op": "rotary", "inverse": False, "batch": 4, "seq": 8192,
         "q_heads": 32, "k_heads": 8, "head": 128, "rotated": 128, "interleaved": False,
         "order": "fused", "scaling": "parts", "type": "bf16", "far": 0},
        # its backward pass: gradients as attention leaves them, heads before tokens
        {"name": "rotary_bwd_10b", "op": "rotary", "inverse": True, "batch": 4, "seq": 8192,
         "q_heads": 32, "k_heads": 8, "head": 128, "rotated": 128, "interleaved": False,
         "order": "heads", "scaling": "parts", "type": "bf16", "far": 0},
        # evaluation token by token: three rows of the 10B set's vocabulary, alternatives
        {"name": "logp_rows", "op": "logp", "rows": 3, "vocab": 128256, "type": "bf16", "pad": 0,
         "top": 8, "entropy": True, "left_out": 0, "masked": 256, "empty": 0},
        # the small model of the repository's example: many short rows
        {"name": "logp_small_vocab", "op": "logp", "rows": 512, "vocab": 512, "type": "bf16",
         "pad": 0, "top": 0, "entropy": False, "left_out": 0, "masked": 0, "empty": 0},
        # the loss of a training microbatch of the 1.1B set, an eighth of it padding
        {"name": "logp_1b", "op": "logp", "rows": 16384, "vocab": 32000, "type": "bf16", "pad": 0,
         "top": 0, "entropy": False, "left_out": 2048, "masked": 0, "empty": 0},
        # scoring a batch with the 10B set's vocabulary: entropy and twenty alternatives
        {"name": "logp_10b", "op": "logp", "rows": 8192, "vocab": 128256, "type": "bf16",
         "pad": 0, "top": 20, "entropy": True, "left_out": 0, "masked": 256, "empty": 0},
        # odd vocabulary inside wider rows, fp32, masked rows among them
        {"name": "logp_odd", "op": "logp", "rows": 1023, "vocab": 32003, "type": "f32", "pad": 5,
         "top": 5, "entropy": True, "left_out": 17, "masked": 1000, "empty": 3},
        # its gradients: of the log probability, the entropy, the log sum and the alternatives
        {"name": "logp_bwd_odd", "op": "logp_bwd", "rows": 1023, "vocab": 32003, "type": "f32",
         "pad": 5, "top": 5, "entropy": True, "left_out": 17, "masked": 1000, "empty": 3},
        # the loss's gradient in the 1.1B set's microbatch
        {"name": "logp_bwd_1b", "op": "logp_bwd", "rows": 16384, "vocab": 32000, "type": "bf16",
         "pad": 0, "top": 0, "entropy": False, "left_out": 2048, "masked": 0, "empty": 0},
        # the 10B set's vocabulary with an entropy term in the loss
        {"name": "logp_bwd_10b", "op": "logp_bwd", "rows": 8192, "vocab": 128256, "type": "bf16",
         "pad": 0, "top": 0, "entropy": True, "left_out": 0, "masked": 256, "empty": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        head = rng.choice([16, 32, 64, 64, 80, 96, 128, 128, 128, 192, 256, rng.randint(2, 256)])
        rotated = max(2, (head if rng.random() < 0.6 else rng.randint(2, head)) // 2 * 2)
        q = _log(rng, 1, 64)
        c = {"op": "rotary", "inverse": rng.random() < 0.5, "batch": _log(rng, 1, 64), "seq": 1,
             "q_heads": q, "k_heads": rng.choice([1, max(1, q // 4), q]), "head": head,
             "rotated": rotated, "interleaved": rng.random() < 0.5,
             "order": rng.choice(["fused", "heads", "plain"]),
             "scaling": rng.choice(["none", "linear", "base", "parts"]),
             "type": rng.choice(["f32", "bf16", "f16"]),
             "far": rng.choice([0, 8192, 100000, 1 << 20])}
        per = (c["q_heads"] + c["k_heads"]) * head * c["batch"] * (2 if c["type"] == "f32" else 1)
        if rng.random() < 0.75:
            c["seq"] = _log(rng, 1, min(16384, max(1, LARGEST_ROTARY // per)))
        if c["rotated"] == 2 and c["scaling"] == "base":
            c["scaling"] = "linear"
        return c
    vocab = _log(rng, 2, 200000)
    if rng.random() < 0.4:
        vocab = max(64, vocab // 64 * 64)
    kind = rng.choice(["f32", "bf16", "f16"])
    rows = _log(rng, 1, min(32768, LARGEST_LOGITS // vocab // (2 if kind == "f32" else 1)))
    some = lambda n: rng.choice([0, 0, rng.randint(0, n)])  # noqa: E731
    return {"op": rng.choice(["logp", "logp_bwd"]), "rows": rows, "vocab": vocab, "type": kind,
            "pad": rng.choice([0, 0, 0, 1, 64]), "top": rng.choice([0, 0, 1, 5, 20, 32]),
            "entropy": rng.random() < 0.5, "left_out": some(rows // 4), "masked": some(vocab // 4),
            "empty": some(rows // 8)}


# ----------------------------------------------------------------------------
# inputs


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] == "rotary":
        return _prepare_rotary(case, g)
    return _prepare_logits(case, g)


SCALING = {"none": {}, "linear": {"factor": 8.0}, "base": {"factor": 8.0},
           "parts": {"factor": 8.0, "context": 8192.0, "low": 1.0, "high": 4.0}}


def _prepare_rotary(case, g):
    B, S, H, K, D = (case[k] for k in ("batch", "seq", "q_heads", "k_heads", "head"))
    dt = TYPES[case["type"]]

    def randn(*shape):
        x = torch.randn(shape, generator=g, device=DEV)
        return x.mul_(1e-3 if case["inverse"] else 1.0).to(dt)
    if case["order"] == "fused":        # one product's rows: queries, keys, values
        rows = randn(B, S, H + 2 * K, D)
        q, k = rows[:, :, :H], rows[:, :, H:H + K]
    elif case["order"] == "heads":      # heads before tokens, seen as tokens before heads
        q, k = randn(B, H, S, D).transpose(1, 2), randn(B, K, S, D).transpose(1, 2)
    else:
        q, k = randn(B, S, H, D), randn(B, S, K, D)
    # sequences of one batch are at positions of their own
    start = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device=DEV)
    positions = start + torch.arange(S, device=DEV)
    # scaled for contexts eight times the trained ones; the amplitude as YaRN (Peng et al.,
    # 2023) sets it
    state = {"case": dict(case), "q": q, "k": k, "positions": positions,
             "amplitude": 0.1 * math.log(8.0) + 1 if case["scaling"] == "parts" else 1.0,
             "base": 500000.0 if case["scaling"] == "parts" else 10000.0}
    if own:
        import pseudo_grad_sync_gb300 as dl
        state["frequencies"] = dl.RotaryFrequencies(
            case["rotated"], base=state["base"], scaling=case["scaling"],
            amplitude=state["amplitude"], device=DEV, **SCALING[case["scaling"]])
    return state


def _prepare_logits(case, g):
    R, V = case["rows"], case["vocab"]
    z = torch.randn(R, V + case["pad"], generator=g, device=DEV)
    # rows of different sharpness and offset, a common profile of frequent tokens
    z.add_(torch.randn(V + case["pad"], generator=g, device=DEV))
    z.mul_(torch.rand(R, 1, generator=g, device=DEV).mul_(2.0).add_(0.5))
    z.add_(torch.randn(R, 1, generator=g, device=DEV), alpha=3.0)
    if case["masked"]:                  # vocabulary entries that no text uses
        z[:, V - min(case["masked"], V - 1):V] = -INF
    order = torch.randperm(R, generator=g, device=DEV)
    if case["empty"]:                   # a mask that leaves nothing
        z[order[case["left_out"]:case["left_out"] + case["empty"]], :V] = -INF
    z = z.to(TYPES[case["type"]])[:, :V]
    tokens = torch.randint(0, V, (R,), generator=g, device=DEV)
    tokens[order[:case["left_out"]]] = -1
    state = {"case": dict(case), "logits": z, "tokens": tokens}
    if case["op"] == "logp":
        return state
    # what the forward pass left: the rows' statistics and alternatives
    s = _statistics(z, tokens, True)
    state["row_max"], state["log_sum"] = s["row_max"], s["log_sum"]
    state["entropy"] = s["entropy"] if case["entropy"] else None

    def grad(*shape):
        return torch.randn(*shape, generator=g, device=DEV).mul_(1 / R)
    state["d_logp"] = grad(R)
    state["d_entropy"] = grad(R) if case["entropy"] else None
    state["d_lse"] = grad(R) if case["entropy"] else None
    state["top_tokens"] = _alternatives(z, s["none"], case["top"]) if case["top"] else None
    state["d_top"] = grad(R, case["top"]) if case["top"] else None
    return state


# ----------------------------------------------------------------------------
# one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rotary": _rotary_own, "logp": _logp_own, "logp_bwd": _bwd_own}[op](state)
    return {"rotary": _rotary_plain, "logp": _logp_plain, "logp_bwd": _bwd_plain}[op](state)


def _rotary_own(s):
    import pseudo_grad_sync_gb300 as dl
    c = s["case"]
    q, k = dl.rotary_apply((s["q"], s["k"]), s["frequencies"], s["positions"],
                           interleaved=c["interleaved"], inverse=c["inverse"])
    return {"q": q, "k": k}


def _logp_own(s):
    import pseudo_grad_sync_gb300 as dl
    c = s["case"]
    r = dl.logprobs_forward(s["logits"], s["tokens"], top=c["top"], entropy=c["entropy"])
    out = {"logp": r.logp, "lse": r.lse}
    if c["entropy"]:
        out["entropy"] = r.entropy
    if c["top"]:
        out["top_tokens"], out["top_logp"] = r.top_tokens, r.top_logp
    return out


def _bwd_own(s):
    import pseudo_grad_sync_gb300 as dl
    return {"dlogits": dl.logprobs_backward(
        s["logits"], s["tokens"], s["row_max"], s["log_sum"], d_logp=s["d_logp"],
        d_entropy=s["d_entropy"], d_lse=s["d_lse"], entropy=s["entropy"],
        top_tokens=s["top_tokens"], d_top=s["d_top"])}


def _frequencies(s):
    """Radians per token of every pair, in 64 bits."""
    c, d = s["case"], s["case"]["rotated"]
    how = SCALING[c["scaling"]]
    base = s["base"]
    if c["scaling"] == "base":
        base = base * how["factor"] ** (d / (d - 2))
    f = base ** (-torch.arange(0, d, 2, dtype=torch.float64, device=DEV) / d)
    if c["scaling"] == "linear":
        f = f / how["factor"]
    if c["scaling"] == "parts":     # fast pairs as trained, slow ones slowed, a ramp between
        turns = how["context"] * f / (2 * math.pi)
        keep = ((turns - how["low"]) / (how["high"] - how["low"])).clamp(0, 1)
        f = f * (keep + (1 - keep) / how["factor"])
    return f


def _rotary_plain(s):
    c = s["case"]
    # in 64 bits: a far position's angle has few digits left in 32
    angle = s["positions"].double()[..., None] * _frequencies(s)
    sign = -s["amplitude"] if c["inverse"] else s["amplitude"]
    cos = (torch.cos(angle) * s["amplitude"]).float()[:, :, None]
    sin = (torch.sin(angle) * sign).float()[:, :, None]
    return {"q": _turn(s["q"], cos, sin, c), "k": _turn(s["k"], cos, sin, c)}


def _turn(x, cos, sin, c):
    d = c["rotated"]
    y = x.float()
    a, b = (y[..., 0:d:2], y[..., 1:d:2]) if c["interleaved"] else (y[..., :d // 2],
                                                                    y[..., d // 2:d])
    first, second = a * cos - b * sin, b * cos + a * sin
    turned = (torch.stack([first, second], -1).flatten(-2) if c["interleaved"]
              else torch.cat([first, second], -1))
    return torch.cat([turned, y[..., d:]], -1).to(x.dtype)


def _statistics(z, tokens, entropy):
    """Row statistics; a left out row has zeros, one that the mask leaves empty no sum."""
    z = z.float()
    top = z.amax(1)
    empty = top == -INF
    top = torch.where(empty, torch.zeros_like(top), top)
    z = z - top[:, None]
    e = torch.exp(z)
    total = e.sum(1)
    log_sum = torch.log(total)
    out = tokens < 0
    none = out | empty
    fill = lambda v, where: torch.where(where, torch.zeros_like(v), v)  # noqa: E731
    s = {"row_max": fill(top, out), "log_sum": fill(log_sum, out), "out": out, "none": none,
         "shifted": z, "lse": fill(top + log_sum, out), "exp": e}
    if entropy:
        mean = (e * z.clamp(min=-1e30)).sum(1) / total
        s["entropy"] = fill(log_sum - mean, none)
    return s


def _alternatives(z, none, k):
    """Tokens of the k largest logits, the lowest first on ties; -1 beyond the finite ones."""
    z = z.float() + 0.0
    bits = z.view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    V = z.shape[1]
    key = (order << 32) | (V - 1 - torch.arange(V, device=z.device))
    got = torch.topk(key, min(k, V), sorted=True).values
    tokens = V - 1 - (got & 0xFFFFFFFF)
    bad = none[:, None] | torch.gather(z, 1, tokens).eq(-INF)
    tokens = torch.where(bad, torch.full_like(tokens, -1), tokens)
    return torch.nn.functional.pad(tokens, (0, k - tokens.shape[1]), value=-1)


def _logp_plain(s):
    c, z, t = s["case"], s["logits"], s["tokens"]
    r = _statistics(z, t, c["entropy"])
    at = torch.gather(r["shifted"], 1, t.clamp(min=0)[:, None])[:, 0]
    logp = torch.where(r["none"], torch.full_like(at, -INF), at - r["log_sum"])
    out = {"logp": torch.where(r["out"], torch.zeros_like(at), logp), "lse": r["lse"]}
    if c["entropy"]:
        out["entropy"] = r["entropy"]
    if c["top"]:
        top = _alternatives(z, r["none"], c["top"])
        at = torch.gather(r["shifted"], 1, top.clamp(min=0)) - r["log_sum"][:, None]
        out["top_tokens"] = top
        out["top_logp"] = torch.where(top < 0, torch.full_like(at, -INF), at)
    return out


def _bwd_plain(s):
    c, t = s["case"], s["tokens"]
    logp = s["logits"].float() - s["row_max"][:, None] - s["log_sum"][:, None]
    factor = -s["d_logp"]
    if s["d_lse"] is not None:
        factor = factor + s["d_lse"]
    if s["d_top"] is not None:
        d_top = torch.where(s["top_tokens"] < 0, torch.zeros_like(s["d_top"]), s["d_top"])
        factor = factor - d_top.sum(1)
    dz = torch.exp(logp)
    if s["d_entropy"] is None:
        dz = dz * factor[:, None]
    else:
        inner = logp.clamp(min=-1e30) + s["entropy"][:, None]
        dz = dz * (factor[:, None] - s["d_entropy"][:, None] * inner)
    dz.scatter_add_(1, t.clamp(min=0)[:, None], s["d_logp"][:, None])
    if s["d_top"] is not None:
        dz.scatter_add_(1, s["top_tokens"].clamp(min=0), d_top)
    # rows left out, and those without a distribution, have no gradient
    none = (t < 0) | (s["log_sum"] == -INF)
    return {"dlogits": torch.where(none[:, None], torch.zeros_like(dz), dz).to(s["logits"].dtype)}


# ----------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    if case["op"] == "rotary":
        tokens = case["batch"] * case["seq"]
        heads = tokens * (case["q_heads"] + case["k_heads"])
        return {"bytes": 2 * heads * case["head"] * SIZE[case["type"]] + 8 * tokens,
                "flops": 3 * heads * case["rotated"]}
    R, V, size = case["rows"], case["vocab"], SIZE[case["type"]]
    read = R - case["left_out"]
    per_row = 8 + 4 * (1 + case["entropy"])
    if case["op"] == "logp":
        return {"bytes": read * V * size + R * (4 + per_row + 12 * case["top"]),
                "flops": read * V * (6 if case["entropy"] else 4)}
    read -= case["empty"]
    return {"bytes": read * V * size + R * (V * size + 8 + per_row + 12 * case["top"]),
            "flops": read * V * (7 if case["entropy"] else 4)}


# ----------------------------------------------------------------------------
# the definition in 64 bits


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "rotary":
        return _exact_rotary(s)
    rows = max(1, (1 << 27) // case["vocab"])
    fn = _exact_logp if case["op"] == "logp" else _exact_bwd
    parts = [fn(s, slice(r, r + rows)) for r in range(0, case["rows"], rows)]
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


def _exact_rotary(s):
    """Pairs as complex numbers, turned by a * exp(i p f)."""
    c, d = s["case"], s["case"]["rotated"]
    how = SCALING[c["scaling"]]
    f = []
    for i in range(d // 2):
        base = s["base"] * how["factor"] ** (d / (d - 2)) if c["scaling"] == "base" else s["base"]
        w = math.exp(-2 * i / d * math.log(base))
        if c["scaling"] == "linear":
            w /= how["factor"]
        if c["scaling"] == "parts":
            r = how["context"] * w / math.tau
            x = min(1.0, max(0.0, (r - how["low"]) / (how["high"] - how["low"])))
            w = x * w + (1 - x) * w / how["factor"]
        f.append(-w if c["inverse"] else w)
    f = torch.tensor(f, dtype=torch.float64, device=DEV)
    turn = torch.polar(torch.full((), s["amplitude"], dtype=torch.float64, device=DEV),
                       s["positions"].double()[..., None] * f)[:, :, None]
    out = {}
    for key in ("q", "k"):
        y = s[key].double()     # a new tensor: its pairs are turned in place
        even, odd = ((slice(0, d, 2), slice(1, d, 2)) if c["interleaved"]
                     else (slice(0, d // 2), slice(d // 2, d)))
        for b in range(y.shape[0]):
            z = torch.complex(y[b, ..., even], y[b, ..., odd]) * turn[b]
            y[b, ..., even], y[b, ..., odd] = z.real, z.imag
        out[key] = y
    return out


def _exact_logp(s, rows):
    c = s["case"]
    z, t = s["logits"][rows].double(), s["tokens"][rows]
    R, V = z.shape
    lse = torch.logsumexp(z, 1)
    none = lse == -INF
    logp = z - torch.where(none, torch.zeros_like(lse), lse)[:, None]
    at = logp[torch.arange(R, device=DEV), t.clamp(min=0)]
    out = {"logp": torch.where(t < 0, torch.zeros_like(at), at),
           "lse": torch.where(t < 0, torch.zeros_like(lse), lse)}
    if c["top"]:
        k = min(c["top"], V)
        index = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
        value = logp.gather(1, index)
        gone = (value == -INF) | (t < 0)[:, None]
        out["top_tokens"] = torch.full((R, c["top"]), -1, device=DEV)
        out["top_tokens"][:, :k] = index.masked_fill(gone, -1)
        out["top_logp"] = torch.full((R, c["top"]), -INF, dtype=torch.float64, device=DEV)
        out["top_logp"][:, :k] = value.masked_fill(gone, -INF)
    if c["entropy"]:
        p = torch.exp(logp)
        h = -(p * logp.masked_fill(p == 0, 0)).sum(1)
        out["entropy"] = torch.where((t < 0) | none, torch.zeros_like(h), h)
    return out


def _exact_bwd(s, rows):
    """The Jacobians' rows, term by term."""
    z, t = s["logits"][rows].double(), s["tokens"][rows]
    part = lambda k: None if s[k] is None else s[k][rows].double()  # noqa: E731
    gone = (t < 0) | (s["log_sum"][rows] == -INF)
    z -= (part("row_max") + part("log_sum"))[:, None]
    p = torch.exp(z)
    g = part("d_logp")
    dz = -g[:, None] * p
    line = torch.arange(z.shape[0], device=DEV)
    dz[line, t.clamp(min=0)] += g
    if s["d_lse"] is not None:
        dz += part("d_lse")[:, None] * p
    if s["d_entropy"] is not None:
        z.masked_fill_(p == 0, 0)
        dz -= part("d_entropy")[:, None] * p * (z + part("entropy")[:, None])
    if s["d_top"] is not None:
        top, q = s["top_tokens"][rows], part("d_top")
        for i in range(top.shape[1]):
            have = (top[:, i] >= 0).double() * q[:, i]
            dz -= have[:, None] * p
            dz[line, top[:, i].clamp(min=0)] += have
    return {"dlogits": dz.masked_fill_(gone[:, None], 0)}
