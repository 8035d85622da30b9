"""Workloads of a learner's inner step: gradient norm, AdamW, layer norm.

Between two outer synchronisations every DiLoCo learner takes many inner steps: the
layers' norms forward and backward, the global gradient norm that clips, and one AdamW
step over all tensors of its fragments. The cases below are these operators at the sizes
of the repository's own tensor sets, and ``draw`` spreads further ones over the same
ranges. With ``own`` false ``run`` computes them with elementary torch operations in
32 bits; with ``own`` true through the library's entry points.

Flat layout (the library's): a fragment is a run of tensors; the buffers of a model's
fragments are slices of one flat buffer, each starting on a multiple of 64 elements.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 128                       # elements that share a scale of the 8-bit states
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
HYPER = {"lr": 4e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1}
SEED = 0xD110C0
LARGEST = 1_100_048_384           # elements of the largest listed 32-bit step
LARGEST8 = 415_260_672            # of the largest listed 8-bit step
LARGEST_NORM = 32768 * 4096       # of the largest listed layer norm


# ----------------------------------------------------------------------------
# cases


def listed():
    return [
        # a fine-tuned head or adapter: few small tensors, the call's latency counts
        {"name": "grad_norm_few", "op": "grad_norm", "model": "ragged", "tensors": 12,
         "elements": 150_001, "shapes": 1, "fragments": 1, "grad": "f32"},
        # the clip of every inner step of the 1.1B decoder set, bf16 gradients, 24 fragments
        {"name": "grad_norm_1b", "op": "grad_norm", "model": "decoder_1b", "fragments": 24,
         "grad": "bf16"},
        # few small tensors, latency
        {"name": "adamw_few", "op": "adamw", "bits": 32, "model": "ragged", "tensors": 12,
         "elements": 150_001, "shapes": 1, "fragments": 1, "grad": "f32", "copy": False},
        # many ragged tensors of odd sizes (norm vectors beside matrices), fp32 gradients
        {"name": "adamw_ragged", "op": "adamw", "bits": 32, "model": "ragged", "tensors": 2000,
         "elements": 48_000_007, "shapes": 2, "fragments": 3, "grad": "f32", "copy": False},
        # one inner step of the whole 1.1B decoder set, mixed precision
        {"name": "adamw_1b", "op": "adamw", "bits": 32, "model": "decoder_1b", "fragments": 24,
         "grad": "bf16", "copy": True},
        # the same step with 8-bit states: few small tensors
        {"name": "adamw8_few", "op": "adamw", "bits": 8, "model": "ragged", "tensors": 12,
         "elements": 150_001, "shapes": 1, "fragments": 1, "grad": "f32", "copy": False},
        # ragged tensors whose blocks end and start at odd places
        {"name": "adamw8_ragged", "op": "adamw", "bits": 8, "model": "ragged", "tensors": 2000,
         "elements": 48_000_007, "shapes": 2, "fragments": 3, "grad": "f32", "copy": False},
        # the median fragment of the 10B decoder set (one learner's share of a step)
        {"name": "adamw8_10b_fragment", "op": "adamw", "bits": 8, "model": "decoder_10b_median",
         "fragments": 1, "grad": "bf16", "copy": True},
        # one row up to a few: evaluation token by token
        {"name": "norm_fwd_rows", "op": "norm_fwd", "rows": 5, "width": 2048, "type": "bf16",
         "param": "f32", "rms": True, "bias": False, "pad": 0},
        # a training microbatch of the 10B set's width
        {"name": "norm_fwd_batch", "op": "norm_fwd", "rows": 32768, "width": 4096, "type": "bf16",
         "param": "f32", "rms": False, "bias": True, "pad": 0},
        # odd width, fp32 activations, rows inside wider ones
        {"name": "norm_bwd_odd", "op": "norm_bwd", "rows": 1023, "width": 2047, "type": "f32",
         "param": "f32", "rms": False, "bias": True, "pad": 5, "accumulate": True},
        # the backward pass of the training microbatch
        {"name": "norm_bwd_batch", "op": "norm_bwd", "rows": 32768, "width": 4096, "type": "bf16",
         "param": "f32", "rms": False, "bias": True, "pad": 0, "accumulate": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["grad_norm", "adamw", "adamw8", "norm_fwd", "norm_bwd"])
    if op in ("norm_fwd", "norm_bwd"):
        width = _log(rng, 16, 16384)
        if rng.random() < 0.5:
            width = max(16, width // 64 * 64)
        c = {"op": op, "rows": _log(rng, 1, min(65536, LARGEST_NORM // width)), "width": width,
             "type": rng.choice(["f32", "bf16", "f16"]), "param": rng.choice(["f32", "bf16"]),
             "rms": rng.random() < 0.5, "bias": rng.random() < 0.5,
             "pad": rng.choice([0, 0, 0, 1, 64])}
        if c["type"] == "f32":
            c["rows"] = max(1, c["rows"] // 2)
        if op == "norm_bwd":
            c["accumulate"] = rng.random() < 0.5
        return c
    most = LARGEST8 if op == "adamw8" else LARGEST
    c = {"op": "grad_norm" if op == "grad_norm" else "adamw", "model": "ragged",
         "tensors": _log(rng, 1, 2000), "shapes": rng.randrange(1 << 20),
         "fragments": rng.randint(1, 24), "grad": rng.choice(["f32", "bf16"])}
    if op != "grad_norm":
        c["bits"], c["copy"] = (8 if op == "adamw8" else 32), rng.random() < 0.5
    c["elements"] = _log(rng, 1000 + c["tensors"], most if c["grad"] == "bf16" else most // 2)
    return c


# ----------------------------------------------------------------------------
# tensor sets


def _decoder(layers, d, ffn, n_q, n_kv, vocab):
    kv = n_kv * (d // n_q)
    out = [vocab * d]
    for _ in range(layers):
        out += [d * d, d * kv, d * kv, d * d, ffn * d, ffn * d, d * ffn, d, d]
    return out + [d, vocab * d]


def _pack(numels, parts):
    """Tensors to fragments, largest first onto the lightest; model order within one."""
    loads, of = [0] * parts, [[] for _ in range(parts)]
    for t in sorted(range(len(numels)), key=lambda t: (-numels[t], t)):
        p = min(range(parts), key=lambda p: (loads[p], p))
        loads[p] += numels[t]
        of[p].append(t)
    return [[numels[t] for t in sorted(f)] for f in of]


def _fragments(case):
    """Tensor sizes of every fragment of the case."""
    if case["model"] == "decoder_1b":
        return _pack(_decoder(22, 2048, 5632, 32, 4, 32000), case["fragments"])
    if case["model"] == "decoder_10b_median":
        return [_pack(_decoder(42, 4096, 14336, 32, 8, 128256), 24)[9]]
    r = random.Random(case["shapes"])
    T, n = case["tensors"], case["elements"]
    w = [math.exp(r.uniform(0, 9)) for _ in range(T)]
    sizes = [1 + int((n - T) * x / sum(w)) for x in w]
    sizes[0] += n - sum(sizes)
    return [f for f in _pack(sizes, min(case["fragments"], T)) if f]


class _Layout:
    """Where the fragments and tensors lie in the flat buffers, and the scale slots of the
    8-bit states: block b of a fragment's tensor t, which starts at element o of the
    fragment, has slot o // 128 + t + b."""

    def __init__(self, frags):
        self.frags = frags
        self.n = [sum(f) for f in frags]
        self.slots = [n // BLOCK + len(f) for n, f in zip(self.n, frags)]
        self.start = [0]
        for n in self.n:
            self.start.append(self.start[-1] + -(-n // 64) * 64)
        self.total = self.start[-1]
        self.slot0 = np.concatenate([[0], np.cumsum(self.slots)]).tolist()
        begin, span, slot, last, pads = [], [], [], [], []
        for j, f in enumerate(frags):
            o = 0
            for t, s in enumerate(f):
                begin.append(self.start[j] + o)
                span.append(s)
                slot.append(self.slot0[j] + o // BLOCK + t)
                last.append(slot[-1] + max(0, (s - 1) // BLOCK))
                o += s
            pads.append((self.start[j] + o, self.start[j + 1]))
            span[-1] += pads[-1][1] - pads[-1][0]
        self.pads = [p for p in pads if p[1] > p[0]]
        to = lambda v: torch.tensor(v, dtype=torch.int64, device=DEV)  # noqa: E731
        self.begin, self.span, self.slot, self.last = to(begin), to(span), to(slot), to(last)
        used = np.zeros(self.slot0[-1] + 1, dtype=np.int64)
        np.add.at(used, slot, 1)
        np.add.at(used, np.asarray(last) + 1, -1)
        self.used = to(np.cumsum(used)[:-1]) > 0    # slots that hold a block

    def slices(self, flat):
        return [flat[s:s + n] for s, n in zip(self.start, self.n)]

    def tensors(self):
        """The tensor of every element."""
        return torch.searchsorted(torch.cumsum(self.span, 0), torch.arange(self.total, device=DEV),
                                  right=True, out_int32=True)


# ----------------------------------------------------------------------------
# inputs


def _randn(n, g, std=1.0):
    return torch.randn(n, generator=g, device=DEV).mul_(std)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] in ("norm_fwd", "norm_bwd"):
        return _prepare_norm(case, g)
    L = _Layout(_fragments(case))
    N, T = L.total, L.span.numel()
    # each tensor's gradients have their own spread, as layers' gradients do
    sigma = torch.exp(torch.rand(T, generator=g, device=DEV) * math.log(100.0)) * 3e-5
    spread = sigma[L.tensors()]
    grad = _randn(N, g).mul_(spread).to(TYPES[case["grad"]])
    state = {"case": dict(case), "layout": L, "grad": grad}
    if case["op"] == "grad_norm":
        for a, b in L.pads:
            grad[a:b] = 0
        state["max_norm"] = 1.0
        state["out"] = torch.zeros(2, device=DEV)
        if own:
            import pseudo_grad_sync_gb300 as dl
            state["grads"] = dl.GradList(L.slices(grad))
            state["workspace"] = dl.new_workspace(dl.grad_norm_workspace_bytes())
        return state
    state["theta"] = _randn(N, g, 0.02)
    flats = [grad, state["theta"]]
    if case["bits"] == 32:
        state["m"] = _randn(N, g, 0.3).mul_(spread)
        state["v"] = _randn(N, g, 0.5).exp_().mul_(spread).mul_(spread)
    else:
        # mid-training codes; the scales follow each tensor's spread
        exps = torch.floor(torch.log2(sigma))
        state["m"] = _randn(N, g, 20.0).clamp_(-250, 250).to(torch.float8_e4m3fn)
        state["v"] = _randn(N, g, 0.5).exp_().mul_(40.0).clamp_(max=250).to(torch.float8_e4m3fn)
        S = L.slot0[-1]
        blocks = torch.zeros(S, dtype=torch.int64, device=DEV)
        blocks[L.slot[1:]] = 1
        of = torch.cumsum(blocks, 0)
        state["m_scale"] = torch.exp2(exps[of] - 6)
        state["v_scale"] = torch.exp2(exps[of] - 5)
    flats += [state["m"], state["v"]]
    for f in flats:
        for a, b in L.pads:
            f[a:b] = torch.zeros(b - a, device=DEV).to(f.dtype)
    state["copy"] = torch.zeros(N, dtype=torch.bfloat16, device=DEV) if case["copy"] else None
    # vectors (norms, biases) are not decayed
    state["decay"] = (L.span > 8192).float()
    state["clip"] = torch.tensor([1.25, 0.8], device=DEV)     # norm, coefficient
    state["step"] = 100
    if own:
        import pseudo_grad_sync_gb300 as dl
        bounds = np.concatenate([[0], np.cumsum([len(f) for f in L.frags])]).tolist()
        S, s0 = L.slot0[-1], L.slot0
        by8 = case["bits"] == 8
        state["jobs"] = dl.AdamWJobs(
            [dl.Fragment(f, DEV) for f in L.frags], L.slices(state["theta"]), L.slices(grad),
            L.slices(state["m"]), L.slices(state["v"]),
            m_scale=[state["m_scale"][a:b] for a, b in zip(s0, s0[1:])] if by8 else None,
            v_scale=[state["v_scale"][a:b] for a, b in zip(s0, s0[1:])] if by8 else None,
            theta_bf16=L.slices(state["copy"]) if case["copy"] else None,
            decay=[state["decay"][a:b].clone() for a, b in zip(bounds, bounds[1:])])
    return state


def _prepare_norm(case, g):
    R, D, pad = case["rows"], case["width"], case["pad"]
    xt, wt = TYPES[case["type"]], TYPES[case["param"]]

    def rows(std):
        whole = torch.randn(R, D + pad, generator=g, device=DEV).mul_(std)
        return whole
    x = rows(1.0)
    # a residual stream: rows of different size, a common offset, a few large channels
    x.mul_(torch.exp(_randn((R, 1), g, 0.7))).add_(0.1)
    x[:, ::max(1, D // 7)] *= 8.0
    x = x.to(xt)[:, :D]
    state = {"case": dict(case), "x": x, "eps": 1e-5,
             "weight": _randn(D, g, 0.2).add_(1.0).to(wt),
             "bias": _randn(D, g, 0.1).to(wt) if case["bias"] else None}
    if case["op"] == "norm_bwd":
        state["dy"] = rows(1e-3).to(xt)[:, :D]
        xf = x.float()
        mean = torch.zeros(R, device=DEV) if case["rms"] else xf.mean(1)
        var = (xf - mean[:, None]).square_().mean(1)
        state["mean"] = None if case["rms"] else mean
        state["rstd"] = torch.rsqrt(var + state["eps"])
        state["dweight"] = _randn(D, g, 1e-2).to(wt)
        state["dbias"] = _randn(D, g, 1e-2).to(wt) if case["bias"] else None
        if own:
            import pseudo_grad_sync_gb300 as dl
            state["workspace"] = dl.new_workspace(dl.layernorm_workspace_bytes(R, D))
    return state


# ----------------------------------------------------------------------------
# one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return {"grad_norm": _norm_plain, "adamw": _adamw_plain, "norm_fwd": _fwd_plain,
            "norm_bwd": _bwd_plain}[op](state)


def _norm_own(s):
    import pseudo_grad_sync_gb300 as dl
    dl.grad_norm(s["grads"], s["max_norm"], out=s["out"], workspace=s["workspace"])
    return {"norm": s["out"][0:1], "coef": s["out"][1:2]}


def _adamw_own(s):
    import pseudo_grad_sync_gb300 as dl
    s["step"] += 1
    dl.adamw_step(s["jobs"], s["step"], lr=HYPER["lr"], betas=(HYPER["beta1"], HYPER["beta2"]),
                  eps=HYPER["eps"], weight_decay=HYPER["weight_decay"], clip=s["clip"], seed=SEED)
    return _updated(s)


def _updated(s):
    out = {"theta": s["theta"], "m": s["m"], "v": s["v"]}
    if s["case"]["bits"] == 8:
        out["m_scale"], out["v_scale"] = s["m_scale"], s["v_scale"]
    if s["copy"] is not None:
        out["copy"] = s["copy"]
    return out


def _fwd_own(s):
    import pseudo_grad_sync_gb300 as dl
    y, mean, rstd = dl.layernorm_forward(s["x"], s["weight"], s["bias"], eps=s["eps"],
                                         rms=s["case"]["rms"])
    return {"y": y, "rstd": rstd} if mean is None else {"y": y, "mean": mean, "rstd": rstd}


def _bwd_own(s):
    import pseudo_grad_sync_gb300 as dl
    dx, dw, db = dl.layernorm_backward(
        s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], dweight=s["dweight"],
        dbias=s["dbias"], rms=s["case"]["rms"], accumulate=s["case"]["accumulate"],
        workspace=s["workspace"])
    return {"dx": dx, "dweight": dw} if db is None else {"dx": dx, "dweight": dw, "dbias": db}


_OWN = {"grad_norm": _norm_own, "adamw": _adamw_own, "norm_fwd": _fwd_own, "norm_bwd": _bwd_own}


def _norm_plain(s):
    norm = torch.sqrt(s["grad"].float().square().sum())
    coef = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm))
    return {"norm": norm.reshape(1), "coef": coef.reshape(1)}


def _adamw_plain(s):
    h, L = HYPER, s["layout"]
    s["step"] += 1
    g = s["grad"].float() * s["clip"][1]
    by8 = s["case"]["bits"] == 8
    if by8:
        place = _places(L)
        slot = place // BLOCK
        m = s["m"].float() * s["m_scale"][slot]
        r = s["v"].float() * s["v_scale"][slot]
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = m * h["beta1"] + g * (1 - h["beta1"])
    v = v * h["beta2"] + (g * g) * (1 - h["beta2"])
    del g
    root = torch.sqrt(v)
    bc1, bc2 = 1 - h["beta1"] ** s["step"], 1 - h["beta2"] ** s["step"]
    keep = (1 - (h["lr"] * h["weight_decay"]) * s["decay"])[L.tensors()]
    theta = s["theta"] * keep - (h["lr"] / bc1) * m / (root * (1 / math.sqrt(bc2)) + h["eps"])
    s["theta"].copy_(theta)
    del keep, theta
    if s["copy"] is not None:
        s["copy"].copy_(s["theta"])
    if not by8:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return _updated(s)
    low, high = _bits(s["step"], L.slot0[-1])
    for key, x, r16, least in (("m", m, low, 0.0), ("v", root, high, 2.0 ** -9)):
        scale = _scales(L, place, x, s[key + "_scale"])
        s[key].copy_(_encode(x / scale[slot], r16[place], least))
        s[key + "_scale"].copy_(scale)
    return _updated(s)


def _places(L):
    """Slot * 128 + place within the block, of every element."""
    of = L.tensors()
    place = torch.arange(L.total, device=DEV) + (L.slot * BLOCK - L.begin)[of]
    return torch.minimum(place, (L.last * BLOCK + BLOCK - 1)[of])


def _scales(L, place, x, old):
    """2^(k-7) for a block whose largest magnitude lies in [2^k, 2^(k+1)), k >= -53; slots
    that no block has keep what they hold."""
    blocks = torch.zeros(old.numel() * BLOCK, device=DEV)
    blocks[place] = x.abs()
    top = blocks.view(-1, BLOCK).amax(1)
    k = (top.view(torch.int32) >> 23) - 127
    new = torch.ldexp(torch.ones_like(top), k.clamp(min=-53) - 7)
    return torch.where(L.used, new, old)


def _i64(v):
    v &= (1 << 64) - 1
    return v - (1 << 64) if v >> 63 else v


GOLDEN, MIX1, MIX2 = (_i64(v) for v in (0x9E3779B97F4A7C15, 0xBF58476D1CE4E5B9,
                                        0x94D049BB133111EB))


def _mix(z):
    """The output function of SplitMix64 (Steele, Lea and Flood, 2014) on int64 tensors."""
    z = (z ^ ((z >> 30) & ((1 << 34) - 1))) * MIX1
    z = (z ^ ((z >> 27) & ((1 << 37) - 1))) * MIX2
    return z ^ ((z >> 31) & ((1 << 33) - 1))


def _key(step):
    z, mask = (SEED + step * (GOLDEN & ((1 << 64) - 1))) & ((1 << 64) - 1), (1 << 64) - 1
    z = ((z ^ (z >> 30)) * (MIX1 & mask)) & mask
    z = ((z ^ (z >> 27)) * (MIX2 & mask)) & mask
    return _i64(z ^ (z >> 31))


def _bits(step, slots):
    """16 random bits for every place's m and for its root of v. Four places of a block share
    the 64 bits of one hash: m takes the low word, the root the high word; of a word, places
    0 and 2 take the low and the high half, 1 and 3 the same halves in reverse bit order."""
    z = _mix(torch.arange(slots * (BLOCK // 4), device=DEV) * GOLDEN + _key(step))
    out = []
    for w in (z & 0xFFFFFFFF, (z >> 32) & 0xFFFFFFFF):
        halves = torch.stack([w & 0xFFFF, w >> 16], 1).to(torch.int32)
        r = ((halves & 0x5555) << 1) | ((halves >> 1) & 0x5555)
        r = ((r & 0x3333) << 2) | ((r >> 2) & 0x3333)
        r = ((r & 0x0F0F) << 4) | ((r >> 4) & 0x0F0F)
        r = ((r & 0x00FF) << 8) | (r >> 8)
        out.append(torch.stack([halves, r], 2).reshape(-1))
    return out


def _encode(x, r16, least):
    """e4m3 with stochastic rounding: the magnitude, in units of its last place, plus
    r16 / 2^16, rounded down. A positive magnitude is at least `least`."""
    a = x.abs()
    a = torch.where(a > 0, a.clamp(min=least), a)
    normal = ((a.view(torch.int32) + (r16 << 4)) >> 20) - 960
    small = (torch.floor(a * 2.0 ** 25).to(torch.int32) + r16) >> 16
    code = torch.where(a < 2.0 ** -6, small, normal).clamp(max=126)
    code = code | ((x.view(torch.int32) >> 24) & 0x80)
    return code.to(torch.uint8).view(torch.float8_e4m3fn)


def _fwd_plain(s):
    c, x = s["case"], s["x"].float()
    mean = None if c["rms"] else x.mean(1, keepdim=True)
    if mean is not None:
        x = x - mean
    rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + s["eps"])
    y = x * rstd * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = y.to(s["x"].dtype)
    if mean is None:
        return {"y": y, "rstd": rstd.reshape(-1)}
    return {"y": y, "mean": mean.reshape(-1), "rstd": rstd.reshape(-1)}


def _bwd_plain(s):
    c, x, dy = s["case"], s["x"].float(), s["dy"].float()
    rstd = s["rstd"][:, None]
    xhat = (x if c["rms"] else x - s["mean"][:, None]) * rstd
    wdy = dy * s["weight"].float()
    dx = wdy - xhat * (wdy * xhat).mean(1, keepdim=True)
    if not c["rms"]:
        dx = dx - wdy.mean(1, keepdim=True)
    out = {"dx": (dx * rstd).to(s["x"].dtype)}
    grads = {"dweight": (dy * xhat).sum(0)}
    if c["bias"]:
        grads["dbias"] = dy.sum(0)
    for k, v in grads.items():
        s[k].copy_(s[k].float() + v if c["accumulate"] else v)
        out[k] = s[k]
    return out


# ----------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    if case["op"] in ("norm_fwd", "norm_bwd"):
        R, D, xs, ps = case["rows"], case["width"], SIZE[case["type"]], SIZE[case["param"]]
        vectors = 1 + case["bias"]
        stats = R * 4 * (1 if case["rms"] else 2)
        if case["op"] == "norm_fwd":
            return {"bytes": 2 * R * D * xs + vectors * D * ps + stats, "flops": 8 * R * D}
        moved = vectors * D * ps * (2 if case["accumulate"] else 1)
        return {"bytes": 3 * R * D * xs + D * ps + moved + stats, "flops": 14 * R * D}
    frags = _fragments(case)
    n = sum(sum(f) for f in frags)
    if case["op"] == "grad_norm":
        return {"bytes": n * SIZE[case["grad"]] + 8, "flops": 2 * n}
    per = 8 + SIZE[case["grad"]] + (2 if case["copy"] else 0) + (16 if case["bits"] == 32 else 4)
    scales = sum(-(-t // BLOCK) for f in frags for t in f) * 16 if case["bits"] == 8 else 0
    return {"bytes": n * per + scales, "flops": (16 if case["bits"] == 32 else 24) * n}


# ----------------------------------------------------------------------------
# the definition in 64 bits


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "grad_norm":
        total = sum(float(p.double().square().sum()) for p in s["grad"].split(1 << 27))
        norm = math.sqrt(total)
        return {"norm": torch.tensor([norm], dtype=torch.float64),
                "coef": torch.tensor([min(1.0, s["max_norm"] / norm)], dtype=torch.float64)}
    if op == "adamw":
        return _exact_adamw(s)
    x = s["x"].double()
    n = x.shape[1]
    w = s["weight"].double()
    if op == "norm_fwd":
        mu = x.sum(1) / n
        var = (x ** 2).sum(1) / n if case["rms"] else ((x.t() - mu) ** 2).sum(0) / n
        r = 1 / (var + s["eps"]) ** 0.5
        y = torch.einsum("rc,r,c->rc", x if case["rms"] else (x.t() - mu).t(), r, w)
        if s["bias"] is not None:
            y += s["bias"].double()
        return {"y": y, "rstd": r} if case["rms"] else {"y": y, "mean": mu, "rstd": r}
    r, dy = s["rstd"].double(), s["dy"].double()
    if not case["rms"]:
        x = x - s["mean"].double().unsqueeze(1)
    x *= r.unsqueeze(1)
    old = 1.0 if case["accumulate"] else 0.0
    out = {"dweight": old * s["dweight"].double() + torch.einsum("rc,rc->c", dy, x)}
    if case["bias"]:
        out["dbias"] = old * s["dbias"].double() + dy.sum(0)
    dy *= w
    along = torch.einsum("rc,rc->r", dy, x) / n
    shift = torch.zeros_like(r) if case["rms"] else dy.sum(1) / n
    out["dx"] = (dy - along.unsqueeze(1) * x - shift.unsqueeze(1)) * r.unsqueeze(1)
    return out


def _exact_adamw(s):
    """Tensor by tensor, in 64 bits. The 8-bit states' codes and scales are rounding itself
    and have no value in 64 bits."""
    h, L = HYPER, s["layout"]
    t = s["step"] + 1
    by8 = s["case"]["bits"] == 8
    theta = torch.zeros(L.total, dtype=torch.float64, device=DEV)
    m_out = None if by8 else torch.zeros_like(theta)
    v_out = None if by8 else torch.zeros_like(theta)
    decay = s["decay"].double().tolist()
    coef = float(s["clip"][1].double())
    begin, span = L.begin.tolist(), L.span.tolist()
    slot, last = L.slot.tolist(), L.last.tolist()
    for i, (a, n) in enumerate(zip(begin, span)):
        g = s["grad"][a:a + n].double() * coef
        if by8:
            def state(key):
                blocks = s[key + "_scale"][slot[i]:last[i] + 1].double()
                per = blocks.repeat_interleave(BLOCK)
                if per.numel() < n:          # the unused elements at a fragment's end
                    per = torch.cat([per, per.new_zeros(n - per.numel())])
                return s[key][a:a + n].double() * per[:n]
            m, v = state("m"), state("v") ** 2
        else:
            m, v = s["m"][a:a + n].double(), s["v"][a:a + n].double()
        m = h["beta1"] * m + (1 - h["beta1"]) * g
        v = h["beta2"] * v + (1 - h["beta2"]) * g ** 2
        step = (m / (1 - h["beta1"] ** t)) / ((v / (1 - h["beta2"] ** t)) ** 0.5 + h["eps"])
        p = s["theta"][a:a + n].double()
        theta[a:a + n] = p - h["lr"] * (h["weight_decay"] * decay[i] * p + step)
        if not by8:
            m_out[a:a + n], v_out[a:a + n] = m, v
    out = {"theta": theta, "m": m_out, "v": v_out}
    if by8:
        out["m_scale"] = out["v_scale"] = None
    if s["copy"] is not None:
        out["copy"] = theta
    return out
