"""Plain implementations of the decoder operators for the tests, in 64 bits.

torch in float64 on the inputs' device, written from the formulas in
include/diloco_sync.h."""
import math
from fractions import Fraction

import torch

INF = math.inf


def frequencies(dim, base=10000.0, scaling="none", factor=1.0, context=0.0, low=1.0, high=4.0):
    """Radians per token of every pair, as Python floats."""
    if scaling == "base":
        base = base * factor ** (dim / (dim - 2))
    out = []
    for i in range(dim // 2):
        f = base ** (-2 * i / dim)
        if scaling == "linear":
            f /= factor
        if scaling == "parts":
            g = min(1.0, max(0.0, (context * f / math.tau - low) / (high - low)))
            f = f * g + (1 - g) * f / factor
        out.append(f)
    return out


def angles(positions, turns):
    """[..., pairs] radians in [0, 2 pi): the fraction of a turn is exact (Python integers)."""
    flat = [[float(Fraction((int(p) * int(t)) % 2**64, 2**64)) * math.tau for t in turns]
            for p in positions.reshape(-1).tolist()]
    return torch.tensor(flat, dtype=torch.float64).view(*positions.shape, len(turns))


def rotate(x, angle, amplitude=1.0, interleaved=False, inverse=False):
    """x [batch, tokens, heads, width]; angle [batch, tokens, pairs]. Returns the
    result and the sum of the terms' magnitudes."""
    y = x.double().clone()
    d = 2 * angle.shape[-1]
    cos = amplitude * torch.cos(angle)[:, :, None]
    sin = (-amplitude if inverse else amplitude) * torch.sin(angle)[:, :, None]
    first, second = ((slice(0, d, 2), slice(1, d, 2)) if interleaved
                     else (slice(0, d // 2), slice(d // 2, d)))
    a, b = y[..., first].clone(), y[..., second].clone()
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    size = torch.zeros_like(y)
    size[..., first] = size[..., second] = (a.abs() + b.abs()) * abs(amplitude)
    return y, size


def logprobs(z, tokens=None, top=0):
    """Every output of the forward call, and `far`, the mean of |z - m|."""
    z = z.double()
    rows, vocab = z.shape
    m = z.max(1).values
    bad = torch.isnan(m) | (m == INF)
    empty = m == -INF
    m = torch.where(empty, torch.zeros_like(m), m)
    d = z - m[:, None]
    e = torch.exp(d)
    S = e.sum(1)
    log_sum = torch.log(S)
    far = -(e * torch.where(e == 0, torch.zeros_like(d), d)).sum(1) / torch.where(empty, torch.ones_like(S), S)
    out = {"row_max": m, "log_sum": log_sum, "lse": m + log_sum,
           "entropy": torch.where(empty, torch.zeros_like(m), log_sum + far)}
    none = empty | bad
    if top:
        k = min(top, vocab)
        order = torch.sort(torch.where(z == z, z, -INF), dim=1, descending=True, stable=True)
        at, value = order.indices[:, :k], order.values[:, :k]
        gone = (value == -INF) | none[:, None]
        pad = lambda v, fill: torch.nn.functional.pad(v, (0, top - k), value=fill)  # noqa: E731
        out["top_tokens"] = pad(at.masked_fill(gone, -1), -1)
        out["top_logp"] = pad((value - m[:, None] - log_sum[:, None]).masked_fill(gone, -INF), -INF)
    if tokens is not None:
        t = tokens.long()
        at = d.gather(1, t.clamp(0, vocab - 1)[:, None])[:, 0]
        logp = torch.where(empty, torch.full_like(at, -INF), at - log_sum)
        out["logp"] = logp.masked_fill(t >= vocab, math.nan)
    for k, v in out.items():
        if k != "top_tokens":
            out[k] = v.masked_fill(bad.view(-1, *[1] * (v.dim() - 1)), math.nan)
    if tokens is not None:
        for k in out:
            fill = {"top_tokens": -1, "top_logp": -INF}.get(k, 0)
            out[k] = out[k].masked_fill((t < 0).view(-1, *[1] * (out[k].dim() - 1)), fill)
    out["far"] = far
    return out


def dlogits(z, tokens, row_max, log_sum, d_logp=None, d_entropy=None, d_lse=None, entropy=None,
            top_tokens=None, d_top=None):
    """The gradient, and the magnitude of each element's terms."""
    z = z.double()
    rows, vocab = z.shape
    zeros = torch.zeros(rows, dtype=torch.float64, device=z.device)
    g, h, l = (zeros if v is None else v.double() for v in (d_logp, d_entropy, d_lse))  # noqa: E741
    t = torch.zeros(rows, dtype=torch.int64, device=z.device) if tokens is None else tokens.long()
    d = z - row_max.double()[:, None]
    lp = d - log_sum.double()[:, None]
    p = torch.exp(lp)
    q = None
    named = zeros.clone()
    if d_top is not None:
        ok = (top_tokens >= 0) & (top_tokens < vocab)
        q = torch.where(ok, d_top.double(), torch.zeros_like(d_top, dtype=torch.float64))
        named = q.sum(1)
    H = zeros if entropy is None else entropy.double()
    inner = torch.where(p == 0, torch.zeros_like(lp), lp + H[:, None])
    dz = p * ((l - g - named)[:, None] - h[:, None] * inner)
    size = p * ((l.abs() + g.abs() + (zeros if q is None else q.abs().sum(1)))[:, None]
                + h.abs()[:, None] * (inner.abs() + H.abs()[:, None] + log_sum.double().abs()[:, None])
                + (h.abs()[:, None] * torch.where(p == 0, torch.zeros_like(d), d.abs())))
    size = size * (1 + torch.where(p == 0, torch.zeros_like(d), d.abs()))
    here = (t >= 0) & (t < vocab)
    dz.scatter_add_(1, t.clamp(0, vocab - 1)[:, None], torch.where(here, g, zeros)[:, None])
    size.scatter_add_(1, t.clamp(0, vocab - 1)[:, None], torch.where(here, g.abs(), zeros)[:, None])
    any_ = (g != 0) | (h != 0) | (l != 0)
    if q is not None:
        dz.scatter_add_(1, top_tokens.clamp(0, vocab - 1), q)
        size.scatter_add_(1, top_tokens.clamp(0, vocab - 1), q.abs())
        any_ = any_ | (q != 0).any(1)
    dz = dz.masked_fill(((t >= vocab) & (g != 0))[:, None], math.nan)
    none = (t < 0) | (log_sum == -INF) | ~any_
    return dz.masked_fill(none[:, None], 0), size.masked_fill(none[:, None], 0)
