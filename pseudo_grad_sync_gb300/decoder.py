"""The two ends of a learner's decoder: rotary positions and token log probabilities.

Argument marshalling of the entry points of libdiloco_sync.so under their C
names (imported into the package):

    rotary_frequencies   turns per token of a head's pairs (host), scaled for
                         long contexts
    rotary_apply         queries and keys turned by their positions
    logprobs_forward     log probabilities of given tokens, log sum, entropy and
                         the most probable alternatives of rows of logits
    logprobs_backward    the logits' gradient

``RotaryFrequencies`` holds a model's table on the device; ``rotary`` and
``token_logprobs`` are torch.autograd operations.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional

import numpy as np
import torch

from . import _check, _cuda, _F32, _I64, DLError, lib
from .inner import _TYPE, _at, _away, _on, _one_device, _rows, _stream_of

DL_I32, DL_I64 = 4, 5
DL_ROTARY_MAX_DIM = 8192
DL_ROTARY_MAX_JOBS = 4
DL_ROTARY_INTERLEAVED = 1
DL_ROTARY_INVERSE = 2
DL_LOGPROBS_MAX_TOP = 32

_SCALING = {"none": 0, "linear": 1, "base": 2, "parts": 3}
_INDEX = {torch.int32: DL_I32, torch.int64: DL_I64}
_FLT_MAX = torch.finfo(torch.float32).max


class _RotaryJob(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p)] + [
        (name, ctypes.c_int64)
        for name in ("x_batch", "x_token", "x_head", "y_batch", "y_token", "y_head")] + [
        ("heads", ctypes.c_int32)]


def declare(L):
    """Argument and result types of the decoder's entry points."""
    vp, i32, i64, f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double
    L.dl_rotary_frequencies.restype = ctypes.c_int
    L.dl_rotary_frequencies.argtypes = [i32, f64, i32, f64, f64, f64, f64, vp]
    L.dl_rotary_apply.restype = ctypes.c_int
    L.dl_rotary_apply.argtypes = [vp, i32, i32, i64, i64, i32, i32, vp, f64,
                                  vp, i32, i64, i64, i32, vp]
    L.dl_logprobs_forward.restype = ctypes.c_int
    L.dl_logprobs_forward.argtypes = [vp, i64, i32, i64, i32, vp, i32, vp, vp, vp, i32, vp, vp, vp,
                                      vp, vp]
    L.dl_logprobs_backward.restype = ctypes.c_int
    L.dl_logprobs_backward.argtypes = [vp, i64, i32, i64, i32, vp, i32, vp, vp, vp, vp, vp, vp, i32,
                                       vp, vp, vp, i64, vp]


def _int32(n, name):
    """n, which ctypes would cut to its low 32 bits."""
    if n >= 2**31:
        raise ValueError(f"{name}: {n}, at most 2^31 - 1")
    return n


# ----------------------------------------------------------------------------
# rotary positions


def rotary_frequencies(dim, base=10000.0, scaling="none", factor=1.0, context=0.0, low=1.0,
                       high=4.0):
    """Turns per token of dim / 2 pairs as uint64 fractions of 2^64
    (dl_rotary_frequencies). scaling: "none", "linear", "base" or "parts"."""
    if scaling not in _SCALING:
        raise ValueError(f"scaling: {scaling!r}, expected one of {', '.join(_SCALING)}")
    dim = int(dim)
    if not 2 <= dim <= DL_ROTARY_MAX_DIM or dim % 2:
        raise ValueError(f"dim: {dim}, expected an even number from 2 to {DL_ROTARY_MAX_DIM}")
    turns = np.empty(dim // 2, dtype=np.uint64)
    _check("dl_rotary_frequencies", lib().dl_rotary_frequencies(
        dim, base, _SCALING[scaling], factor, context, low, high, turns.ctypes.data))
    return turns


class RotaryFrequencies:
    """A model's rotary table: turns per token of the pairs of a head's first
    ``dim`` elements, on the device, and the amplitude of the rotated pairs.

    base, scaling, factor, context, low, high: as rotary_frequencies takes
    them. amplitude: of cos and sin (1, or what a scaling for long contexts
    prescribes). frequencies: radians per token of every pair (a sequence or
    host array, each at least 0 and below 2 pi) in place of the formulas."""

    def __init__(self, dim, base=10000.0, scaling="none", factor=1.0, context=0.0, low=1.0,
                 high=4.0, amplitude=1.0, frequencies=None, device="cuda"):
        self.dim, self.amplitude = int(dim), float(amplitude)
        if not abs(self.amplitude) <= _FLT_MAX:
            raise ValueError(f"amplitude: {amplitude}, must be finite in float32")
        turns = rotary_frequencies(dim, base, scaling, factor, context, low, high)
        if frequencies is not None:
            f = np.asarray(frequencies, dtype=np.float64)
            if f.shape != turns.shape:
                raise ValueError(f"frequencies: shape {f.shape}, expected {turns.shape}")
            if not ((f >= 0) & (f < 2 * math.pi)).all():
                raise ValueError("frequencies: must be at least 0 and below 2 pi")
            turns = np.array([round(x / (2 * math.pi) * 2.0**64) & (2**64 - 1)
                              for x in f.tolist()], dtype=np.uint64)
        self.turns = torch.from_numpy(turns.view(np.int64)).to(device)
        self.device = self.turns.device


def _refuse_heads(t, name, like):
    """The error of a tensor that _heads does not take."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in _TYPE or t.dtype is not like.dtype:
        want = like.dtype if like is not t else "float32, bfloat16 or float16"
        raise TypeError(f"{name}: dtype {t.dtype}, expected {want}")
    if t.dim() not in (3, 4):
        raise ValueError(f"{name}: {t.dim()} dimensions, expected [batch, tokens, heads, "
                         "head_dim] or [tokens, heads, head_dim]")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    raise ValueError(f"{name}: shape {tuple(t.shape)} does not go with {tuple(like.shape)}")


def _heads(t, name, i, like, shape):
    """Strides (batch, token, head, ...) of [batch][tokens][heads][head_dim],
    which must go with `like` of that shape; a tensor of three dimensions has a
    batch of one. name and i name it where it does not."""
    if isinstance(t, torch.Tensor) and t.dtype is like.dtype and t.dtype in _TYPE:
        d, s = t.shape, t.stride()
        if len(d) == len(shape) and d[-1] == shape[-1] and (s[-1] == 1 or d[-1] == 1):
            if len(d) == 4:
                if d[1] == shape[1] and d[0] == shape[0]:
                    return s
            elif len(d) == 3 and d[0] == shape[0]:
                return (0, *s)
    _refuse_heads(t, f"{name}[{i}]", like)


def _positions(positions, batch, tokens):
    """(tensor kept alive, type code, stride between batches) of the positions."""
    if not isinstance(positions, torch.Tensor):
        raise TypeError(f"positions: expected a torch.Tensor, got {type(positions).__name__}")
    if positions.dtype not in _INDEX:
        raise TypeError(f"positions: dtype {positions.dtype}, expected int32 or int64")
    shape = positions.shape
    if shape not in ((tokens,), (1, tokens), (batch, tokens)):
        raise ValueError(f"positions: shape {tuple(shape)}, expected ({tokens},) or "
                         f"({batch}, {tokens})")
    if tokens > 1 and positions.stride(-1) != 1:
        positions = positions.contiguous()
    stride = positions.stride(0) if len(shape) == 2 and shape[0] > 1 else 0
    return positions, _INDEX[positions.dtype], stride


def rotary_apply(xs, frequencies, positions=None, first=0, interleaved=False, inverse=False,
                 out=None, stream=None):
    """Rotary positions of a tensor or of up to four together (dl_rotary_apply).

    xs: [batch, tokens, heads, head_dim] or [tokens, heads, head_dim], of one
    type (float32, bfloat16 or float16), batch, tokens and head_dim; any
    strides with a contiguous last dimension, so heads before tokens are
    x.transpose(1, 2) and parts of a fused product slices of it.
    frequencies: a RotaryFrequencies; its dim elements of a head are rotated,
    the others copied. positions: int32 or int64, [batch, tokens] or [tokens];
    without them token s of every sequence is at first + s. inverse: by the
    negative angle (the gradient). out: where to write (xs themselves for in
    place). Returns a tensor for a tensor, a tuple for a sequence. Autograd
    records neither the call nor what it writes into out; rotary is for that."""
    single = isinstance(xs, torch.Tensor)
    xs = (xs,) if single else tuple(xs)
    if not 1 <= len(xs) <= DL_ROTARY_MAX_JOBS:
        raise ValueError(f"xs: {len(xs)} tensors, expected 1 to {DL_ROTARY_MAX_JOBS}")
    x0 = xs[0]
    if not isinstance(x0, torch.Tensor):
        _refuse_heads(x0, "xs[0]", x0)
    device = x0.device
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream, device)):
            return rotary_apply(x0 if single else xs, frequencies, positions, first, interleaved,
                                inverse, out)
    at = x0.get_device()
    if _away(at):
        with torch.cuda.device(device):
            return rotary_apply(x0 if single else xs, frequencies, positions, first, interleaved,
                                inverse, out)
    if not isinstance(frequencies, RotaryFrequencies):
        raise TypeError(f"frequencies: expected RotaryFrequencies, got {type(frequencies).__name__}")
    shape, n = x0.shape, len(xs)
    ys = None
    if out is not None:
        ys = (out,) if isinstance(out, torch.Tensor) else tuple(out)
        if len(ys) != n:
            raise ValueError(f"out: {len(ys)} tensors for {n}")
    jobs = (_RotaryJob * n)()
    turns = frequencies.turns
    here = turns.get_device() == at >= 0
    given = []
    for i, x in enumerate(xs):
        s = _heads(x, "xs", i, x0, shape)
        heads = x.shape[-2]
        if ys is None:
            y = torch.empty_like(x)
            r = y.stride()
            if r[-1] != 1:  # windows that overlap may come back in another order
                y = torch.empty(x.shape, dtype=x.dtype, device=device)
                r = y.stride()
            if len(r) == 3:
                r = (0, *r)
        else:
            y = ys[i]
            r = _heads(y, "out", i, x0, shape)
            if y.shape[-2] != heads:
                raise ValueError(f"out[{i}]: shape {tuple(y.shape)}, expected {tuple(x.shape)}")
            here = here and y.get_device() == at
        here = here and x.get_device() == at
        if heads >= 2**31:
            _int32(heads, "heads")
        jobs[i] = (x.data_ptr(), y.data_ptr(), s[0], s[1], s[2], r[0], r[1], r[2], heads)
        given.append(y)
    ys = tuple(given)
    batch, tokens, width = shape[0] if len(shape) == 4 else 1, shape[-3], _int32(shape[-1], "head_dim")
    if width < frequencies.dim:
        raise ValueError(f"xs[0]: heads of {width} elements, frequencies rotate {frequencies.dim}")
    pp, ptype, pstride = None, DL_I64, 0
    if positions is not None:
        positions, ptype, pstride = _positions(positions, batch, tokens)
        pp = positions.data_ptr()
        here = here and positions.get_device() == at
    elif not -2**63 <= first < 2**63:
        raise ValueError(f"first: {first} does not fit 64 bits")
    if not here:
        _cuda(*xs, *ys, turns, positions)
        _one_device(*xs, *ys, turns, positions)
    flags = (DL_ROTARY_INTERLEAVED if interleaved else 0) | (DL_ROTARY_INVERSE if inverse else 0)
    st = lib().dl_rotary_apply(jobs, n, _TYPE[x0.dtype], batch, tokens, width, frequencies.dim,
                               turns.data_ptr(), frequencies.amplitude, pp, ptype, pstride, first,
                               flags, _on(None, device))
    if st:
        raise DLError("dl_rotary_apply", st)
    return ys[0] if single else ys


class _Rotary(torch.autograd.Function):
    """A rotation is linear: its gradient is the rotation back, which may be
    differentiated in its turn."""

    @staticmethod
    def forward(ctx, frequencies, positions, first, interleaved, inverse, *xs):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(positions)
        ctx.how = frequencies, first, interleaved, inverse
        return rotary_apply(xs, frequencies, positions, first, interleaved, inverse)

    @staticmethod
    def backward(ctx, *dys):
        frequencies, first, interleaved, inverse = ctx.how
        positions, = ctx.saved_tensors
        # outputs that nothing used have no gradient, and some inputs need none
        asked = [dy is not None and need for dy, need in zip(dys, ctx.needs_input_grad[5:])]
        # a broadcast gradient may have any stride
        given = [dy if dy.stride(-1) == 1 else dy.contiguous() for dy, ask in zip(dys, asked) if ask]
        dxs = iter(_Rotary.apply(frequencies, positions, first, interleaved, not inverse, *given)
                   if given else ())
        return (None,) * 5 + tuple([next(dxs) if ask else None for ask in asked])


def rotary(xs, frequencies, positions=None, first=0, interleaved=False):
    """rotary_apply as a torch.autograd operation: a tensor or a sequence of up
    to four (queries and keys) turned by their positions, into new tensors."""
    if isinstance(xs, torch.Tensor):
        return _Rotary.apply(frequencies, positions, first, interleaved, False, xs)[0]
    return _Rotary.apply(frequencies, positions, first, interleaved, False, *xs)


# ----------------------------------------------------------------------------
# token log probabilities


class LogProbs(NamedTuple):
    """What logprobs_forward computed; None for what was not asked for.
    statistics: [2, ...], the rows' row_max and log_sum for logprobs_backward."""
    logp: Optional[torch.Tensor]
    lse: torch.Tensor
    entropy: Optional[torch.Tensor]
    top_tokens: Optional[torch.Tensor]
    top_logp: Optional[torch.Tensor]
    statistics: torch.Tensor

    @property
    def row_max(self):
        return self.statistics[0]

    @property
    def log_sum(self):
        return self.statistics[1]


class TokenLogProbs(NamedTuple):
    """The outputs of token_logprobs; None for what was not asked for."""
    logp: Optional[torch.Tensor]
    lse: torch.Tensor
    entropy: Optional[torch.Tensor]
    top_tokens: Optional[torch.Tensor]
    top_logp: Optional[torch.Tensor]


def _tokens(tokens, shape):
    """Type code of the rows' tokens."""
    if not isinstance(tokens, torch.Tensor):
        raise TypeError(f"tokens: expected a torch.Tensor, got {type(tokens).__name__}")
    if tokens.dtype not in _INDEX:
        raise TypeError(f"tokens: dtype {tokens.dtype}, expected int32 or int64")
    if tokens.shape != shape:
        raise ValueError(f"tokens: shape {tuple(tokens.shape)}, expected {tuple(shape)}")
    return _INDEX[tokens.dtype]


def _per_row(t, shape, name, dtypes=_F32):
    """A contiguous tensor of a value (or of the alternatives) per row."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtypes[0]}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _all_on(at, *tensors):
    """Refuses tensors of the host or of another device than index `at`."""
    for t in tensors:
        if t is not None and t.get_device() != at:
            at = -1
    if at < 0:
        _cuda(*tensors)
        _one_device(*tensors)


def logprobs_forward(logits, tokens=None, top=0, entropy=False, stream=None):
    """Log probabilities over the last dimension of logits (dl_logprobs_forward).

    logits: float32, bfloat16 or float16, [..., vocabulary]; leading dimensions
    that fold into rows, the last one contiguous. tokens: int32 or int64 of the
    leading shape, or None for no logp; a negative token leaves its row out
    (outputs 0, not read). top: how many of the most probable tokens (up to 32)
    to return with their log probabilities; -1 and -inf past the possible ones.
    entropy: whether to compute it. Returns LogProbs, its fields float32 of the
    leading shape (top_tokens int64 and top_logp with a last dimension of top)."""
    zp, zs = _rows(logits, "logits")
    device = logits.device
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream, device)):
            return logprobs_forward(logits, tokens, top, entropy)
    at = logits.get_device()
    if _away(at):
        with torch.cuda.device(device):
            return logprobs_forward(logits, tokens, top, entropy)
    lead, vocab = logits.shape[:-1], logits.shape[-1]
    rows = logits.numel() // vocab
    if not 0 <= top <= DL_LOGPROBS_MAX_TOP:
        raise ValueError(f"top: {top}, expected 0 to {DL_LOGPROBS_MAX_TOP}")
    ttype = DL_I64
    if tokens is not None:
        ttype = _tokens(tokens, lead)
        if not tokens.is_contiguous():
            tokens = tokens.contiguous()
    _all_on(at, logits, tokens)
    lse = torch.empty(lead, dtype=torch.float32, device=device)
    # both statistics in one allocation; what a caller may change in place has its own
    statistics = torch.empty((2, *lead), dtype=torch.float32, device=device)
    sp = statistics.data_ptr()
    logp = torch.empty_like(lse) if tokens is not None else None
    h = torch.empty_like(lse) if entropy else None
    top_tokens = top_logp = None
    if top:
        top_tokens = torch.empty((*lead, top), dtype=torch.int64, device=device)
        top_logp = torch.empty((*lead, top), dtype=torch.float32, device=device)
    st = lib().dl_logprobs_forward(zp, zs, _TYPE[logits.dtype], rows, vocab, _at(tokens), ttype,
                                   _at(logp), _at(h), lse.data_ptr(), top, _at(top_tokens),
                                   _at(top_logp), sp, sp + 4 * rows, _on(None, device))
    if st:
        raise DLError("dl_logprobs_forward", st)
    return LogProbs(logp, lse, h, top_tokens, top_logp, statistics)


def logprobs_backward(logits, tokens, row_max, log_sum, d_logp=None, d_entropy=None, d_lse=None,
                      entropy=None, top_tokens=None, d_top=None, out=None, stream=None):
    """The logits' gradient (dl_logprobs_backward) from the statistics of
    logprobs_forward and the gradients of its outputs, contiguous float32, any
    of them None. entropy: the forward call's, with d_entropy. top_tokens:
    the forward call's, with d_top. out: where to write, logits themselves for
    in place (unseen by autograd). A row whose gradients are all zero gets zeros
    and is not read."""
    zp, zs = _rows(logits, "logits")
    device = logits.device
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream, device)):
            return logprobs_backward(logits, tokens, row_max, log_sum, d_logp, d_entropy, d_lse,
                                     entropy, top_tokens, d_top, out)
    at = logits.get_device()
    if _away(at):
        with torch.cuda.device(device):
            return logprobs_backward(logits, tokens, row_max, log_sum, d_logp, d_entropy, d_lse,
                                     entropy, top_tokens, d_top, out)
    lead, vocab = logits.shape[:-1], logits.shape[-1]
    rows = logits.numel() // vocab
    ttype = DL_I64
    if tokens is not None:
        ttype = _tokens(tokens, lead)
        if not tokens.is_contiguous():
            tokens = tokens.contiguous()
    elif d_logp is not None:
        raise ValueError("d_logp: needs the tokens")
    if row_max is None or log_sum is None:
        raise ValueError("row_max, log_sum: missing")
    if d_entropy is not None and entropy is None:
        raise ValueError("d_entropy: needs the entropy")
    for t, name in ((row_max, "row_max"), (log_sum, "log_sum"), (d_logp, "d_logp"),
                    (d_entropy, "d_entropy"), (d_lse, "d_lse"), (entropy, "entropy")):
        _per_row(t, lead, name)
    top = 0
    if d_top is not None:
        if top_tokens is None:
            raise ValueError("d_top: needs the top_tokens")
        top = top_tokens.shape[-1] if top_tokens.dim() else 0
        if not 0 <= top <= DL_LOGPROBS_MAX_TOP:
            raise ValueError(f"top_tokens: {top} of a row, at most {DL_LOGPROBS_MAX_TOP}")
        _per_row(top_tokens, (*lead, top), "top_tokens", _I64)
        _per_row(d_top, (*lead, top), "d_top")
    if out is None:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=device)
    yp, ys = _rows(out, "out", logits)
    tops = (top_tokens, d_top) if top else (None, None)
    _all_on(at, logits, tokens, row_max, log_sum, d_logp, d_entropy, d_lse, entropy, out, *tops)
    st = lib().dl_logprobs_backward(
        zp, zs, _TYPE[logits.dtype], rows, vocab, _at(tokens), ttype, row_max.data_ptr(),
        log_sum.data_ptr(), _at(entropy), _at(d_logp), _at(d_entropy), _at(d_lse), top,
        _at(tops[0]), _at(tops[1]), yp, ys, _on(None, device))
    if st:
        raise DLError("dl_logprobs_backward", st)
    return out


class _TokenLogProbsGradient(torch.autograd.Function):
    """logprobs_backward in a graph that may be differentiated again
    (create_graph=True): a second derivative is an error, not a silent zero."""

    @staticmethod
    def forward(ctx, logits, tokens, row_max, log_sum, d_logp, d_entropy, d_lse, entropy, top_tokens,
                d_top):
        return logprobs_backward(logits, tokens, row_max, log_sum, d_logp, d_entropy, d_lse,
                                 entropy, top_tokens, d_top)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("token_logprobs: second derivatives are not implemented")


class _TokenLogProbs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, top, entropy):
        r = logprobs_forward(logits, tokens, top, entropy)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(logits, tokens, r.statistics, r.entropy, r.top_tokens)
        if top:
            ctx.mark_non_differentiable(r.top_tokens)
        return r.logp, r.lse, r.entropy, r.top_tokens, r.top_logp

    @staticmethod
    def backward(ctx, d_logp, d_lse, d_entropy, _, d_top):
        logits, tokens, statistics, entropy, top_tokens = ctx.saved_tensors
        # broadcast gradients (as of a mean) have one value for every row
        d_logp, d_lse, d_entropy, d_top = (
            None if d is None else d.contiguous() for d in (d_logp, d_lse, d_entropy, d_top))
        args = (logits, tokens, *statistics.unbind(0), d_logp, d_entropy, d_lse, entropy,
                top_tokens, d_top)
        if torch.is_grad_enabled():
            dz = _TokenLogProbsGradient.apply(*args)
        else:
            dz = logprobs_backward(*args)
        return dz, None, None, None


def token_logprobs(logits, tokens=None, top=0, entropy=False):
    """logprobs_forward as a torch.autograd operation: TokenLogProbs, with
    gradients of logp, lse, entropy and top_logp. First derivatives only:
    differentiating its gradients again (create_graph=True) raises. The logits
    are kept for the backward pass and must not change before it."""
    return TokenLogProbs(*_TokenLogProbs.apply(logits, tokens, top, entropy))
