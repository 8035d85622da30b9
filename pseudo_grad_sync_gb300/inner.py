"""A learner's inner step: layer norms, gradient clipping and AdamW.

Argument marshalling of the inner-step entry points of libdiloco_sync.so under
their C names (imported into the package):

    grad_norm            global gradient norm and clip coefficient
    adamw_step           AdamW over every tensor of a list of fragments, with
                         states in 32 or in 8 bits
    layernorm_forward    layer norm (or RMS norm) of rows
    layernorm_backward   its input's and its parameters' gradients

``GradList`` and ``AdamWJobs`` check and marshal a list of buffers once, for a
program that steps the same buffers again and again. ``InnerAdamW`` bundles
the clip and the step with their states; ``layer_norm`` is the norm as a
torch.autograd operation.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import (Fragment, _cuda, _Fragment, _need, _need_all, _F32, _U8, DLError, lib,
               new_workspace)

DL_F32, DL_BF16, DL_F16, DL_E4M3 = 0, 1, 2, 3
DL_NORM_RMS = 1
DL_NORM_ACCUMULATE = 2
DL_ADAMW_BLOCK = 128

_TYPE = {torch.float32: DL_F32, torch.bfloat16: DL_BF16, torch.float16: DL_F16}
_GRADS = (torch.float32, torch.bfloat16)
_PARAMS = (torch.float32, torch.bfloat16)


# These calls run at every layer and step, some for microseconds: their own
# time counts. Handles are therefore taken as integers (the declared argument
# types convert them), and the current stream without making a Stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


# The library launches on the current device. A call whose buffers live on
# another one makes it current first (one comparison of indexes when not).


def _away(index):
    """Whether a GPU (its index; -1 for the host) is not the current one."""
    return index >= 0 and index != _current()


def _stream_of(stream, device):
    """stream, which must be one of a call's device."""
    if device.type == "cuda" and stream.device != device:
        raise ValueError(f"stream of {stream.device}, buffers on {device}")
    return stream


def _one_device(*items):
    """After _cuda: every tensor given (or in a list given) on one device."""
    first = None
    for it in items:
        for t in (it if isinstance(it, (list, tuple)) else [it]):
            if t is None:
                continue
            if first is None:
                first = t.device
            elif t.device != first:
                raise ValueError(f"tensors must be on one device, found {first} and {t.device}")
    return first


def _on(stream, device):
    """cudaStream_t of stream, or of the device's current stream."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None or device.index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return _raw_stream(device.index)


def _at(t):
    return None if t is None else t.data_ptr()


def _buffer(t, dtype, n, name, device):
    """_need and the device check of one buffer, for the frequent case."""
    if (type(t) is torch.Tensor and t.dtype is dtype and t.get_device() == device.index
            and t.numel() >= n and t.is_contiguous()):
        return
    _need(t, (dtype,), n, name)
    _cuda(t)
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, the other buffers on {device}")


class _AdamWJob(ctypes.Structure):
    _fields_ = [("frag", ctypes.POINTER(_Fragment))] + [
        (name, ctypes.c_void_p)
        for name in ("theta", "grad", "m", "v", "m_scale", "v_scale", "theta_bf16", "d_decay")]


class _AdamWConfig(ctypes.Structure):
    _fields_ = [(name, ctypes.c_double)
                for name in ("lr", "beta1", "beta2", "eps", "weight_decay")] + [
        ("step", ctypes.c_int64), ("seed", ctypes.c_uint64)]


def declare(L):
    """Argument and result types of the inner-step entry points."""
    vp, i32, i64, f64, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double,
                             ctypes.c_size_t)
    L.dl_grad_norm_workspace_bytes.restype = sz
    L.dl_grad_norm_workspace_bytes.argtypes = []
    L.dl_grad_norm.restype = ctypes.c_int
    L.dl_grad_norm.argtypes = [vp, vp, i32, i32, f64, vp, vp, sz, vp]
    L.dl_adamw_scale_slots.restype = i64
    L.dl_adamw_scale_slots.argtypes = [ctypes.POINTER(_Fragment)]
    L.dl_adamw_step.restype = ctypes.c_int
    L.dl_adamw_step.argtypes = [ctypes.POINTER(_AdamWJob), i32, i32, i32,
                                ctypes.POINTER(_AdamWConfig), vp, vp]
    L.dl_layernorm_forward.restype = ctypes.c_int
    L.dl_layernorm_forward.argtypes = [vp, i64, i32, i64, i32, vp, vp, i32, f64, i32, vp, i64, vp,
                                       vp, vp]
    L.dl_layernorm_workspace_bytes.restype = sz
    L.dl_layernorm_workspace_bytes.argtypes = [i64, i32]
    L.dl_layernorm_backward.restype = ctypes.c_int
    L.dl_layernorm_backward.argtypes = [vp, i64, vp, i64, i32, i64, i32, vp, i32, vp, vp, i32, vp,
                                        i64, vp, vp, vp, sz, vp]


# ----------------------------------------------------------------------------
# gradient norm


def grad_norm_workspace_bytes() -> int:
    return int(lib().dl_grad_norm_workspace_bytes())


class GradList:
    """Gradient buffers (contiguous, one element type), checked once."""

    def __init__(self, grads):
        self.grads = list(grads)
        dtype = self.grads[0].dtype if self.grads else torch.float32
        if dtype not in _GRADS:
            raise TypeError(f"grads[0]: dtype {dtype}, expected float32 or bfloat16")
        _need_all(self.grads, (dtype,), 0, "grads")
        _cuda(self.grads)
        self.device = _one_device(self.grads)  # None for an empty list
        self._index = -1 if self.device is None else self.device.index
        n = len(self.grads)
        self.type = _TYPE[dtype]
        self._ptrs = (ctypes.c_void_p * max(n, 1))(*[g.data_ptr() for g in self.grads])
        self._numel = (ctypes.c_int64 * max(n, 1))(*[g.numel() for g in self.grads])


def grad_norm(grads, max_norm=math.inf, out=None, workspace=None, stream=None):
    """Norm over all gradient buffers and the clip coefficient (dl_grad_norm).

    grads: a list of device tensors, or a ``GradList``. Returns ``out``, a
    device float32 tensor (norm, coefficient), the ``clip`` of adamw_step.
    workspace: of grad_norm_workspace_bytes(), zeroed when allocated
    (new_workspace); calls on different streams need their own."""
    G = grads if isinstance(grads, GradList) else GradList(grads)
    if G.device is None and out is None:
        raise ValueError("grad_norm: an empty list needs an out tensor")
    device = G.device or out.device
    if stream is not None:  # what is allocated here belongs to that stream
        with torch.cuda.stream(_stream_of(stream, device)):
            return grad_norm(G, max_norm, out, workspace)
    if _away(G._index if G._index >= 0 else out.get_device()):
        with torch.cuda.device(device):
            return grad_norm(G, max_norm, out, workspace)
    if out is None:
        out = torch.empty(2, dtype=torch.float32, device=device)
    if workspace is None:
        workspace = new_workspace(grad_norm_workspace_bytes(), device)
    _buffer(out, torch.float32, 2, "out", device)
    _buffer(workspace, torch.uint8, 0, "workspace", device)
    st = lib().dl_grad_norm(G._ptrs, G._numel, len(G.grads), G.type, max_norm, out.data_ptr(),
                            workspace.data_ptr(), workspace.numel(), _on(None, device))
    if st:
        raise DLError("dl_grad_norm", st)
    return out


# ----------------------------------------------------------------------------
# AdamW


def adamw_scale_slots(frag: Fragment) -> int:
    """Scale slots of a fragment's 8-bit states (dl_adamw_scale_slots)."""
    return int(lib().dl_adamw_scale_slots(frag.c))


class AdamWJobs:
    """The buffers of an AdamW step over a list of fragments, checked once.

    Per-fragment lists: theta (float32), grad (float32 or bfloat16), m and v
    (float32, or float8_e4m3fn with m_scale and v_scale, float32 of
    adamw_scale_slots(frag) elements), and optionally theta_bf16 (bfloat16
    copies that every step writes) and decay (device float32 [T] factors on
    the weight decay). Entries of the optional lists may be None."""

    def __init__(self, frags, theta, grad, m, v, m_scale=None, v_scale=None, theta_bf16=None,
                 decay=None):
        self.frags = list(frags)
        P = len(self.frags)
        lists = {"theta": theta, "grad": grad, "m": m, "v": v, "m_scale": m_scale,
                 "v_scale": v_scale, "theta_bf16": theta_bf16, "decay": decay}
        lists = {k: [None] * P if x is None else list(x) for k, x in lists.items()}
        for name, x in lists.items():
            if len(x) != P:
                raise ValueError(f"{name}: {len(x)} buffers for {P} fragments")
        gtype = next((g.dtype for g in lists["grad"] if g is not None), torch.float32)
        stype = next((s.dtype for s in lists["m"] if s is not None), torch.float32)
        if gtype not in _GRADS:
            raise TypeError(f"grad[0]: dtype {gtype}, expected float32 or bfloat16")
        if stype not in (torch.float32, torch.float8_e4m3fn):
            raise TypeError(f"m[0]: dtype {stype}, expected float32 or float8_e4m3fn")
        by8 = stype == torch.float8_e4m3fn
        self.grad_type, self.state_type = _TYPE[gtype], DL_E4M3 if by8 else DL_F32
        self._jobs = (_AdamWJob * max(P, 1))()
        for j, F in enumerate(self.frags):
            slots = adamw_scale_slots(F) if by8 else 0
            for name, dtypes, n, needed in (
                    ("theta", _F32, F.n, True), ("grad", (gtype,), F.n, True),
                    ("m", (stype,), F.n, True), ("v", (stype,), F.n, True),
                    ("m_scale", _F32, slots, by8), ("v_scale", _F32, slots, by8),
                    ("theta_bf16", (torch.bfloat16,), F.n, False), ("decay", _F32, F.T, False)):
                t = lists[name][j]
                if t is None and needed and F.n > 0:
                    raise ValueError(f"{name}[{j}]: missing")
                _need(t, dtypes, n, f"{name}[{j}]")
                setattr(self._jobs[j], "d_decay" if name == "decay" else name,
                        None if t is None else t.data_ptr())
            self._jobs[j].frag = ctypes.pointer(F._c)
        offsets = [F.d_offsets for F in self.frags]
        _cuda(*lists.values(), offsets)
        self.buffers = lists
        self._cfg = _AdamWConfig()
        self._cfg_ref = ctypes.byref(self._cfg)
        self.device = _one_device(*lists.values(), offsets) or torch.device(
            "cuda", torch.cuda.current_device())
        self._index = self.device.index


def adamw_step(jobs: AdamWJobs, step, lr=4e-4, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1,
               clip=None, seed=0, stream=None):
    """One AdamW step over every job, in place (dl_adamw_step). step counts
    from 1. clip: device float32 (norm, coefficient) as grad_norm returns it;
    a coefficient that is not finite skips the step on the device. seed: of
    the 8-bit states' rounding; it may stay the same over a run."""
    if _away(jobs._index):
        with torch.cuda.device(jobs.device):
            return adamw_step(jobs, step, lr, betas, eps, weight_decay, clip, seed, stream)
    if stream is not None:
        _stream_of(stream, jobs.device)
    if clip is not None:
        _buffer(clip, torch.float32, 2, "clip", jobs.device)
    c = jobs._cfg
    c.lr, (c.beta1, c.beta2), c.eps, c.weight_decay = lr, betas, eps, weight_decay
    c.step, c.seed = step, seed & (2**64 - 1)
    st = lib().dl_adamw_step(jobs._jobs, len(jobs.frags), jobs.grad_type, jobs.state_type,
                             jobs._cfg_ref, _at(clip), _on(stream, jobs.device))
    if st:
        raise DLError("dl_adamw_step", st)


class InnerAdamW:
    """AdamW over a learner's fragments with its states, clipping first.

    theta and grad: per-fragment lists of flat device buffers (a learner's
    replica and the gradients that its backward passes write); what lies behind
    a fragment's n elements is neither read nor written. bits: 32 or 8,
    the width of the states. max_norm: clip by the global gradient norm; a
    step whose gradients are not all finite is then skipped on the device
    (``steps`` still counts it). decay: per-fragment lists or arrays of T
    factors on the weight decay (0 for norms and biases). theta_bf16: buffers
    that receive a rounded copy of the parameters every step."""

    def __init__(self, frags, theta, grad, bits=32, lr=4e-4, betas=(0.9, 0.95), eps=1e-8,
                 weight_decay=0.1, decay=None, theta_bf16=None, max_norm=None, seed=0):
        if bits not in (32, 8):
            raise ValueError(f"bits: {bits}, expected 32 or 8")
        frags, theta, grad = list(frags), list(theta), list(grad)
        dev = theta[0].device
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.max_norm, self.seed, self.steps = max_norm, seed, 0
        dtype = torch.float32 if bits == 32 else torch.float8_e4m3fn

        def zeros(sizes, dt):  # e4m3's code 0 is the value 0
            return [torch.zeros(max(n, 1), dtype=torch.uint8 if dt == torch.float8_e4m3fn else dt,
                                device=dev).view(dt) for n in sizes]
        self.m, self.v = (zeros([F.n for F in frags], dtype) for _ in range(2))
        self.m_scale = self.v_scale = None
        if bits == 8:
            self.m_scale, self.v_scale = (zeros([adamw_scale_slots(F) for F in frags],
                                                torch.float32) for _ in range(2))
        if decay is not None:
            decay = [None if d is None else torch.as_tensor(d, dtype=torch.float32, device=dev)
                     for d in decay]
        self.jobs = AdamWJobs(frags, theta, grad, self.m, self.v, self.m_scale, self.v_scale,
                              theta_bf16, decay)
        # the norm of what is stepped: a buffer may be longer than its fragment
        self.grads = GradList([g.view(-1)[:F.n] for F, g in zip(frags, grad) if F.n])
        self.clip = torch.ones(2, dtype=torch.float32, device=dev)
        self.workspace = new_workspace(grad_norm_workspace_bytes(), dev)

    def step(self, lr=None, stream=None):
        """Clip (with max_norm) and step; returns ``clip``, the device tensor
        (norm, coefficient), or, without max_norm, None. The next step writes
        the same tensor: clone() what is to be kept. A call that raises is not
        counted."""
        clip = None
        if self.max_norm is not None:
            clip = grad_norm(self.grads, self.max_norm, self.clip, self.workspace, stream)
        adamw_step(self.jobs, self.steps + 1, self.lr if lr is None else lr, self.betas, self.eps,
                   self.weight_decay, clip, self.seed, stream)
        self.steps += 1
        return clip


# ----------------------------------------------------------------------------
# layer norm


def layernorm_workspace_bytes(rows: int, width: int) -> int:
    return int(lib().dl_layernorm_workspace_bytes(rows, width))


def _rows(t, name, like=None):
    """(device address, row stride) of rows of a last dimension with stride 1;
    the leading dimensions must fold into one."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in _TYPE or (like is not None and t.dtype is not like.dtype):
        want = like.dtype if like is not None else "float32, bfloat16 or float16"
        raise TypeError(f"{name}: dtype {t.dtype}, expected {want}")
    if like is not None and t.shape != like.shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(like.shape)}")
    if t.dim() == 0:
        raise ValueError(f"{name}: needs at least one dimension")
    width = t.shape[-1]
    if width < 1:
        raise ValueError(f"{name}: the last dimension is empty")
    if width >= 2**31:  # ctypes would pass its low 32 bits
        raise ValueError(f"{name}: a last dimension of {width}, at most 2^31 - 1")
    stride = width
    if not t.is_contiguous():
        if t.dim() != 2:
            try:
                t = t.view(-1, width)
            except RuntimeError:
                raise ValueError(f"{name}: the leading dimensions do not fold into rows") from None
        if t.stride(1) != 1 and width > 1:
            raise ValueError(f"{name}: the last dimension must be contiguous")
        if t.shape[0] > 1 and t.stride(0) < width:
            raise ValueError(f"{name}: rows overlap (stride {t.stride(0)}, width {width})")
        stride = max(t.stride(0), width)
    if not t.is_cuda:
        return None, stride  # refused by the caller, after its other checks
    return t.data_ptr(), stride


def _empty_like(x):
    """A contiguous tensor of x's shape and type."""
    return torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype,
                                                                     device=x.device)


def _params(weight, bias, width):
    """Type code of the parameters; their device is checked by the caller."""
    if not isinstance(weight, torch.Tensor) or weight.numel() != width:
        raise ValueError(f"weight: expected {width} elements")
    if weight.dtype not in _PARAMS or not weight.is_contiguous():
        _need(weight, _PARAMS, width, "weight")
    if bias is not None and (bias.dtype is not weight.dtype or bias.numel() < width
                             or not bias.is_contiguous()):
        _need(bias, (weight.dtype,), width, "bias")
    return _TYPE[weight.dtype]


def _stats(mean, rstd, rows, rms):
    """Checks of the rows' statistics; returns mean, or None for the RMS norm."""
    if rms:
        mean = None
    elif mean is None:
        raise ValueError("mean: missing (rms=False)")
    else:
        _need(mean, _F32, rows, "mean")
    _need(rstd, _F32, rows, "rstd")
    return mean


def layernorm_forward(x, weight, bias=None, eps=1e-5, rms=False, y=None, mean=None, rstd=None,
                      stream=None):
    """Layer norm over the last dimension (dl_layernorm_forward). Returns
    (y, mean, rstd), mean None with rms=True. x: float32, bfloat16 or float16
    with a contiguous last dimension; weight, bias: float32 or bfloat16."""
    xp, xs = _rows(x, "x")
    device = x.device
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream, device)):
            return layernorm_forward(x, weight, bias, eps, rms, y, mean, rstd)
    at = x.get_device()
    if _away(at):
        with torch.cuda.device(device):
            return layernorm_forward(x, weight, bias, eps, rms, y, mean, rstd)
    shape = x.shape
    width = shape[-1]
    rows = x.numel() // width
    ptype = _params(weight, bias, width)
    if y is None:
        y = _empty_like(x)
        yp, ys = (y.data_ptr() if xp is not None else None), width
    else:
        yp, ys = _rows(y, "y", x)
    given = rstd is not None or mean is not None
    if rstd is None:
        rstd = torch.empty(shape[:-1], dtype=torch.float32, device=device)
    if rms:
        mean = None
    elif mean is None:
        mean = torch.empty(shape[:-1], dtype=torch.float32, device=device)
    if given:
        mean = _stats(mean, rstd, rows, rms)
    if xp is None or not (
            y.get_device() == at and weight.get_device() == at and rstd.get_device() == at
            and (bias is None or bias.get_device() == at)
            and (mean is None or mean.get_device() == at)):
        _cuda(x, weight, bias, y, mean, rstd)
        _one_device(x, weight, bias, y, mean, rstd)
    st = lib().dl_layernorm_forward(xp, xs, _TYPE[x.dtype], rows, width, weight.data_ptr(),
                                    _at(bias), ptype, eps, DL_NORM_RMS if rms else 0, yp, ys,
                                    _at(mean), rstd.data_ptr(), _on(None, device))
    if st:
        raise DLError("dl_layernorm_forward", st)
    return y, mean, rstd


def layernorm_backward(dy, x, weight, mean, rstd, dweight=None, dbias=None, rms=False,
                       accumulate=False, dx=None, workspace=None, bias=True, stream=None):
    """Gradients of layernorm_forward (dl_layernorm_backward). Returns (dx,
    dweight, dbias). dweight and dbias may be slices of a fragment's flat
    gradient buffer; with accumulate=True the sums are added to what they
    hold. Without a dweight both are allocated (dbias only with bias=True);
    a call that passes dweight alone computes no dbias. A copy that timed out
    is reported by read_device_status(None), and by the workspace's status
    word when the caller passed one."""
    xp, xs = _rows(x, "x")
    device = x.device
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream, device)):
            return layernorm_backward(dy, x, weight, mean, rstd, dweight, dbias, rms, accumulate,
                                      dx, workspace, bias)
    at = x.get_device()
    if _away(at):
        with torch.cuda.device(device):
            return layernorm_backward(dy, x, weight, mean, rstd, dweight, dbias, rms, accumulate,
                                      dx, workspace, bias)
    dyp, ds = _rows(dy, "dy", x)
    width = x.shape[-1]
    rows = x.numel() // width
    ptype = _params(weight, None, width)
    if dweight is None:
        if accumulate:
            raise ValueError("accumulate: needs the dweight to add to")
        dweight = torch.empty(width, dtype=weight.dtype, device=device)
        if dbias is None and bias:
            dbias = torch.empty(width, dtype=weight.dtype, device=device)
    if dx is None:
        dx = _empty_like(x)
        dxp, os = (dx.data_ptr() if xp is not None else None), width
    else:
        dxp, os = _rows(dx, "dx", x)
    if workspace is None:
        workspace = torch.empty(layernorm_workspace_bytes(rows, width), dtype=torch.uint8,
                                device=device)
    mean = _stats(mean, rstd, rows, rms)
    _need(dweight, (weight.dtype,), width, "dweight")
    _need(dbias, (weight.dtype,), width, "dbias")
    _need(workspace, _U8, 0, "workspace")
    if xp is None or not (
            dy.get_device() == at and dx.get_device() == at and weight.get_device() == at
            and rstd.get_device() == at and dweight.get_device() == at
            and workspace.get_device() == at and (mean is None or mean.get_device() == at)
            and (dbias is None or dbias.get_device() == at)):
        _cuda(dy, x, weight, mean, rstd, dx, dweight, dbias, workspace)
        _one_device(dy, x, weight, mean, rstd, dx, dweight, dbias, workspace)
    flags = (DL_NORM_RMS if rms else 0) | (DL_NORM_ACCUMULATE if accumulate else 0)
    st = lib().dl_layernorm_backward(
        dyp, ds, xp, xs, _TYPE[x.dtype], rows, width, weight.data_ptr(), ptype, _at(mean),
        rstd.data_ptr(), flags, dxp, os, dweight.data_ptr(), _at(dbias), workspace.data_ptr(),
        workspace.numel(), _on(None, device))
    if st:
        raise DLError("dl_layernorm_backward", st)
    return dx, dweight, dbias


class _LayerNormGradient(torch.autograd.Function):
    """layernorm_backward in a graph that may be differentiated again
    (create_graph=True): a second derivative is an error, not a silent zero.
    Its inputs carry the history, so this holds for a constant dy too."""

    @staticmethod
    def forward(ctx, dy, x, weight, mean, rstd, rms, bias):
        return layernorm_backward(dy, x, weight, mean, rstd, rms=rms, bias=bias)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("layer_norm: second derivatives are not implemented")


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, rms):
        y, mean, rstd = layernorm_forward(x, weight, bias, eps, rms)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.rms, ctx.bias = rms, bias is not None
        ctx.shapes = weight.shape, None if bias is None else bias.shape
        return y

    @staticmethod
    def backward(ctx, dy):
        # a broadcast gradient (as of a sum) has rows that overlap
        args = (dy.contiguous(), *ctx.saved_tensors)
        if torch.is_grad_enabled():
            dx, dw, db = _LayerNormGradient.apply(*args, ctx.rms, ctx.bias)
        else:
            dx, dw, db = layernorm_backward(*args, rms=ctx.rms, bias=ctx.bias)
        w_shape, b_shape = ctx.shapes  # the parameters may have leading ones
        return dx, dw.view(w_shape), None if db is None else db.view(b_shape), None, None


def layer_norm(x, weight, bias=None, eps=1e-5, rms=False):
    """layernorm_forward as a torch.autograd operation. First derivatives only:
    differentiating its gradients again (create_graph=True) raises. It always
    takes a weight; parameters are float32 or bfloat16; x's leading dimensions
    must fold into rows that do not overlap (x.contiguous() where not)."""
    if bias is not None and bias.numel() != weight.numel():  # its gradient would not fit it
        raise ValueError(f"bias: {bias.numel()} elements, expected {weight.numel()}")
    return _LayerNorm.apply(x, weight, bias, eps, rms)
