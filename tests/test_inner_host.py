"""The inner-step entry points on the host (no GPU): refusals of the C ABI
before any launch, the binding's own checks, scale slots, and the reference
that the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import inner_ref as ref
import pseudo_grad_sync_gb300 as dl
from pseudo_grad_sync_gb300 import _build, inner

FAKE = 1 << 20  # a 256-byte aligned device address that is never dereferenced


@pytest.fixture(scope="module")
def L():
    _build.build()
    return dl.lib()


def _frag(numels):
    off = np.concatenate([[0], np.cumsum(numels)]).astype(np.int64)
    return dl._Fragment(off.ctypes.data, FAKE, len(numels)), off


# ----------------------------------------------------------------------------
# C ABI


def test_grad_norm_refusals(L):
    ws = L.dl_grad_norm_workspace_bytes()
    assert ws > 256
    ptrs, n = (ctypes.c_void_p * 2)(FAKE, FAKE), (ctypes.c_int64 * 2)(4, 4)

    def call(p=ptrs, k=n, count=2, kind=0, max_norm=1.0, out=FAKE, w=FAKE, nbytes=ws):
        return L.dl_grad_norm(p, k, count, kind, max_norm, out, w, nbytes, None)
    assert call(count=-1) == -1 and call(p=None) == -1 and call(k=None) == -1
    assert call(kind=2) == -1 and call(kind=3) == -1          # fp16 and e4m3 gradients
    assert call(max_norm=0.0) == -1 and call(max_norm=-1.0) == -1 and call(max_norm=math.nan) == -1
    assert call(out=None) == -1 and call(out=FAKE + 2) == -2
    assert call(k=(ctypes.c_int64 * 2)(4, -1)) == -1
    assert call(p=(ctypes.c_void_p * 2)(FAKE, None)) == -1
    assert call(p=(ctypes.c_void_p * 2)(FAKE, FAKE + 2)) == -2
    assert call(p=(ctypes.c_void_p * 2)(FAKE, FAKE + 1), kind=1) == -2
    assert call(w=None) == -6 and call(nbytes=ws - 1) == -6 and call(w=FAKE + 128) == -2


def _job(numels, **put):
    f, off = _frag(numels)
    job = (inner._AdamWJob * 1)()
    job[0].frag = ctypes.pointer(f)
    for k in ("theta", "grad", "m", "v", "m_scale", "v_scale"):
        setattr(job[0], k, FAKE)
    for k, v in put.items():
        setattr(job[0], k, v)
    return job, (f, off)


def _adamw(L, job, n=1, gtype=0, stype=0, clip=None, **put):
    c = inner._AdamWConfig(1e-3, 0.9, 0.95, 1e-8, 0.1, 1, 0)
    for k, v in put.items():
        setattr(c, k, v)
    return L.dl_adamw_step(job, n, gtype, stype, ctypes.byref(c), clip, None)


def test_adamw_refusals(L):
    job, keep = _job([10, 20])
    assert _adamw(L, job, n=-1) == -1 and _adamw(L, None) == -1
    assert _adamw(L, job, gtype=2) == -1 and _adamw(L, job, gtype=3) == -1
    assert _adamw(L, job, stype=1) == -1 and _adamw(L, job, stype=2) == -1
    assert L.dl_adamw_step(job, 1, 0, 0, None, None, None) == -1
    for bad in ({"lr": -1.0}, {"lr": math.nan}, {"lr": math.inf}, {"beta1": 1.0}, {"beta1": -0.1},
                {"beta2": 1.0}, {"beta2": math.nan}, {"eps": 0.0}, {"eps": 1e-40},
                {"eps": math.nan}, {"weight_decay": -1.0}, {"weight_decay": math.inf},
                {"lr": 1e30, "weight_decay": 1e30}, {"lr": 1e38}, {"step": 0}, {"step": -5}):
        assert _adamw(L, job, **bad) == -1, bad
    assert _adamw(L, job, clip=FAKE + 2) == -2
    for k in ("theta", "grad", "m", "v"):
        job, keep = _job([10, 20], **{k: None})
        assert _adamw(L, job) == -1, k
        job, keep = _job([10, 20], **{k: FAKE + 4})
        assert _adamw(L, job) == -2, k
    for k in ("m_scale", "v_scale"):
        job, keep = _job([10, 20], **{k: None})
        assert _adamw(L, job, stype=3) == -1, k
        job, keep = _job([10, 20], **{k: FAKE + 2})
        assert _adamw(L, job, stype=3) == -2, k
    job, keep = _job([10, 20], theta_bf16=FAKE + 2)
    assert _adamw(L, job) == -2
    job, keep = _job([10, 20], d_decay=FAKE + 2)
    assert _adamw(L, job) == -2
    job, keep = _job([10, 20])
    keep[1][1] = 40  # decreasing offsets
    assert _adamw(L, job) == -5
    assert L.dl_adamw_scale_slots(job[0].frag) == -5
    # nothing to do: no launch, whatever the pointers
    job, keep = _job([0, 0], theta=None, grad=None, m=None, v=None)
    assert _adamw(L, job) == 0 and _adamw(L, job, n=0) == 0 and _adamw(L, None, n=0) == 0


def test_layernorm_refusals(L):
    def fwd(x=FAKE, xs=64, kind=1, rows=4, width=64, w=FAKE, b=None, pt=0, eps=1e-5, flags=0,
            y=FAKE, ys=64, mean=FAKE, rstd=FAKE):
        return L.dl_layernorm_forward(x, xs, kind, rows, width, w, b, pt, eps, flags, y, ys, mean,
                                      rstd, None)
    for bad in ({"kind": 3}, {"kind": -1}, {"pt": 2}, {"rows": -1}, {"width": 0}, {"xs": 63},
                {"ys": 63}, {"eps": -1.0}, {"eps": math.nan}, {"eps": math.inf}, {"flags": 2},
                {"flags": 4}, {"x": None}, {"y": None}, {"w": None}, {"mean": None},
                {"rstd": None}):
        assert fwd(**bad) == -1, bad
    for bad in ({"x": FAKE + 1}, {"y": FAKE + 1}, {"w": FAKE + 2}, {"b": FAKE + 2},
                {"b": FAKE + 1, "pt": 1}, {"mean": FAKE + 2}, {"rstd": FAKE + 2},
                {"x": FAKE + 2, "kind": 0}):
        assert fwd(**bad) == -2, bad
    assert fwd(rows=0, x=None, y=None, w=None, mean=None, rstd=None) == 0
    assert L.dl_layernorm_workspace_bytes(-1, 64) == 0 and L.dl_layernorm_workspace_bytes(4, 0) == 0
    ws = L.dl_layernorm_workspace_bytes(4, 64)

    def bwd(dy=FAKE, ds=64, x=FAKE, xs=64, kind=1, rows=4, width=64, w=FAKE, pt=0, mean=FAKE,
            rstd=FAKE, flags=0, dx=FAKE, os=64, dw=FAKE, db=None, work=FAKE, nbytes=ws):
        return L.dl_layernorm_backward(dy, ds, x, xs, kind, rows, width, w, pt, mean, rstd, flags,
                                       dx, os, dw, db, work, nbytes, None)
    for bad in ({"kind": 3}, {"pt": 2}, {"rows": -1}, {"width": 0}, {"ds": 63}, {"xs": 63},
                {"os": 63}, {"flags": 4}, {"dy": None}, {"x": None}, {"dx": None}, {"w": None},
                {"mean": None}, {"rstd": None}, {"dw": None}):
        assert bwd(**bad) == -1, bad
    for bad in ({"dy": FAKE + 1}, {"x": FAKE + 1}, {"dx": FAKE + 1}, {"w": FAKE + 2},
                {"dw": FAKE + 2}, {"db": FAKE + 2}, {"mean": FAKE + 2}, {"rstd": FAKE + 2},
                {"work": FAKE + 16}):
        assert bwd(**bad) == -2, bad
    assert bwd(work=None) == -6 and bwd(nbytes=ws - 1) == -6


# ----------------------------------------------------------------------------
# binding


def test_binding_checks_before_any_call(L):
    F = dl.Fragment([100, 28], device="cpu")
    f32, e4 = torch.zeros(128), torch.zeros(128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    slots = dl.adamw_scale_slots(F)
    assert slots == 128 // 128 + 2
    sc = torch.zeros(slots)
    with pytest.raises(TypeError, match=r"grads\[0\]: dtype"):
        dl.grad_norm([f32.half()])
    with pytest.raises(TypeError, match=r"grads\[1\]: dtype"):
        dl.grad_norm([f32, f32.bfloat16()])
    with pytest.raises(ValueError, match="must be contiguous"):
        dl.grad_norm([torch.zeros(64)[::2]])
    with pytest.raises(ValueError, match="CUDA device"):
        dl.grad_norm([f32])
    with pytest.raises(ValueError, match="empty list"):
        dl.grad_norm([])
    J = dl.AdamWJobs
    with pytest.raises(TypeError, match=r"grad\[0\]: dtype"):
        J([F], [f32], [f32.half()], [f32], [f32])
    with pytest.raises(TypeError, match=r"m\[0\]: dtype"):
        J([F], [f32], [f32], [f32.half()], [f32])
    with pytest.raises(TypeError, match=r"v\[0\]: dtype"):
        J([F], [f32], [f32], [e4], [f32], [sc], [sc])
    with pytest.raises(ValueError, match=r"m_scale\[0\]: missing"):
        J([F], [f32], [f32], [e4], [e4])
    with pytest.raises(ValueError, match=r"v_scale\[0\]: .* need at least 3"):
        J([F], [f32], [f32], [e4], [e4], [sc], [sc[:2]])
    with pytest.raises(ValueError, match=r"theta\[0\]: 127 elements"):
        J([F], [f32[:127]], [f32], [f32], [f32])
    with pytest.raises(ValueError, match="theta: 1 buffers for 2 fragments"):
        J([F, F], [f32], [f32, f32], [f32, f32], [f32, f32])
    with pytest.raises(ValueError, match=r"decay\[0\]: .* need at least 2"):
        J([F], [f32], [f32], [f32], [f32], decay=[torch.zeros(1)])
    with pytest.raises(ValueError, match="CUDA device"):
        J([F], [f32], [f32], [f32], [f32])
    with pytest.raises(ValueError, match="bits: 16"):
        dl.InnerAdamW([F], [f32], [f32], bits=16)


def test_layernorm_binding_checks(L):
    x, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(TypeError, match="x: dtype"):
        dl.layernorm_forward(x.double(), w)
    with pytest.raises(TypeError, match="weight: dtype"):
        dl.layernorm_forward(x, w.half())
    with pytest.raises(ValueError, match="weight: expected 64 elements"):
        dl.layernorm_forward(x, torch.ones(65))
    with pytest.raises(TypeError, match="bias: dtype"):
        dl.layernorm_forward(x, w, w.bfloat16())
    with pytest.raises(ValueError, match="last dimension must be contiguous"):
        dl.layernorm_forward(torch.zeros(64, 4).t(), w)
    with pytest.raises(ValueError, match="rows overlap"):
        dl.layernorm_forward(torch.zeros(1, 64).expand(4, 64), w)
    with pytest.raises(ValueError, match="do not fold"):
        dl.layernorm_forward(torch.zeros(4, 3, 64)[:, :2], w)
    with pytest.raises(ValueError, match="last dimension is empty"):
        dl.layernorm_forward(torch.zeros(4, 0), w)
    with pytest.raises(ValueError, match="y: shape"):
        dl.layernorm_forward(x, w, y=torch.zeros(4, 65))
    with pytest.raises(ValueError, match="CUDA device"):
        dl.layernorm_forward(x, w)
    r = torch.zeros(4)
    with pytest.raises(TypeError, match="dy: dtype"):
        dl.layernorm_backward(x.half(), x, w, r, r)
    with pytest.raises(ValueError, match="mean: missing"):
        dl.layernorm_backward(x, x, w, None, r)
    with pytest.raises(ValueError, match="rstd: 3 elements"):
        dl.layernorm_backward(x, x, w, r, r[:3])
    with pytest.raises(ValueError, match="accumulate"):
        dl.layernorm_backward(x, x, w, r, r, accumulate=True)
    with pytest.raises(TypeError, match="dweight: dtype"):
        dl.layernorm_backward(x, x, w, r, r, w.bfloat16())
    with pytest.raises(ValueError, match="CUDA device"):
        dl.layernorm_backward(x, x, w, r, r)


def test_scale_slots_cover_every_block_once(L):
    rng = np.random.default_rng(0)
    for _ in range(200):
        numels = [int(x) for x in rng.integers(0, 600, rng.integers(0, 12))]
        f, off = _frag(numels)
        slots = L.dl_adamw_scale_slots(ctypes.byref(f))
        assert slots == ref.slots_of(numels)
        seen = set()
        for _, a, b, s in ref.spans(numels):
            for k in range(-(-(b - a) // ref.BLOCK)):
                assert 0 <= s + k < slots and s + k not in seen
                seen.add(s + k)


# ----------------------------------------------------------------------------
# the reference itself


def test_reference_rounding_is_e4m3_and_unbiased():
    vals = ref.E4M3[:127]
    assert vals[0] == 0 and vals[126] == 448 and np.all(np.diff(vals) > 0)
    # torch reads the same values
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(t[:127], vals.astype(np.float32))
    assert np.array_equal(t[128:255], -vals.astype(np.float32))
    # an exact value keeps its code whatever the bits; between two codes the
    # upper one is taken in exactly the fraction's share of the 2^16 bits
    r = np.arange(65536, dtype=np.uint32)
    for c in (0, 1, 7, 8, 9, 63, 100, 126):
        assert np.all(ref.encode(np.full(65536, vals[c], np.float32), r) == c)
        if c < 126:
            for k in (1, 777, 32768, 65535):
                x = vals[c] + (vals[c + 1] - vals[c]) * (k / 65536)
                up = ref.encode(np.full(65536, x, np.float32), r) == c + 1
                assert up.sum() == k
    assert np.all(ref.encode(np.float32([449, 1e30]), np.uint32([0, 0])) == 126)
    assert np.all(ref.encode(np.float32([-448, -0.0]), np.uint32([9, 9])) == [254, 128])


def test_reference_adamw_against_torch():
    """The 64-bit reference against torch's own AdamW in double precision."""
    rng = np.random.default_rng(1)
    p = torch.tensor(rng.standard_normal(50), dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    th, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for step in range(1, 6):
        g = rng.standard_normal(50)
        p.grad = torch.tensor(g)
        opt.step()
        th, m, v, _ = ref.adamw64(th, g, m, v, [50], step, 1e-2, 0.9, 0.95, 1e-8, 0.1)
        assert np.allclose(th, p.detach().numpy(), rtol=1e-12, atol=1e-14)


def test_reference_norms_against_torch_autograd():
    rng = np.random.default_rng(2)
    x, w, b = (torch.tensor(rng.standard_normal(s), dtype=torch.float64, requires_grad=True)
               for s in ((4, 9), 9, 9))
    dy = torch.tensor(rng.standard_normal((4, 9)))
    y = torch.nn.functional.layer_norm(x, (9,), w, b, 1e-5)
    y.backward(dy)
    args = [t.detach().numpy() for t in (x, w, b)]
    yr, mean, rstd = ref.norm64(*args, 1e-5, False)
    dx, dw, db, _ = ref.norm64_backward(dy.numpy(), args[0], args[1], mean, rstd, False)
    for a, t in ((yr, y), (dx, x.grad), (dw, w.grad), (db, b.grad)):
        assert np.allclose(a, t.detach().numpy(), rtol=1e-12, atol=1e-13)
    x.grad = w.grad = None
    (x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-5) * w).backward(dy)
    yr, mean, rstd = ref.norm64(args[0], args[1], None, 1e-5, True)
    dx, dw, _, _ = ref.norm64_backward(dy.numpy(), args[0], args[1], mean, rstd, True)
    assert np.allclose(dx, x.grad.numpy(), rtol=1e-12) and np.allclose(dw, w.grad.numpy(), rtol=1e-12)
