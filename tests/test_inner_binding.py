"""The inner-step binding on the host (no GPU): sizes that do not fit the ABI's
arguments, what it passes on, and the autograd operation with the two norm
calls replaced by their formulas in torch."""
import ctypes

import pytest
import torch

import pseudo_grad_sync_gb300 as dl
from pseudo_grad_sync_gb300 import _build, inner


@pytest.fixture(scope="module", autouse=True)
def library():
    _build.build()
    return dl.lib()


def test_widths_beyond_the_abi_are_refused():
    """A 32-bit width would be cut: 2^32 + 64 columns taken as 64."""
    for width in (2**31, 2**32 + 64):
        x, w = (torch.empty(s, dtype=torch.bfloat16, device="meta") for s in ((2, width), (width,)))
        r = torch.empty(2, device="meta")
        with pytest.raises(ValueError, match="at most 2\\^31 - 1"):
            dl.layernorm_forward(x, w)
        with pytest.raises(ValueError, match="at most 2\\^31 - 1"):
            dl.layernorm_backward(x, x, w, r, r)
        with pytest.raises(ValueError, match="at most 2\\^31 - 1"):
            dl.layer_norm(x, w)
    x, w = (torch.empty(s, dtype=torch.bfloat16, device="meta") for s in ((2, 2**31 - 1), (2**31 - 1,)))
    with pytest.raises(ValueError, match="CUDA device"):  # the widest that fits: the next check
        dl.layernorm_forward(x, w)


def test_adamw_refuses_an_eps_whose_quotient_is_lost(library):
    """Beyond 2^126 the approximate quotient is 0, whatever the moment: with
    lr = eps = 2e38 the update would be m, and was nothing."""
    off = torch.tensor([0, 4], dtype=torch.int64)
    f = dl._Fragment(off.data_ptr(), 1 << 20, 1)
    for state in (0, 3):
        for eps, refused in ((2.0 ** 125, False), (2.0 ** 125 * 1.01, True), (2e38, True), (3.4e38, True)):
            job = (inner._AdamWJob * 1)()
            job[0].frag = ctypes.pointer(f)
            for k in ("theta", "grad", "m", "v", "m_scale", "v_scale"):
                setattr(job[0], k, (1 << 20) + (4 if k == "theta" else 0))  # theta off 16 bytes
            c = inner._AdamWConfig(1e-3, 0.9, 0.95, eps, 0.1, 1, 0)
            got = library.dl_adamw_step(job, 1, 0, state, ctypes.byref(c), None, None)
            assert got == (-1 if refused else -2), eps  # -2: the next check, of theta's alignment


# ----------------------------------------------------------------------------
# layer_norm under autograd


@pytest.fixture
def formulas(monkeypatch):
    """The two calls by their formulas, on any device, without history as theirs."""
    def forward(x, weight, bias=None, eps=1e-5, rms=False, **kw):
        with torch.no_grad():
            mean = None if rms else x.mean(-1)
            d = x if rms else x - mean[..., None]
            rstd = torch.rsqrt(d.square().mean(-1) + eps)
            y = d * rstd[..., None] * weight.reshape(-1)
            return (y if bias is None else y + bias.reshape(-1)), mean, rstd

    def backward(dy, x, weight, mean, rstd, dweight=None, dbias=None, rms=False, bias=True, **kw):
        with torch.no_grad():
            h = (x if rms else x - mean[..., None]) * rstd[..., None]
            wdy = dy * weight.reshape(-1)
            dx = wdy - h * (wdy * h).mean(-1, keepdim=True)
            if not rms:
                dx = dx - wdy.mean(-1, keepdim=True)
            rows = tuple(range(x.dim() - 1))
            return dx * rstd[..., None], (dy * h).sum(rows), dy.sum(rows) if bias else None
    monkeypatch.setattr(inner, "layernorm_forward", forward)
    monkeypatch.setattr(inner, "layernorm_backward", backward)


def _case(rms):
    gen = torch.Generator().manual_seed(1)
    x, w, b, c = (torch.randn(s, generator=gen, dtype=torch.float64) for s in ((3, 5), 5, 5, (3, 5)))
    leaves = [t.requires_grad_() for t in (x, w, b)]

    def norm(x, w, b):
        d = x if rms else x - x.mean(-1, keepdim=True)
        return d * torch.rsqrt(d.square().mean(-1, keepdim=True) + 1e-5) * w + b
    return leaves, c, norm


@pytest.mark.parametrize("rms", [False, True])
def test_layer_norm_first_derivatives(formulas, rms):
    leaves, c, norm = _case(rms)
    want = torch.autograd.grad((norm(*leaves) * c).sum(), leaves)
    for create_graph in (False, True):
        got = torch.autograd.grad((dl.layer_norm(*leaves, rms=rms) * c).sum(), leaves,
                                  create_graph=create_graph)
        assert all(torch.allclose(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("constant", [False, True])
@pytest.mark.parametrize("of", [0, 1])
def test_layer_norm_second_derivatives_are_refused(formulas, rms, constant, of):
    """A gradient penalty: torch's own formula has a second derivative, this
    operation says that it has none, whether dy has a history or not."""
    leaves, c, norm = _case(rms)

    def penalty(y):
        loss = (y * c).sum() if constant else y.pow(3).sum()
        g, = torch.autograd.grad(loss, leaves[of], create_graph=True)
        return loss + g.square().sum()
    assert torch.isfinite(torch.autograd.grad(penalty(norm(*leaves)), leaves[0])[0]).all()
    with pytest.raises(RuntimeError, match="second derivatives are not implemented"):
        torch.autograd.grad(penalty(dl.layer_norm(*leaves, rms=rms)), leaves[0])


def test_layer_norm_parameters_with_leading_ones(formulas):
    """Their gradients have their shapes."""
    leaves, c, norm = _case(False)
    x, w, b = leaves
    want = torch.autograd.grad((norm(x, w, b) * c).sum(), leaves)
    for create_graph in (False, True):
        w2, b2 = (t.detach().reshape(1, 1, 5).requires_grad_() for t in (w, b))
        got = torch.autograd.grad((dl.layer_norm(x, w2, b2) * c).sum(), (x, w2, b2),
                                  create_graph=create_graph)
        assert got[1].shape == got[2].shape == (1, 1, 5)
        assert all(torch.allclose(a.reshape(b.shape), b) for a, b in zip(got, want))


def test_a_bias_of_another_length_has_no_gradient(formulas):
    x, w = torch.zeros(4, 64), torch.ones(64)
    for n in (1, 63, 65):
        with pytest.raises(ValueError, match=f"bias: {n} elements, expected 64"):
            dl.layer_norm(x, w, torch.zeros(n))


# ----------------------------------------------------------------------------
# devices: tensors that say that they live on a GPU, a library that notes where
# it was called


class _Placed(torch.Tensor):
    """A host tensor that gives a GPU as its device."""
    @staticmethod
    def on(t, index):
        t = t.as_subclass(_Placed)
        t._index = index
        return t

    device = property(lambda self: torch.device("cuda", self._index))
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self._index

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        with torch._C.DisableTorchFunctionSubclass():
            return func(*args, **(kwargs or {}))


class _Stream:
    def __init__(self, index):
        self.device, self.cuda_stream = torch.device("cuda", index), 100 + index


@pytest.fixture
def machine(monkeypatch):
    """Two GPUs, the first one current, as far as the binding can see."""
    state = {"current": 0, "calls": []}

    class Device:
        def __init__(self, device):
            self.index = torch.device(device).index

        def __enter__(self):
            self.before, state["current"] = state["current"], self.index

        def __exit__(self, *a):
            state["current"] = self.before

    class On(Device):
        def __init__(self, stream):
            self.index = stream.device.index

    class Library:
        def __getattr__(self, name):
            if name.endswith(("_bytes", "_slots")):
                return getattr(real, name)

            def call(*args):
                state["calls"].append((name, state["current"], args[-1]))
                return 0
            return call
    real = dl.lib()
    monkeypatch.setattr(inner, "lib", lambda: Library())
    monkeypatch.setattr(inner, "_current", lambda: state["current"])
    monkeypatch.setattr(inner, "_raw_stream", lambda index: 10 + index)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "stream", On)
    return state


def _on(index, *sizes, dtype=torch.float32):
    return [_Placed.on(torch.zeros(s, dtype=dtype), index) for s in sizes]


def _fragment(numels, index):
    F = dl.Fragment(numels, device="cpu")
    F.d_offsets = _Placed.on(F.d_offsets, index)
    return F


def _calls(index):
    """Every inner-step call, with all its buffers on one GPU."""
    x, y, w, mean, rstd = _on(index, (4, 8), (4, 8), 8, 4, 4)
    dw, db, out, grad, theta, m, v = _on(index, 8, 8, 2, 12, 12, 12, 12)
    ws, = _on(index, max(inner.grad_norm_workspace_bytes(), inner.layernorm_workspace_bytes(4, 8)),
              dtype=torch.uint8)
    J = dl.AdamWJobs([_fragment([5, 7], index)], [theta], [grad], [m], [v])
    return {
        "dl_grad_norm": lambda **k: dl.grad_norm([grad], 1.0, **{"out": out, "workspace": ws, **k}),
        "dl_adamw_step": lambda **k: dl.adamw_step(J, 1, **{"clip": out, **k}),
        "dl_layernorm_forward": lambda **k: dl.layernorm_forward(
            x, **{"weight": w, "bias": db, "y": y, "mean": mean, "rstd": rstd, **k}),
        "dl_layernorm_backward": lambda **k: dl.layernorm_backward(
            y, x, **{"weight": w, "mean": mean, "rstd": rstd, "dweight": dw, "dbias": db, "dx": y,
                     "workspace": ws, **k}),
    }


CALLS = ["dl_grad_norm", "dl_adamw_step", "dl_layernorm_forward", "dl_layernorm_backward"]


@pytest.mark.parametrize("name", CALLS)
def test_a_call_runs_on_its_buffers_device(machine, name):
    for index in (0, 1):
        _calls(index)[name]()
        assert machine["calls"].pop() == (name, index, 10 + index) and machine["current"] == 0
        _calls(index)[name](stream=_Stream(index))
        got, at, stream = machine["calls"].pop()
        assert (got, at) == (name, index) and machine["current"] == 0 and not machine["calls"]
        assert stream in (100 + index, 10 + index)  # given, or made current with its device


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(machine, name):
    for index in (0, 1):
        with pytest.raises(ValueError, match=f"stream of cuda:{1 - index}, buffers on cuda:{index}"):
            _calls(index)[name](stream=_Stream(1 - index))
    assert not machine["calls"]


@pytest.mark.parametrize("name,arg,size", [
    ("dl_grad_norm", "out", 2), ("dl_grad_norm", "workspace", 1 << 16), ("dl_adamw_step", "clip", 2),
    ("dl_layernorm_forward", "weight", 8), ("dl_layernorm_forward", "bias", 8),
    ("dl_layernorm_forward", "y", (4, 8)), ("dl_layernorm_forward", "mean", 4),
    ("dl_layernorm_forward", "rstd", 4), ("dl_layernorm_backward", "weight", 8),
    ("dl_layernorm_backward", "mean", 4), ("dl_layernorm_backward", "rstd", 4),
    ("dl_layernorm_backward", "dweight", 8), ("dl_layernorm_backward", "dbias", 8),
    ("dl_layernorm_backward", "dx", (4, 8)), ("dl_layernorm_backward", "workspace", 1 << 16)])
def test_buffers_of_two_devices_are_refused(machine, name, arg, size):
    for index in (0, 1):
        other, = _on(1 - index, size, dtype=torch.uint8 if arg == "workspace" else torch.float32)
        with pytest.raises(ValueError, match="cuda:0.*cuda:1|cuda:1.*cuda:0"):
            _calls(index)[name](**{arg: other})
    assert not machine["calls"]


def test_lists_of_two_devices_are_refused(machine):
    (a, b, c, d), (e,) = _on(0, 12, 12, 12, 12), _on(1, 12)
    with pytest.raises(ValueError, match="one device"):
        dl.GradList([a, e])
    F = _fragment([5, 7], 0)
    with pytest.raises(ValueError, match="one device"):
        dl.AdamWJobs([F], [a], [b], [c], [e])
    with pytest.raises(ValueError, match="one device"):  # the offsets, which the kernels read
        dl.AdamWJobs([_fragment([5, 7], 1)], [a], [b], [c], [d])
    with pytest.raises(ValueError, match="CUDA device"):
        dl.AdamWJobs([dl.Fragment([5, 7], device="cpu")], [a], [b], [c], [d])
