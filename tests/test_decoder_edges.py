"""The decoder operators' binding on the host (no GPU), with the library call
replaced by its formula on host memory: what the binding hands over is what a
caller gets back."""
import ctypes

import numpy as np
import pytest
import torch

import decoder_ref as ref
import pseudo_grad_sync_gb300 as dl
from pseudo_grad_sync_gb300 import _build, decoder


class Formula:
    """dl_rotary_apply on host memory, from its jobs' pointers and strides."""

    def __init__(self, library):
        self.calls = []
        self.dl_rotary_frequencies = library.dl_rotary_frequencies

    def dl_rotary_apply(self, jobs, n, kind, batch, tokens, width, dim, turns, amplitude, positions, ptype, pstride,
                        first, flags, stream):
        assert kind == dl.DL_F32 and positions is None
        pairs = np.ctypeslib.as_array((ctypes.c_uint64 * (dim // 2)).from_address(turns))
        angle = ref.angles((first + torch.arange(tokens)).expand(batch, tokens), pairs)
        for j in jobs[:n]:
            shape = (batch, tokens, j.heads, width)
            x = self._view(j.x, shape, (j.x_batch, j.x_token, j.x_head, 1))
            y = self._view(j.y, shape, (j.y_batch, j.y_token, j.y_head, 1))
            y.copy_(ref.rotate(x, angle, amplitude, bool(flags & 1), bool(flags & 2))[0])
        self.calls.append((n, flags))
        return 0

    @staticmethod
    def _view(at, shape, strides):
        size = 1 + sum((n - 1) * s for n, s in zip(shape, strides))
        return torch.frombuffer((ctypes.c_float * size).from_address(at), dtype=torch.float32).as_strided(shape, strides)


@pytest.fixture
def formula(monkeypatch):
    _build.build()
    fake = Formula(dl.lib())
    monkeypatch.setattr(decoder, "lib", lambda: fake)
    for name in ("_cuda", "_one_device"):
        monkeypatch.setattr(decoder, name, lambda *items: None)
    monkeypatch.setattr(decoder, "_on", lambda stream, device: None)
    return fake


def layouts():
    """name -> [batch, tokens, heads, 16] inputs of every kind of strides with a contiguous last dimension."""
    v = torch.randn(4000, generator=torch.Generator().manual_seed(1))
    return {
        "contiguous": v[:2 * 5 * 3 * 16].view(2, 5, 3, 16),
        "heads first": v[:2 * 5 * 3 * 16].view(2, 3, 5, 16).transpose(1, 2),
        "fused": v[:2 * 5 * 9 * 16].view(2, 5, 9, 16)[:, :, 3:6],
        "a shared head": v[:2 * 5 * 16].view(2, 5, 1, 16).expand(2, 5, 3, 16),
        "all shared": v[:16].expand(2, 5, 3, 16),
        "windows": v.unfold(0, 16, 1)[:10].view(2, 5, 16).unsqueeze(2),
        "windows of heads": v.as_strided((2, 5, 3, 16), (1, 16, 1, 1)),
        "halves of windows": v.as_strided((2, 5, 3, 16), (100, 8, 8, 1)),
    }


@pytest.mark.parametrize("name", layouts())
def test_rotary_of_any_layout(formula, name):
    """The result is the formula's, whatever the strides; also those of windows that overlap."""
    x = layouts()[name]
    F = dl.RotaryFrequencies(12, amplitude=1.5, device="cpu")
    want = ref.rotate(x, ref.angles(torch.arange(3, 8).expand(2, 5), dl.rotary_frequencies(12)), 1.5)[0]
    y = dl.rotary_apply(x, F, first=3)
    assert y.stride(-1) == 1 and torch.allclose(y.double(), want, rtol=0, atol=1e-6)
    flat = dl.rotary_apply(x[1], F, first=3)
    assert flat.stride(-1) == 1 and torch.allclose(flat.double(), want[1], rtol=0, atol=1e-6)


def test_rotary_turns_back_what_is_asked_for(formula):
    """Only gradients of inputs that need one are computed, in one call."""
    F = dl.RotaryFrequencies(16, device="cpu")
    q, k = (torch.randn(2, 5, h, 16, generator=torch.Generator().manual_seed(h)) for h in (3, 1))
    for needs in ((True, True), (True, False), (False, True)):
        xs = [x.clone().requires_grad_(need) for x, need in zip((q, k), needs)]
        formula.calls.clear()
        sum(y.sum() for y in dl.rotary(xs, F)).backward()
        assert formula.calls == [(2, 0), (sum(needs), dl.DL_ROTARY_INVERSE)]
        for x, need in zip(xs, needs):
            want = dl.rotary_apply(torch.ones_like(x), F, inverse=True)
            assert torch.equal(x.grad, want) if need else x.grad is None
    w = torch.randn_like(q).requires_grad_()  # a derivative of the gradient
    x = q.clone().requires_grad_()
    dx, = torch.autograd.grad((dl.rotary((x, k), F)[0] * w).sum(), x, create_graph=True)
    dw, = torch.autograd.grad(dx.sum(), w)
    assert torch.equal(dw, dl.rotary_apply(torch.ones_like(q), F))
