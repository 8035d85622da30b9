"""The inner-step binding on the host (no GPU): sizes that do not fit the ABI's
arguments, what it passes on, and the autograd operation with the two norm
calls replaced by their formulas in torch."""
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
