"""The decoder operators on the host (no GPU): the entry points' refusals, the
frequency tables, the binding's checks, and the references against torch."""
import ctypes
import math

import numpy as np
import pytest
import torch

import decoder_ref as ref
import pseudo_grad_sync_gb300 as dl
from pseudo_grad_sync_gb300 import _build, decoder

FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    _build.build()
    return dl.lib()


@pytest.fixture(scope="module", autouse=True)
def _built(L):
    pass


# ----------------------------------------------------------------------------
# frequencies


@pytest.mark.parametrize("dim", [2, 4, 50, 64, 128, 8192])
@pytest.mark.parametrize("how", [
    {}, {"base": 500000.0}, {"scaling": "linear", "factor": 8.0}, {"scaling": "base", "factor": 4.0},
    {"scaling": "parts", "factor": 8.0, "context": 8192.0, "low": 1.0, "high": 4.0, "base": 500000.0}])
def test_frequencies_follow_the_formula(dim, how):
    if dim == 2 and how.get("scaling") == "base":
        with pytest.raises(dl.DLError):
            dl.rotary_frequencies(dim, **how)
        return
    got = dl.rotary_frequencies(dim, **how)
    want = ref.frequencies(dim, **how)
    assert got.dtype == np.uint64 and got.shape == (dim // 2,)
    # a power and a few operations in 64 bits: its exponent's rounding is up to
    # ln(base) units of 2^-53, a handful more for the rest; the last 2^-64 turn
    for t, f in zip(got.tolist(), want):
        assert abs(t - f / math.tau * 2.0**64) <= 64 * 2.0**-53 * f / math.tau * 2.0**64 + 1


def test_frequencies_refusals(L):
    turns = np.empty(8, dtype=np.uint64)

    def call(dim=16, base=1e4, scaling=0, factor=2.0, context=64.0, low=1.0, high=4.0,
             out=turns.ctypes.data):
        return L.dl_rotary_frequencies(dim, base, scaling, factor, context, low, high, out)
    for bad in ({"dim": 0}, {"dim": 15}, {"dim": -2}, {"dim": 8194}, {"base": 0.5}, {"base": math.nan},
                {"base": math.inf}, {"scaling": 4}, {"scaling": -1}, {"out": None},
                {"scaling": 1, "factor": 0.5}, {"scaling": 1, "factor": math.nan},
                {"scaling": 2, "factor": math.inf}, {"scaling": 2, "base": 1e300, "factor": 1e300},
                {"scaling": 3, "context": 0.0}, {"scaling": 3, "low": -1.0}, {"scaling": 3, "high": 1.0},
                {"scaling": 3, "high": math.inf}, {"scaling": 3, "context": math.nan}):
        assert call(**bad) == -1, bad
    assert call() == 0 and call(scaling=3) == 0
    with pytest.raises(ValueError, match="scaling"):
        dl.rotary_frequencies(16, scaling="other")
    for dim in (0, 3, 8194, 2**32 + 16):
        with pytest.raises(ValueError, match="dim"):
            dl.rotary_frequencies(dim)


def test_given_frequencies():
    f = [1.0, 0.25, 0.0, 6.0]
    F = dl.RotaryFrequencies(8, frequencies=f, amplitude=2.0, device="cpu")
    for t, want in zip(F.turns.numpy().view(np.uint64).tolist(), f):
        assert abs(t - want / math.tau * 2**64) <= 2.0**-50 * 2**64
    plain = dl.RotaryFrequencies(8, device="cpu")
    assert np.array_equal(plain.turns.numpy().view(np.uint64), dl.rotary_frequencies(8))
    for bad in ([1.0], [1.0, 2.0, 3.0, 7.0], [1.0, -1.0, 0.0, 0.0], [1.0, math.nan, 0.0, 0.0]):
        with pytest.raises(ValueError, match="frequencies"):
            dl.RotaryFrequencies(8, frequencies=bad, device="cpu")
    for bad in (math.nan, math.inf, 1e39):
        with pytest.raises(ValueError, match="amplitude"):
            dl.RotaryFrequencies(8, amplitude=bad, device="cpu")


# ----------------------------------------------------------------------------
# refusals of the entry points


def test_rotary_apply_refusals(L):
    def call(n_jobs=1, kind=1, batch=2, tokens=3, width=64, dim=64, turns=FAKE, amplitude=1.0,
             positions=FAKE, ptype=5, pstride=3, first=0, flags=0, jobs=True, other=None, **put):
        arr = (decoder._RotaryJob * 5)()
        for j in arr:
            j.x, j.y, j.heads = FAKE, FAKE + (1 << 19), 4
            j.x_batch, j.x_token, j.x_head = 768, 256, 64
            j.y_batch, j.y_token, j.y_head = 768, 256, 64
        for k, v in put.items():
            setattr(arr[0], k, v)
        for k, v in (other or {}).items():
            setattr(arr[1], k, v)
        return L.dl_rotary_apply(arr if jobs else None, n_jobs, kind, batch, tokens, width, dim, turns,
                                 amplitude, positions, ptype, pstride, first, flags, None)
    for bad in ({"jobs": False}, {"n_jobs": 0}, {"n_jobs": 5}, {"kind": 3}, {"kind": -1}, {"batch": -1},
                {"tokens": -1}, {"width": 1}, {"dim": 0}, {"dim": 63}, {"dim": 66}, {"width": 9000, "dim": 8194},
                {"turns": None}, {"amplitude": math.nan}, {"amplitude": math.inf}, {"amplitude": 1e39},
                {"ptype": 0}, {"ptype": 3}, {"pstride": -1}, {"flags": 4}, {"flags": -1}, {"heads": -1},
                {"x": None}, {"y": None}, {"x_head": -1}, {"y_token": -256},
                {"y_head": 63},                       # heads overlap
                {"y_token": 0}, {"y_batch": 256},     # tokens, batches overlap
                {"y_token": 2**62, "tokens": 2**33},  # beyond 64 bits
                {"y": FAKE, "x_head": 128},           # in place with other strides
                {"batch": 2**33, "tokens": 2**33},
                {"n_jobs": 2},                        # two tensors to one place
                {"n_jobs": 2, "other": {"y": FAKE}}):  # one into the other's input
        assert call(**bad) == -1, bad
    for bad in ({"turns": FAKE + 4}, {"positions": FAKE + 4}, {"positions": FAKE + 2, "ptype": 4},
                {"x": FAKE + 1}, {"y": FAKE + (1 << 19) + 1}, {"x": FAKE + 2, "kind": 0}):
        assert call(**bad) == -2, bad
    for none in ({"batch": 0}, {"tokens": 0}, {"heads": 0}):
        assert call(turns=None, x=None, y=None, **none) == 0


def test_logprobs_refusals(L):
    def fwd(z=FAKE, stride=64, kind=1, rows=4, vocab=64, tokens=FAKE, ttype=5, logp=FAKE, h=FAKE, lse=FAKE,
            top=3, tt=FAKE, tl=FAKE, m=FAKE, ls=FAKE):
        return L.dl_logprobs_forward(z, stride, kind, rows, vocab, tokens, ttype, logp, h, lse, top, tt, tl, m,
                                     ls, None)
    for bad in ({"kind": 3}, {"kind": -1}, {"rows": -1}, {"vocab": 0}, {"stride": 63}, {"ttype": 1}, {"top": -1},
                {"top": 33}, {"z": None}, {"tokens": None}, {"logp": None}, {"tt": None}, {"tl": None},
                {"m": None}, {"ls": None}):
        assert fwd(**bad) == -1, bad
    for bad in ({"z": FAKE + 1}, {"z": FAKE + 2, "kind": 0}, {"tokens": FAKE + 4}, {"tokens": FAKE + 2, "ttype": 4},
                {"logp": FAKE + 2}, {"h": FAKE + 1}, {"lse": FAKE + 2}, {"tt": FAKE + 4}, {"tl": FAKE + 2},
                {"m": FAKE + 2}, {"ls": FAKE + 2}):
        assert fwd(**bad) == -2, bad
    assert fwd(rows=0, z=None, tokens=None, logp=None) == 0

    def bwd(z=FAKE, stride=64, kind=1, rows=4, vocab=64, tokens=FAKE, ttype=5, m=FAKE, ls=FAKE, h=FAKE, g=FAKE,
            dh=FAKE, dl_=FAKE, top=3, tt=FAKE, dt=FAKE, out=FAKE, ostride=64):
        return L.dl_logprobs_backward(z, stride, kind, rows, vocab, tokens, ttype, m, ls, h, g, dh, dl_, top, tt,
                                      dt, out, ostride, None)
    for bad in ({"kind": 3}, {"rows": -1}, {"vocab": 0}, {"stride": 63}, {"ostride": 63}, {"ttype": 1}, {"top": -1},
                {"top": 33}, {"z": None}, {"out": None}, {"m": None}, {"ls": None}, {"h": None}, {"tokens": None},
                {"tt": None}, {"dt": None}, {"ostride": 128}):
        assert bwd(**bad) == -1, bad
    for bad in ({"z": FAKE + 1}, {"out": FAKE + 1}, {"tokens": FAKE + 4}, {"m": FAKE + 2}, {"ls": FAKE + 2},
                {"h": FAKE + 2}, {"g": FAKE + 2}, {"dh": FAKE + 2}, {"dl_": FAKE + 2}, {"tt": FAKE + 4},
                {"dt": FAKE + 2}):
        assert bwd(**bad) == -2, bad
    assert bwd(rows=0, z=None, out=None, m=None, ls=None) == 0


# ----------------------------------------------------------------------------
# the binding's checks


def meta(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_rotary_binding_checks():
    F = dl.RotaryFrequencies(16, device="cpu")
    x = torch.zeros(2, 3, 4, 16)
    for bad, error, text in (
            (dict(xs=[]), ValueError, "1 to 4"), (dict(xs=[x] * 5), ValueError, "1 to 4"),
            (dict(xs=[3]), TypeError, "torch.Tensor"), (dict(xs=x.double()), TypeError, "float64"),
            (dict(xs=x[0, 0]), ValueError, "dimensions"), (dict(xs=x[..., ::2]), ValueError, "contiguous"),
            (dict(xs=x[..., :8]), ValueError, "heads of 8"), (dict(xs=(x, x.bfloat16())), TypeError, "bfloat16"),
            (dict(xs=(x, x[:1])), ValueError, "does not go with"), (dict(xs=(x, x[:, :2])), ValueError, "does not"),
            (dict(xs=(x, x[0])), ValueError, "does not go"), (dict(xs=x, frequencies=7), TypeError, "Rotary"),
            (dict(xs=x, out=x[:1]), ValueError, "shape"), (dict(xs=(x, x), out=x), ValueError, "1 tensors for 2"),
            (dict(xs=x, positions=[1, 2, 3]), TypeError, "positions"),
            (dict(xs=x, positions=torch.zeros(3)), TypeError, "int32 or int64"),
            (dict(xs=x, positions=torch.zeros(2, dtype=torch.int64)), ValueError, "positions"),
            (dict(xs=x, positions=torch.zeros(3, 3, dtype=torch.int64)), ValueError, "positions"),
            (dict(xs=x, first=2**63), ValueError, "64 bits"), (dict(xs=x), ValueError, "CUDA device")):
        with pytest.raises(error, match=text):
            dl.rotary_apply(**{"frequencies": F, **bad})
    with pytest.raises(ValueError, match="2\\^31"):
        dl.rotary_apply(meta(1, 1, 2**31), F)
    with pytest.raises(ValueError, match="2\\^31"):
        dl.rotary_apply(meta(1, 2**31 + 4, 16), F)


def test_logprobs_binding_checks():
    z, t = torch.zeros(4, 50), torch.zeros(4, dtype=torch.int64)
    r = torch.zeros(4)
    for bad, error, text in (
            (dict(logits=3), TypeError, "torch.Tensor"), (dict(logits=z.double()), TypeError, "float64"),
            (dict(logits=z[:, ::2]), ValueError, "contiguous"), (dict(logits=z[:, :0]), ValueError, "empty"),
            (dict(top=33), ValueError, "top"), (dict(top=-1), ValueError, "top"),
            (dict(tokens=[1]), TypeError, "tokens"), (dict(tokens=r), TypeError, "int32 or int64"),
            (dict(tokens=t[:3]), ValueError, "tokens"), (dict(), ValueError, "CUDA device")):
        with pytest.raises(error, match=text):
            dl.logprobs_forward(**{"logits": z, "tokens": t, **bad})
    tt = torch.zeros(4, 2, dtype=torch.int64)
    for bad, error, text in (
            (dict(tokens=None), ValueError, "needs the tokens"), (dict(row_max=None), ValueError, "missing"),
            (dict(log_sum=r[:3]), ValueError, "log_sum"), (dict(d_logp=r.double()), TypeError, "d_logp"),
            (dict(d_entropy=r), ValueError, "needs the entropy"), (dict(d_logp=r[:1].expand(4)), ValueError, "contig"),
            (dict(d_top=tt.float()), ValueError, "needs the top"),
            (dict(d_top=tt.float(), top_tokens=tt.int()), TypeError, "top_tokens"),
            (dict(d_top=r, top_tokens=tt), ValueError, "d_top"), (dict(out=z[:3]), ValueError, "out"),
            (dict(d_top=torch.zeros(4, 33), top_tokens=torch.zeros(4, 33, dtype=torch.int64)), ValueError, "at most"),
            (dict(out=z.bfloat16()), TypeError, "out"), (dict(), ValueError, "CUDA device")):
        with pytest.raises(error, match=text):
            dl.logprobs_backward(**{"logits": z, "tokens": t, "row_max": r, "log_sum": r, "d_logp": r, **bad})
    for vocab in (2**31, 2**32 + 64):
        with pytest.raises(ValueError, match="2\\^31"):
            dl.logprobs_forward(meta(2, vocab, dtype=torch.bfloat16))


# ----------------------------------------------------------------------------
# the references, and the autograd operations with the calls by their formulas


def test_reference_logprobs_against_torch():
    torch.manual_seed(0)
    z = (torch.randn(7, 40, dtype=torch.float64) * 3).requires_grad_()
    t = torch.randint(0, 40, (7,))
    w = ref.logprobs(z.detach(), t, 5)
    lp = torch.log_softmax(z, 1)
    H = torch.distributions.Categorical(logits=z).entropy()
    lse = torch.logsumexp(z, 1)
    at = lp.gather(1, t[:, None])[:, 0]
    top = torch.topk(lp, 5)
    for got, want in ((w["logp"], at), (w["entropy"], H), (w["lse"], lse), (w["top_logp"], top.values)):
        assert torch.allclose(got, want.detach(), rtol=1e-12, atol=1e-12)
    assert torch.equal(w["top_tokens"], top.indices)
    g, h, l, q = (torch.randn(s, dtype=torch.float64) for s in ((7,), (7,), (7,), (7, 5)))
    want, = torch.autograd.grad((at * g + H * h + lse * l).sum() + (top.values * q).sum(), z)
    got, size = ref.dlogits(z.detach(), t, w["row_max"], w["log_sum"], g, h, l, w["entropy"], w["top_tokens"], q)
    assert torch.allclose(got, want, rtol=1e-10, atol=1e-12) and bool((size >= got.abs() * (1 - 1e-9)).all())


def test_reference_rotation_keeps_lengths_and_relative_angles():
    turns = dl.rotary_frequencies(8)
    x = torch.randn(1, 6, 2, 10, dtype=torch.float64)
    p = torch.tensor([[0, 1, 5, 1000, 2**33, -7]])
    for interleaved in (False, True):
        y, _ = ref.rotate(x, ref.angles(p, turns), interleaved=interleaved)
        back, _ = ref.rotate(y, ref.angles(p, turns), interleaved=interleaved, inverse=True)
        assert torch.allclose(back, x, rtol=0, atol=1e-12) and torch.equal(y[..., 8:], x[..., 8:])
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1), rtol=1e-12)
        moved, _ = ref.rotate(x, ref.angles(p + 12345, turns), interleaved=interleaved)
        a, b = (torch.einsum("bshd,bthd->bhst", v, v) for v in (y, moved))
        assert torch.allclose(a, b, rtol=0, atol=1e-9)  # only differences of positions count


def test_angles_are_those_of_the_frequencies():
    f = ref.frequencies(32)
    angle = ref.angles(torch.arange(0, 4000, 37), dl.rotary_frequencies(32))
    want = torch.arange(0, 4000, 37, dtype=torch.float64)[:, None] * torch.tensor(f, dtype=torch.float64)
    # 4000 radians to some units of 2^-53
    assert float((torch.sin(angle) - torch.sin(want)).abs().max()) <= 64 * 4000 * 2.0**-53


@pytest.fixture
def formulas(monkeypatch):
    """The calls by their formulas, on the host."""
    def forward(logits, tokens=None, top=0, entropy=False, **kw):
        with torch.no_grad():
            w = ref.logprobs(logits, tokens, top)
            return dl.LogProbs(w.get("logp"), w["lse"], w["entropy"] if entropy else None, w.get("top_tokens"),
                               w.get("top_logp"), torch.stack([w["row_max"], w["log_sum"]]))

    def backward(logits, tokens, row_max, log_sum, d_logp=None, d_entropy=None, d_lse=None, entropy=None,
                 top_tokens=None, d_top=None, **kw):
        for d in (d_logp, d_entropy, d_lse, d_top):
            assert d is None or d.is_contiguous()
        with torch.no_grad():
            return ref.dlogits(logits, tokens, row_max, log_sum, d_logp, d_entropy, d_lse, entropy, top_tokens,
                               d_top)[0]

    def apply(xs, frequencies, positions=None, first=0, interleaved=False, inverse=False, **kw):
        with torch.no_grad():
            turns = frequencies.turns.numpy().view(np.uint64)
            if positions is None:
                positions = (first + torch.arange(xs[0].shape[1])).expand(xs[0].shape[:2])
            return tuple(ref.rotate(x, ref.angles(positions, turns), frequencies.amplitude, interleaved, inverse)[0]
                         for x in xs)
    monkeypatch.setattr(decoder, "logprobs_forward", forward)
    monkeypatch.setattr(decoder, "logprobs_backward", backward)
    monkeypatch.setattr(decoder, "rotary_apply", apply)


def test_autograd_passes_every_gradient(formulas):
    torch.manual_seed(1)
    z = torch.randn(4, 9, dtype=torch.float64, requires_grad=True)
    t = torch.tensor([1, 8, -1, 3])

    def f(z):
        r = dl.token_logprobs(z, t, top=2, entropy=True)
        return r.logp, r.lse, r.entropy, r.top_logp[:2]
    assert torch.autograd.gradcheck(f, (z,), atol=1e-7)
    # only some outputs used; a mean's gradient has one value for all rows
    dz, = torch.autograd.grad(dl.token_logprobs(z, t, top=2, entropy=True).entropy.mean(), z)
    assert dz.shape == z.shape
    r = dl.token_logprobs(z)
    assert r.logp is None and r.entropy is None and r.top_tokens is None and r.top_logp is None
    dz, = torch.autograd.grad(r.lse.sum(), z)
    assert torch.allclose(dz, torch.softmax(z.detach(), 1))
    with pytest.raises(RuntimeError, match="second derivatives"):
        dz, = torch.autograd.grad(dl.token_logprobs(z, t).logp.sum(), z, create_graph=True)
        dz.sum().backward()


def test_rotary_autograd(formulas):
    torch.manual_seed(2)
    F = dl.RotaryFrequencies(6, amplitude=1.5, device="cpu")
    q = torch.randn(2, 3, 2, 8, dtype=torch.float64, requires_grad=True)
    k = torch.randn(2, 3, 1, 8, dtype=torch.float64, requires_grad=True)
    p = torch.tensor([[3, 1, 2], [100, 7, 0]])
    for interleaved in (False, True):
        f = lambda q, k: dl.rotary((q, k), F, p, interleaved=interleaved)  # noqa: E731
        assert torch.autograd.gradcheck(f, (q, k)) and torch.autograd.gradgradcheck(f, (q, k))
        assert torch.autograd.gradcheck(lambda q: dl.rotary(q, F, first=5, interleaved=interleaved), (q,))
    only = torch.autograd.grad(dl.rotary((q, k), F, p)[0].sum(), (q, k), allow_unused=True)
    assert only[0] is not None and only[1] is None


def test_job_layout_matches_the_header(L):
    """sizeof and the field order of the struct that crosses the ABI."""
    assert ctypes.sizeof(decoder._RotaryJob) == 72
    assert [n for n, _ in decoder._RotaryJob._fields_] == [
        "x", "y", "x_batch", "x_token", "x_head", "y_batch", "y_token", "y_head", "heads"]
