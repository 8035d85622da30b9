"""The decoder operators at the edges of what they take, against plain
implementations in 64 bits. Bounds as in test_gpu_decoder.py: U = 2^-24 is half
a unit in the last place of fp32."""
import math

import pytest

import test_gpu_decoder as base
from test_gpu_decoder import TYPES, dl, gen, logits_of, near, randn  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

INF = math.inf


# ----------------------------------------------------------------------------
# rotary positions


def test_rotary_most_heads(dl):
    """One token of 2^31 - 1 heads, in place: the last ones are turned, and nothing beside them."""
    heads, pad = 2**31 - 1, 64
    room = torch.full((2 * heads + 2 * pad,), 7.0, dtype=torch.float16, device="cuda")
    x = room[pad:pad + 2 * heads].view(1, heads, 2)
    x[..., 0] = 1
    x[..., 1] = 0
    F = dl.RotaryFrequencies(2, frequencies=[1.0])
    dl.rotary_apply(x, F, first=1, out=x)
    for i, want in enumerate((math.cos(1.0), math.sin(1.0))):
        low, high = x[0, :, i].aminmax()
        near(torch.stack([low, high]), torch.full((2,), want, device="cuda").double(), base.ROTARY_TOL + base.UT["f16"])
    assert bool((room[:pad] == 7).all()) and bool((room[-pad:] == 7).all())


def test_rotary_widest_head(dl):
    """One head of 2^31 - 1 elements, 16 of them rotated: the others are copied to the last."""
    width, pad = 2**31 - 1, 64
    x = torch.empty(width + 1, dtype=torch.float16, device="cuda").normal_(generator=gen(1))
    room = torch.full((width + 1 + pad,), 7.0, dtype=torch.float16, device="cuda")
    # strides of whole packs: the widest ones are used
    view = lambda t: t.as_strided((1, 1, width), (2**31, 2**31, 1))  # noqa: E731
    F = dl.RotaryFrequencies(16)
    dl.rotary_apply(view(x), F, first=3, out=view(room))
    assert torch.equal(room[:16], dl.rotary_apply(x[:16].view(1, 1, 16), F, first=3).view(16))
    assert torch.equal(room[16:width], x[16:width])
    assert bool((room[width:] == 7).all())


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_of_windows(dl, kind, interleaved):
    """Inputs and gradients whose rows overlap give what copies of them do."""
    v = randn((4000,), 1, kind)
    F = dl.RotaryFrequencies(48)
    for x in (v.unfold(0, 64, 1)[:8].unsqueeze(1), v.unfold(0, 64, 1)[:30].view(2, 15, 64).unsqueeze(2),
              v.as_strided((2, 5, 3, 64), (1, 64, 1, 1)), v.as_strided((2, 5, 3, 64), (400, 32, 32, 1))):
        want = dl.rotary_apply(x.contiguous(), F, first=9, interleaved=interleaved)
        got = dl.rotary_apply(x, F, first=9, interleaved=interleaved)
        assert got.stride(-1) == 1 and torch.equal(got, want)
        leaf = x.contiguous().clone().requires_grad_()  # (a clone of windows may be laid out otherwise)
        dx, = torch.autograd.grad(dl.rotary(leaf, F, first=9, interleaved=interleaved), leaf, x)
        assert torch.equal(dx, dl.rotary_apply(x.contiguous(), F, first=9, interleaved=interleaved, inverse=True))


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("limit", ["1", "5"])
def test_rotary_many_tiles_per_block(dl, kind, interleaved, limit, monkeypatch):
    """Few blocks for many tiles, of several sequences too: the same bits as with a block for each."""
    for batch, tokens, heads, width, dim in ((3, 700, 2, 64, 64), (5, 131, 40, 128, 96), (2, 99, 3, 75, 50),
                                             (700, 1, 4, 64, 64), (1, 2000, 1, 8, 6), (2, 7, 2, 2060, 2048)):
        F = dl.RotaryFrequencies(dim)
        xs = randn((batch, tokens, heads, width), 1, kind), randn((batch, tokens, 1, width), 2, kind)
        positions = torch.randint(0, 9999, (batch, tokens), generator=gen(3), device="cuda")
        for p in (None, positions):
            monkeypatch.delenv("DL_GRID_LIMIT", raising=False)
            want = dl.rotary_apply(xs, F, p, interleaved=interleaved)
            monkeypatch.setenv("DL_GRID_LIMIT", limit)
            got = dl.rotary_apply(xs, F, p, interleaved=interleaved)
            here = [x.clone() for x in xs]
            dl.rotary_apply(here, F, p, interleaved=interleaved, out=here)
            assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, got, here))


# ----------------------------------------------------------------------------
# token log probabilities


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,vocab", [(600, 40), (600, 1000), (300, 2048), (4096, 5000), (40, 20001), (300, 20001),
                                        (600, 32000)])
def test_logprobs_certain_tokens(dl, kind, rows, vocab):
    """One token has all of a row's probability: its log probability is at most 0
    (so 1 - exp of it is no negative number) and the entropy at least 0, whatever the
    logit; masks and logits far below beside it."""
    at = base.tokens_of(rows, vocab, 1)
    top_logit = (torch.rand(rows, generator=gen(2), device="cuda") * 2 - 1) * 60
    top_logit[::7] *= 100
    top_logit = top_logit.to(TYPES[kind])
    for below in (None, 30.0, 90.0):
        z = torch.full((rows, vocab), -INF, dtype=TYPES[kind], device="cuda")
        if below is not None:
            z[:, :] = (top_logit - below)[:, None]
        z[torch.arange(rows), at] = top_logit
        # The others are at d below the row's token: `below` after the rounding to the type, which
        # near 2^12 moves bf16 values by up to 16. Their terms sum to s = (vocab - 1) e^-d, so that
        # -logp = ln S = ln(1 + s) <= s and entropy = ln S + s d / S <= s + s d; beside them the
        # bounds of check_logprobs, with far <= s d and |ln S| <= s.
        d = (top_logit.double() - z[torch.arange(rows), (at + 1) % vocab].double())
        s = (vocab - 1) * torch.exp(-d)
        far = torch.nan_to_num(s * d)
        tol = s + far + base.sum_tol(far) * (1 + 2 * far) + 4 * base.U * (s + far)
        for top, entropy in ((0, False), (0, True), (1, True), (4, False)):
            r = dl.logprobs_forward(z, at, top=top, entropy=entropy)
            values = [r.logp, -r.log_sum] + ([-r.entropy] if entropy else []) + ([r.top_logp[:, 0]] if top else [])
            for v in values:
                assert float(v.max()) <= 0.0
                assert bool((v.double() >= -tol).all())
            if top:
                assert torch.equal(r.top_tokens[:, 0], at)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,vocab", [(61, 40), (61, 1000), (23, 5003), (5, 70001)])
@pytest.mark.parametrize("limit", ["1", "5"])
def test_logprobs_gradient_many_chunks_per_block(dl, kind, rows, vocab, limit, monkeypatch):
    """Few blocks for many rows and chunks, rows left out and without gradients among
    them, dlogits aligned as the logits and otherwise, and in place: the same bits as
    with warps for all."""
    z, tokens = logits_of(rows, vocab, kind, 1), base.tokens_of(rows, vocab, 2)
    tokens[torch.rand(rows, generator=gen(3), device="cuda") < 0.3] = -1
    r = dl.logprobs_forward(z, tokens, top=5, entropy=True)
    g, h, q = randn((rows,), 4), randn((rows,), 5), randn((rows, 5), 6)
    for d in (g, h, q):
        d[::4] = 0
    for args in (dict(d_logp=g), dict(d_logp=g, d_entropy=h, entropy=r.entropy, top_tokens=r.top_tokens, d_top=q)):
        def dlogits(out):
            return dl.logprobs_backward(z, tokens, r.row_max, r.log_sum, out=out, **args)
        monkeypatch.delenv("DL_GRID_LIMIT", raising=False)
        want = dlogits(torch.empty_like(z))
        monkeypatch.setenv("DL_GRID_LIMIT", limit)
        assert torch.equal(dlogits(torch.empty_like(z)), want)
        room = torch.full((rows, vocab + 3), 9.0, dtype=z.dtype, device="cuda")
        assert torch.equal(dlogits(room[:, 1:vocab + 1]), want)
        assert bool((room[:, 0] == 9).all()) and bool((room[:, vocab + 1:] == 9).all())
        here = z.clone()
        dl.logprobs_backward(here, tokens, r.row_max, r.log_sum, out=here, **args)
        assert torch.equal(here, want)
