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


def forms(packs, narrow):
    """(rows of a call, blocks or a warp per row, threads per row) of every form of the kernel that rows of
    that many packs of 16 bytes are computed by."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if packs <= 256:
        return [(300, 1, 32)]
    out = [(3 * sms // ranks, ranks, 256) for ranks in (2, 4, 8) if packs // ranks >= 256]
    out.append((3 * sms // 2 + 1, 1, 128))
    return out + [(4096, 1, 32)] if narrow else out


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("off", [0, 3])
@pytest.mark.parametrize("vocab", [700, 2040, 5003, 20011, 131077])
def test_logprobs_counts_every_border_once(dl, kind, off, vocab):
    """Rows with a single finite column, at every border between threads, stages and
    blocks that share a row: a sum of 1, which twice that column would make 2 and
    without it nothing; the gradient likewise."""
    n = 16 // TYPES[kind].itemsize
    stride = (vocab + 3 + n - 1) // n * n  # every row as the first one on its 16-byte boundary
    packs = (vocab + off % n + n - 1) // n
    for rows, ranks, threads in forms(packs, vocab < 6000):
        each = -(-packs // ranks)
        starts = {b for r in range(ranks) for b in range(r * each, min(r * each + each, packs), threads)}
        columns = {p * n - off % n + d for p in starts for d in (-1, 0, n - 1)} | {0, vocab // 3, vocab - 1}
        columns = torch.tensor(sorted(c for c in columns if 0 <= c < vocab), device="cuda")
        room = torch.empty((rows, stride), dtype=TYPES[kind], device="cuda")
        for first in range(0, len(columns), rows):
            at = columns[first:first + rows]
            at = torch.cat([at, at[-1:].expand(rows - len(at))])  # the form goes by the number of rows
            room.fill_(math.nan)
            z = room[:, off:off + vocab]
            z.fill_(-INF)
            z[torch.arange(rows), at] = 1.5
            zero = torch.zeros(rows, device="cuda")
            for top, entropy in ((0, False), (3, True)):
                r = dl.logprobs_forward(z, at, top=top, entropy=entropy)
                assert bool((r.row_max == 1.5).all())
                near(r.logp, zero, base.SUM_TOL, "logp")
                near(r.log_sum, zero, base.SUM_TOL, "log_sum")
                if top:
                    near(r.entropy, zero, base.SUM_TOL, "entropy")
                    assert torch.equal(r.top_tokens[:, 0], at) and bool((r.top_tokens[:, 1:] == -1).all())
            other, g = (at + 1) % vocab, randn((rows,), 1)
            dz = dl.logprobs_backward(z, other, r.row_max, r.log_sum, g)
            # e^0 / S: the bound of S, and of 1 / S
            near(dz[torch.arange(rows), at], -g, (base.SUM_TOL + 4 * base.U + base.UT[kind]) * g.abs().double(), "dz")
            assert torch.equal(dz[torch.arange(rows), other], g.to(dz.dtype))
            assert bool((torch.count_nonzero(dz, 1) == 2).all())


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_logprobs_with_and_without_alternatives(dl, kind):
    """The order of a row's sums goes by what else a call asks for and by its number
    of rows: each result is within the bound of the others."""
    n = 16 // TYPES[kind].itemsize
    for packs in (95, 96, 97, 112, 127, 128, 129, 200, 255, 256, 257, 600):
        vocab = packs * n
        z, tokens = logits_of(4100, vocab, kind, packs), base.tokens_of(4100, vocab, 2)
        want = dl.logprobs_forward(z[:40], tokens[:40])
        far = base.ref.logprobs(z[:40], None)["far"]
        for rows in (40, 300, 4100):
            for top, entropy in ((0, False), (0, True), (1, False), (9, True)):
                r = dl.logprobs_forward(z[:rows], tokens[:rows], top=top, entropy=entropy)
                assert torch.equal(r.row_max[:40], want.row_max)
                tol = 2 * (base.sum_tol(far) + 8 * base.U * (want.lse.abs() + want.logp.abs()).double())
                near(r.logp[:40], want.logp, tol, (packs, rows, top, entropy))
                near(r.lse[:40], want.lse, tol, (packs, rows, top, entropy))
