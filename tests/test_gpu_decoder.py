"""The decoder operators against plain implementations in 64 bits.

Tolerances are worst-case bounds of the operators' fp32 arithmetic (u = 2^-24
is half a unit in the last place), per element; tokens are compared exactly."""
import importlib.util
import math
import os

import pytest

import decoder_ref as ref
from conftest import ROOT

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
UT = {"f32": U, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# Below the normal range: fp16 results round to a multiple of 2^-24, probabilities under
# 2^-126 are zero (times gradients of some units: 64 of them allowed)
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -30}
INF = math.inf


@pytest.fixture(scope="module")
def dl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import pseudo_grad_sync_gb300 as dl
    dl.lib()
    return dl


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, seed, kind="f32"):
    return torch.randn(shape, generator=gen(seed), device="cuda").to(TYPES[kind])


def near(got, want, tol, what=""):
    """Equal where want is not finite, else within tol, element by element."""
    got, want = got.double(), want.double()
    want = torch.where(want.abs() > torch.finfo(torch.float32).max, want.sign() * INF, want)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    rest = ~fine & ~torch.isnan(want)
    assert torch.equal(got[rest], want[rest]), what
    tol = torch.as_tensor(tol, dtype=torch.float64, device=got.device).expand(got.shape)
    off = (got - want).abs()[fine] - tol[fine]
    assert off.numel() == 0 or float(off.max()) <= 0, (what, float(off.max()))


# ----------------------------------------------------------------------------
# rotary positions

# cos and sin: the angle rounds once (at most pi/4: 0.8 u), the function is off
# by two units (2 u below 1), its product with the amplitude and the amplitude
# itself round (2 u); a product and the sum round (2 u): under 8 u of |a| + |b|.
ROTARY_TOL = 8 * U


def check_rotary(x, y, angle, kind, **how):
    want, size = ref.rotate(x, angle.to(x.device), **how)
    near(y, want, ROTARY_TOL * size + UT[kind] * want.abs() + TINY[kind])


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("batch,tokens,heads,width,dim", [
    (1, 1, 1, 2, 2), (2, 3, 5, 64, 64), (3, 17, 4, 128, 128), (2, 9, 3, 75, 50), (1, 33, 2, 96, 32),
    (5, 1, 36, 64, 64), (2, 5, 3, 83, 16), (1, 4, 2, 257, 256), (2, 301, 3, 40, 24),
    (1, 2, 2, 2060, 2048), (1, 3, 1, 8193, 8192), (7, 1, 300, 8, 6), (2, 7, 5, 96, 52), (1, 9, 3, 256, 2),
    (2, 4, 3, 16, 14), (1, 5, 2, 24, 18), (1, 5, 2, 64, 62)])
def test_rotary(dl, kind, interleaved, batch, tokens, heads, width, dim):
    F = dl.RotaryFrequencies(dim, amplitude=1.25)
    q, k = randn((batch, tokens, heads, width), 1, kind), randn((batch, tokens, 1, width), 2, kind)
    positions = torch.randint(-50, 100000, (batch, tokens), generator=gen(3), device="cuda")
    angle = ref.angles(positions, dl.rotary_frequencies(dim))
    for inverse in (False, True):
        a, b = dl.rotary_apply((q, k), F, positions, interleaved=interleaved, inverse=inverse)
        how = {"amplitude": 1.25, "interleaved": interleaved, "inverse": inverse}
        check_rotary(q, a, angle, kind, **how)
        check_rotary(k, b, angle, kind, **how)
        assert torch.equal(a[..., dim:], q[..., dim:])  # behind the rotated part: copied
    # in place, 32-bit positions: the same bits
    again = q.clone()
    assert dl.rotary_apply(again, F, positions.int(), interleaved=interleaved, inverse=True,
                           out=again) is again
    assert torch.equal(again, a)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_rotary_layouts_and_strides(dl, kind):
    """Every layout of the same values gives the same bits: fused rows, heads
    before tokens, offsets of any alignment, broadcast inputs, outputs within
    wider rows whose rest stays as it was."""
    B, S, H, D, R = 3, 29, 6, 64, 48
    F = dl.RotaryFrequencies(R)
    x = randn((B, S, H, D), 5, kind)
    positions = torch.randint(0, 5000, (B, S), generator=gen(6), device="cuda")
    for interleaved in (False, True):
        y = dl.rotary_apply(x, F, positions, interleaved=interleaved)
        check_rotary(x, y, ref.angles(positions, dl.rotary_frequencies(R)), kind,
                     interleaved=interleaved)
        heads_first = x.transpose(1, 2).contiguous().transpose(1, 2)
        got = dl.rotary_apply(heads_first, F, positions, interleaved=interleaved)
        assert torch.equal(got, y) and got.stride() == heads_first.stride()
        for pad in (1, 2, 4, 8):
            rows = torch.full((B, S, H * D + 3 * pad), 7.0, device="cuda", dtype=TYPES[kind])
            view = rows.as_strided((B, S, H, D), (rows.stride(0), rows.stride(1), D, 1), pad)
            view.copy_(x)
            assert torch.equal(dl.rotary_apply(view, F, positions, interleaved=interleaved), y)
            dl.rotary_apply(view, F, positions, interleaved=interleaved, out=view)
            assert torch.equal(view, y)
            assert bool((rows[:, :, :pad] == 7).all()) and bool((rows[:, :, pad + H * D:] == 7).all())
            rows.fill_(7)
            dl.rotary_apply(x, F, positions, interleaved=interleaved, out=view)
            assert torch.equal(view, y)
            assert bool((rows[:, :, :pad] == 7).all()) and bool((rows[:, :, pad + H * D:] == 7).all())
        one = x[:, :, :1].expand(B, S, H, D)  # a shared head
        assert torch.equal(dl.rotary_apply(one, F, positions, interleaved=interleaved),
                           dl.rotary_apply(one.contiguous(), F, positions, interleaved=interleaved))
        flat = dl.rotary_apply(x[1], F, positions[1], interleaved=interleaved)
        assert torch.equal(flat, y[1])


def test_rotary_positions(dl):
    """Shared and given positions, a first one, and far ones: the angle is exact."""
    B, S, H, D = 2, 5, 2, 32
    F, turns = dl.RotaryFrequencies(D), dl.rotary_frequencies(D)
    x = randn((B, S, H, D), 8)
    row = torch.arange(S, device="cuda")
    y = dl.rotary_apply(x, F)
    for p in (row, row[None], row.expand(B, S), row.int()):
        assert torch.equal(dl.rotary_apply(x, F, p), y)
    wide = torch.stack([row, row + 100], 1)
    assert torch.equal(dl.rotary_apply(x, F, wide[:, 0]), y)  # a column: not contiguous
    for first in (0, 7, -3, 2**31 - 2, 2**40 + 1, -2**62, 2**63 - S):
        got = dl.rotary_apply(x, F, first=first)
        p = torch.tensor([first + s for s in range(S)])
        check_rotary(x, got, ref.angles(p.expand(B, S), turns), "f32")
        assert torch.equal(dl.rotary_apply(x, F, p.cuda()), got)
    assert torch.equal(dl.rotary_apply(x, F, positions=torch.zeros(S, dtype=torch.int64).cuda()), x)


def test_rotary_empty_and_many_tensors(dl):
    F = dl.RotaryFrequencies(16)
    for shape in ((0, 3, 2, 16), (2, 0, 2, 16), (2, 3, 0, 16)):
        assert dl.rotary_apply(torch.empty(shape, device="cuda"), F).shape == shape
    xs = [randn((2, 9, h, 24), h) for h in (1, 0, 3, 5)]
    for x, y in zip(xs, dl.rotary_apply(xs, F, first=11)):
        assert torch.equal(y, dl.rotary_apply(x, F, first=11))


def test_rotary_long(dl):
    """Offsets beyond 2^31 elements, and more tokens than a grid's blocks hold at once."""
    F = dl.RotaryFrequencies(128)
    rows = torch.empty((2**31 // 128 + 70, 1, 128), dtype=torch.bfloat16, device="cuda")
    rows[-100:].copy_(randn((100, 1, 128), 1, "bf16"))
    rows[:100].copy_(rows[-100:])
    S = rows.shape[0]
    last = rows[-100:].clone()
    dl.rotary_apply(rows, F, out=rows)
    assert torch.equal(rows[-100:], dl.rotary_apply(last, F, first=S - 100))
    assert torch.equal(rows[:100], dl.rotary_apply(last, F))


def test_rotary_gradient(dl):
    """The gradient is the rotation back; against the formula and against differences."""
    F = dl.RotaryFrequencies(12, scaling="linear", factor=4.0, amplitude=1.5)
    q, k = randn((2, 5, 3, 16), 1).requires_grad_(), randn((2, 5, 1, 16), 2).requires_grad_()
    p = torch.randint(0, 99, (2, 5), generator=gen(3), device="cuda")
    a, b = dl.rotary((q, k), F, p)
    da, db = randn(a.shape, 4), randn(b.shape, 5)
    dq, dk = torch.autograd.grad((a, b), (q, k), (da, db))
    angle = ref.angles(p, dl.rotary_frequencies(12, scaling="linear", factor=4.0))
    check_rotary(da, dq, angle, "f32", amplitude=1.5, inverse=True)
    check_rotary(db, dk, angle, "f32", amplitude=1.5, inverse=True)
    # differences: the map is linear, so a step of any size will do
    step = randn(q.shape, 6)
    moved = (dl.rotary(q + step, F, p) - dl.rotary(q, F, p)).detach().double()
    got, want = float((moved * da.double()).sum()), float((dq.double() * step.double()).sum())
    terms = float((moved * da.double()).abs().sum())
    # q + step rounds (u of it), as do both results (16 u of their terms)
    assert abs(got - want) <= 64 * U * (terms + float(((q.detach().abs() + step.abs()) * dq.abs()).double().sum()))
    # one output unused; a broadcast gradient; a gradient's gradient
    only = torch.autograd.grad(dl.rotary((q, k), F, p)[1].sum(), (q, k), allow_unused=True)
    assert only[0] is None
    check_rotary(torch.ones_like(b), only[1], angle, "f32", amplitude=1.5, inverse=True)
    w = randn(q.shape, 7).requires_grad_()
    first, = torch.autograd.grad((dl.rotary(q, F, p) * w).sum(), q, create_graph=True)
    second, = torch.autograd.grad((first * step).sum(), w)
    check_rotary(step, second, angle, "f32", amplitude=1.5)
    shared = randn((1, 5, 1, 16), 8).requires_grad_()  # a broadcast input
    dl.rotary(shared.expand(2, 5, 3, 16), F, p).backward(da)
    assert torch.allclose(shared.grad, dq.sum((0, 2), keepdim=True), rtol=0, atol=1e-5)


# ----------------------------------------------------------------------------
# token log probabilities

# S = sum e^(z - m), relative: every term's exponent is off by 3 u |z - m| (the
# difference, its product, log2 e) and its power by 4 u; up to 128 additions
# and 64 changes of the maximum (each a power and a product, 5 u) in a thread's
# and the joined sums.
SUM_TOL = (4 + 128 + 64 * 5) * U


def sum_tol(far):
    return SUM_TOL + 3 * U * far


def check_logprobs(r, z, tokens, top, entropy):
    want = ref.logprobs(z, tokens, top)
    far = torch.nan_to_num(want["far"])
    log = sum_tol(far)
    scale = lambda *v: 4 * U * sum(torch.nan_to_num(x, 0, 0, 0).abs() for x in v)  # noqa: E731
    ls = want["log_sum"]
    near(r.row_max, want["row_max"], 0, "row_max")
    near(r.log_sum, ls, log + scale(ls), "log_sum")
    near(r.lse, want["lse"], log + scale(ls, want["row_max"], want["lse"]), "lse")
    if tokens is None:
        assert r.logp is None
    else:
        near(r.logp, want["logp"], log + scale(ls, want["logp"]), "logp")
    if entropy:
        near(r.entropy, want["entropy"], log + far * 2 * log + scale(ls, far), "entropy")
    else:
        assert r.entropy is None
    if top:
        assert torch.equal(r.top_tokens, want["top_tokens"])
        near(r.top_logp, want["top_logp"], log[:, None] + scale(ls)[:, None] + scale(want["top_logp"]),
             "top_logp")
    else:
        assert r.top_tokens is None and r.top_logp is None


def logits_of(rows, vocab, kind, seed, pad=0, spread=3.0, offset=0.0):
    z = torch.randn((rows, vocab + pad), generator=gen(seed), device="cuda") * spread + offset
    return z.to(TYPES[kind])[:, :vocab]


def tokens_of(rows, vocab, seed):
    return torch.randint(0, vocab, (rows,), generator=gen(seed), device="cuda")


def check_backward(dl, z, tokens, r, kind, seed, top=0, entropy=False, zero_rows=(), out=None):
    rows = z.shape[0]
    d_logp = None if tokens is None else randn((rows,), seed)
    d_lse = randn((rows,), seed + 1)
    d_entropy = randn((rows,), seed + 2) if entropy else None
    d_top = randn((rows, top), seed + 3) if top else None
    for d in (d_logp, d_lse, d_entropy, d_top):
        if d is not None:
            d[list(zero_rows)] = 0
    args = dict(d_logp=d_logp, d_entropy=d_entropy, d_lse=d_lse, entropy=r.entropy if entropy else None,
                top_tokens=r.top_tokens if top else None, d_top=d_top)
    want, size = ref.dlogits(z, tokens, r.row_max, r.log_sum, **args)
    got = dl.logprobs_backward(z, tokens, r.row_max, r.log_sum, out=out, **args)
    # a power (4 u), its exponent (3 u |z - m|, in size), 1 / S (3 u) and six sums and products
    near(got, want, 16 * U * torch.nan_to_num(size) + UT[kind] * want.abs() + 64 * TINY[kind], "dlogits")
    return got


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,vocab", [
    (1, 1), (3, 2), (5, 7), (2, 31), (4, 33), (1, 64), (9, 129), (70, 255), (2, 1000), (33, 1025), (3, 2047),
    (2, 4097), (5, 8192), (2, 20001), (40, 32000), (1, 32003), (1, 128256), (3, 131073), (700, 513),
    (4100, 5001), (4097, 2560)])
def test_logprobs(dl, kind, rows, vocab):
    z, tokens = logits_of(rows, vocab, kind, rows + vocab), tokens_of(rows, vocab, 1)
    for top, entropy in ((0, False), (0, True), (1, False), (7, True), (32, False)):
        r = dl.logprobs_forward(z, tokens, top=top, entropy=entropy)
        check_logprobs(r, z, tokens, top, entropy)
        check_backward(dl, z, tokens, r, kind, vocab, top, entropy)
    none = dl.logprobs_forward(z, top=3, entropy=True)
    check_logprobs(none, z, None, 3, True)
    check_backward(dl, z, None, none, kind, 9, 3, True)
    small = dl.logprobs_forward(z, tokens.int())
    assert torch.equal(small.logp, dl.logprobs_forward(z, tokens).logp)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [5, 63, 1000, 32003])
def test_logprobs_strides_and_alignment(dl, kind, vocab):
    """Rows inside wider ones, at every offset, NaN between them; what lies
    between stays as it was."""
    rows = 6
    tokens = tokens_of(rows, vocab, 2)
    whole = logits_of(rows, vocab, kind, 3)
    want = dl.logprobs_forward(whole, tokens, top=4, entropy=True)
    grad = check_backward(dl, whole, tokens, want, kind, 4, 4, True)
    for pad, off in ((1, 0), (3, 1), (8, 3), (8, 8), (16, 5)):
        room = torch.full((rows, vocab + pad), math.nan, device="cuda", dtype=TYPES[kind])
        z = room[:, min(off, pad):min(off, pad) + vocab]
        z.copy_(whole)
        r = dl.logprobs_forward(z, tokens, top=4, entropy=True)
        check_logprobs(r, z, tokens, 4, True)
        assert torch.equal(r.top_tokens, want.top_tokens) and torch.equal(r.row_max, want.row_max)
        # outputs of other strides and offsets than the logits'
        for opad, ooff in ((0, 0), (pad, min(off, pad)), (5, 2)):
            place = torch.full((rows, vocab + opad), 9.0, device="cuda", dtype=TYPES[kind])
            out = place[:, ooff:ooff + vocab]
            check_backward(dl, z, tokens, r, kind, 4, 4, True, out=out)
            assert bool((place[:, :ooff] == 9).all()) and bool((place[:, ooff + vocab:] == 9).all())
        # in place
        r = dl.logprobs_forward(whole, tokens, top=4, entropy=True)
        z.copy_(whole)
        got = check_backward(dl, z.clone(), tokens, r, kind, 4, 4, True)
        assert torch.equal(got, grad)
        here = z.clone() if pad == 1 else z
        seeds = [randn((rows,), 4 + i) for i in range(3)]
        dl.logprobs_backward(here, tokens, r.row_max, r.log_sum, seeds[0], seeds[2], seeds[1], r.entropy,
                             r.top_tokens, randn((rows, 4), 7), out=here)
        assert torch.equal(here, grad)
        if here is z:
            rest = torch.ones(vocab + pad, dtype=torch.bool)
            rest[min(off, pad):min(off, pad) + vocab] = False
            assert bool(torch.isnan(room[:, rest.cuda()]).all())


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_logprobs_slices(dl, kind):
    """One row and two, of a few columns, anywhere in a buffer: a single pack may
    hold both ends of the tensor."""
    room = torch.full((64,), math.nan, device="cuda", dtype=TYPES[kind])
    for vocab in (1, 2, 3, 5, 7, 8, 9, 16, 17):
        for off in range(17):
            for rows in (1, 2):
                room.fill_(math.nan)
                z = room[off:off + rows * vocab].view(rows, vocab)
                z.copy_(logits_of(rows, vocab, kind, vocab + off))
                tokens = tokens_of(rows, vocab, off)
                r = dl.logprobs_forward(z, tokens, top=2, entropy=True)
                check_logprobs(r, z, tokens, 2, True)
                check_backward(dl, z, tokens, r, kind, off, 2, True)
                check_logprobs(dl.logprobs_forward(z, tokens), z, tokens, 0, False)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [40, 3000, 70001])
def test_logprobs_masks(dl, kind, vocab):
    """Masked entries, rows with one entry and none, the lowest values, NaN and
    infinities, tokens left out and out of range."""
    low = torch.finfo(TYPES[kind]).min
    z = logits_of(16, vocab, kind, 5).clone()
    z[0] = -INF                                # a row that the mask leaves empty
    z[1] = -INF
    z[1, vocab // 2] = 1.5                     # one entry
    z[2, vocab // 3:] = -INF
    z[3] = low                                 # the lowest value everywhere: uniform
    z[4, 5:] = low
    z[5] = -INF
    z[5, 3::7] = low
    z[6, vocab - 1] = INF
    z[7, vocab // 2] = math.nan
    z[8] = math.nan
    z[9, 1::2] = math.nan                      # a row left out: not read
    z[10] = 0.0
    z[10, 1::3] = -0.0                         # equal zeros: the lower token first
    z[11, ::2] = -INF
    z[12] = -torch.finfo(TYPES[kind]).max
    z[12, 0] = torch.finfo(TYPES[kind]).max
    z[13] = INF
    tokens = tokens_of(16, vocab, 6)
    tokens[1], tokens[2], tokens[9], tokens[14], tokens[15] = vocab // 2, vocab - 1, -100, vocab, 2**40
    for top in (0, 5, 32):
        r = dl.logprobs_forward(z, tokens, top=top, entropy=True)
        check_logprobs(r, z, tokens, top, True)
        got = check_backward(dl, z, tokens, r, kind, 8, top, True, zero_rows=(7, 13))
        assert float(got[[0, 7, 9, 13]].float().abs().sum()) == 0.0
        assert bool(torch.isnan(got[[6, 8, 14, 15]].float()).all())
    narrow = torch.where(tokens > 2**31 - 1, torch.full_like(tokens, 2**31 - 1), tokens).int()
    near(dl.logprobs_forward(z, narrow).logp, r.logp, 0)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab,rows,limit", [
    (100, 90, 1), (100, 90, 5), (1500, 61, 1), (1500, 61, 5), (9001, 4200, 24), (20011, 160, 1),
    (20011, 160, 24), (70001, 21, 5), (131073, 9, 1), (131073, 9, 24)])
def test_logprobs_many_rows_per_block(dl, kind, vocab, rows, limit, monkeypatch):
    """Few blocks for many rows: runs of rows through the rings and the handovers, rows
    left out at every place among them, masks that leave some empty."""
    monkeypatch.setenv("DL_GRID_LIMIT", str(limit))
    z = logits_of(rows, vocab, kind, limit)
    z[torch.rand(rows, generator=gen(1), device="cuda") < 0.1] = -INF
    z[torch.rand(rows, generator=gen(2), device="cuda") < 0.3, vocab // 2:] = -INF
    tokens = tokens_of(rows, vocab, 3)
    tokens[torch.rand(rows, generator=gen(4), device="cuda") < 0.4] = -1
    for out in (tokens, torch.full_like(tokens, -1), torch.where(tokens < 0, tokens + 2, tokens)):
        for top, entropy in ((0, False), (6, True)):
            r = dl.logprobs_forward(z, out, top=top, entropy=entropy)
            check_logprobs(r, z, out, top, entropy)
    check_backward(dl, z, out, r, kind, 5, 6, True)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_logprobs_offset(dl, kind):
    """Logits on a common offset lose nothing: the statistics keep the maximum
    and the sum apart."""
    z = logits_of(5, 5000, kind, 3, offset=1000.0)
    tokens = tokens_of(5, 5000, 2)
    r = dl.logprobs_forward(z, tokens, top=3, entropy=True)
    check_logprobs(r, z, tokens, 3, True)
    check_backward(dl, z, tokens, r, kind, 4, 3, True)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("order", ["up", "down", "equal", "steps", "one pack", "one thread"])
def test_logprobs_alternatives(dl, kind, order):
    """Orders that gather the alternatives where a split of the row would rather not have them."""
    vocab = 40000
    z = logits_of(3, vocab, kind, 1, spread=0.01)
    if order in ("up", "down"):
        z = (torch.arange(vocab, device="cuda") * (1e-3 if order == "up" else -1e-3)).to(TYPES[kind])
        z = z.expand(3, vocab).contiguous()
    elif order == "equal":
        z = torch.full_like(z, 0.25)
    elif order == "steps":
        z = (torch.arange(vocab, device="cuda") // 5000).to(TYPES[kind]).expand(3, vocab).contiguous()
    elif order == "one pack":
        z[:, 16000:16032] += 5
    else:
        z[:, 3::2048] += 5
        z[1:, 4::2048] += 5
    for top in (1, 20, 32):
        r = dl.logprobs_forward(z, None, top=top)
        check_logprobs(r, z, None, top, False)
        again = dl.logprobs_forward(z, None, top=top)
        assert torch.equal(r.top_tokens, again.top_tokens) and torch.equal(r.lse, again.lse)


def test_logprobs_named_twice(dl):
    """Tokens that repeat among the alternatives add up; entries out of range have no gradient."""
    z, tokens = logits_of(4, 3000, "f32", 1), tokens_of(4, 3000, 2)
    r = dl.logprobs_forward(z, tokens)
    named = tokens[:, None] + torch.tensor([0, 0, 1, -5000, 0, 4000, 1], device="cuda")
    named[:, 2] = named[:, 6] = 7
    q, g = randn((4, 7), 3), randn((4,), 4)
    want, size = ref.dlogits(z, tokens, r.row_max, r.log_sum, d_logp=g, top_tokens=named, d_top=q)
    got = dl.logprobs_backward(z, tokens, r.row_max, r.log_sum, g, top_tokens=named, d_top=q)
    near(got, want, 16 * U * size + U * want.abs() + TINY["f32"])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", list(range(1018, 1031)) + [1, 2, 3, 6, 9, 15, 2047, 2048, 2049, 2056, 4099])
def test_logprobs_named_at_the_edges(dl, kind, vocab):
    """Tokens and alternatives at both ends of rows of every alignment, where a
    row's chunks and its 16-byte packs end; dlogits aligned as the logits and
    otherwise."""
    rows = 34
    for pad, opad in ((0, 0), (1, 0), (0, 3), (8, 8)):
        z = logits_of(rows, vocab, kind, vocab, pad=pad)
        near_ends = torch.arange(rows, device="cuda") // 2 % vocab
        tokens = torch.where(torch.arange(rows, device="cuda") % 2 == 0, near_ends, vocab - 1 - near_ends)
        r = dl.logprobs_forward(z, tokens, top=1)
        named = torch.stack([vocab - 1 - near_ends, near_ends, tokens, near_ends * 0, near_ends * 0 + vocab - 1], 1)
        g, q = randn((rows,), 3), randn((rows, 5), 4)
        for d_top in (None, q):
            out = torch.empty((rows, vocab + opad), device="cuda", dtype=TYPES[kind])[:, :vocab]
            args = dict(top_tokens=named if d_top is not None else None, d_top=d_top)
            want, size = ref.dlogits(z, tokens, r.row_max, r.log_sum, g, **args)
            dl.logprobs_backward(z, tokens, r.row_max, r.log_sum, g, out=out, **args)
            near(out, want, 16 * U * size + UT[kind] * want.abs() + 64 * TINY[kind], (pad, opad))


def test_logprobs_shapes(dl):
    z = logits_of(12, 100, "bf16", 1).view(3, 4, 100)
    t = tokens_of(12, 100, 2).view(3, 4)
    r = dl.logprobs_forward(z, t, top=2, entropy=True)
    assert r.logp.shape == r.entropy.shape == (3, 4) and r.top_tokens.shape == (3, 4, 2)
    flat = dl.logprobs_forward(z.view(12, 100), t.view(12), top=2, entropy=True)
    assert torch.equal(flat.logp, r.logp.view(12)) and torch.equal(flat.top_logp, r.top_logp.view(12, 2))
    one = dl.logprobs_forward(z[0, 0], t[0, 0])
    assert one.logp.shape == () and torch.equal(one.logp, r.logp[0, 0])
    none = dl.logprobs_forward(z[:0], t[:0], top=2, entropy=True)
    assert none.logp.shape == (0, 4) and none.top_logp.shape == (0, 4, 2)
    assert dl.logprobs_backward(z[:0], t[:0], none.row_max, none.log_sum, none.logp).shape == (0, 4, 100)


def test_logprobs_long(dl):
    """Rows whose offsets pass 2^31 elements, more rows than a grid holds at once."""
    rows, vocab = 70000, 32003
    z = torch.zeros((rows, vocab), dtype=torch.bfloat16, device="cuda")
    few = torch.tensor([0, 1, 35000, rows - 2, rows - 1], device="cuda")
    z[few] = logits_of(5, vocab, "bf16", 1)
    tokens = tokens_of(rows, vocab, 2)
    r = dl.logprobs_forward(z, tokens, top=2)
    part = dl.logprobs_forward(z[few], tokens[few], top=2)
    # alone these rows lie otherwise on the 16-byte boundaries and may be split otherwise:
    # other orders of the same sums, each within the bound
    near(r.logp[few], part.logp, 2 * (sum_tol(20.0) + 12 * U * part.logp.abs().double()))
    assert torch.equal(r.top_tokens[few], part.top_tokens)
    g = randn((rows,), 3)
    got = dl.logprobs_backward(z, tokens, r.row_max, r.log_sum, g, out=z)
    want, size = ref.dlogits(logits_of(5, vocab, "bf16", 1), tokens[few], part.row_max, part.log_sum, g[few])
    near(got[few], want, 16 * U * size + UT["bf16"] * want.abs() + 64 * TINY["bf16"])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_logprobs_widest(dl, kind):
    """A row of 2^31 - 1 columns, all masked but seven."""
    vocab = 2**31 - 1
    z = torch.full((1, vocab), -INF, device="cuda", dtype=TYPES[kind])
    at = torch.tensor([0, 1, 7, 2**30 + 3, 2**31 - 9, 2**31 - 3, vocab - 1], device="cuda")
    v = torch.tensor([1.0, -2.0, 3.0, 0.5, 3.0, 2.0, -1.0], device="cuda")
    z[0, at] = v.to(z.dtype)
    tokens = at[-1:]
    r = dl.logprobs_forward(z, tokens, top=9, entropy=True)
    lp = torch.log_softmax(v.double(), 0)
    order = torch.sort(v, descending=True, stable=True).indices
    assert r.top_tokens[0].tolist() == at[order].tolist() + [-1, -1]
    near(r.top_logp[0, :7], lp[order], sum_tol(4.0) + 16 * U)
    near(r.logp[0], lp[-1], sum_tol(4.0) + 16 * U)
    near(r.entropy[0], -(lp.exp() * lp).sum(), 9 * sum_tol(4.0) + 16 * U)
    g = torch.ones(1, device="cuda")
    dz = dl.logprobs_backward(z, tokens, r.row_max, r.log_sum, g, out=z)
    want = -lp.exp()
    want[-1] += 1
    near(dz[0, at], want, 64 * U + UT[kind] * want.abs())
    assert int(torch.count_nonzero(dz)) == 7


def test_token_logprobs_gradient(dl):
    """Every output's gradient together, against 64-bit autograd and differences."""
    z = logits_of(6, 301, "f32", 1).requires_grad_()
    t = tokens_of(6, 301, 2)
    t[3] = -1
    r = dl.token_logprobs(z, t, top=3, entropy=True)
    assert r.top_tokens.requires_grad is False
    w = [randn((6,), 3), randn((6,), 4), randn((6,), 5), randn((6, 3), 6)]
    loss = (r.logp * w[0]).sum() + (r.lse * w[1]).sum() + (r.entropy * w[2]).sum() + (r.top_logp[:3] * w[3][:3]).sum()
    got, = torch.autograd.grad(loss, z)

    def plain(z):
        lp = torch.log_softmax(z, 1)
        keep = (t >= 0).double()
        top = lp.gather(1, r.top_tokens.clamp(min=0))
        return ((lp.gather(1, t.clamp(min=0)[:, None])[:, 0] * w[0] + torch.logsumexp(z, 1) * w[1]
                 - (lp.exp() * lp).sum(1) * w[2]) * keep).sum() + (top * w[3])[:3].sum()
    zd = z.detach().double().requires_grad_()
    want, = torch.autograd.grad(plain(zd), zd)
    assert float((got.double() - want).abs().max()) <= 1e-5 * float(want.abs().max())
    step = torch.randn(z.shape, generator=gen(9), device="cuda", dtype=torch.float64)
    eps = 1e-4
    slope = float((plain(zd + eps * step) - plain(zd - eps * step)).detach()) / (2 * eps)
    assert abs(slope - float((got.double() * step).sum())) <= 1e-4 * float((got.double() * step).abs().sum())
    # a mean's gradient is one value for all rows
    z2 = z.detach().to(torch.bfloat16).requires_grad_()
    (-dl.token_logprobs(z2, t).logp.mean()).backward()
    keep = t >= 0
    p = torch.softmax(z2.detach().double(), 1)
    p[torch.arange(6), t.clamp(min=0)] -= 1
    want = p * keep[:, None] / 6
    near(z2.grad, want, UT["bf16"] * want.abs() + 64 * U / 6)
    with pytest.raises(RuntimeError, match="second derivatives"):
        gz, = torch.autograd.grad(dl.token_logprobs(z, t).logp.sum(), z, create_graph=True)
        gz.sum().backward()
    with pytest.raises(RuntimeError, match="inplace|in-place"):
        a = (z2 * 1).clone()
        s = dl.token_logprobs(a, t).logp.sum()
        a.add_(1)
        s.backward()
    # an output may be changed in place
    r = dl.token_logprobs(z, t)
    r.logp.mul_(2).sum().backward()
    zero = z.grad.clone()
    z.grad = None
    (dl.token_logprobs(z, t).logp * 2).sum().backward()
    assert torch.equal(zero, z.grad)


# ----------------------------------------------------------------------------
# streams, graphs, both operators together


def test_streams_and_graphs(dl):
    """On a given stream, and captured once and replayed on new values."""
    F = dl.RotaryFrequencies(64)
    x = randn((2, 33, 4, 64), 1, "bf16")
    z, t = logits_of(9, 32003, "bf16", 2), tokens_of(9, 32003, 3)
    g = randn((9,), 4)

    def both():
        y = dl.rotary_apply(x, F, positions)
        r = dl.logprobs_forward(z, t, top=4, entropy=True)
        return y, r, dl.logprobs_backward(z, t, r.row_max, r.log_sum, g)
    positions = torch.randint(0, 999, (2, 33), generator=gen(5), device="cuda")
    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = dl.rotary_apply(x, F, positions, stream=side)
    r = dl.logprobs_forward(z, t, top=4, entropy=True, stream=side)
    d = dl.logprobs_backward(z, t, r.row_max, r.log_sum, g, stream=side)
    side.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(d, want[2])
    assert all(torch.equal(a, b) for a, b in zip(r, want[1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    x.copy_(randn(x.shape, 11, "bf16"))
    z.copy_(logits_of(9, 32003, "bf16", 12))
    t.copy_(tokens_of(9, 32003, 13))
    positions.add_(5)
    want = both()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    assert all(torch.equal(a, b) for a, b in zip(got[1], want[1]))


def test_calls_at_once(dl):
    """Calls of two streams at the same time, many of them, share nothing."""
    F = dl.RotaryFrequencies(64)
    work = []
    for i in range(2):
        z, t = logits_of(300, 32003 + 17 * i, "bf16", i), tokens_of(300, 32003, i)
        x = randn((2, 400, 9, 64), 5 + i, "bf16")
        r = dl.logprobs_forward(z, t, top=6, entropy=True)
        work.append((z, t, x, r, dl.logprobs_backward(z, t, r.row_max, r.log_sum, r.logp), dl.rotary_apply(x, F)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(10):
        got = []
        for s, (z, t, x, *_) in zip(streams, work):
            with torch.cuda.stream(s):
                r = dl.logprobs_forward(z, t, top=6, entropy=True)
                got.append((r, dl.logprobs_backward(z, t, r.row_max, r.log_sum, r.logp), dl.rotary_apply(x, F)))
        torch.cuda.synchronize()
        for (r, d, y), (_, _, _, want, wd, wy) in zip(got, work):
            assert all(torch.equal(a, b) for a, b in zip(r, want)) and torch.equal(d, wd) and torch.equal(y, wy)


def _attend(x, w, F, apply):
    """A layer of causal attention on rotary queries and keys with grouped heads."""
    B, S, E = x.shape
    qkv = (x @ w.t()).view(B, S, 8, 16)
    q, k = apply((qkv[:, :, :4], qkv[:, :, 4:6]), F)
    v = qkv[:, :, 6:]
    k, v = (t.repeat_interleave(2, 2) for t in (k, v))
    a = torch.einsum("bshd,bthd->bhst", q, k) / 4
    a = a.masked_fill(torch.ones(S, S, dtype=torch.bool, device=x.device).triu(1), -INF).softmax(-1)
    return torch.einsum("bhst,bthd->bshd", a, v).reshape(B, S, E)


def test_decoder_step(dl):
    """A small decoder's loss and every gradient: norm, rotary attention, log
    probabilities, against the same model in 64-bit torch."""
    B, S, E, V = 2, 11, 64, 333
    w = {"embed": (V, E), "norm": (E,), "qkv": (128, E), "last": (E,), "out": (V, E)}
    p = {n: (randn(s, i) * 0.2 + (n in ("norm", "last"))).requires_grad_() for i, (n, s) in enumerate(w.items())}
    tokens = tokens_of(B * S, V, 20).view(B, S)
    targets = tokens_of(B * S, V, 21).view(B, S)
    targets[0, :3] = -1
    F = dl.RotaryFrequencies(16)

    def model(p, norm, rotate, loss):
        x = p["embed"][tokens]
        x = x + _attend(norm(x, p["norm"]), p["qkv"], F, rotate)
        return loss(norm(x, p["last"]) @ p["out"].t())

    def ours(z):
        r = dl.token_logprobs(z, targets, entropy=True)
        return -r.logp.sum() + 1e-2 * r.lse.square().sum() - 0.1 * r.entropy.sum()
    loss = model(p, lambda x, w: dl.layer_norm(x, w, rms=True), dl.rotary, ours)
    got = torch.autograd.grad(loss, list(p.values()))

    angle = ref.angles(torch.arange(S).expand(B, S), dl.rotary_frequencies(16)).cuda()

    def rotate64(xs, F):
        c, s = torch.cos(angle)[:, :, None], torch.sin(angle)[:, :, None]
        return [torch.cat([x[..., :8] * c - x[..., 8:] * s, x[..., 8:] * c + x[..., :8] * s], -1) for x in xs]

    def theirs(z):
        keep = (targets >= 0).double()
        lp = torch.log_softmax(z, -1)
        nll = -lp.gather(-1, targets.clamp(min=0)[..., None])[..., 0]
        return ((nll + 1e-2 * torch.logsumexp(z, -1).square() + 0.1 * (lp.exp() * lp).sum(-1)) * keep).sum()
    p64 = {n: v.detach().double().requires_grad_() for n, v in p.items()}
    want_loss = model(p64, lambda x, w: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5) * w, rotate64, theirs)
    want = torch.autograd.grad(want_loss, list(p64.values()))
    # products of 333, 128 and 64 terms in fp32, a few in a row: 2000 u of the norm
    assert abs(loss.item() - want_loss.item()) <= 2000 * U * abs(want_loss.item())
    for n, a, b in zip(p, got, want):
        assert float((a.double() - b).norm()) <= 2000 * U * float(b.norm()), n


@pytest.mark.parametrize("bits", [8, 32])
def test_example_with_attention(dl, bits):
    """examples/inner_outer.py with rotary attention: it runs, its losses are
    numbers, and every parameter has a gradient."""
    spec = importlib.util.spec_from_file_location(
        "inner_outer", os.path.join(ROOT, "examples", "inner_outer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.main(["--learners", "2", "--rounds", "1", "--inner", "2", "--bits", str(bits),
                           "--attention"])
    assert all(math.isfinite(v) for v in losses)
    p = {n: (torch.randn(s, generator=gen(i), device="cuda") * 0.05 + ("norm.w" in n)).requires_grad_()
         for i, (n, s) in enumerate(example.shapes(True).items())}
    tokens = tokens_of(2 * example.SEQ, example.VOCAB, 1)
    example.loss_of(p, tokens, tokens.flip(0), dl.RotaryFrequencies(example.HEAD)).backward()
    assert all(float(v.grad.abs().sum()) > 0 for v in p.values())


# ----------------------------------------------------------------------------
# refusals on the device


def test_refusals(dl):
    x = randn((2, 3, 4, 16), 1)
    F = dl.RotaryFrequencies(16)
    with pytest.raises(ValueError, match="CUDA|cpu"):
        dl.rotary_apply(x, F, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        dl.rotary_apply(x, dl.RotaryFrequencies(16, device="cpu"))
    shared = x[:, :, :1].expand(2, 3, 4, 16)
    with pytest.raises(dl.DLError):  # in place on a broadcast head: elements share places
        dl.rotary_apply(shared, F, out=shared)
    with pytest.raises(dl.DLError):  # the same tensor twice in place
        dl.rotary_apply((x, x), F, out=(x, x))
    z, t = logits_of(4, 50, "f32", 1), tokens_of(4, 50, 2)
    with pytest.raises(ValueError, match="CUDA"):
        dl.logprobs_forward(z, t.cpu())
    with pytest.raises(ValueError, match="overlap"):
        dl.logprobs_forward(z[:1].expand(4, 50), t)
    r = dl.logprobs_forward(z, t)
    with pytest.raises(ValueError, match="CUDA"):
        dl.logprobs_backward(z, t, r.row_max, r.log_sum, r.logp.cpu())
