"""The inner-step operators where they are easily wrong: geometries and paths
that small cases do not reach, values at the ends of their ranges, and what a
call leaves behind. Plain implementations in 64 bits, tolerances per element
from the operators' fp32 arithmetic (u = 2^-24)."""
import numpy as np
import pytest

import inner_ref as ref
import test_gpu_inner as base
from test_gpu_inner import HYPER, NORM_TOL, U, codes, dl, np64, to_cuda  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


# ----------------------------------------------------------------------------
# layer norm: every launch geometry, in its aligned, partial and plain forms

# rows of 129..256 and of 4097..6144 columns have threads per row of their own
MORE_WIDTHS = [130, 200, 256, 4104, 5632, 6144]


@pytest.mark.parametrize("width", MORE_WIDTHS)
@pytest.mark.parametrize("kind,param", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"),
                                        ("f16", "f32")])
def test_layernorm_of_more_widths(dl, width, kind, param):
    base.test_layernorm(dl, width, kind, param)


@pytest.mark.parametrize("width", MORE_WIDTHS)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_long_runs_of_rows_of_more_widths(dl, width, kind, monkeypatch):
    base.test_layernorm_long_runs_of_rows(dl, width, kind, monkeypatch)


@pytest.mark.parametrize("width", [5, 61, 101, 203, 501, 1001, 2047, 4001, 5001, 6143, 8190, 11_007])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("limit", [None, "2"])
def test_aligned_rows_that_end_inside_a_pack(dl, width, kind, limit, monkeypatch):
    """Rows that start on 16 bytes and whose width is no multiple of a pack,
    loaded straight (each row its own round) and through the copies' ring."""
    if limit:
        monkeypatch.setenv("DL_GRID_LIMIT", limit)
    rng = np.random.default_rng(width)
    pad, rows = -width % 8, 150
    for rms in (False, True):
        x = base._rows(rng, rows, width, kind, pad)
        assert x.data_ptr() % 16 == 0 and x.stride(0) % 8 == 0
        w, b = (to_cuda(rng.standard_normal(width)) for _ in range(2))
        y, mean, rstd = dl.layernorm_forward(x, w, b, base.EPS, rms)
        x64, w64, b64 = np64(x), np64(w), np64(b)
        yr, mr, rr = ref.norm64(x64, w64, b64, base.EPS, rms)
        h = (x64 - mr[:, None]) * rr[:, None]
        assert np.all(abs(np64(y) - yr) <= base._forward_tol(x64, w64, b64, yr, h, rr, kind)), rms
        base._backward_case(dl, rng, x, w, mean, rstd, rms, True, kind, "f32", pad, False, 64 + rows)


@pytest.mark.parametrize("width", [64, 256, 1024, 2048, 4096, 5632, 8192, 16_384])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_outputs_off_16_bytes_beside_aligned_inputs(dl, width, kind, monkeypatch):
    """The outputs' rows may be aligned to their elements only while the
    inputs come in whole packs: the same bits, and nothing beside them."""
    rng = np.random.default_rng(width)
    rows = 41
    x, dy = base._rows(rng, rows, width, kind, 0), base._rows(rng, rows, width, kind, 0, 1e-2)
    w, b = (to_cuda(rng.standard_normal(width)) for _ in range(2))
    for limit in (None, "2"):
        if limit:
            monkeypatch.setenv("DL_GRID_LIMIT", limit)
        want, mean, rstd = dl.layernorm_forward(x, w, b)
        dx, dw, db = dl.layernorm_backward(dy, x, w, mean, rstd)
        out = torch.full((rows, width + 3), 3.0, dtype=x.dtype, device="cuda")
        y = out[:, 1:1 + width]
        dl.layernorm_forward(x, w, b, y=y)
        assert torch.equal(y, want)
        _, dw2, db2 = dl.layernorm_backward(dy, x, w, mean, rstd, dx=y)
        assert torch.equal(y, dx) and torch.equal(dw, dw2) and torch.equal(db, db2)
        assert (out[:, 0] == 3).all() and (out[:, 1 + width:] == 3).all()


# ----------------------------------------------------------------------------
# 8-bit AdamW: long runs of blocks at every offset from four elements

# tensors of more than ten blocks that start 0, 1, 3, 2, 2 and 0 elements past
# a multiple of four, whole and partial last blocks, small ones between
RUNS = [128 * 41 + 1, 128 * 37 + 2, 128 * 50 + 3, 128 * 45, 5, 1, 128 * 39 + 126, 0, 128 * 64, 130]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("limit", ["1", "2"])
@pytest.mark.parametrize("copy", [True, False])
def test_adamw8_long_runs_of_blocks(dl, kind, limit, copy, monkeypatch):
    """One or two blocks of threads: runs of many blocks per warp, so that the
    rings refill and wrap, and blocks that start inside a group of four follow
    one another. Codes and scales bit for bit from old states, theta and its
    copy as ever."""
    monkeypatch.setenv("DL_GRID_LIMIT", limit)
    monkeypatch.setattr(base, "SHAPES", [RUNS, RUNS])
    base.test_adamw_8(dl, kind, 0 if copy else 1)


@pytest.mark.parametrize("start", [0, 1, 2, 3])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_adamw8_one_tensor_at_every_offset(dl, kind, start, monkeypatch):
    """Runs of 32 blocks that end in the middle of the tensor: the next warp
    goes on from there."""
    monkeypatch.setenv("DL_GRID_LIMIT", "1")
    monkeypatch.setattr(base, "SHAPES", [[start, 128 * 700 + 77]])
    base.test_adamw_8(dl, kind, 0)


def test_adamw8_long_runs_over_many_jobs(dl, monkeypatch):
    monkeypatch.setenv("DL_GRID_LIMIT", "1")
    base.test_adamw_many_jobs_counts_slots_and_splits_launches(dl)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_adamw8_long_runs_write_nothing_outside(dl, kind, monkeypatch):
    monkeypatch.setenv("DL_GRID_LIMIT", "1")
    base.test_adamw_writes_nothing_outside_its_buffers(dl, 8, kind)
    # several long tensors between bytes of one value
    F = dl.Fragment(RUNS)
    pad, n, slots = 64, F.n, dl.adamw_scale_slots(F)

    def guarded(count, dtype):
        size = torch.empty(0, dtype=dtype).element_size()
        raw = torch.full(((count + 2 * pad) * size,), 0x3C, dtype=torch.uint8, device="cuda")
        return raw, raw.view(dtype)[pad:pad + count]
    e4 = torch.float8_e4m3fn
    raws, bufs = zip(*(guarded(c, d) for c, d in (
        (n, torch.float32), (n, base.TYPES[kind]), (n, e4), (n, e4), (slots, torch.float32),
        (slots, torch.float32), (n, torch.bfloat16))))
    dl.adamw_step(dl.AdamWJobs([F], *([b] for b in bufs)), 1, **HYPER)
    for raw, inside in zip(raws, bufs):
        edge = pad * inside.element_size()
        assert (raw[:edge] == 0x3C).all() and (raw[-edge:] == 0x3C).all()
    slot = ref.places(RUNS) // ref.BLOCK
    free = sorted(set(range(slots)) - set(slot.tolist()))
    for b in bufs[4:6]:
        assert (b[free].view(torch.int32) == 0x3C3C3C3C).all()


# ----------------------------------------------------------------------------
# bounded waits


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("width", [64, 1000, 4096, 5632, 11_008])
def test_a_wait_that_runs_out_is_reported(dl, kind, width, monkeypatch):
    """With waits of no polls every wait for a copy runs out. The calls end and
    say so: in the library's status word, and backward also in the workspace's.
    The next calls are as ever."""
    monkeypatch.setenv("DL_GRID_LIMIT", "2")
    rng = np.random.default_rng(width)
    x, dy = (base._rows(rng, 700, width, kind, 0) for _ in range(2))
    w = to_cuda(rng.standard_normal(width))
    y, mean, rstd = dl.layernorm_forward(x, w)
    want = dl.layernorm_backward(dy, x, w, mean, rstd)
    assert dl.read_device_status(None) == 0
    monkeypatch.setenv("DL_WAIT_POLLS", "0")
    dl.layernorm_forward(x, w)
    assert dl.read_device_status(None) == 1 and dl.read_device_status(None) == 0
    dl.layernorm_backward(dy, x, w, mean, rstd)
    assert dl.read_device_status(None) == 1 and dl.read_device_status(None) == 0
    ws = dl.new_workspace(dl.layernorm_workspace_bytes(700, width))
    dl.layernorm_backward(dy, x, w, mean, rstd, workspace=ws)
    assert dl.read_device_status(ws) == 1 and dl.read_device_status(None) == 1
    monkeypatch.delenv("DL_WAIT_POLLS")
    assert torch.equal(dl.layernorm_forward(x, w)[0], y)
    again = dl.layernorm_backward(dy, x, w, mean, rstd, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    assert dl.read_device_status(None) == 0 and dl.read_device_status(ws) == 0


def test_a_gradient_pass_that_ran_out_is_reported(dl, monkeypatch):
    """The same through the autograd operation, which has no workspace of its
    caller's."""
    monkeypatch.setenv("DL_GRID_LIMIT", "2")
    x = torch.randn(300, 512, device="cuda", requires_grad=True)
    w = torch.ones(512, device="cuda", requires_grad=True)
    y = dl.layer_norm(x, w)
    assert dl.read_device_status(None) == 0
    monkeypatch.setenv("DL_WAIT_POLLS", "0")
    y.sum().backward()
    assert dl.read_device_status(None) == 1


def test_layernorm_of_the_widest_row(dl):
    """2^31 - 1 columns: a constant row's deviations are zero, and nothing lies
    beside it. (Sums of equal values are exact; the width and the sum both
    round to powers of two, so the mean is the constant.)"""
    width = 2 ** 31 - 1
    x = torch.full((width,), 2.0, dtype=torch.bfloat16, device="cuda")
    w = torch.full((width,), 0.5, dtype=torch.bfloat16, device="cuda")
    out = torch.full((width + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = dl.layernorm_forward(x, w, y=out[:width])
    assert float(mean) == 2.0 and abs(float(rstd) * base.EPS ** 0.5 - 1) < 1e-6
    assert int(out[:width].count_nonzero()) == 0 and bool((out[width:] == 3).all())


# ----------------------------------------------------------------------------
# InnerAdamW


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("behind", [float("nan"), float("inf"), 1e3])
def test_the_clip_reads_the_fragments_only(dl, bits, behind):
    """Buffers longer than their fragments (rounded up to 64 elements): what
    lies behind enters neither the norm nor the step."""
    rng = np.random.default_rng(3)
    numels = [[100, 33], [0], [257]]
    results = []
    for extra in (False, True):
        F = [dl.Fragment(n) for n in numels]
        r = np.random.default_rng(4)
        size = [-(-f.n // 64) * 64 if extra else f.n for f in F]
        th, g = [], []
        for f, s in zip(F, size):
            for to, fill in ((th, 0.25), (g, behind)):
                t = torch.full((s,), fill, device="cuda")
                t[:f.n] = to_cuda(r.standard_normal(f.n))
                to.append(t)
        opt = dl.InnerAdamW(F, th, g, bits=bits, max_norm=0.5, **HYPER)
        clip = opt.step()
        norm = base._norm64([t[:f.n] for f, t in zip(F, g)])
        assert abs(float(clip[0]) - norm) <= NORM_TOL * norm
        results.append([clip] + [t[:f.n].clone() for f, t in zip(F, th)])
        assert all((t[f.n:] == 0.25).all() for f, t in zip(F, th))
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_inner_adamw_takes_generators_and_missing_buffers(dl):
    """Buffers given as generators clip as lists do; an empty fragment needs no
    gradient buffer."""
    rng = np.random.default_rng(6)
    numels = [[64], [0], [40]]
    vals = [rng.standard_normal(sum(n)) for n in numels]
    out = []
    for lazily in (False, True):
        F = [dl.Fragment(n) for n in numels]
        th = [torch.ones(f.n, device="cuda") for f in F]
        g = [to_cuda(v) if v.size else None for v in vals]
        opt = dl.InnerAdamW(iter(F) if lazily else F, iter(th) if lazily else th,
                            iter(g) if lazily else g, max_norm=0.1, **HYPER)
        out.append([opt.step()] + th)
        norm = base._norm64([t for t in g if t is not None])
        assert abs(float(out[-1][0][0]) - norm) <= NORM_TOL * norm
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_a_step_that_raised_is_not_counted(dl):
    F = dl.Fragment([100])
    th, g = torch.zeros(100, device="cuda"), torch.ones(100, device="cuda")
    opt = dl.InnerAdamW([F], [th], [g], max_norm=1.0, **HYPER)
    opt.step()
    before = th.clone()
    with pytest.raises(dl.DLError):
        opt.step(lr=-1.0)
    assert opt.steps == 1 and torch.equal(th, before)
    opt.step()
    assert opt.steps == 2


def test_a_step_returns_the_clip_that_the_next_one_writes(dl):
    F = dl.Fragment([1000])
    th, g = torch.zeros(1000, device="cuda"), torch.ones(1000, device="cuda")
    opt = dl.InnerAdamW([F], [th], [g], max_norm=1.0, **HYPER)
    kept = []
    for k in range(3):
        g.fill_(k + 1.0)
        clip = opt.step()
        assert clip is opt.clip
        kept.append(clip.clone())
    for k, c in enumerate(kept):
        n = (k + 1) * 1000 ** 0.5
        assert abs(float(c[0]) / n - 1) <= NORM_TOL and abs(float(c[1]) * n - 1) <= 2 * NORM_TOL


# ----------------------------------------------------------------------------
# layer norm backward: rows on a large offset


@pytest.mark.parametrize("offset", [0.0, 10.0, 100.0, 1000.0])
@pytest.mark.parametrize("width", [100, 512, 4096, 11_008, 20_000])
def test_dx_of_rows_on_an_offset(dl, width, offset):
    """dy along xhat, so that dx is small against its terms. From the same
    statistics: x - mean is rounded once (u of the difference, whatever the
    offset) and xhat is off by 2 u; w dy by u; the row sums by 85 u of their
    terms, so their means by 91 u with 1/width and their products; the products
    of the last steps by 5 u of their terms, and the result by u."""
    rng = np.random.default_rng(width)
    rows = 16
    x = to_cuda(offset + rng.standard_normal((rows, width)))
    w = to_cuda(1 + 0.3 * rng.standard_normal(width))
    _, mean, rstd = dl.layernorm_forward(x, w)
    r = np64(rstd)[:, None]
    h = (np64(x) - np64(mean)[:, None]) * r
    dy = to_cuda((h + 0.05 * rng.standard_normal(h.shape)) / np64(w))
    dx, _, _ = dl.layernorm_backward(dy, x, w, mean, rstd)
    want, _, _, h = ref.norm64_backward(np64(dy), np64(x), np64(w), np64(mean), np64(rstd), False)
    wdy = abs(np64(dy) * np64(w))
    along = (wdy * abs(h)).mean(1, keepdims=True)
    tol = U * (2 * abs(want) + r * (5 * wdy + 95 * wdy.mean(1, keepdims=True) + 100 * abs(h) * along))
    assert np.all(abs(np64(dx) - want) <= tol), float((abs(np64(dx) - want) / tol).max())


# ----------------------------------------------------------------------------
# the ends of the ranges


@pytest.mark.parametrize("b2", [1e-9, 0.003, 0.0, 0.95])
def test_adamw8_smallest_scales_and_small_betas(dl, b2):
    """The smallest scale's square times a small beta2 lies below fp32's normal
    range; the moments are those of value = code * scale all the same, codes
    and scales bit for bit."""
    rng = np.random.default_rng(1)
    n = [128 * 9 + 5, 128 * 4]
    F = dl.Fragment(n)
    g = to_cuda(rng.standard_normal(F.n) * 1e-22)
    g[::3] = 0
    th = torch.zeros(F.n, device="cuda")
    e4 = torch.float8_e4m3fn
    m, v = (torch.from_numpy(rng.integers(0, 0x78, F.n).astype(np.uint8)).cuda().view(e4)
            for _ in range(2))
    slots = dl.adamw_scale_slots(F)
    msc, ssc = (torch.full((slots,), 2.0 ** -60, device="cuda") for _ in range(2))
    old = (codes(m), codes(v), msc.cpu().numpy(), ssc.cpu().numpy())
    dl.adamw_step(dl.AdamWJobs([F], [th], [g], [m], [v], [msc], [ssc]), 5, lr=1e-3, betas=(0.9, b2),
                  seed=4)
    want = ref.adamw8_codes(g.cpu().numpy(), *old, n, 5, 0.9, b2, 1.0, 4)
    for got, w in zip((codes(m), msc.cpu().numpy(), codes(v), ssc.cpu().numpy()), want):
        assert np.array_equal(got, w)


def test_adamw8_a_root_beyond_fp32_squares(dl):
    """code * scale = 2^64: its square is Inf, so the block's new scale is NaN;
    its neighbours' are not."""
    F = dl.Fragment([384])
    th, g = torch.zeros(384, device="cuda"), torch.zeros(384, device="cuda")
    e4 = torch.float8_e4m3fn
    m = torch.zeros(384, dtype=torch.uint8, device="cuda").view(e4)
    v = torch.zeros(384, dtype=torch.uint8, device="cuda")
    v[130] = 0x78  # 256
    v[5] = 0x70    # 128
    v = v.view(e4)
    slots = dl.adamw_scale_slots(F)
    msc, ssc = (torch.full((slots,), 2.0 ** 56, device="cuda") for _ in range(2))
    old = (codes(m), codes(v), msc.cpu().numpy(), ssc.cpu().numpy())
    dl.adamw_step(dl.AdamWJobs([F], [th], [g], [m], [v], [msc], [ssc]), 2, seed=1, **HYPER)
    want = ref.adamw8_codes(g.cpu().numpy(), *old, [384], 2, 0.9, 0.95, 1.0, 1)
    assert np.isnan(want[3][1]) and np.isfinite(want[3][[0, 2]]).all()
    assert np.array_equal(ssc.cpu().numpy(), want[3], equal_nan=True)
    keep = np.r_[0:128, 256:384]
    assert np.array_equal(codes(v)[keep], want[2][keep])


def test_grad_norm_after_an_interrupted_call(dl):
    """A call of several launches that stopped halfway (its error was reported)
    leaves a running total behind; the next call does not add to it."""
    rng = np.random.default_rng(9)
    for count in (1, 200):
        bufs = [to_cuda(rng.standard_normal(500)) for _ in range(count)]
        ws = dl.new_workspace(dl.grad_norm_workspace_bytes())
        want = dl.grad_norm(bufs, 1.0, workspace=ws).clone()
        ws[256:264].view(torch.float64).fill_(1e6)  # the workspace's running total
        assert torch.equal(dl.grad_norm(bufs, 1.0, workspace=ws), want)
        assert torch.equal(dl.grad_norm(bufs, 1.0, workspace=ws), want)


@pytest.mark.parametrize("width", [5, 64, 300, 1000, 4096, 5632, 8192, 16_384, 20_000])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_the_mean_of_a_row_with_an_infinity(dl, width, kind):
    """It is that infinity, NaN only where both signs meet; y is NaN."""
    x = base._rows(np.random.default_rng(width), 6, width, kind, 0)
    inf = float("inf")
    x[0, 0], x[1, width - 1], x[2, 1], x[2, 2], x[3, 3] = inf, -inf, inf, -inf, float("nan")
    w = to_cuda(np.ones(width))
    y, mean, rstd = dl.layernorm_forward(x, w)
    m = mean.tolist()
    assert m[0] == inf and m[1] == -inf and np.isnan(m[2:4]).all() and np.isfinite(m[4:]).all()
    assert bool(torch.isnan(y[:4]).all()) and bool(torch.isfinite(y[4:]).all())
    assert np.isnan(rstd.tolist()[:4]).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_grad_norm_of_mostly_zeros(dl, kind):
    """Rows that no token met (an embedding's gradient): zeros of both signs
    beside values in fp32's range of squares, below and above it."""
    rng = np.random.default_rng(5)
    g = to_cuda(np.zeros((600, 4096)), kind)
    g[::7] = -0.0
    assert dl.grad_norm([g], 1.0).tolist() == [0.0, 1.0]
    for scale in (1.0, 1e-30, 1e25):
        g[3::50] = to_cuda(rng.standard_normal((12, 4096)) * scale, kind)
        g[17, 5] = scale
        want = base._norm64([g])
        got = float(dl.grad_norm([g])[0])
        assert abs(got - want) <= NORM_TOL * want
    g[400, 4095] = float("nan")
    assert np.isnan(dl.grad_norm([g], 1.0).tolist()).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_grad_norm_of_zeros_takes_no_longer(dl, kind):
    """Half again as long as dense values at most (4 GB, beyond L2); read
    twice, as groups outside the range are, zeros took two to seven times."""
    n = 1 << (30 if kind == "f32" else 31)
    G = dl.GradList([torch.ones(n, dtype=base.TYPES[kind], device="cuda")])
    ws, out = dl.new_workspace(dl.grad_norm_workspace_bytes()), torch.zeros(2, device="cuda")
    took = []
    for fill in (1.0, 0.0):
        G.grads[0].fill_(fill)
        dl.grad_norm(G, 1.0, out, ws)
        best = float("inf")
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            dl.grad_norm(G, 1.0, out, ws)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        took.append(best)
        norm = n ** 0.5 * fill
        assert abs(float(out[0]) - norm) <= NORM_TOL * norm
    assert took[1] <= 1.5 * took[0], took
