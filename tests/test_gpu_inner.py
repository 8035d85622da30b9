"""The inner-step operators against plain implementations in 64 bits.

Tolerances are worst-case bounds of the operators' fp32 arithmetic (u = 2^-24
is half a unit in the last place), per element; the 8-bit states are compared
bit for bit."""
import numpy as np
import pytest

import inner_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
UT = {"f32": U, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # 2^-p, p bits of precision
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def dl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import pseudo_grad_sync_gb300 as dl
    dl.lib()
    return dl


def np64(t):
    return t.detach().double().cpu().numpy()


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


def to_cuda(a, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(TYPES[dtype])


# ----------------------------------------------------------------------------
# gradient norm

# A thread adds up to 64 squares in fp32 before it goes on in fp64: relative
# error of the sum at most 64 u, of its root half of that, plus the rounding
# of the result.
NORM_TOL = 33 * U


def _norm64(bufs):
    return float(np.sqrt(sum(float(np.sum(np64(b) ** 2)) for b in bufs)))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", [[1], [3, 0, 7], [17], [8191, 8192, 8193, 1], [100_003],
                                   [64] * 200, [5_000_001, 2, 131_072]])
def test_grad_norm(dl, kind, sizes):
    rng = np.random.default_rng(len(sizes) + sizes[0])
    bufs = [to_cuda(rng.standard_normal(n) * 10.0 ** rng.uniform(-3, 1), kind) for n in sizes]
    ws = dl.new_workspace(dl.grad_norm_workspace_bytes())
    want = _norm64(bufs)
    for max_norm in (want * 0.37, want * 2.0, float("inf")):
        out = dl.grad_norm(bufs, max_norm, workspace=ws)
        norm, coef = np64(out)
        assert abs(norm - want) <= NORM_TOL * want
        assert abs(coef - min(1.0, max_norm / want)) <= (NORM_TOL + U) * 1.0
        again = dl.grad_norm(dl.GradList(bufs), max_norm, workspace=ws)
        assert torch.equal(out, again)
    assert int(ws.count_nonzero()) == int(ws[256:].count_nonzero())  # status word untouched


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [1, 2, 3, 5, 7])
def test_grad_norm_of_unaligned_slices(dl, kind, shift):
    rng = np.random.default_rng(shift)
    flat = to_cuda(rng.standard_normal(30_000), kind)
    bufs = [flat[shift:shift + 1], flat[shift + 1:shift + 9], flat[10 + shift:29_990 + shift % 3]]
    out = dl.grad_norm(bufs)
    want = _norm64(bufs)
    assert abs(float(out[0]) - want) <= NORM_TOL * want and float(out[1]) == 1.0


@pytest.mark.parametrize("value", [3e25, 2e-30, 1e-42])
def test_grad_norm_beyond_the_range_of_fp32_squares(dl, value):
    g = torch.full((70_001,), value, device="cuda")
    want = float(np.float32(value)) * np.sqrt(70_001)
    out = np64(dl.grad_norm([g], 1.0))
    assert abs(out[0] - want) <= NORM_TOL * want + 2.0 ** -150
    assert abs(out[1] - min(1.0, 1.0 / want)) <= 2 * NORM_TOL * min(1.0, 1.0 / want)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_grad_norm_not_finite(dl, bad, kind):
    g = to_cuda(np.ones(20_000), kind)
    g[12_345] = bad
    out = dl.grad_norm([torch.ones(5, device="cuda", dtype=g.dtype), g], 1.0)
    assert not np.isfinite(np64(out)[0]) and np.isnan(np64(out)[1])


def test_grad_norm_of_nothing_and_zeros(dl):
    out = torch.full((2,), 7.0, device="cuda")
    dl.grad_norm([], 1.0, out=out)
    assert out.tolist() == [0.0, 1.0]
    z = torch.zeros(40_000, device="cuda")
    assert dl.grad_norm([z], 1.0).tolist() == [0.0, 1.0]


# ----------------------------------------------------------------------------
# AdamW

HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
SHAPES = [[1], [5, 0, 3], [128], [127, 129, 1], [4096, 4096 * 3 + 4], [1000, 24, 2047, 2049, 8192],
          [7] * 300, [300_001, 3, 70_000]]


def _problem(dl, frags, kind, bits, seed, copy=False, decay=True):
    rng = np.random.default_rng(seed)
    P = {"frags": [dl.Fragment(n) for n in frags], "numels": frags}
    sizes = [sum(n) for n in frags]
    P["theta"] = [to_cuda(rng.standard_normal(n) * 0.02) for n in sizes]
    P["grad"] = [to_cuda(rng.standard_normal(n) * np.exp(rng.uniform(-9, -4, n)), kind)
                 for n in sizes]
    if bits == 32:
        P["m"] = [to_cuda(rng.standard_normal(n) * 1e-3) for n in sizes]
        P["v"] = [to_cuda(rng.uniform(0, 1, n) ** 4 * 1e-6) for n in sizes]
        P["msc"] = P["ssc"] = None
    else:
        def some(n, sign):
            c = rng.integers(0, 0x78, n).astype(np.uint8) | (rng.integers(0, 2, n) * 128 * sign
                                                             ).astype(np.uint8)
            return torch.from_numpy(c).cuda().view(torch.float8_e4m3fn)
        P["m"] = [some(n, 1) for n in sizes]
        P["v"] = [some(n, 0) for n in sizes]
        slots = [dl.adamw_scale_slots(F) for F in P["frags"]]
        P["msc"], P["ssc"] = ([to_cuda(2.0 ** rng.integers(-20, -10, s)) for s in slots]
                              for _ in range(2))
    P["copy"] = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in sizes] if copy else None
    P["decay"] = [to_cuda(rng.integers(0, 2, len(n)) * 1.0) for n in frags] if decay else None
    P["jobs"] = dl.AdamWJobs(P["frags"], P["theta"], P["grad"], P["m"], P["v"], P["msc"], P["ssc"],
                             P["copy"], P["decay"])
    return P


def _theta_tol(old, new, g, m_old, m_new, denom, step):
    """u per rounding: theta * keep (keep itself rounded twice), the update's
    factors (step size, root, its scale, eps, the division, three each at
    most), m' with its own error, and the final fma."""
    b1 = HYPER["betas"][0]
    size = HYPER["lr"] / (1 - b1 ** step)
    err_m = 6 * U * (b1 * abs(m_old) + (1 - b1) * abs(g))
    return 5 * U * abs(old) + size / denom * (err_m + 20 * U * abs(m_new)) + 2 * U * abs(new)


def _check_theta(P, j, before, m_old, v_old, step, coef):
    g = np64(P["grad"][j])
    b1, b2 = HYPER["betas"]
    decay = None if P["decay"] is None else np64(P["decay"][j])
    th, m, v, denom = ref.adamw64(before, g, m_old, v_old, P["numels"][j], step, HYPER["lr"], b1,
                                  b2, HYPER["eps"], HYPER["weight_decay"], decay, coef)
    got = np64(P["theta"][j])
    tol = _theta_tol(before, th, g * coef, m_old, m, denom, step)
    assert np.all(abs(got - th) <= tol), float(np.max(abs(got - th) / np.maximum(tol, 1e-300)))
    if P["copy"] is not None:  # the copy is the new theta, rounded
        assert torch.equal(P["copy"][j], P["theta"][j].to(torch.bfloat16))
    return m, v


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_adamw_32(dl, kind, shape):
    P = _problem(dl, [SHAPES[shape]], kind, 32, shape, copy=shape % 2 == 0, decay=shape % 3 != 1)
    clip = torch.tensor([9.0, 0.3], device="cuda") if shape % 2 else None
    coef = float(np.float32(0.3)) if shape % 2 else 1.0
    for step in (1, 2, 1000):
        before, m_old, v_old = (np64(P[k][0]) for k in ("theta", "m", "v"))
        dl.adamw_step(P["jobs"], step, clip=clip, **HYPER)
        m, v = _check_theta(P, 0, before, m_old, v_old, step, coef)
        g = np64(P["grad"][0]) * coef
        b1, b2 = HYPER["betas"]
        # the rounded constants, the products and the sum: at most 6 u of each term
        assert np.all(abs(np64(P["m"][0]) - m) <= 6 * U * (b1 * abs(m_old) + (1 - b1) * abs(g)))
        assert np.all(abs(np64(P["v"][0]) - v) <= 8 * U * v + 2.0 ** -148)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_adamw_8(dl, kind, shape):
    P = _problem(dl, [SHAPES[shape]], kind, 8, 50 + shape, copy=shape % 2 == 0)
    clip = torch.tensor([9.0, 0.3], device="cuda") if shape % 2 else None
    coef = np.float32(0.3) if shape % 2 else np.float32(1)
    b1, b2 = HYPER["betas"]
    numels = SHAPES[shape]
    slot = ref.places(numels) // ref.BLOCK
    for step in (1, 2, 1000):
        before = np64(P["theta"][0])
        m8, s8 = codes(P["m"][0]), codes(P["v"][0])
        msc, ssc = (P[k][0].cpu().numpy() for k in ("msc", "ssc"))
        dl.adamw_step(P["jobs"], step, clip=clip, seed=77, **HYPER)
        grad = P["grad"][0].float().cpu().numpy()
        want = ref.adamw8_codes(grad, m8, s8, msc, ssc, numels, step, b1, b2, coef, 77)
        assert np.array_equal(codes(P["m"][0]), want[0])
        assert np.array_equal(P["msc"][0].cpu().numpy(), want[1])
        assert np.array_equal(codes(P["v"][0]), want[2])
        assert np.array_equal(P["ssc"][0].cpu().numpy(), want[3])
        m_old = ref.E4M3[m8] * msc[slot]
        v_old = (ref.E4M3[s8] * ssc[slot].astype(np.float64)) ** 2
        m, v = _check_theta(P, 0, before, m_old, v_old, step, float(coef))
        # each stored value lies within one unit of its code's last place of the moment
        for key, sc, x in (("m", "msc", m), ("v", "ssc", np.sqrt(v))):
            scale = np64(P[sc][0])[slot]
            val = ref.E4M3[codes(P[key][0])] * scale
            unit = np.maximum(abs(x) * 2.0 ** -3, scale * 2.0 ** -9)
            assert np.all(abs(val - x) <= unit * (1 + 1e-5))


def test_adamw_many_jobs_counts_slots_and_splits_launches(dl):
    """More jobs than one launch takes, empty ones among them: as if each
    fragment were stepped alone, and the random bits follow the slots of all
    jobs before."""
    rng = np.random.default_rng(3)
    frags = [[int(x) for x in rng.integers(0, 400, rng.integers(1, 5))] for _ in range(70)]
    frags[5], frags[40] = [0], [0, 0]
    P = _problem(dl, frags, "bf16", 8, 9)
    old = [(codes(P["m"][j]), codes(P["v"][j]), P["msc"][j].cpu().numpy(), P["ssc"][j].cpu().numpy())
           for j in range(70)]
    dl.adamw_step(P["jobs"], 3, seed=5, **HYPER)
    slot0 = 0
    for j, n in enumerate(frags):
        if sum(n):
            want = ref.adamw8_codes(P["grad"][j].float().cpu().numpy(), *old[j], n, 3, 0.9, 0.95, 1.0,
                                    5, slot0)
            got = (codes(P["m"][j]), P["msc"][j].cpu().numpy(), codes(P["v"][j]),
                   P["ssc"][j].cpu().numpy())
            for a, b in zip(got, want):
                assert np.array_equal(a, b), j
        slot0 += ref.slots_of(n)
    Q = _problem(dl, frags, "f32", 32, 10)
    before = [[np64(Q[k][j]) for k in ("theta", "m", "v")] for j in range(70)]
    dl.adamw_step(Q["jobs"], 3, **HYPER)
    for j, n in enumerate(frags):
        if sum(n):
            _check_theta(Q, j, *before[j], 3, 1.0)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("coef", [float("nan"), float("inf")])
def test_a_coefficient_that_is_not_finite_skips_the_step(dl, bits, coef):
    P = _problem(dl, [[5000, 77]], "f32", bits, 1, copy=True)
    keys = [k for k in ("theta", "m", "v", "msc", "ssc", "copy") if P[k] is not None]
    before = {k: P[k][0].view(torch.uint8).clone() for k in keys}
    dl.adamw_step(P["jobs"], 1, clip=torch.tensor([1.0, coef], device="cuda"), **HYPER)
    for k in keys:
        assert torch.equal(P[k][0].view(torch.uint8), before[k]), k


def test_adamw8_extreme_moments(dl):
    """Blocks of zeros, of one value, of tiny and of huge gradients, from
    zeroed states: codes bit for bit, zeros stay zeros, and a positive root
    never becomes zero."""
    blocks = [np.zeros(128), np.full(128, 1e-22), np.full(128, 1e15), np.full(128, 1e-38)]
    one = np.zeros(128)
    one[77] = 0.5
    mixed = np.geomspace(1e-12, 1.0, 128)
    g = np.concatenate(blocks + [one, mixed]).astype(np.float32)
    n = [g.size]
    F = dl.Fragment(n)
    slots = dl.adamw_scale_slots(F)
    th, gr = torch.zeros(g.size, device="cuda"), torch.from_numpy(g).cuda()
    m, v = (torch.zeros(g.size, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            for _ in range(2))
    msc, ssc = (torch.zeros(slots, device="cuda") for _ in range(2))
    jobs = dl.AdamWJobs([F], [th], [gr], [m], [v], [msc], [ssc])
    old = (codes(m), codes(v), msc.cpu().numpy(), ssc.cpu().numpy())
    dl.adamw_step(jobs, 1, seed=1, **HYPER)
    want = ref.adamw8_codes(g, *old, n, 1, 0.9, 0.95, 1.0, 1)
    assert np.array_equal(codes(m), want[0]) and np.array_equal(codes(v), want[2])
    assert np.array_equal(msc.cpu().numpy(), want[1]) and np.array_equal(ssc.cpu().numpy(), want[3])
    root = np.sqrt(want[5])
    assert np.array_equal(codes(v) > 0, root > 0)
    assert np.isfinite(np64(th)).all() and np.all(np64(th)[:128] == 0)


def test_adamw8_not_finite_stays_in_its_block(dl):
    """Without a clip a NaN or Inf gradient turns its own block to NaN and no
    other, not even one of a tensor that begins beside it."""
    numels = [200, 130, 128]
    P = _problem(dl, [numels], "f32", 8, 4)
    P["grad"][0][130] = float("nan")     # second block of the first tensor
    P["grad"][0][340] = float("inf")     # the third tensor's only block
    dl.adamw_step(P["jobs"], 2, **HYPER)
    slot = ref.places(numels) // ref.BLOCK
    val = ref.E4M3[codes(P["m"][0])] * np64(P["msc"][0])[slot]
    bad = np.isin(slot, [slot[130], slot[340]])
    assert np.all(np.isnan(val[bad])) and np.all(np.isfinite(val[~bad]))
    th = np64(P["theta"][0])
    assert np.isnan(th[130]) and np.isfinite(np.delete(th, [130, 340])).all()


def test_adamw8_rounding_is_unbiased_over_steps(dl):
    """With a constant squared gradient the root decays towards it; each
    step's relative change (0.05%) is far below a code's spacing (6 to 12%).
    Nearest rounding would keep the root where it started; here its mean over
    the elements follows the exact sequence. One step's rounding is at most
    half a unit (6%) in standard deviation, decayed by 0.1% a step: over 1000
    steps the deviation of one element stays below 0.06 * sqrt(1000), and of
    the mean of 65536 elements below 0.06 * sqrt(1000) / 256 = 0.75%; five of
    those is 3.7%."""
    n = 65536
    F = dl.Fragment([n])
    g = torch.full((n,), 1e-3, device="cuda")
    th = torch.zeros(n, device="cuda")
    m = torch.zeros(n, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v = torch.full((n,), 4.0, device="cuda").to(torch.float8_e4m3fn)
    msc = torch.full((dl.adamw_scale_slots(F),), 2.0 ** -10, device="cuda")
    ssc = msc.clone()
    jobs = dl.AdamWJobs([F], [th], [g], [m], [v], [msc], [ssc])
    b2 = 0.999
    v64 = (4.0 * 2.0 ** -10) ** 2
    for step in range(1, 1001):
        dl.adamw_step(jobs, step, lr=0.0, betas=(0.9, b2), seed=11)
        v64 = b2 * v64 + (1 - b2) * float(np.float32(1e-3)) ** 2
    val = ref.E4M3[codes(v)] * np.repeat(np64(ssc)[:n // 128], 128)
    assert abs(np.mean(val ** 2) / v64 - 1) < 2 * 0.037
    first = (4.0 * 2.0 ** -10) ** 2
    assert v64 < 0.5 * first  # the sequence did move


def test_adamw_beyond_2_31_elements(dl):
    """Offsets that pass 32 bits: a fragment of 2^31 + 4099 elements, its
    last tensor checked."""
    big, last = 2 ** 31 + 3, 4096
    numels = [big, last]
    F = dl.Fragment(numels)
    n = F.n
    th = torch.zeros(n, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            for _ in range(2))
    slots = dl.adamw_scale_slots(F)
    msc, ssc = (torch.zeros(slots, device="cuda") for _ in range(2))
    rng = np.random.default_rng(0)
    tail = to_cuda(rng.standard_normal(last + 64), "bf16")
    g[-(last + 64):] = tail
    dl.adamw_step(dl.AdamWJobs([F], [th], [g], [m], [v], [msc], [ssc]), 1, seed=3, **HYPER)
    t0 = big // 128 + 1
    want = ref.adamw8_codes(tail[64:].float().cpu().numpy(), np.zeros(last, np.uint8),
                            np.zeros(last, np.uint8), np.zeros(33, np.float32),
                            np.zeros(33, np.float32), [last], 1, 0.9, 0.95, 1.0, 3, t0)
    assert np.array_equal(codes(m[big:]), want[0]) and np.array_equal(codes(v[big:]), want[2])
    b1, b2 = HYPER["betas"]
    gt = np64(tail)
    upd, mm, _, denom = ref.adamw64(0 * gt, gt, 0 * gt, 0 * gt, [gt.size], 1, HYPER["lr"], b1, b2,
                                    HYPER["eps"], HYPER["weight_decay"])
    tol = _theta_tol(0 * gt, upd, gt, 0 * gt, mm, denom, 1)
    assert np.all(abs(np64(th[-(last + 64):]) - upd) <= tol)
    del m, v, msc, ssc
    assert float(th[:2 ** 31 - 64].abs().max()) == 0.0
    m, v = (torch.zeros(n, device="cuda") for _ in range(2))
    th.zero_()
    dl.adamw_step(dl.AdamWJobs([F], [th], [g], [m], [v]), 1, **HYPER)
    assert np.all(abs(np64(th[-(last + 64):]) - upd) <= tol)
    assert float(th[:2 ** 31 - 64].abs().max()) == 0.0


def test_inner_adamw_clips_and_steps(dl):
    rng = np.random.default_rng(8)
    numels = [[4096, 33], [257]]
    for bits in (32, 8):
        F = [dl.Fragment(n) for n in numels]
        th = [to_cuda(rng.standard_normal(f.n)) for f in F]
        g = [to_cuda(rng.standard_normal(f.n)) for f in F]
        before = [np64(t) for t in th]
        opt = dl.InnerAdamW(F, th, g, bits=bits, max_norm=0.5, decay=[[1, 0], None], **HYPER)
        clip = opt.step()
        norm = _norm64(g)
        assert abs(float(clip[0]) - norm) <= NORM_TOL * norm
        coef = float(clip[1])
        for j, n in enumerate(numels):
            zero = np.zeros(F[j].n)
            want, m, _, denom = ref.adamw64(before[j], np64(g[j]), zero, zero, n, 1, HYPER["lr"], 0.9,
                                            0.95, HYPER["eps"], HYPER["weight_decay"],
                                            [1, 0] if j == 0 else None, coef)
            tol = _theta_tol(before[j], want, np64(g[j]) * coef, zero, m, denom, 1)
            assert np.all(abs(np64(th[j]) - want) <= tol)
        g[0][5] = float("nan")
        now = [t.clone() for t in th]
        assert np.isnan(float(opt.step()[1]))
        assert all(torch.equal(a, b) for a, b in zip(th, now))


# ----------------------------------------------------------------------------
# layer norm

EPS = 1e-5


def _rows(rng, R, D, kind, pad, scale=1.0):
    whole = rng.standard_normal((R, D + pad)) * scale
    whole[:, ::5] *= 6
    return to_cuda(whole * np.exp(rng.uniform(-2, 2, (R, 1))) + 0.3 * scale, kind)[:, :D]


def _forward_tol(x, w, b, y, h, rstd, kind):
    """Sums of a row: no chain of additions longer than 80, so the mean is off
    by at most 80 u mean|x| and the variance by 85 u of itself (its root by
    43 u); then at most 4 roundings of the product and one of the sum."""
    mean_abs = abs(x).mean(1, keepdims=True)
    hw = abs(h * w)
    bias = 0 if b is None else abs(b)
    return UT[kind] * abs(y) + U * (50 * hw + 2 * bias + 90 * rstd[:, None] * abs(w) * mean_abs) \
        + 2.0 ** -24 * (kind == "f16") + 2.0 ** -130


WIDTHS = [1, 2, 3, 8, 31, 33, 64, 100, 257, 512, 1000, 1024, 2047, 2048, 4096, 5001, 8192, 11008,
          16384, 16390, 40_001]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("kind,param", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"),
                                        ("f16", "f32")])
def test_layernorm(dl, width, kind, param):
    rng = np.random.default_rng(width)
    for rows, pad, rms, bias in ((1, 0, False, True), (5, 1, True, False), (37, 64, False, False),
                                 (23, 2, False, True),
                                 (300 if width <= 5001 else 160, 0, True, True)):
        x = _rows(rng, rows, width, kind, pad)
        w = to_cuda(1 + 0.3 * rng.standard_normal(width), param)
        b = to_cuda(0.2 * rng.standard_normal(width), param) if bias else None
        y, mean, rstd = dl.layernorm_forward(x, w, b, EPS, rms)
        x64, w64, b64 = np64(x), np64(w), None if b is None else np64(b)
        yr, mr, rr = ref.norm64(x64, w64, b64, EPS, rms)
        h = (x64 - mr[:, None]) * rr[:, None]
        tol = _forward_tol(x64, w64, b64, yr, h, rr, kind)
        assert np.all(abs(np64(y) - yr) <= tol), (rows, pad, rms)
        assert np.all(abs(np64(rstd) - rr) <= 50 * U * rr)
        if rms:
            assert mean is None
        else:
            assert np.all(abs(np64(mean) - mr) <= 81 * U * abs(x64).mean(1) + 2.0 ** -140)
        _backward_case(dl, rng, x, w, mean, rstd, rms, bias, kind, param, pad, rows == 37)


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_layernorm_long_runs_of_rows(dl, width, kind, monkeypatch):
    """The same with two blocks, so that each takes many rounds: the rings of
    copies wrap around, the last round is partial, and the statistics are
    fetched in several pieces."""
    monkeypatch.setenv("DL_GRID_LIMIT", "2")
    rng = np.random.default_rng(1000 + width)
    for rows, pad, rms in ((1337 if width <= 2048 else 203, 0, False), (90, 64, True)):
        x = _rows(rng, rows, width, kind, pad)
        w, b = (to_cuda(rng.standard_normal(width)) for _ in range(2))
        y, mean, rstd = dl.layernorm_forward(x, w, b, EPS, rms)
        x64, w64, b64 = np64(x), np64(w), np64(b)
        yr, mr, rr = ref.norm64(x64, w64, b64, EPS, rms)
        h = (x64 - mr[:, None]) * rr[:, None]
        assert np.all(abs(np64(y) - yr) <= _forward_tol(x64, w64, b64, yr, h, rr, kind)), (rows, pad)
        # two blocks: a chain of additions is at most half of the rows
        _backward_case(dl, rng, x, w, mean, rstd, rms, True, kind, "f32", pad, False, 64 + rows / 2)


def _backward_case(dl, rng, x, w, mean, rstd, rms, bias, kind, param, pad, accumulate, chain=None):
    rows, width = x.shape
    dy = _rows(rng, rows, width, kind, pad, 1e-2)
    flat = to_cuda(rng.standard_normal(2 * width + 9), param)
    dw, db = flat[3:3 + width], flat[4 + width:4 + 2 * width] if bias else None  # as in a fragment
    start = flat.clone()
    dx, gw, gb = dl.layernorm_backward(dy, x, w, mean, rstd, dw, db, rms=rms, accumulate=accumulate)
    assert gw is dw and gb is db
    x64, w64, dy64 = np64(x), np64(w), np64(dy)
    m64 = None if mean is None else np64(mean)
    want, dwr, dbr, h = ref.norm64_backward(dy64, x64, w64, m64, np64(rstd), rms)
    # the two row sums are off by 85 u of their terms' magnitudes; xhat by 3 u
    # of |x| + |mean| times rstd, which the subtraction may leave
    r = np64(rstd)[:, None]
    wdy = abs(dy64 * w64)
    herr = 3 * r * (abs(x64) + (0 if rms else abs(m64)[:, None]))
    along = (wdy * abs(h)).mean(1, keepdims=True)
    off_along = 85 * along + (wdy * herr).mean(1, keepdims=True)
    tol = UT[kind] * abs(want) + U * r * (8 * wdy + 90 * wdy.mean(1, keepdims=True)
                                          + abs(h) * (off_along + 4 * along) + herr * along)
    assert np.all(abs(np64(dx) - want) <= tol + 2.0 ** -24 * (kind == "f16") + 2.0 ** -130)
    # sums over rows: no chain of additions longer than 64 + rows / 8
    chain = chain or 64 + rows / 8
    up = UT[param]
    old = np64(start[3:3 + width]) if accumulate else 0.0
    tw = U * (chain * (abs(dy64) * abs(h)).sum(0) + (abs(dy64) * herr).sum(0) + 2 * abs(old))
    assert np.all(abs(np64(dw) - (dwr + old)) <= tw + up * abs(dwr + old) + 2.0 ** -130)
    if bias:
        old = np64(start[4 + width:4 + 2 * width]) if accumulate else 0.0
        tb = U * (chain * abs(dy64).sum(0) + 2 * abs(old))
        assert np.all(abs(np64(db) - (dbr + old)) <= tb + up * abs(dbr + old) + 2.0 ** -130)
    keep = torch.ones(flat.numel(), dtype=torch.bool, device="cuda")
    keep[3:3 + width] = False
    if bias:
        keep[4 + width:4 + 2 * width] = False
    assert torch.equal(flat[keep], start[keep])  # nothing beside the gradients is written


def test_layernorm_rows_zero_and_one_dimension(dl):
    w, b = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")
    y, mean, rstd = dl.layernorm_forward(torch.empty(0, 64, device="cuda"), w, b)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dw, db = torch.full((64,), 3.0, device="cuda"), torch.full((64,), 4.0, device="cuda")
    e = torch.empty(0, 64, device="cuda")
    dl.layernorm_backward(e, e, w, mean, rstd, dw, db, accumulate=True)
    assert (dw == 3).all() and (db == 4).all()
    dl.layernorm_backward(e, e, w, mean, rstd, dw, db)
    assert (dw == 0).all() and (db == 0).all()
    x = torch.randn(64, device="cuda")
    y, mean, rstd = dl.layernorm_forward(x, w, b)
    y2, _, _ = dl.layernorm_forward(x[None, None], w, b)
    assert y.shape == (64,) and mean.shape == () and torch.equal(y, y2[0, 0])


@pytest.mark.parametrize("width", [96, 2048, 20_000])
def test_layernorm_bad_rows_stay_alone(dl, width):
    rng = np.random.default_rng(1)
    x = _rows(rng, 40, width, "bf16", 0)
    w = to_cuda(np.ones(width))
    good, gm, gr = dl.layernorm_forward(x, w)
    x2 = x.clone()
    x2[3, 5], x2[17, width - 1], x2[39, 0] = float("nan"), float("inf"), -float("inf")
    y, mean, rstd = dl.layernorm_forward(x2, w)
    ok = [r for r in range(40) if r not in (3, 17, 39)]
    assert torch.equal(y[ok], good[ok])
    assert all(bool(torch.isnan(y[r]).any()) for r in (3, 17, 39))
    dy = _rows(rng, 40, width, "bf16", 0, 1e-2)
    a, _, _ = dl.layernorm_backward(dy, x, w, gm, gr, bias=False)
    c, _, _ = dl.layernorm_backward(dy, x2, w, mean, rstd, bias=False)
    assert torch.equal(a[ok], c[ok])


def test_layernorm_constant_rows_and_large_offsets(dl):
    """A constant row has variance 0: y is the bias, and rstd 1/sqrt(eps).
    A row of small spread on a large offset keeps its spread."""
    w, b = torch.full((512,), 2.0, device="cuda"), torch.full((512,), 0.5, device="cuda")
    y, mean, rstd = dl.layernorm_forward(torch.full((3, 512), 7.0, device="cuda"), w, b, EPS)
    assert (y == 0.5).all() and (mean == 7).all()
    assert abs(float(rstd[0]) * np.sqrt(EPS) - 1) < 1e-6
    x = to_cuda(1000.0 + np.random.default_rng(0).integers(-8, 9, (4, 512)) / 8.0)
    y, mean, rstd = dl.layernorm_forward(x, w, b, 0.0)
    yr, mr, rr = ref.norm64(np64(x), np64(w), np64(b), 0.0, False)
    h = (np64(x) - mr[:, None]) * rr[:, None]
    assert np.all(abs(np64(y) - yr) <= _forward_tol(np64(x), np64(w), np64(b), yr, h, rr, "f32"))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("width", [100, 2048, 18_000])
def test_layernorm_in_place(dl, kind, width):
    rng = np.random.default_rng(2)
    x, dy = _rows(rng, 33, width, kind, 0), _rows(rng, 33, width, kind, 0, 1e-2)
    w, b = to_cuda(rng.standard_normal(width)), to_cuda(rng.standard_normal(width))
    y, mean, rstd = dl.layernorm_forward(x, w, b)
    dx, dw, db = dl.layernorm_backward(dy, x, w, mean, rstd)
    dx2, dw2, db2 = dl.layernorm_backward(dy, x, w, mean, rstd, dx=dy)
    assert dx2 is dy and torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)
    y2, _, _ = dl.layernorm_forward(x, w, b, y=x)
    assert y2 is x and torch.equal(y, y2)


def test_layernorm_repeats_bit_for_bit(dl):
    rng = np.random.default_rng(5)
    x, dy = _rows(rng, 3000, 1024, "bf16", 0), _rows(rng, 3000, 1024, "bf16", 0, 1e-2)
    w = to_cuda(rng.standard_normal(1024))
    _, mean, rstd = dl.layernorm_forward(x, w)
    a = dl.layernorm_backward(dy, x, w, mean, rstd)
    for _ in range(5):
        c = dl.layernorm_backward(dy, x, w, mean, rstd)
        assert all(torch.equal(p, q) for p, q in zip(a, c))


def test_layernorm_beyond_2_31_elements(dl):
    rows, width = 70_001, 32_768
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(6)
    tail = _rows(rng, 3, width, "bf16", 0)
    x[-3:] = tail
    w = to_cuda(rng.standard_normal(width))
    y, mean, rstd = dl.layernorm_forward(x, w)
    want, wm, wr = dl.layernorm_forward(tail, w)
    assert torch.equal(y[-3:], want) and torch.equal(mean[-3:], wm) and torch.equal(rstd[-3:], wr)
    assert int(y[:-3].count_nonzero()) == 0
    dy = y.zero_()
    dy[-3:] = _rows(rng, 3, width, "bf16", 0, 1e-2)
    part, pw, pb = dl.layernorm_backward(dy[-3:].clone(), tail, w, wm, wr)
    dx, dw, db = dl.layernorm_backward(dy, x, w, mean, rstd, dx=dy)
    assert torch.equal(dx[-3:], part)
    # three rows that are not zero: any order of their sum is within 3 u of the terms' magnitudes
    for a, p, t in ((dw, pw, abs(np64(pw))), (db, pb, abs(np64(pb)))):
        assert np.all(abs(np64(a) - np64(p)) <= 1e-4 * (t + t.mean()))


@pytest.mark.parametrize("rms", [False, True])
def test_layer_norm_gradients_against_differences(dl, rms):
    """The autograd operation's gradients against central differences of the
    64-bit forward pass. Differences: step 1e-4, error at most step^2 times a
    third derivative of order one, 1e-7; fp32 gradients: 1e-5 of their scale."""
    rng = np.random.default_rng(7)
    x, w, b = rng.standard_normal((3, 17)), rng.standard_normal(17), rng.standard_normal(17)
    c = rng.standard_normal((3, 17))
    xt, wt, bt = (to_cuda(t).requires_grad_() for t in (x, w, b))
    (dl.layer_norm(xt, wt, bt, EPS, rms) * to_cuda(c)).sum().backward()
    x, w, b, c = (np64(t) for t in (xt, wt, bt, to_cuda(c)))

    def f(x, w, b):
        return float((ref.norm64(x, w, b, EPS, rms)[0] * c).sum())
    for t, args in ((xt, 0), (wt, 1), (bt, 2)):
        base = [x, w, b]
        got = np64(t.grad)
        for i in np.ndindex(got.shape):
            up, dn = [v.copy() for v in base], [v.copy() for v in base]
            up[args][i] += 1e-4
            dn[args][i] -= 1e-4
            d = (f(*up) - f(*dn)) / 2e-4
            assert abs(got[i] - d) <= 1e-5 * max(1.0, abs(got).max()), (args, i)


def test_layer_norm_takes_broadcast_gradients_and_leading_dimensions(dl):
    x = torch.randn(2, 3, 65, device="cuda", requires_grad=True)
    w = torch.randn(65, device="cuda", requires_grad=True)
    dl.layer_norm(x, w).sum().backward()          # dy is one value, expanded
    g, gw = x.grad.clone(), w.grad.clone()
    x.grad = w.grad = None
    dl.layer_norm(x, w).backward(torch.ones(2, 3, 65, device="cuda"))
    assert torch.equal(g, x.grad) and torch.equal(gw, w.grad)


# ----------------------------------------------------------------------------
# streams, canaries


def test_inner_calls_on_another_stream(dl):
    rng = np.random.default_rng(12)
    s = torch.cuda.Stream()
    P, Q = (_problem(dl, [[70_000, 31]], "bf16", 8, 2) for _ in range(2))
    x = _rows(rng, 500, 1536, "bf16", 0)
    w = to_cuda(rng.standard_normal(1536))
    wsa, wsb = (dl.new_workspace(dl.grad_norm_workspace_bytes()) for _ in range(2))
    torch.cuda.synchronize()
    clip = dl.grad_norm(P["grad"], 0.1, workspace=wsa)
    dl.adamw_step(P["jobs"], 4, clip=clip, seed=1, **HYPER)
    y, mean, rstd = dl.layernorm_forward(x, w)
    d = dl.layernorm_backward(x, x, w, mean, rstd)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        clip2 = dl.grad_norm(Q["grad"], 0.1, workspace=wsb)
        dl.adamw_step(Q["jobs"], 4, clip=clip2, seed=1, **HYPER)
        y2, mean2, rstd2 = dl.layernorm_forward(x, w, stream=s)
        d2 = dl.layernorm_backward(x, x, w, mean2, rstd2)
    s.synchronize()
    assert torch.equal(clip, clip2) and torch.equal(y, y2) and torch.equal(rstd, rstd2)
    assert all(torch.equal(a, b) for a, b in zip(d, d2))
    for k in ("theta", "m", "v", "msc", "ssc"):
        assert torch.equal(P[k][0].view(torch.uint8), Q[k][0].view(torch.uint8)), k


def test_what_a_call_allocates_belongs_to_its_stream(dl):
    """A call on a given stream without a workspace or outputs, while the
    current stream is busy: its scratch is zeroed and used on that stream."""
    s = torch.cuda.Stream()
    g = to_cuda(np.random.default_rng(3).standard_normal(300_000))
    x, w = g[:65536].view(64, 1024), to_cuda(np.ones(1024))
    want, (y, mean, rstd) = dl.grad_norm([g], 1.0), dl.layernorm_forward(x, w)
    d = dl.layernorm_backward(x, x, w, mean, rstd)
    dl.grad_norm([g], 1.0, stream=s)  # the stream's first allocations
    dl.layernorm_backward(x, x, w, *dl.layernorm_forward(x, w, stream=s)[1:], stream=s)
    for size in (256, dl.grad_norm_workspace_bytes(), 1 << 20):  # blocks that are not zero when reused
        torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    a = dl.grad_norm([g], 1.0, stream=s)
    y2, mean2, rstd2 = dl.layernorm_forward(x, w, stream=s)
    d2 = dl.layernorm_backward(x, x, w, mean2, rstd2, stream=s)
    s.synchronize()
    busy = not torch.cuda.current_stream().query()
    with torch.cuda.stream(s):
        assert torch.equal(a, want) and torch.equal(y, y2) and torch.equal(rstd, rstd2)
        assert all(torch.equal(p, q) for p, q in zip(d, d2))
    assert busy  # the comparison did not wait for the current stream
    torch.cuda.synchronize()


def test_inner_calls_in_a_graph(dl):
    """Captured once and replayed: the clip, a step and a norm give what the
    same calls give outside a graph."""
    rng = np.random.default_rng(13)
    P, Q = (_problem(dl, [[30_000, 5]], "f32", 32, 3) for _ in range(2))
    x = _rows(rng, 64, 512, "f32", 0)
    w = to_cuda(rng.standard_normal(512))
    ws = dl.new_workspace(dl.grad_norm_workspace_bytes())
    clip = torch.zeros(2, device="cuda")
    dl.grad_norm(P["grad"], 0.1, clip, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dl.grad_norm(P["grad"], 0.1, clip, ws)
        dl.adamw_step(P["jobs"], 2, clip=clip, **HYPER)
        y, _, _ = dl.layernorm_forward(x, w)
    for _ in range(3):
        graph.replay()
        dl.adamw_step(Q["jobs"], 2, clip=dl.grad_norm(Q["grad"], 0.1), **HYPER)
    torch.cuda.synchronize()
    for k in ("theta", "m", "v"):
        assert torch.equal(P[k][0], Q[k][0]), k
    assert torch.equal(y, dl.layernorm_forward(x, w)[0])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_adamw_writes_nothing_outside_its_buffers(dl, bits, kind):
    pad = 64
    for numels in ([1], [3, 126, 130], [5000, 1, 2]):
        F = dl.Fragment(numels)
        n = F.n
        slots = dl.adamw_scale_slots(F)
        state = torch.float32 if bits == 32 else torch.float8_e4m3fn

        def guarded(count, dtype):
            size = torch.empty(0, dtype=dtype).element_size()
            raw = torch.full(((count + 2 * pad) * size,), 0x3C, dtype=torch.uint8, device="cuda")
            return raw, raw.view(dtype)[pad:pad + count]
        bufs = {k: guarded(c, d) for k, c, d in (
            ("theta", n, torch.float32), ("grad", n, TYPES[kind]), ("m", n, state), ("v", n, state),
            ("msc", slots, torch.float32), ("ssc", slots, torch.float32),
            ("copy", n, torch.bfloat16))}
        by8 = bits == 8
        dl.adamw_step(dl.AdamWJobs(
            [F], [bufs["theta"][1]], [bufs["grad"][1]], [bufs["m"][1]], [bufs["v"][1]],
            [bufs["msc"][1]] if by8 else None, [bufs["ssc"][1]] if by8 else None,
            [bufs["copy"][1]]), 1, **HYPER)
        for k, (raw, inside) in bufs.items():
            size = inside.element_size()
            assert (raw[:pad * size] == 0x3C).all() and (raw[-pad * size:] == 0x3C).all(), (k, numels)
        if by8:  # slots without a block stay as they were
            slot = ref.places(numels) // ref.BLOCK
            free = [s for s in range(slots) if s not in set(slot.tolist())]
            for k in ("msc", "ssc"):
                assert (bufs[k][1][free].view(torch.int32) == 0x3C3C3C3C).all()


@pytest.mark.parametrize("width", [1, 7, 130, 2048, 2050])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_layernorm_writes_nothing_outside_its_rows(dl, width, kind):
    """Rows inside wider ones: the columns between them keep their values."""
    rng = np.random.default_rng(width)
    for extra in (1, 8):
        R = 19
        x, dy = _rows(rng, R, width, kind, extra), _rows(rng, R, width, kind, extra)
        out = torch.full((R + 2, width + extra), 3.0, dtype=TYPES[kind], device="cuda")
        y = out[1:-1, :width]
        w = to_cuda(rng.standard_normal(width))
        want, mean, rstd = dl.layernorm_forward(x, w)
        dl.layernorm_forward(x, w, y=y)
        assert torch.equal(y, want)
        dx, _, _ = dl.layernorm_backward(dy, x, w, mean, rstd)
        assert (out[0] == 3).all() and (out[-1] == 3).all() and (out[:, width:] == 3).all()
        dl.layernorm_backward(dy, x, w, mean, rstd, dx=y)
        assert torch.equal(y, dx)
        assert (out[0] == 3).all() and (out[-1] == 3).all() and (out[:, width:] == 3).all()


# ----------------------------------------------------------------------------
# the path that uses them together


@pytest.mark.parametrize("bits", [8, 32])
def test_example_trains(dl, bits):
    """examples/inner_outer.py: inner steps through the norms, the clip and
    AdamW, then the outer step; the loss falls from ln(512) = 6.24."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "inner_outer.py")
    spec = importlib.util.spec_from_file_location("inner_outer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.main(["--learners", "2", "--rounds", "5", "--inner", "20", "--bits", str(bits)])
    assert losses[0] < 6.5 and losses[-1] < 0.5 * losses[0], losses
