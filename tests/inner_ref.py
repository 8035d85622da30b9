"""Plain implementations of the inner-step operators for the tests.

numpy only, written from the formulas in include/diloco_sync.h. The AdamW and
layer norm references work in 64 bits; ``adamw8_codes`` also restates the 8-bit
states' fp32 arithmetic and rounding operation by operation, so that codes and
scales can be compared bit for bit."""
import numpy as np

BLOCK = 128
M64 = (1 << 64) - 1
GOLDEN = 0x9E3779B97F4A7C15


# ----------------------------------------------------------------------------
# e4m3 and its stochastic rounding


def e4m3_values():
    """The value of every e4m3 code (NaN for 0x7f and 0xff)."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if (c & 0x7F) == 0x7F else (-v if c & 0x80 else v)
    return out


E4M3 = e4m3_values()


def mix(z):
    z = np.asarray(z, dtype=np.uint64)
    with np.errstate(over="ignore"):
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
    return z ^ (z >> np.uint64(31))


def reverse16(x):
    return np.array([int(f"{int(v):016b}"[::-1], 2) for v in range(65536)], np.uint32)[x]


def random16(seed, step, place):
    """(for m, for s): 16 bits of every place (slot * 128 + element of the block)."""
    place = np.asarray(place, dtype=np.uint64)
    key = mix(np.uint64((seed + step * GOLDEN) & M64))
    with np.errstate(over="ignore"):
        z = mix(key + (place >> np.uint64(2)) * np.uint64(GOLDEN))
    p = (place & np.uint64(3)).astype(np.int64)
    out = []
    for w in (z & np.uint64(0xFFFFFFFF), z >> np.uint64(32)):
        w = w.astype(np.uint32)
        half = np.where(p < 2, w & 0xFFFF, w >> 16)
        out.append(np.where(p & 1, reverse16(half), half).astype(np.uint32))
    return out


def encode(x, r16):
    """e4m3 codes of fp32 values: the magnitude in units of the code's last
    place plus r16 / 2^16, rounded down; at most 448."""
    x = np.asarray(x, dtype=np.float32)
    a = np.abs(x).astype(np.float64)
    _, e = np.frexp(a)                       # a in [2^(e-1), 2^e)
    e = np.where(a > 0, np.maximum(e - 1, -6), -6)
    units = np.floor(a / 2.0 ** (e - 3.0) * 65536.0).astype(np.int64)  # exact
    code = 8 * (e + 6) + ((units + r16.astype(np.int64)) >> 16)
    code = np.minimum(code, 126) | (np.signbit(x).astype(np.int64) << 7)
    return code.astype(np.uint8)


# ----------------------------------------------------------------------------
# AdamW


def spans(numels):
    """(tensor, first element, end, first slot) of every tensor."""
    o = 0
    for t, n in enumerate(numels):
        yield t, o, o + n, o // BLOCK + t
        o += n


def places(numels, slot0=0):
    """slot0 * 128 + the place of every element of a fragment."""
    out = np.empty(sum(numels), dtype=np.int64)
    for _, a, b, s in spans(numels):
        out[a:b] = (slot0 + s) * BLOCK + np.arange(b - a)
    return out


def slots_of(numels):
    return sum(numels) // BLOCK + len(numels)


def per_element(numels, decay):
    return np.repeat(np.ones(len(numels)) if decay is None else np.asarray(decay, np.float64),
                     numels)


def adamw64(theta, g, m, v, numels, step, lr, b1, b2, eps, wd, decay=None, coef=1.0):
    """One step in 64 bits; v may be given as it is (not its root)."""
    theta, g, m, v = (np.asarray(x, np.float64) for x in (theta, g, m, v))
    g = g * float(coef)
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    keep = 1 - lr * wd * per_element(numels, decay)
    root = np.sqrt(v)
    denom = root / np.sqrt(1 - b2 ** step) + eps
    return theta * keep - lr / (1 - b1 ** step) * m / denom, m, v, denom


def adamw8_codes(g, m8, s8, msc, ssc, numels, step, b1, b2, coef, seed, slot0=0):
    """The new codes and scales, in fp32 with every operation rounded once.
    m8, s8: uint8 codes; msc, ssc: fp32 scales per slot (copied, updated)."""
    f = np.float32
    place = places(numels)
    slot = place // BLOCK
    with np.errstate(all="ignore"):
        gi = g.astype(f) * f(coef)
        m = (E4M3[m8].astype(f) * msc[slot]) * f(b1) + gi * f(1 - b1)
        s = E4M3[s8].astype(f) * ssc[slot]
        v = (s * s) * f(b2) + (gi * gi) * f(1 - b2)
        root = np.sqrt(v)
        rm, rs = random16(seed, step, place + slot0 * BLOCK)
        out = []
        for x, r, old, least in ((m, rm, msc, 0.0), (root, rs, ssc, 2.0 ** -9)):
            top = np.zeros(old.size, f)
            np.maximum.at(top, slot, np.abs(x))
            k = np.maximum((top.view(np.int32) >> 23) - 127, -53)
            scale = np.where(np.isfinite(top), np.ldexp(f(1), k - 7).astype(f), f(np.nan))
            used = np.zeros(old.size, bool)
            used[slot] = True
            y = x / np.ldexp(f(1), k - 7).astype(f)[slot]
            y = np.where(y > 0, np.maximum(y, f(least)), y)
            out += [encode(np.nan_to_num(y, nan=0.0, posinf=0.0, neginf=0.0), r),
                    np.where(used, scale, old).astype(f)]
    return out[0], out[1], out[2], out[3], m, v


# ----------------------------------------------------------------------------
# layer norm


def norm64(x, w, b, eps, rms):
    x, w = x.astype(np.float64), w.astype(np.float64)
    mean = np.zeros(len(x)) if rms else x.mean(1)
    d = x - mean[:, None]
    rstd = 1 / np.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None] * w
    return (y if b is None else y + b.astype(np.float64)), mean, rstd


def norm64_backward(dy, x, w, mean, rstd, rms):
    """From the saved statistics, as the operator does."""
    dy, x, w, rstd = (t.astype(np.float64) for t in (dy, x, w, rstd))
    mean = np.zeros(len(x)) if rms else mean.astype(np.float64)
    h = (x - mean[:, None]) * rstd[:, None]
    wdy = dy * w
    dx = wdy - h * (wdy * h).mean(1, keepdims=True)
    if not rms:
        dx = dx - wdy.mean(1, keepdims=True)
    return dx * rstd[:, None], (dy * h).sum(0), dy.sum(0), h
