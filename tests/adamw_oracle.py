"""fp64 oracle of the AdamW step and integer oracle of its 8-bit states, written from the formats'
definition (include/xtvxy.h) on the CPU."""
import numpy as np

BLOCK = 128


def m_value(code):
    """e4m3 without infinities."""
    code = np.asarray(code, dtype=np.int64)
    e, f = (code >> 3) & 15, code & 7
    mag = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    return np.where((code & 127) == 127, np.nan, np.where(code & 128, -mag, mag))


def v_value(code):
    code = np.asarray(code, dtype=np.int64)
    e, f = code >> 4, code & 15
    return np.where(e == 0, f * 2.0 ** -18, (1 + f / 16.0) * 2.0 ** (e - 15.0))


def decode(codes, exps, value):
    return value(codes) * np.exp2(np.repeat(exps.astype(np.float64), BLOCK)[:len(codes)] - 127)


def random_bits(first, n, seed, step):
    mask = 0xffffffff
    salt = (seed * 0xBB67AE85 + step * 0x3C6EF373) & mask
    x = ((np.arange(first, first + n, dtype=np.uint64) & mask) * 0x9E3779B1 + salt) & mask
    x = ((x ^ (x >> 16)) * 0xBB67AE85) & mask
    x = ((x ^ (x >> 15)) * 0x3C6EF373) & mask
    return (x ^ (x >> 16)).astype(np.int64)


def smallest_exponent(top, limit):
    """Smallest biased e in 1..253 with top <= limit 2^(e - 127)."""
    e = np.arange(1, 254)
    fits = top[:, None] <= limit * np.exp2(e - 127.0)[None, :]
    return np.where(fits.any(1), e[fits.argmax(1)], 253)


def codes_and_fractions(x, bits, least):
    """|x| in steps of `bits` mantissa bits (subnormal below 2^least): (code, remainder in [0, 1))."""
    e = np.frexp(np.maximum(x, 2.0 ** least))[1] - 1.0  # floor(log2), exact
    steps = x / 2.0 ** (e - bits)
    whole = np.floor(steps)
    normal = steps >= 2 ** bits
    code = np.where(normal, (e - least + 1) * 2 ** bits + whole - 2 ** bits, whole)
    return code.astype(np.int64), steps - whole


def encode(m, v, first, seed, step):
    """(m codes, v codes, m exponents, v exponents) and, per element, how near each remainder is to the
    random threshold that decides its rounding."""
    n = len(m)
    pad = (-n) % BLOCK
    mb, vb = np.pad(m, (0, pad)).reshape(-1, BLOCK), np.pad(v, (0, pad)).reshape(-1, BLOCK)
    me = np.maximum(smallest_exponent(np.nanmax(np.where(np.isfinite(mb), np.abs(mb), 0), 1), 1.75) - 8, 1)
    ve = smallest_exponent(np.nanmax(np.where(np.isfinite(vb), vb, 0), 1), 1.9375)
    rnd = random_bits(first, n, seed, step)
    xm = np.abs(m) / np.exp2(np.repeat(me, BLOCK)[:n] - 127.0)
    xv = v / np.exp2(np.repeat(ve, BLOCK)[:n] - 127.0)
    with np.errstate(invalid="ignore"):
        cm, fm = codes_and_fractions(np.where(np.isfinite(xm), xm, 0), 3, -6)
        cv, fv = codes_and_fractions(np.where(np.isfinite(xv), xv, 0), 4, -14)
    um = ((rnd >> 19) + 0.5) / 2.0 ** 13
    uv = (rnd & 0x7ffff) / 2.0 ** 19
    qm, qv = cm + (fm + um >= 1), cv + (fv + uv >= 1)
    qv = np.where((v > 0) & (qv < 1), 1, qv)
    qm = np.where(np.isfinite(m), qm + np.where(m < 0, 128, 0), 127)
    qv = np.where(np.isfinite(v), qv, 255)
    return qm, qv, me, ve, np.abs(fm + um - 1), np.abs(fv + uv - 1)


def update(p, g, m, v, t, lr, b1, b2, eps, wd):
    """The step in fp64: new (p, m, v), and a bound of fp32's roundings in each."""
    m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    den = np.sqrt(v1) / np.sqrt(1 - b2 ** t) + eps
    upd = lr / (1 - b1 ** t) * m1 / den
    p1 = p * (1 - lr * wd) - upd
    u = 2.0 ** -24
    em = 3 * u * (np.abs(b1 * m) + np.abs((1 - b1) * g)) + 1e-44
    ev = 4 * u * (b2 * v + (1 - b2) * g * g) + 1e-44
    # sums that cancel in m leave its error next to a small value: carried through absolutely; the
    # square root halves v's relative error, root, reciprocal and products add a few units each
    ep = 4 * u * np.abs(p) + lr / (1 - b1 ** t) * em / den + 16 * u * np.abs(upd) + 2 * u * np.abs(p1) + 1e-44
    return p1, m1, v1, ep, em, ev
