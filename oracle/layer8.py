"""The attention layer in 8 bits from its definitions, in numpy: the rotation's
frequencies and turns, block-scaled caches (codes with a power of two for each 16
tokens and head) and int8 linear layers.  TEST INFRASTRUCTURE ONLY (see
``oracle/__init__.py``)."""
import numpy as np

from oracle.formats import E4M3_POSITIVE, E4M3_TABLE

BLOCK = 16
MOST = {"e4m3": 448.0, "int8": 127.0}           # largest code
MOST_BYTE = {"e4m3": 246, "int8": 240}


# ------------------------------------------------------------- rotation ----

def turns(rotary_dim, base=10000.0, scaling="none", factor=1.0, original=8192.0, slow=1.0, fast=None, pair_factors=None):
    """(turns a position of every pair, in extended precision, amplitude)."""
    L = np.longdouble
    d, pi2 = rotary_dim, 2 * L("3.14159265358979323846264338327950288")
    fast = (32.0 if scaling == "yarn" else 4.0) if fast is None else fast
    b = L(base) * L(factor) ** (L(d) / (d - 2)) if scaling == "ntk" else L(base)
    i = np.arange(d // 2, dtype=np.longdouble)
    w = b ** (-2 * i / d)                       # radians
    if scaling == "linear":
        w = w / L(factor)
    elif scaling == "yarn":
        pair = lambda t: d * np.log(L(original) / (t * pi2)) / (2 * np.log(b))  # noqa: E731
        lo, hi = max(np.floor(pair(fast)), 0), min(np.ceil(pair(slow)), d - 1)
        r = np.clip((i - lo) / max(hi - lo, L("0.001")), 0, 1)
        w = w / L(factor) * r + w * (1 - r)
    elif scaling == "wavelength":
        k = np.clip((L(original) * w / pi2 - slow) / (L(fast) - slow), 0, 1)
        w = w * k + w / L(factor) * (1 - k)
    if pair_factors is not None:
        w = w / np.asarray(pair_factors, np.longdouble)
    return w / pi2, 0.1 * np.log(factor) + 1.0 if scaling == "yarn" else 1.0


def rotate(x, positions, turn, layout, amplitude=1.0):
    """x [T, heads, dim] float64 rotated; rows of a negative position as they are.

    Returns (y, tol): tol bounds fp32 evaluation before the last rounding.  The angle within an eighth of a turn is off
    by 3 units of fp32 (2^-24) of at most pi / 4 and the series' rounding is 2 units more, so cosine and sine are off by
    less than 3e-7; the two products, their sum and the amplitude add 4 units: 6e-7 of |a| + |b| in all."""
    n = len(turn)
    rot = 2 * n
    y, tol = x.copy(), np.zeros_like(x)
    frac = np.mod(np.asarray(positions, np.longdouble)[:, None] * turn, 1)
    angle = (frac * 2 * np.longdouble("3.14159265358979323846264338327950288")).astype(np.float64)
    c, s = amplitude * np.cos(angle)[:, None], amplitude * np.sin(angle)[:, None]
    ia, ib = (slice(0, n), slice(n, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., ia], x[..., ib]
    live = (np.asarray(positions) >= 0)[:, None, None]
    y[..., ia] = np.where(live, a * c - b * s, a)
    y[..., ib] = np.where(live, b * c + a * s, b)
    bound = np.where(live, 6e-7 * abs(amplitude) * (np.abs(a) + np.abs(b)), 0.0)
    tol[..., ia], tol[..., ib] = bound, bound
    return y, tol


# --------------------------------------------------- block-scaled caches ----

def round_codes(x, kind):
    """Values in steps of their scale to codes (as float64 values): nearest, ties to even, clamped."""
    if kind == "int8":
        return np.where(np.isnan(x), 0.0, np.clip(np.rint(x), -127, 127))
    mag = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(E4M3_POSITIVE, mag, side="left"), 1, 126)
    lo = hi - 1
    dl, dh = mag - E4M3_POSITIVE[lo], E4M3_POSITIVE[hi] - mag
    v = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), E4M3_POSITIVE[hi], E4M3_POSITIVE[lo])
    return np.where(np.isnan(x), np.nan, np.copysign(v, x))


def scale_byte(top, kind):
    """Smallest byte e with top <= MOST * 2^(e - 127), within 1 .. the largest."""
    if top == 0:
        return 1
    m, e = np.frexp(top / MOST[kind])           # float64: exact enough that no fp32 value can cross
    return int(np.clip(127 + e - (m == 0.5), 1, MOST_BYTE[kind]))


def code_values(raw, kind):
    """Cache bytes as the codes' values."""
    return E4M3_TABLE[raw.astype(np.int64)] if kind == "e4m3" else raw.view(np.int8).astype(np.float64)


def append(rows, slots, codes, scales, kind):
    """codes [pages, heads, page, dim] (values) and scales [pages, heads, page / 16] (bytes) after one call wrote rows
    [T, heads, dim] (float64) at slots."""
    codes, scales = codes.copy(), scales.copy()
    pages, heads, page, dim = codes.shape
    runs, last = [], None
    for t, s in enumerate(slots):
        if not 0 <= s < pages * page:
            last = None
            continue
        if last is None or s != last + 1 or s % BLOCK == 0:
            runs.append([])
        runs[-1].append((t, int(s)))
        last = s
    for run in runs:
        s0 = run[0][1]
        pg, first = s0 // page, s0 % page // BLOCK * BLOCK
        fresh = s0 % BLOCK == 0
        t = [x for x, _ in run]
        at = [x % page - first for _, x in run]
        others = np.setdiff1d(np.arange(BLOCK), at)
        for h in range(heads):
            x = rows[t, h]
            fin = np.abs(x[np.isfinite(x)])
            need = scale_byte(fin.max() if fin.size else 0.0, kind)
            old = 1 if fresh else int(np.clip(scales[pg, h, first // BLOCK], 1, MOST_BYTE[kind]))
            e = max(need, old)
            blk = codes[pg, h, first:first + BLOCK]
            if fresh:
                blk[others] = 0.0
            elif e > old:
                blk[others] = round_codes(blk[others] * 2.0 ** (old - e), kind)
            blk[at] = round_codes(x * 2.0 ** (127 - e), kind)
            scales[pg, h, first // BLOCK] = e
    return codes, scales


def block_values(codes, scales):
    """What a block-scaled cache stands for."""
    return codes * np.repeat(2.0 ** (scales.astype(np.float64) - 127), BLOCK, axis=2)[..., None]


def fill(x, kind):
    """(code values, scale bytes) of values x [pages, heads, page, dim], every block as one run."""
    pages, heads, page, dim = x.shape
    b = x.reshape(pages, heads, page // BLOCK, BLOCK, dim)
    top = np.abs(b).max((-1, -2))
    e = np.vectorize(lambda t: scale_byte(t, kind))(top).astype(np.uint8)
    return round_codes(b * 2.0 ** (127.0 - e.astype(np.float64))[..., None, None], kind).reshape(x.shape), e


# ---------------------------------------------------- int8 linear layers ----

def int8_quantize(x):
    """(codes, scales fp32) of the rows of x (values of bf16, as fp32): every step one fp32 operation."""
    x = np.asarray(x, np.float32)
    top = np.abs(x).max(1)
    bad, small = ~np.isfinite(top), top < np.float32(2.0 ** -120)
    safe = np.where(bad | small, np.float32(1), top)
    by = np.where(bad | small, np.float32(0), np.float32(127) / safe)
    scale = np.where(bad, np.float32(np.nan), np.where(small, np.float32(0), safe / np.float32(127)))
    return np.rint(np.where((bad | small)[:, None], np.float32(0), x) * by[:, None]).astype(np.int8), scale.astype(np.float32)


def gemm_w8a8(a, a_scale, w, w_scale):
    """fp32 y: the exact sum rounded to fp32, then one fp32 product with each scale."""
    s = a.astype(np.int64) @ w.astype(np.int64).T
    return (s.astype(np.float32) * a_scale[:, None]) * w_scale[None]
