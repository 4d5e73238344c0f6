"""The quantised cache in plain 64-bit numpy (test infrastructure), written
from the definitions in include/indexcache.h, with the tolerances of the
attention over it.

Tolerance of the attention, elementwise, for a row with softmax weights p_s
(normalised), cache scales g_s and values V_s = g_s * code_s:

    2^-8 |ref|                    the output's rounding to bfloat16 (half a
                                  step is 2^-8 relative at worst)
  + sum_s err_s |code_s|          the rounding of the weights: w_s = p_s g_s
                                  is kept as an e4m3 number and an e5m2 number
                                  for the rest: half a step is 2^-4 of a
                                  number and 2^-3 of the rest, 2^-7 in all.
                                  The largest weight stands at 2^2 or more.
                                  Weights below e4m3's normal range (2^-6)
                                  leave at most half its smallest step, 2^-10,
                                  to the rest, an error of 2^-13, 2^-15 of the
                                  largest weight; those below 2^-10 are the
                                  rest alone, off by 2^-3 of themselves, or by
                                  half of e5m2's smallest step, 2^-17, 2^-19
                                  of the largest: err_s = max(2^-7 w,
                                  min(2^-15 max w, 2^-3 w), 2^-19 max w)
  + 2 d (sum_s p_s |V_s|)           the logits' error d (natural units):
                                    float32 sums of 576 products, each
                                    rounding 2^-24, in units of the sum of
                                    absolute terms; q kept to 2^-17 of its
                                    row's largest value; 2^-21 of the logit
                                    for its scaling, and 2^-21 for exp.  A
                                    weight is off by d, and so is the
                                    normaliser: twice d.
"""
import numpy as np

ROW, WIDTH, VALUES, KEYS = 640, 576, 512, 128


def decode_e4m3(codes):
    """Values of e4m3 codes: 4 exponent bits (bias 7), 3 of mantissa, no
    infinities, 0x7f and 0xff are NaN."""
    c = np.asarray(codes, dtype=np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


_GRID = decode_e4m3(np.arange(127))             # 0 .. 448, ascending


def encode_e4m3(x):
    """Nearest e4m3 code, ties to the even mantissa, saturating; NaN -> 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=448.0)), 448.0)
    hi = np.searchsorted(_GRID, a)              # first grid value >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _GRID[lo], _GRID[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isnan(x), 127, code | (np.signbit(x) << 7)).astype(np.uint8)


def row_scale(x):
    """Smallest power of two s >= 2^-32 with max|x| <= 448 s over the finite
    values of each row; 1 for a row without any other than 0."""
    x = np.asarray(x, dtype=np.float64)
    out = np.ones(x.shape[:-1])
    for at in np.ndindex(out.shape):
        r = x[at]
        top = np.abs(r[np.isfinite(r)]).max(initial=0.0)
        if top > 0:
            e = -32
            while top > 448.0 * 2.0 ** e:
                e += 1
            out[at] = 2.0 ** e
    return out


def quantise(x):
    """(codes, scales) of rows."""
    s = row_scale(x)
    return encode_e4m3(np.asarray(x, dtype=np.float64) / s[..., None]), s


def bf16_bits(x):
    """Round float64/32 values to bfloat16 (nearest, ties to even): uint16 bits."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    nan = (u & 0x7FFFFFFF) > 0x7F800000
    return np.where(nan, ((u >> 16) | 0x40).astype(np.uint16), r)


def bf16_value(bits):
    return (np.asarray(bits, dtype=np.uint32) << 16).view(np.float32).astype(np.float64)


def pack_rows(kv):
    """Cache rows [n, 640] uint8 and scales [n] of latent rows [n, 576]."""
    codes, scales = quantise(np.asarray(kv)[:, :VALUES])
    with np.errstate(over="ignore"):
        rest = bf16_bits(np.asarray(kv, dtype=np.float64)[:, VALUES:] / scales[:, None])
    rows = np.concatenate([codes, np.ascontiguousarray(rest).view(np.uint8)], axis=1)
    return rows, scales.astype(np.float32)


def unpack_rows(rows, scales):
    """float64 [n, 576] of cache rows."""
    rows = np.ascontiguousarray(rows)
    rest = bf16_value(np.ascontiguousarray(rows[:, VALUES:]).view(np.uint16))
    return np.concatenate([decode_e4m3(rows[:, :VALUES]), rest], axis=1) * np.asarray(scales, np.float64)[:, None]


def seen_positions(length, Lq, node, mask, idx):
    """Positions that a row sees, in the order it lists them (idx None: all)."""
    ctx = length - Lq
    listed = range(length) if idx is None else [int(s) for s in idx]
    return [s for s in listed if 0 <= s < length and (s < ctx or mask >> (s - ctx) & 1)]


def chain(node):
    return (2 << node) - 1


def attend(q, kv, scales, seen, scale):
    """One query row's heads q [Hq, 576] over rows `seen` of the logical cache
    kv [T, 576] (unpacked values), scales [T].  Returns (out, tolerance)."""
    q = np.asarray(q, np.float64)
    Hq = q.shape[0]
    if not seen:
        return np.zeros((Hq, VALUES)), np.zeros((Hq, VALUES))
    k = kv[seen]
    g = np.asarray(scales, np.float64)[seen]
    s = q @ k.T * scale
    p = np.exp(s - s.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    ref = p @ k[:, :VALUES]
    v = np.abs(k[:, :VALUES])
    w = p * g
    top = w.max(axis=1, keepdims=True)
    err = np.maximum(np.maximum(2.0 ** -7 * w, np.minimum(2.0 ** -15 * top, 2.0 ** -3 * w)), 2.0 ** -19 * top)
    terms = np.abs(q) @ np.abs(k).T * abs(scale)
    floor = np.abs(q).max(axis=1, keepdims=True) * np.abs(k).sum(axis=1) * abs(scale)
    d = (576 * 2.0 ** -24 * terms + 2.0 ** -17 * floor + 2.0 ** -21 * np.abs(s) + 2.0 ** -21).max(axis=1)
    tol = 2.0 ** -8 * np.abs(ref) + err @ (v / g[:, None]) + 2 * d[:, None] * (p @ v)
    return ref, tol


def check_rows(got, ref, tol, what):
    got = np.asarray(got, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), "%s: NaN in other places" % what
    ok = ~np.isnan(ref)
    over = np.abs(got - ref)[ok] - tol[ok]
    assert over.size == 0 or over.max() <= 0, "%s: %.3g over the tolerance" % (what, over.max())
