"""Plain 64-bit forms of what the 4-bit cache and the step before it compute, for their tests.

Tolerances, counted before any run.

normed and rotated rows (rotated()): the result is rounded to bf16 once, half a step, 2^-8 of |y|.  Before that in fp32: the
sum of d <= 128 squares in 16 + 3 steps, 1/sqrt within 2 units, two products, then two products and a sum of the rotation: below
32 roundings of 2^-24 each on terms of at most |x_a c| + |x_b s|, so 2^-19 of that sum.

attention (attend()): with weights p_j and COLD values lo + code * span / 15, the kernel rounds p_j span_j to fp16 (half a step,
2^-11 of the term) and holds the rest in fp32; over a HOT prefix it rounds p_j to bf16 (2^-8 of the term); the output is rounded to
bf16 (2^-8 of |O|).  fp32 errors as counted for the prompt attention's tests (scores below 2^9, at most 2^13 keys): 2^-12 of the
absolute terms.  Weights are relative to a score that the request's largest passes by at most 2^4, so that they add up to 1 or
more, and the spans they meet are scaled so that the largest so far lies between 2^10 and 2^11; a product below fp16's normal range is
off by half a step of 2^-24, 2^-35 of the largest span, and at most 2^13 of them by 2^-22.  With H = sum p |v| over HOT,
C = sum p (|lo| + span) over COLD, both over Z:
  |O - O*| <= 2^-8 |O*| + (2^-8 + 2^-12) H + (2^-11 + 2^-12) C + 2^-22 max span,     |LSE - LSE*| <= 2e-4.
"""
import numpy as np

LSE_ABS = 2e-4


def bf16_bits(x):
    """fp32 array -> bf16 bits, to nearest even (finite values)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_value(bits):
    return (np.asarray(bits, np.uint32) << 16).view(np.float32)


def rotated(x, pos, table, rot, interleaved, weight=None, eps=1e-6):
    """x [n, heads, d] fp64 -> y and the sum of absolute terms of each channel."""
    y = x.astype(np.float64).copy()
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    size = np.abs(y)
    if rot:
        row = table[pos].astype(np.float64)[:, None]
        c, s = row[..., :rot // 2], row[..., rot // 2:]
        i = np.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        ya, yb = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
        size[..., a] = np.abs(ya * c) + np.abs(yb * s)
        size[..., b] = np.abs(yb * c) + np.abs(ya * s)
    return y, size


def check_rotated(got, want, what=""):
    y, size = want
    over = np.abs(got.astype(np.float64) - y) - (2.0 ** -8 * np.abs(y) + 2.0 ** -19 * size)
    assert over.size == 0 or over.max() <= 0, f"{what}: off by {over.max():.3g} over its bound"


def encode(x):
    """bf16 values [..., d] -> codes [..., d], lo, span [..., d / 64] and how near each code's border is (in codes), in 64 bits."""
    g = x.astype(np.float64).reshape(*x.shape[:-1], -1, 64)
    lo = g.min(-1, keepdims=True)
    span = bf16_value(bf16_bits(g.max(-1, keepdims=True) - lo)).astype(np.float64)
    span = np.where(span < 2.0 ** -100, 0, span)
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.where(span > 0, (g - lo) * 15 / span, 0)
    border = np.abs(r - np.floor(r) - 0.5)
    return np.minimum(np.rint(r), 15).reshape(x.shape).astype(int), lo[..., 0], span[..., 0], border.reshape(x.shape)


def fields(rows, hkv, d):
    """rows [n, bytes] -> codes [n, hkv, 2, d], lo and span bits [n, hkv, 2, d / 64] by the layout as gk.h words it."""
    n = len(rows)
    codes, scales = np.zeros((n, hkv, 2, d), int), np.zeros((n, hkv, 2, d // 64, 2), np.uint16)
    for h in range(hkv):
        for part in range(2):
            at = h * d + part * d // 2
            words = rows[:, at:at + d // 2].copy().view("<u4")
            for w in range(d // 8):
                c0 = 8 * w if d == 64 else 8 * (w // 2) + 64 * (w % 2)
                for i in range(8):
                    codes[:, h, part, c0 + i] = (words[:, w] >> np.uint32(4 * i)) & np.uint32(15)
            groups = d // 64
            at = hkv * d + h * 2 * groups * 4 + part * groups * 4
            scales[:, h, part] = rows[:, at:at + 4 * groups].copy().view("<u2").reshape(n, groups, 2)
    return codes, scales[..., 0], scales[..., 1]


def values(rows, hkv, d):
    """rows [n, bytes] -> K, V [n, hkv, d] in 64 bits, and |lo| + span of V."""
    codes, lo, span = fields(rows, hkv, d)
    lo, span = (np.repeat(bf16_value(x).astype(np.float64), 64, -1) for x in (lo, span))
    x = lo + codes * span / 15
    return x[:, :, 0], x[:, :, 1], (np.abs(lo) + span)[:, :, 1]


def attend(q, hot, cold):
    """One request: q [hq, d] fp64, hot (K, V) [n, hkv, d], cold (K, V, |lo| + span) [m, hkv, d] -> O, LSE, bound."""
    hq, d = q.shape
    hkv = cold[0].shape[1]
    O, L, E = np.zeros((hq, d)), np.full(hq, -np.inf), np.zeros((hq, d))
    for h in range(hq):
        k = h * hkv // hq
        keys = np.concatenate([hot[0][:, k], cold[0][:, k]])
        if not len(keys):
            continue
        s = keys @ q[h] / np.sqrt(d)
        m = s.max()
        p = np.exp(s - m)
        z = p.sum()
        p /= z
        n = len(hot[0])
        O[h] = p @ np.concatenate([hot[1][:, k], cold[1][:, k]])
        L[h] = m + np.log(z)
        size = cold[2][:, k]
        E[h] = 2.0 ** -8 * np.abs(O[h]) + (2.0 ** -8 + 2.0 ** -12) * (p[:n] @ np.abs(hot[1][:, k])) + \
            (2.0 ** -11 + 2.0 ** -12) * (p[n:] @ size) + (2.0 ** -22 * size.max() if len(size) else 0)
    return O, L, E


def check_attention(out, lse, want, what=""):
    O, L, E = want
    out, nan = np.asarray(out, np.float64), np.isnan(O)      # values that are held as NaN
    assert (np.isnan(out) == nan).all(), f"{what}: NaN in other places than expected"
    over = (np.abs(out - O) - E)[~nan]
    assert over.size == 0 or over.max() <= 0, f"{what}: output off by {over.max():.3g} over its bound"
    if lse is not None:
        empty = np.isneginf(L)
        assert (np.isneginf(lse) == empty).all(), f"{what}: lse of rows without a token"
        off = np.abs(np.asarray(lse, np.float64)[~empty] - L[~empty])
        assert off.size == 0 or off.max() <= LSE_ABS, f"{what}: lse off by {off.max():.3g}"
