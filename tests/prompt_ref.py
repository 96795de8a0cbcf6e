"""Plain 64-bit attention of packed prompts, for the tests of gk_prompt_attn.

expected() walks the definition request by request with numpy on fp64 copies of
the inputs; errors() measures a result row by row against it.

Tolerance (OUT_REL, LSE_ABS), counted before any run.  The inputs are bf16 and
exact in fp64.  A row's output is O = sum p_j v_j / Z; the kernel rounds each p_j
to bf16 (relative error at most u = 2^-8, half a step of finfo(bf16).eps = 2^-7)
and the result to bf16 (again at most u per channel).  The rest is fp32: scores
of up to 2^9 in log2 units are off by a few 2^9 * 2^-24, below 2^-13; the tensor
core adds 16 keys at a time, so the tests' at most 2^13 keys are 2^9 steps of at
most 2^-23 each, 2^-14; Z and exp2 are better than that.  Together below 2^-12, so
  |O - O*|  <=  u * sum_j p_j |v_j| / Z  +  u * |O*|  +  2^-12 * sum_j p_j |v_j| / Z
channel by channel: with A = sum_j p_j |v_j| / Z (computed beside O*), at most
(2 u + 2^-12) A, as |O*| <= A.  LSE = m + ln Z: 2^-13 from the scores (times ln 2)
and a relative error of Z below 2^-14: below 2e-4 absolute.
"""
import numpy as np

U = 2.0 ** -8
OUT_REL = 2 * U + 2.0 ** -12
LSE_ABS = 2e-4


def expected(q, k, v, new_len, past):
    """q [T, Hq, d], k, v [T, Hkv, d] fp64; past: per request (K, V) [tokens, Hkv, d] -> O, A [T, Hq, d], LSE [T, Hq]."""
    T, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    O, A, L = np.zeros((T, hq, d)), np.zeros((T, hq, d)), np.full((T, hq), -np.inf)
    t0 = 0
    for n, (pk, pv) in zip(new_len, past):
        for h in range(hq if n else 0):
            keys = np.concatenate([pk[:, h // g], k[t0:t0 + n, h // g]])
            vals = np.concatenate([pv[:, h // g], v[t0:t0 + n, h // g]])
            c = len(pk)
            with np.errstate(invalid="ignore", over="ignore"):
                s = q[t0:t0 + n, h] @ keys.T / np.sqrt(d)
            s[np.arange(c + n)[None] > c + np.arange(n)[:, None]] = -np.inf
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            z = p.sum(1, keepdims=True)
            p /= z
            dead = p == 0
            finite = np.isfinite(vals).all(1)
            O[t0:t0 + n, h] = p[:, finite] @ vals[finite]
            A[t0:t0 + n, h] = p[:, finite] @ np.abs(vals[finite])
            for j in np.flatnonzero(~finite):      # 0 times an infinity of a masked key is nothing
                rows = ~dead[:, j]
                O[t0:t0 + n, h][rows] += p[rows, j:j + 1] * vals[j]
                A[t0:t0 + n, h][rows] += p[rows, j:j + 1] * np.abs(vals[j])
            L[t0:t0 + n, h] = (m + np.log(z))[:, 0]
        t0 += n
    return O, A, L


def check(out, lse, want, what=""):
    """Every channel of every row within the counted tolerance."""
    O, A, L = want
    out, lse = np.asarray(out, np.float64), np.asarray(lse, np.float64)
    fin = np.isfinite(O)
    assert (np.isfinite(out) == fin).all(), f"{what}: infinities or NaN in other places than expected"
    over = np.abs(out - O)[fin] - OUT_REL * A[fin]
    assert over.size == 0 or over.max() <= 0, f"{what}: output off by {over.max():.3g} over its bound"
    off = np.abs(lse - L)
    assert off.size == 0 or off.max() <= LSE_ABS, f"{what}: lse off by {off.max():.3g}"
