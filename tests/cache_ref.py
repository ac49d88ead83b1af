"""Plain 64-bit forms of the 8-bit cache's operations and of rotary positions with
several axes, on numpy arrays, one sequence and head at a time: the definitions
written out, against which the kernels are tested."""
import math

import numpy as np

MIN_SCALE = 2.0 ** -126


def _code_values():
    """Value of each of the 256 e4m3 codes (1 sign, 4 exponent bits with bias 7, 3 mantissa bits; 0x7F, 0xFF: NaN)."""
    v = np.empty(256)
    for c in range(256):
        sign, e, m = (-1.0 if c & 128 else 1.0), (c >> 3) & 15, c & 7
        v[c] = sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    v[0x7F] = v[0xFF] = np.nan
    return v


CODES = _code_values()
_FINITE = CODES[:0x7F]  # ascending, 0 .. 448


def encode(x):
    """e4m3 codes of x (|x| <= 448 or NaN): the nearest value, the even code on ties."""
    x = np.asarray(x, dtype=np.float64)
    a = np.where(np.isnan(x), 0.0, np.abs(x))
    hi = np.searchsorted(_FINITE, a, side="left").clip(0, 0x7E)
    lo = (hi - 1).clip(0)
    down, up = a - _FINITE[lo], _FINITE[hi] - a
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def smallest_scale(amax):
    p = -126
    while amax > 448.0 * 2.0 ** p:
        p += 1
    return 2.0 ** p


def append(K, codes, scale, L, s):
    """New rows K [n, d] at position L of one head's codes [T, d] (uint8) and scales [nb], in place.  Returns the
    blocks that became complete."""
    n, done = K.shape[0], []
    at = L
    while at < L + n:
        j = at // s
        to = min(L + n, (j + 1) * s)
        x = K[at - L:to - L]
        finite = np.abs(x[np.isfinite(x)])
        want = smallest_scale(finite.max() if finite.size else 0.0)
        if at > j * s:
            old = scale[j]
            want = max(want, old)
            if want > old:
                codes[j * s:at] = encode(CODES[codes[j * s:at]] * (old / want))
        with np.errstate(invalid="ignore"):
            codes[at:to] = encode(np.where(np.isfinite(x), x / want, np.nan))
        scale[j] = want
        if to == (j + 1) * s:
            done.append(j)
        at = to
    return done


def dequantise(codes, scale, s):
    return CODES[codes] * np.repeat(np.asarray(scale, dtype=np.float64), s)[:codes.shape[0], None]


def select(q, Kbar, bt, k):
    """Own block bt and the k - 1 highest-scoring blocks before it: q [G, d], Kbar [nb, d]; ascending, -1 behind."""
    r = (Kbar[:bt].astype(np.float64) @ q.astype(np.float64).sum(0)).astype(np.float32)
    best = sorted(range(bt), key=lambda j: (-r[j], j))[:k - 1]
    out = sorted(best) + [bt]
    return out + [-1] * (k - len(out))


def attend(q, K, V, tokens, scale):
    """q [G, d] over the rows `tokens` of K, V [T, d]: o [G, d], lse [G], weights [G, n], and per head the largest
    sum of magnitudes that a logit is made of."""
    z = q @ K[tokens].T * scale
    size = (np.abs(q) @ np.abs(K[tokens]).T * scale).max(1)
    m = z.max(1, keepdims=True)
    p = np.exp(z - m)
    l = p.sum(1, keepdims=True)
    return (p / l) @ V[tokens], (m + np.log(l))[:, 0], p / l, size


def evict_order(weight, whole, keep, sink, recent):
    """Complete blocks that stay, ascending."""
    if whole <= keep:
        return list(range(whole))
    always = [j for j in range(whole) if j < sink or j >= whole - recent]
    w = [-math.inf if math.isnan(x) else x for x in weight[:whole]]
    nan = [math.isnan(x) for x in weight[:whole]]
    rest = sorted((j for j in range(whole) if j not in always), key=lambda j: (-w[j], nan[j], j))
    return sorted(always + rest[:keep - len(always)])


def rope_axes(x, pos, sections, base, factor, interleaved=False, own_ladder=False, transpose=False):
    """x [B, heads, T, d], pos [axes, B, T]: every pair turned by its angle, in 64 bits."""
    d = x.shape[-1]
    half, rank, owner, a = d // 2, [0] * len(sections), [], 0
    while len(owner) < half:
        if interleaved:
            if rank[a] < sections[a]:
                owner.append((a, rank[a]))
                rank[a] += 1
            a = (a + 1) % len(sections)
        else:
            while rank[a] == sections[a]:
                a += 1
            owner.append((a, rank[a]))
            rank[a] += 1
    y = np.empty(x.shape)
    for i, (a, r) in enumerate(owner):
        f = base ** (-r / sections[a]) if own_ladder else base ** (-i / half)
        t = pos[a].astype(np.float64) * f / factor * (-1.0 if transpose else 1.0)
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        y[..., i] = x[..., i] * c - x[..., i + half] * s
        y[..., i + half] = x[..., i] * s + x[..., i + half] * c
    return y
