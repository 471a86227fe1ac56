"""Plain fp64 restatements (numpy) of the rotary positions, the 4-bit rows, the paged cache and the
attention over it, for the tests.  Written from the definitions in include/osm_attn.h."""
import numpy as np

GROUP = 64


def rates(rot, base=10000.0):
    return [float(base) ** (-2.0 * i / rot) for i in range(rot // 2)]


def rotate(x, positions, w, layout, amplitude=1.0, inverse=False):
    """x [B, H, N, d] float64, positions [B, N] int, rates w; the angle in extended precision, since
    a far position times a rate keeps no fraction in 64 bits."""
    rot = 2 * len(w)
    a = positions.astype(np.longdouble)[..., None] * np.array(w, dtype=np.longdouble)
    a = np.fmod(a, 2 * np.longdouble("3.14159265358979323846264338327950288"))
    c = np.cos(a).astype(np.float64)[:, None] * amplitude
    s = np.sin(a).astype(np.float64)[:, None] * amplitude * (-1 if inverse else 1)
    y = x.copy()
    i0 = np.arange(len(w)) * (2 if layout == "interleaved" else 1)
    i1 = i0 + (1 if layout == "interleaved" else rot // 2)
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i1] * c + x[..., i0] * s
    return y


def step3(need):
    """The least number of three significant bits that is at least `need` (0 below 2^-126)."""
    m, e = np.frexp(need)
    s = np.ldexp(np.ceil(m * 8) / 8, e)
    return np.where(need < 2.0 ** -126, 0.0, s)


def quantise(x):
    """(codes [..., d], steps [..., d/64], bases [..., d/64]) of finite x [..., d]."""
    g = x.reshape(x.shape[:-1] + (-1, GROUP))
    lo, hi = g.min(-1), g.max(-1)
    s = step3(np.maximum((hi - lo) / 15, np.abs(lo) / 31))
    by = np.where(s > 0, s, 1.0)
    n = np.where(s[..., None] > 0, np.rint(g / by[..., None]), 0.0)
    b = np.where(s > 0, np.rint(lo / by), 0.0)
    codes = np.minimum(n - b[..., None], 15)
    return codes.reshape(x.shape).astype(np.int64), s, b.astype(np.int64)


def stored(x):
    """What a 4-bit row gives back for x [..., d]."""
    codes, s, b = quantise(x)
    g = codes.reshape(x.shape[:-1] + (-1, GROUP))
    return ((g + b[..., None]) * s[..., None]).reshape(x.shape)


def head_bytes(x):
    """The bytes of page heads of values x [..., page, d] in 4 bits: uint8 [..., bytes]."""
    codes, s, b = quantise(x)
    lead, (P, d) = x.shape[:-2], x.shape[-2:]
    body = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8).reshape(lead + (-1,))
    bits = (s.astype(np.float32).view(np.uint32) >> 21).astype(np.int64)
    words = ((bits << 6) | (b & 63)).astype("<u2")
    tail = np.ascontiguousarray(words.reshape(lead + (P * d // GROUP,))).view(np.uint8)
    return np.concatenate((body, tail), -1)


def head_values(raw, P, d):
    """Values [..., P, d] of 4-bit page heads uint8 [..., bytes]."""
    lead = raw.shape[:-1]
    body = raw[..., : P * d // 2].reshape(lead + (P, d // 2)).astype(np.int64)
    codes = np.stack((body & 15, body >> 4), -1).reshape(lead + (P, d // GROUP, GROUP))
    w = np.ascontiguousarray(raw[..., P * d // 2:]).view("<u2").astype(np.int64)
    w = w.reshape(lead + (P, d // GROUP))
    s = ((w >> 6) << 21).astype(np.uint32).view(np.float32).astype(np.float64)
    b = ((w & 63) ^ 32) - 32
    return ((codes + b[..., None]) * s[..., None]).reshape(lead + (P, d))


def head_steps(raw, P, d):
    """The steps of 4-bit page heads, spread over the values: [..., P, d]."""
    w = np.ascontiguousarray(raw[..., P * d // 2:]).view("<u2").astype(np.int64)
    w = w.reshape(raw.shape[:-1] + (P, d // GROUP))
    return np.repeat(((w >> 6) << 21).astype(np.uint32).view(np.float32).astype(np.float64), GROUP,
                     axis=-1)


def dense(pages, table, n):
    """Tokens 0 .. n - 1 of one sequence, [heads, n, d], from pages [num, heads, P, d]."""
    P = pages.shape[2]
    ids = table[: (n + P - 1) // P]
    x = pages[ids].transpose(1, 0, 2, 3)
    return x.reshape(x.shape[0], -1, x.shape[3])[:, :n]


def attend(q, k, v, kmag, vstep, scale, causal, q_len):
    """One sequence: q [H, Nq, d], k, v [H_kv, n, d] -> (O, LSE, tolerance of O, tolerance of LSE).
    kmag, vstep: the steps of a 4-bit cache spread over the values, 136 of K and one of V; |k| and 0
    for bf16.

    Tolerances.  The kernel's scores are fp32 sums of exact products: at most 8 roundings of sums of
    terms |q_c| kmag_c (4 bits: codes below 16 and bases below 32 are summed apart, each at most a
    third of 136 steps), each at most 2^-23 of the sum, d_s = scale sum |q_c| kmag_c 2^-20 in all;
    two roundings of 2^-23 of |s| follow in the exponent.  The exponentials are off by 2^-21, and
    sums over n keys by 2^-23 a step of at most n / 16 + 16 steps.
    The shares are rounded to bf16 (2^-8 at most).  In 4 bits V = s b + s code is summed as two sums
    of terms up to 31 p s and 15 p s, so a step's rounding is relative to those, not to V (which may
    be 0 where they are not): 46 p s 2^-23 a step; and p s is rounded to fp16, 2^-11 of itself (less
    than the 2^-8 already counted, and counted with V as both sums take the same p s) or, where that
    is less, half an fp16 subnormal, 2^-25 in units that put the largest step at 2^6 or more:
    2^-31 max(s) for each key, times |b + code| <= 46.  (These p are relative to a reference at or
    below the row's maximum, as is their sum, so the share's error is at most that over l.)
    The codes are subnormal fp16 numbers, code 2^-24.  A product of 16 terms aligns them to the
    largest, with a subnormal's exponent counted as -14, and drops what lies more than 25 bits below
    (seen with single terms: 2^-24 x 2^11 beside 2^-24 x 2^(11 - j) is exact up to j = 15).  With x
    the largest other factor of the 16, each of them and the sum so far lose less than 2^(-14 - 25) x,
    2^-15 of code 1 times x: 17 x 2^-15 x in all.  For V x is a p s, at most the sum of the 16; for the
    d / 16 products of a score x is at most max |q_c| (and the step follows).
    O is rounded to bf16 once more."""
    H, Nq, d = q.shape
    Hkv, n, _ = k.shape
    kstep = kmag / 136 if vstep.any() else 0 * kmag
    O, L = np.zeros((H, Nq, d)), np.full((H, Nq), -np.inf)
    tO, tL = np.zeros((H, Nq, d)), np.zeros((H, Nq))
    for h in range(H):
        g = h // (H // Hkv)
        for i in range(min(q_len, Nq)):
            end = n - q_len + i + 1 if causal else n
            if end <= 0:
                continue
            s = scale * (k[g, :end] @ q[h, i])
            if np.all(np.isneginf(s)):
                continue
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            p /= l
            O[h, i] = p @ v[g, :end]
            L[h, i] = m + np.log(l)
            ds = (scale * (kmag[g, :end] @ np.abs(q[h, i]))).max() * 2.0 ** -20 + \
                np.abs(s).max() * 2.0 ** -22 + \
                scale * np.abs(q[h, i]).max() * kstep[g, :end].max() * d / 16 * 17 * 2.0 ** -15
            steps = (end / 16 + 16) * 2.0 ** -23
            tO[h, i] = 2.0 ** -8 * np.abs(O[h, i]) + \
                (p @ np.abs(v[g, :end])) * (2.0 ** -8 + 2 * ds + 2.0 ** -20 + steps) * 1.01 + \
                46 * ((p @ vstep[g, :end]) * steps + end / l * 2.0 ** -31 * vstep[g, :end].max()) + \
                17 * 2.0 ** -15 * (p @ vstep[g, :end])
            tL[h, i] = ds + 2.0 ** -20 + steps + 2.0 ** -22 * abs(L[h, i])
    return O, L, tO, tL
