"""Plain 64-bit forms of the MXFP4 operators and of the 8-bit cache (numpy,
one element at a time where that is clearest), and their error bounds."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
E4M3 = np.empty(256)
for _c in range(256):
    _e, _m = (_c >> 3) & 15, _c & 7
    _v = np.ldexp(1 + _m / 8, _e - 7) if _e else np.ldexp(_m / 8, -6)
    E4M3[_c] = np.nan if (_c & 127) == 127 else (-_v if _c & 128 else _v)


# ---------------------------------------------------------------- MXFP4


def mx_quantize(X):
    """X [rows][K] (float64 values of bf16 / fp32 numbers) -> (codes [rows][K], exponent bytes [rows][K/32])."""
    rows, K = X.shape
    codes = np.zeros((rows, K), np.uint8)
    bytes_ = np.zeros((rows, K // 32), np.uint8)
    for r in range(rows):
        for b in range(K // 32):
            x = X[r, 32 * b:32 * b + 32]
            if not np.all(np.isfinite(x)):
                bytes_[r, b] = 255
                continue
            a = np.abs(x).max()
            e = -127 if a == 0 else max(int(np.frexp(a)[1]) - 1 - 2, -127)
            bytes_[r, b] = e + 127
            t = np.abs(np.ldexp(x, -e))
            # count the midpoints passed; a tie goes to the even code
            c = ((t > .25).astype(int) + (t >= .75) + (t > 1.25) + (t >= 1.75) + (t > 2.5) + (t >= 3.5) + (t > 5))
            codes[r, 32 * b:32 * b + 32] = c | np.where(np.signbit(x), 8, 0)
    return codes, bytes_


def mx_values(codes, bytes_):
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(bytes_ == 255, np.nan, np.ldexp(1.0, bytes_.astype(int) - 127))
    return v * np.repeat(s, 32, axis=1)


def mx_pack(codes, bytes_):
    """The tiled layout, straight from its definition."""
    rows, K = codes.shape
    NB, G = -(-rows // 16), -(-K // 128)
    GQ = -(-G // 4)
    pc = np.zeros(NB * G * 1024, np.uint8)
    ps = np.full(NB * GQ * 256, 127, np.uint8)
    n = np.arange(rows)[:, None]
    k = np.arange(0, K, 2)[None]
    at = (((n // 16) * G + k // 128) * 64 + n % 16 + 16 * ((k // 32) % 4)) * 16 + (k % 32) // 2
    pc[at] = codes[:, 0::2] | (codes[:, 1::2] << 4)
    b = np.arange(K // 32)[None]
    ps[(((n // 16) * GQ + b // 16) * 64 + n % 16 + 16 * (b % 4)) * 4 + (b // 4) % 4] = bytes_
    return pc, ps


def product_tolerance(absY, yref, K, bf16_out):
    """K exact products added in fp32 in some order: each addition is off by at
    most one step (2^-23, truncation allowed) of a partial sum that is at most
    sum |w x|; never more than the library's 1e-3 sum |w x|.  bf16 output: half
    a step, 2^-8 |y|."""
    t = min(1e-3, K * 2.0 ** -23) * absY
    return t + 2.0 ** -8 * np.abs(yref) if bf16_out else t


# ------------------------------------------------------------- 8-bit cache


def e4m3_nearest(x):
    """Nearest e4m3 number, ties to even; +-448 beyond; NaN stays."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    step = np.ldexp(1.0, np.maximum(np.frexp(np.where(a > 0, a, 1.0))[1] - 1, -6) - 3)
    return np.where(np.isnan(x), np.nan, np.copysign(np.rint(a / step) * step, x))


def page_exponent(a):
    e = -127
    while a > np.ldexp(448.0, e):
        e += 1
    return e


def append(kv, scales, page, tokens, lo, transposed):
    """Write `tokens` [n][H][D] at slots lo .. of `page` into kv (e4m3 values, float64) and scales (exponents)."""
    H = tokens.shape[1]
    for h in range(H):
        view = kv[page, h].T if transposed else kv[page, h]  # [P][D]
        x = tokens[:, h].astype(np.float64)
        fin = np.abs(x[np.isfinite(x)])
        e = page_exponent(fin.max() if fin.size else 0.0)
        if lo > 0:
            old = int(scales[page, h])
            e = max(e, old)
            if e > old:
                view[:lo] = e4m3_nearest(np.ldexp(view[:lo], old - e))
        view[lo:lo + len(x)] = e4m3_nearest(np.ldexp(x, -e))
        scales[page, h] = e


def attention(q, K, V, first, scale, causal, window):
    """q [n][Hq][D], K and V [T][H][D] (values); query i stands at first + i.
    Returns O, lse, and the bound's ingredients A = sum p |v| and the scores' error bound."""
    n, Hq, D = q.shape
    T, H = K.shape[:2]
    G = Hq // H
    O, A = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, eps = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for i in range(n):
        p0 = first + i
        hi = min(T, p0 + 1) if causal else T
        lo = max(0, p0 - window + 1) if window else 0
        if hi <= lo:
            continue
        for hq in range(Hq):
            k, v = K[lo:hi, hq // G], V[lo:hi, hq // G]
            s = k @ q[i, hq] * scale
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            O[i, hq] = (p[:, None] * v).sum(0) / l
            A[i, hq] = (p[:, None] * np.abs(v)).sum(0) / l
            # a weight below 2^-126 of the largest may become 0 (at most 2^-126 max|v|
            # each, as l >= 1), and so may weight times 2^ev (then times a code of at
            # most 448); the bound takes 2^-8 A and more, hence the 2^8
            A[i, hq] += 2.0 ** 8 * len(p) * (np.abs(v).max() + 448) * 2.0 ** -126
            lse[i, hq] = m + np.log(l)
            mag = (np.abs(k) @ np.abs(q[i, hq])).max() * abs(scale)
            # D products added in fp32, then one scaling and one exponential
            eps[i, hq] = (D * 2.0 ** -23 + 2.0 ** -22) * mag + 2.0 ** -22
    return O, lse, A, eps


def attention_tolerance(O, A, eps, T):
    """Weights off by 2 eps (they and their sum), rounded to bf16 (half a step,
    2^-8), T of them added in fp32, the output rounded to bf16 (2^-8 |o|)."""
    return (2.5 * eps[..., None] + 2.0 ** -8 * 1.01 + (T + 64) * 2.0 ** -22) * A + 2.0 ** -8 * np.abs(O)


def lse_tolerance(lse, eps, T):
    return 2 * eps + (T + 64) * 2.0 ** -23 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))
