"""float64 definitions of the paged cache's formats and of attention over it.

Test infrastructure only.  Written from the row formats and the formula in
include/kvzip.h; rows are float64 arrays that hold bf16 values.
"""
from __future__ import annotations

import numpy as np


def bf16_round(x):
    """Nearest bf16 value (ties to even) of float64 values, as float64; overflow to inf."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        _, e = np.frexp(x)
        ulp = np.ldexp(1.0, np.maximum(e - 8, -133))       # 8 significant bits; smallest step 2^-133
        r = np.rint(x / ulp) * ulp
    r = np.where(np.abs(r) >= 2.0 ** 128, np.sign(x) * np.inf, r)
    return np.where(np.isfinite(x), r, x)


def bf16_bits(x):
    return (np.asarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint32)


def e4m3_value(code):
    """Value of e4m3 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits; 127 is NaN."""
    code = np.asarray(code).astype(np.int64)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.ldexp(1.0, e - 10))
    v = np.where(code & 128, -v, v)
    return np.where((code & 127) == 127, np.nan, v)


_E4M3 = e4m3_value(np.arange(127))            # 0 .. 448, ascending


def e4m3_code(y):
    """Nearest code of |y| <= 448, ties to the even code, by search over all values."""
    y = np.asarray(y, dtype=np.float64)
    a = np.abs(y)
    hi = np.clip(np.searchsorted(_E4M3, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _E4M3[lo], _E4M3[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.where(np.signbit(y), c + 128, c)


def quantise(x, fmt):
    """Rows [n][d] -> (codes, parameter words).  fp8: codes 0..255; int4: codes
    0..15 (one per element).  Rows the format marks as NaN get zero codes for fp8
    and None-like codes of -1 for int4 (unspecified)."""
    x = np.asarray(x, dtype=np.float64)
    n = x.shape[0]
    if fmt == "fp8":
        codes, par = np.zeros(x.shape, np.int64), np.zeros(n, np.uint32)
        for i in range(n):
            if not np.all(np.isfinite(x[i])):
                par[i] = 0x7FC00000
                continue
            top, e = np.max(np.abs(x[i])), 0
            if top > 0:
                e = -126
                while top > 448.0 * 2.0 ** e:
                    e += 1
            codes[i] = e4m3_code(x[i] / 2.0 ** e)
            par[i] = np.array(2.0 ** e, np.float32).view(np.uint32)
        return codes, par
    codes, par = np.full(x.shape, -1, np.int64), np.zeros(n, np.uint32)
    for i in range(n):
        if not np.all(np.isfinite(x[i])) or np.max(np.abs(x[i])) >= 2.0 ** 126:
            par[i] = 0x7FC07FC0
            continue
        z = np.min(x[i])
        s = float(bf16_round((np.max(x[i]) - z) / 15.0))
        codes[i] = 0 if s == 0 else np.clip(_rint_ratio(x[i], z, s), 0, 15)
        par[i] = int(bf16_bits(s)) | (int(bf16_bits(z)) << 16)
    return codes, par


def _rint_ratio(x, z, s):
    """round((x - z) / s) half to even, decided in whole numbers."""
    from fractions import Fraction
    t = np.rint((x - z) / s)
    near = np.abs(np.abs((x - z) / s - t) - 0.5) < 1e-6
    for i in np.nonzero(near)[0]:
        t[i] = round((Fraction(float(x[i])) - Fraction(float(z))) / Fraction(float(s)))
    return t


def values(codes, par, fmt):
    """float64 values of stored rows (codes as quantise gives them)."""
    par = np.asarray(par, np.uint32)
    if fmt == "fp8":
        return e4m3_value(codes) * par.view(np.float32).astype(np.float64)[:, None]
    s = (par << np.uint32(16)).view(np.float32).astype(np.float64)[:, None]
    z = (par & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64)[:, None]
    return s * codes + z


def attention(q, k, v, m, scale):
    """q [G][n_q][d], k, v [len][d] float64, the unit's m newest tokens are its
    last m rows: (out [G][m][d], weight [G][m][d] = sum p |v|, reach [G][m] = the
    largest scale * sum |q| |k| of a seen row)."""
    G, _, d = q.shape
    n = k.shape[0]
    out, wt = np.zeros((G, m, d)), np.zeros((G, m, d))
    reach = np.zeros((G, m))
    for i in range(m):
        seen = n - m + i + 1
        if seen <= 0:
            continue
        x = scale * (q[:, i] @ k[:seen].T)
        p = np.exp(x - x.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        out[:, i] = p @ v[:seen]
        wt[:, i] = p @ np.abs(v[:seen])
        reach[:, i] = scale * (np.abs(q[:, i]) @ np.abs(k[:seen]).T).max(1)
    return out, wt, reach
