"""How far attention over the paged cache may be from its float64 definition.

Everything here is float64 torch, on any device; stored rows come as the two parts that
the formats are made of (values = a + b: 4 bits a = s c and b = z, else a = value, b = 0).

Per output element, p the true weights of the rows a token sees:

    half |out|                      the output's rounding, half = eps / 2
  + 2 (e^delta - 1) sum p |v|       logits off by delta: a relative error of each weight
                                    and of their sum
  + w sum p |r|                     the rounding of a weight to fewer bits, r what it multiplies
  + 2^-11 sum p |v| + 2^-13 sum p |v|_max       4 bits, many rows: s c + z as fp16, and what
                                    fp16 has no digits for (15 steps of s beside z, a row
                                    beside one 2^8 above it: 15 * 2^8 * 2^-25)
  + (1e-5 + n 2^-26) sum p (|a| + |b|)          exponentials (2^-22 each, their arguments'
                                    rounding) and float32 sums over n rows: an MMA adds 16
                                    products with one rounding of at most 2^-23, and the
                                    weights' sum takes as many steps
  + n 2^-28 max p |v|_max           quantised: fp16 has steps of 2^-24; weights times their
                                    rows' power of two are lifted so that the largest is
                                    2^7 or more, and rows up to 2^4 apart may share one

delta = d 2^-24 reach (float32 sums of d products, reach = scale sum |q| (|a| + |b|));
with many rows and quantised pages also 2^-34 reach (one power of two for 64 rows) and, in
4 bits, 2^-11 scale sum |q| |k| (k as fp16).
w: fp16 weights for quantised pages 2^-11; bf16 pages 2^-8 with many rows, two bf16 parts
with few (2^-16).
"""
import torch


class Rows:
    """Rows [n][d] of K or of V as the cache holds them."""

    def __init__(self, a, b=None):
        self.a = a
        self.b = torch.zeros_like(a) if b is None else b
        self.value = self.a + self.b
        self.parts = self.a.abs() + self.b.abs()


def attention(q, k, v, m, scale, fmt, tc, half):
    """q [G][m][d] of the m newest tokens -> (out, tolerance), [G][m][d]."""
    G, _, d = q.shape
    n = k.value.shape[0]
    i = torch.arange(m, device=q.device).view(1, m, 1)
    j = torch.arange(n, device=q.device).view(1, 1, n)
    hidden = j > n - m + i
    none = (n - m + i + 1 <= 0).expand(G, m, 1)
    x = scale * torch.einsum("gid,jd->gij", q, k.value)
    p = torch.softmax(x.masked_fill(hidden, float("-inf")), 2) if n else x
    p = torch.where(none, torch.zeros_like(p), p)
    def seen_most(t):          # the largest sum |q| t of a row that is seen
        r = scale * torch.einsum("gid,jd->gij", q.abs(), t)
        return r.masked_fill(hidden, 0.0).amax(2, keepdim=True) if n else r.sum(2, keepdim=True)
    mean = lambda t: torch.einsum("gij,jd->gid", p, t)  # noqa: E731
    quant = fmt != "bf16"
    w = 2.0 ** -11 if quant else (2.0 ** -8 if tc else 2.0 ** -16)
    delta = d * 2.0 ** -24 * seen_most(k.parts)
    if tc and quant:
        delta = delta + 2.0 ** -34 * seen_most(k.parts)
    if tc and fmt == "int4":
        delta = delta + 2.0 ** -11 * seen_most(k.value.abs())
    out = mean(v.value)
    wv = mean(v.value.abs())
    tol = half * out.abs() + 2 * torch.expm1(delta) * wv + w * (wv if tc or fmt != "int4" else mean(v.a.abs()))
    tol = tol + (1e-5 + n * 2.0 ** -26) * mean(v.parts)
    if n and quant:
        top = v.value.abs().amax(1)
        tol = tol + n * 2.0 ** -28 * (p * top).amax(2, keepdim=True)
        if tc and fmt == "int4":
            tol = tol + 2.0 ** -11 * wv + 2.0 ** -13 * (p @ top[:, None])
    return out, tol


def close(got, want, tol, alike=True, common=0.0):
    """None, or what is wrong.  alike: rows of one size in random directions, whose
    errors are as good as independent; each query row's error is then below 2^-8 of its
    length (bf16 outputs and weights, 2^-9 / sqrt(3) of an element each, are 2^-8.8 together).
    common: a relative error that all elements of a row may share beside that."""
    if not bool(torch.isfinite(got).all()):
        return "not finite"
    err = (got - want).abs()
    if bool((err > tol).any()):
        return f"off by {float(err.max()):.3g}, {float((err - tol).max()):.3g} too far"
    if alike and got.numel():
        far = err.norm(dim=-1) - (2.0 ** -8 + common) * want.norm(dim=-1)
        if float(far.max()) > 0:
            return f"a row is {float((err.norm(dim=-1) / want.norm(dim=-1)).max()):.3g} of its length off"
    return None
