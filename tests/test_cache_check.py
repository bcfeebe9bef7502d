"""The attention check of tests/cache_check.py itself, on the CPU: rounded definitions
pass, and wrong results of each kind do not, for every format and kernel path."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co
from tests import cache_check as cc


def rows_bf16(seed, *shape, keys=False):
    x = torch.randn(*shape, generator=torch.Generator().manual_seed(seed))
    if keys:
        x[..., ::37] *= 5.0
    return x.to(torch.bfloat16)


def held(x, fmt):
    x = x.double().numpy()
    if fmt == "bf16":
        return cc.Rows(torch.from_numpy(x))
    codes, par = co.quantise(x, fmt)
    if fmt == "fp8":
        return cc.Rows(torch.from_numpy(co.values(codes, par, fmt)))
    z = co.values(np.zeros_like(codes), par, fmt)
    return cc.Rows(torch.from_numpy(co.values(codes, par, fmt) - z), torch.from_numpy(z))


@pytest.mark.parametrize("tc", [False, True])
@pytest.mark.parametrize("d,n,m", [(128, 700, 130), (256, 2000, 40), (128, 9000, 7), (128, 300, 1)])
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int4"])
def test_wrong_results_are_noticed(fmt, d, n, m, tc):
    k, v = held(rows_bf16(1, n, d, keys=True), fmt), held(rows_bf16(2, n, d), fmt)
    q = rows_bf16(3, 2, m, d).double()
    half, scale = torch.finfo(torch.bfloat16).eps / 2, d ** -0.5
    want, tol = cc.attention(q, k, v, m, scale, fmt, tc, half)
    ref, _, _ = co.attention(q.numpy(), k.value.numpy(), v.value.numpy(), m, scale)
    assert np.allclose(want.numpy(), ref, rtol=1e-12, atol=1e-12)
    good = want.to(torch.bfloat16).double()
    assert cc.close(good, want, tol) is None
    swapped = cc.Rows(v.a.view(n, -1, 2).flip(2).reshape(n, d), v.b)      # nibbles exchanged
    late = cc.attention(q, k, v, m, scale, fmt, tc, half)[0].roll(1, 1) if m > 1 else -want
    far = cc.Rows(torch.where((torch.arange(n) // 64 % 20 == 3)[:, None], 2 * v.a, v.a), v.b)
    wrong = {
        "zeros": torch.zeros_like(want), "rotated channels": good.roll(1, -1), "other token": late,
        "scale": cc.attention(q, k, v, m, 0.9 * scale, fmt, tc, half)[0],
        "nibbles": cc.attention(q, k, swapped, m, scale, fmt, tc, half)[0],
        "power of two of a tile": cc.attention(q, k, far, m, scale, fmt, tc, half)[0],
        "one row less": cc.attention(q, cc.Rows(k.a[:-1], k.b[:-1]), cc.Rows(v.a[:-1], v.b[:-1]), m, scale,
                                     fmt, tc, half)[0],
        "half a percent": good * 1.005,
        "nan": torch.full_like(good, float("nan")),
    }
    for what, x in wrong.items():
        assert cc.close(x.to(torch.bfloat16).double(), want, tol) is not None, what
    for what in ("zeros", "rotated channels", "nan"):      # element by element as well
        assert cc.close(wrong[what], want, tol, alike=False) is not None, what
