"""Host-side checks of the paged cache: the formats' definitions against brute
force, and every refusal of the C calls and of PagedCache before the GPU is touched."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import cache_oracle as co


@pytest.fixture(scope="module")
def kz():
    from attention_score_reduction_b200 import build
    build.build()
    from attention_score_reduction_b200 import kvzip
    return kvzip


# ------------------------------------------------------------- the definitions

def test_e4m3_matches_torch():
    codes = np.arange(256)
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    got = co.e4m3_value(codes)
    assert np.array_equal(got, want, equal_nan=True)
    y = np.concatenate([np.linspace(-448, 448, 40001), co._E4M3, -co._E4M3,
                        (co._E4M3[1:] + co._E4M3[:-1]) / 2])
    want = torch.from_numpy(y).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    ok = torch.from_numpy(y).float().double().numpy() == y       # exact in float32
    assert ok.sum() > 300
    assert np.array_equal(co.e4m3_code(y)[ok], want[ok])


def test_bf16_round_matches_torch():
    x = torch.randn(20000, generator=torch.Generator().manual_seed(3)) * 10
    x = torch.cat([x, x * 1e-38, torch.tensor([0.0, 3.39e38, 3.4e38, 1e-40])])
    assert np.array_equal(co.bf16_round(x.double().numpy()), x.to(torch.bfloat16).double().numpy())


def _row(seed, d=128, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(1, d, generator=g) * spread).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("spread", [1e-30, 1.0, 1e30])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_int4_definition(seed, spread):
    """Codes are the nearest of the 16 values s c + z (by exact fractions), and the
    scale is the bf16 nearest to range / 15."""
    x = _row(seed, spread=spread)
    codes, par = co.quantise(x, "int4")
    s = float((par << np.uint32(16)).view(np.float32)[0])
    z = float((par & np.uint32(0xFFFF0000)).view(np.float32)[0])
    assert z == x.min()
    ideal = (Fraction(float(x.max())) - Fraction(z)) / 15
    assert abs(Fraction(s) - ideal) <= ideal / 256
    for e, c in zip(x[0], codes[0]):
        dist = [abs(Fraction(s) * k + Fraction(z) - Fraction(float(e))) for k in range(16)]
        assert dist[c] == min(dist)


def test_fp8_definition():
    for seed, spread in ((1, 1.0), (2, 1e-36), (3, 1e36)):
        x = _row(seed, spread=spread)
        codes, par = co.quantise(x, "fp8")
        s = float(par.view(np.float32)[0])
        top = np.abs(x).max()
        assert top <= 448 * s and (s == 2.0 ** -126 or top > 448 * s / 2)
        err = np.abs(co.values(codes, par, "fp8") - x)
        assert np.all(err <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10 * s))


def test_attention_definition():
    g = np.random.default_rng(5)
    q, k, v = g.normal(size=(2, 3, 8)), g.normal(size=(7, 8)), g.normal(size=(7, 8))
    out, wt, _ = co.attention(q, k, v, 3, 0.5)
    for h in range(2):
        for i in range(3):
            n = 7 - 3 + i + 1
            w = [np.exp(0.5 * np.dot(q[h, i], k[j])) for j in range(n)]
            want = sum(w[j] * v[j] for j in range(n)) / sum(w)
            assert np.allclose(out[h, i], want, rtol=1e-12, atol=1e-12)
    out, _, _ = co.attention(q, k[:2], v[:2], 3, 0.5)      # token 0 sees nothing
    assert np.all(out[:, 0] == 0) and np.allclose(out[:, 1], v[0])


# ------------------------------------------------------------- refusals of the C calls

FAKE = 1 << 20      # aligned, never dereferenced by a refused call
FIELDS = dict(format=1, d=128, page_rows=64, max_pages=10, n_pages=100, units=4, k_pages=FAKE,
              v_pages=FAKE, k_params=FAKE, v_params=FAKE, page_table=FAKE, lens=FAKE, status=FAKE)

BAD_CACHE = [
    (dict(format=3), 1), (dict(format=-1), 1), (dict(d=64), 2), (dict(d=0), 1), (dict(d=-128), 1),
    (dict(page_rows=8), 2), (dict(page_rows=48), 2), (dict(page_rows=256), 2), (dict(page_rows=0), 1),
    (dict(units=-1), 1), (dict(n_pages=0), 1), (dict(max_pages=0), 1), (dict(max_pages=-4), 1),
    (dict(n_pages=(1 << 31) // 64), 2), (dict(max_pages=(1 << 31) // 64), 2),
    (dict(units=(1 << 24) + 1), 2), (dict(k_pages=None), 1), (dict(v_pages=None), 1),
    (dict(k_params=None), 1), (dict(v_params=None), 1), (dict(page_table=None), 1),
    (dict(lens=None), 1), (dict(status=None), 1), (dict(k_pages=FAKE + 8), 1),
    (dict(v_pages=FAKE + 2), 1), (dict(k_params=FAKE + 4), 1), (dict(page_table=FAKE + 2), 1),
    (dict(lens=FAKE + 1), 1), (dict(status=FAKE + 2), 1),
]


def _cache(kz, **over):
    return kz.CacheStruct(**{**FIELDS, **over})


def _write(kz, c, **o):
    a = dict(k=FAKE, v=FAKE, ku=1280, kr=128, vu=1280, vr=128, n=10, starts=None, counts=None,
             offsets=None)
    a.update(o)
    return kz.library().kvzip_cache_write(c, a["k"], a["v"], a["ku"], a["kr"], a["vu"], a["vr"],
                                          a["n"], a["starts"], a["counts"], a["offsets"], None)


def _read(kz, c, **o):
    a = dict(k=FAKE, v=FAKE, n=10, starts=None, offsets=None)
    a.update(o)
    return kz.library().kvzip_cache_read(c, a["k"], a["v"], a["n"], a["starts"], a["offsets"], None)


def _attend(kz, c, **o):
    a = dict(q=FAKE, qu=4096, qh=1024, qr=128, out=FAKE, f32=0, ou=4096, oh=1024, orow=128,
             q_lens=None, n_q=8, G=4, scale=0.0, ws=FAKE, ws_bytes=1 << 40)
    a.update(o)
    return kz.library().kvzip_cache_attention(
        c, a["q"], a["qu"], a["qh"], a["qr"], a["out"], a["f32"], a["ou"], a["oh"], a["orow"],
        a["q_lens"], a["n_q"], a["G"], a["scale"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("over,want", BAD_CACHE)
def test_bad_cache_is_refused(kz, over, want):
    c = _cache(kz, **over)
    assert _write(kz, c) == want
    assert _read(kz, c) == want
    assert _attend(kz, c) == want
    assert kz.cache_attention_workspace_size(c, 4, 8) == 0


def test_null_cache_is_refused(kz):
    null = ctypes.POINTER(kz.CacheStruct)()
    assert _write(kz, null) == kz.ERR_INVALID_ARG
    assert _read(kz, null) == kz.ERR_INVALID_ARG
    assert _attend(kz, null) == kz.ERR_INVALID_ARG


@pytest.mark.parametrize("over,want", [
    (dict(n=-1), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(k=FAKE + 8), 1),
    (dict(v=FAKE + 4), 1), (dict(kr=12), 1), (dict(vu=-128), 1), (dict(vr=-8), 1), (dict(ku=4), 1),
    (dict(starts=FAKE + 1), 1), (dict(counts=FAKE + 2), 1), (dict(offsets=FAKE + 4), 1),
    (dict(counts=FAKE, offsets=FAKE), 1), (dict(n=1 << 31), 2)])
def test_write_refuses(kz, over, want):
    assert _write(kz, _cache(kz), **over) == want


@pytest.mark.parametrize("over,want", [
    (dict(n=-1), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(k=FAKE + 8), 1),
    (dict(starts=FAKE + 2), 1), (dict(offsets=FAKE + 4), 1), (dict(n=1 << 31), 2)])
def test_read_refuses(kz, over, want):
    assert _read(kz, _cache(kz), **over) == want


@pytest.mark.parametrize("over,want", [
    (dict(G=0), 1), (dict(G=-1), 1), (dict(G=65), 2), (dict(n_q=-1), 1), (dict(n_q=(1 << 24) + 1), 2),
    (dict(q=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(q=FAKE + 8), 1),
    (dict(out=FAKE + 8), 1), (dict(ws=FAKE + 16), 1), (dict(q_lens=FAKE + 2), 1), (dict(qr=4), 1),
    (dict(qh=-128), 1), (dict(orow=0), 1), (dict(oh=64), 1), (dict(ou=0), 1), (dict(orow=132), 1),
    (dict(ws_bytes=1024), 1)])
def test_attention_refuses(kz, over, want):
    assert _attend(kz, _cache(kz), **over) == want


def test_nothing_to_do_is_ok(kz):
    assert _write(kz, _cache(kz, units=0)) == kz.OK
    assert _read(kz, _cache(kz), n=0) == kz.OK
    assert _attend(kz, _cache(kz), n_q=0) == kz.OK
    assert _attend(kz, _cache(kz, units=0)) == kz.OK
    # a bf16 cache needs no parameter words: refused only for what comes after them
    assert _attend(kz, _cache(kz, format=0, k_params=None, v_params=None), q=None) == kz.ERR_INVALID_ARG


def test_workspace_size_grows_with_the_call(kz):
    c = _cache(kz)
    a, b = kz.cache_attention_workspace_size(c, 4, 1), kz.cache_attention_workspace_size(c, 4, 64)
    assert 0 < a < b < 1 << 30
    assert kz.cache_attention_workspace_size(c, 0, 1) == 0
    assert kz.cache_attention_workspace_size(c, 65, 1) == 0


def test_paged_cache_refuses_host_tensors():
    from attention_score_reduction_b200 import cache
    pages = torch.zeros(4, 16, 128, dtype=torch.bfloat16)
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        cache.PagedCache("bf16", pages, pages, None, None, one.view(1, 1), one, one)
    with pytest.raises(ValueError):
        cache.PagedCache("int3", pages, pages, None, None, one.view(1, 1), one, one)
    with pytest.raises(ValueError):
        cache.PagedCache.allocate("fp4", 1, 128, 4, device="cpu")
