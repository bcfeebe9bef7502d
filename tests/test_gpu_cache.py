"""The paged cache on the GPU: writing (with quantisation), reading back, and
attention, against the float64 definitions in oracle/cache_oracle.py.

Codes, parameters and lengths must be equal.  Values read back are one rounding
to bf16 away from the definition.  Attention's tolerance per output element:

    half(out) |out| + (w + 2 (e^delta - 1) + 1e-5) * sum_j p_j |v_j|

half(out) = eps/2 of the output type (the final rounding).  w = the rounding of a
weight: fp16 for quantised caches (2^-11); bf16 on the tensor-memory path (2^-8)
and two bf16 parts where few query rows read the cache (2^-16) otherwise.  On the
tensor-memory path an int4 row is rounded to fp16 as well (2^-11 more in v, and in
k: a logit error of 2^-11 * reach), and keys carry one power of two per 64 rows
(2^-38 of the largest reach).  delta bounds the logit: d float32
additions of products whose magnitudes add up to `reach`, d * 2^-24 * reach; a
relative error e^delta - 1 of each weight and of their sum.  1e-5 covers the
exponentials and the sums over rows.  For int4 the products are with s c and z
apart, so magnitudes are taken over both.
"""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu
FMTS = ("bf16", "fp8", "int4")


@pytest.fixture(scope="module")
def kz():
    from attention_score_reduction_b200 import build
    build.build()
    from attention_score_reduction_b200 import kvzip
    return kvzip


@pytest.fixture(scope="module")
def kc(kz):
    from attention_score_reduction_b200 import cache
    return cache


def f64(t):
    return t.detach().cpu().double().numpy()


def rows_bf16(seed, *shape, keys=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g)
    if keys:
        x[..., ::37] *= 5.0
    return x.to(torch.bfloat16)


def make_cache(kc, fmt, lens, d, page_rows, capacity, seed=0, spare=3):
    """A cache whose pages are scattered over the pool and whose every byte outside
    the rows to come is junk (NaN in bf16, NaN parameters otherwise)."""
    units = len(lens)
    max_pages = max(1, -(-capacity // page_rows))
    n_pages = units * max_pages + spare
    g = torch.Generator().manual_seed(seed)
    table = torch.randperm(n_pages, generator=g)[:units * max_pages].to(torch.int32)
    width = {"bf16": d, "fp8": d, "int4": d // 2}[fmt]
    if fmt == "bf16":
        pool = lambda: torch.full((n_pages, page_rows, width), float("nan"),  # noqa: E731
                                  dtype=torch.bfloat16, device="cuda")
        par = lambda: None  # noqa: E731
    else:
        pool = lambda: torch.full((n_pages, page_rows, width), 0x7F, dtype=torch.uint8,  # noqa: E731
                                  device="cuda")
        par = lambda: torch.full((n_pages, page_rows), 0x7FC07FC0, dtype=torch.int32,  # noqa: E731
                                 device="cuda")
    return kc.PagedCache(fmt, pool(), pool(), par(), par(),
                         table.view(units, max_pages).cuda(),
                         torch.tensor(lens, dtype=torch.int32, device="cuda"))


def slots(cache, u, first, n):
    pos = np.arange(first, first + n)
    table = cache.page_table[u].cpu().numpy()
    return table[pos // cache.page_rows].astype(np.int64) * cache.page_rows + pos % cache.page_rows


def stored(cache, side, u, first, n):
    """(codes, parameter words) of stored rows, codes one per element."""
    s = torch.from_numpy(slots(cache, u, first, n)).cuda()
    pages = getattr(cache, side + "_pages")
    raw = pages.view(-1, pages.shape[2])[s].cpu()
    if cache.fmt == "bf16":
        return raw, None
    par = getattr(cache, side + "_params").view(-1)[s].cpu().numpy().view(np.uint32)
    raw = raw.numpy().astype(np.int64)
    if cache.fmt == "int4":
        raw = np.stack((raw & 15, raw >> 4), 2).reshape(n, cache.d)
    return raw, par


def held_values(cache, side, u, n):
    codes, par = stored(cache, side, u, 0, n)
    return f64(codes) if par is None else co.values(codes, par, cache.fmt)


def check_stored(cache, side, u, first, rows):
    codes, par = stored(cache, side, u, first, rows.shape[0])
    if cache.fmt == "bf16":
        assert torch.equal(codes.view(torch.int16), rows.cpu().view(torch.int16))
        return
    want, wpar = co.quantise(f64(rows), cache.fmt)
    assert np.array_equal(par, wpar)
    want = np.where(want < 0, codes, want)          # rows of NaN: codes unspecified for int4
    bad = np.argwhere(codes != want)
    assert bad.size == 0, (bad[:5], codes[tuple(bad[0])], want[tuple(bad[0])])


# ------------------------------------------------------------------ writing

@pytest.mark.parametrize("page_rows", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("fmt", FMTS)
def test_write_dense_append(kc, fmt, d, page_rows):
    lens, n = [0, 1, 17, 63, 130], 37
    c = make_cache(kc, fmt, lens, d, page_rows, 260, seed=d + page_rows)
    before = c.k_pages.clone(), c.v_pages.clone()
    k, v = rows_bf16(1, 5, n, d, keys=True).cuda(), rows_bf16(2, 5, n, d).cuda()
    c.write(k, v)
    assert c.lens.tolist() == [x + n for x in lens]
    c.write(k[:, :5], v[:, :5])                     # a second, small append, from views
    assert c.lens.tolist() == [x + n + 5 for x in lens]
    c.check_status()
    used = np.zeros(c.n_pages * page_rows, bool)
    for u, first in enumerate(lens):
        for side, x in (("k", k), ("v", v)):
            check_stored(c, side, u, first, x[u])
            check_stored(c, side, u, first + n, x[u, :5])
        used[slots(c, u, first, n + 5)] = True
    free = torch.from_numpy(~used).cuda()            # nothing else was touched
    for side, old in zip(("k", "v"), before):
        new = getattr(c, side + "_pages")
        assert torch.equal(new.view(-1, new.shape[2])[free].view(torch.uint8),
                           old.view(-1, old.shape[2])[free].view(torch.uint8))
        if fmt != "bf16":
            assert bool((getattr(c, side + "_params").view(-1)[free] == 0x7FC07FC0).all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [1, 2, 32, 33, 200])
def test_write_counts_and_starts(kc, fmt, n):
    lens = [5, 40, 0, 9]
    c = make_cache(kc, fmt, lens, 128, 32, 450)
    k, v = rows_bf16(3, 4, n, 128).cuda(), rows_bf16(4, 4, n, 128).cuda()
    counts = [n, 0, 1, (n + 1) // 2]
    ct = torch.tensor(counts, dtype=torch.int32, device="cuda")
    c.write(k, v, counts=ct)
    assert c.lens.tolist() == [a + b for a, b in zip(lens, counts)]
    starts = [0, 3, 7, 50]                            # rewriting earlier rows, and a gap
    c.write(v, k, starts=torch.tensor(starts, dtype=torch.int32, device="cuda"), counts=ct)
    assert c.lens.tolist() == [a + b for a, b in zip(starts, counts)]
    c.write(v, k, starts=c.lens, counts=ct)           # the lengths themselves: an append
    assert c.lens.tolist() == [a + 2 * b for a, b in zip(starts, counts)]
    c.check_status()
    for u in range(4):
        check_stored(c, "k", u, starts[u], v[u, :counts[u]])
        check_stored(c, "v", u, starts[u] + counts[u], k[u, :counts[u]])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("given", [False, True])
def test_write_packed(kc, fmt, given):
    """Rows as compaction leaves them: ragged, empty heads first, amid and last."""
    counts = [0, 300, 0, 0, 1, 77, 0]
    off = np.concatenate(([0], np.cumsum(counts))).astype(np.int64)
    c = make_cache(kc, fmt, [2] * 7, 128, 64, 320)
    k, v = rows_bf16(5, 378, 128, keys=True).cuda(), rows_bf16(6, 378, 128).cuda()
    starts = torch.arange(7, dtype=torch.int32, device="cuda") if given else None
    c.write(k, v, offsets=torch.from_numpy(off).cuda(), starts=starts)
    first = list(range(7)) if given else [2] * 7
    assert c.lens.tolist() == [a + b for a, b in zip(first, counts)]
    c.check_status()
    for u in range(7):
        check_stored(c, "k", u, first[u], k[off[u]:off[u + 1]])
        check_stored(c, "v", u, first[u], v[off[u]:off[u + 1]])


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("fmt", FMTS)
def test_write_strides(kc, fmt, d):
    """Token-major rows as a projection leaves them, and one row for every unit."""
    c = make_cache(kc, fmt, [0, 0, 0], d, 16, 64)
    kv = rows_bf16(7, 20, 3, 2, d).cuda()             # [token][head][k or v][d]
    c.write(kv[:, :, 0].transpose(0, 1), kv[:, :, 1].transpose(0, 1))
    one = rows_bf16(8, d).cuda()
    c.write(one.expand(3, 2, d), one.expand(3, 2, d))
    assert c.lens.tolist() == [22] * 3
    for u in range(3):
        check_stored(c, "k", u, 0, kv[:, u, 0])
        check_stored(c, "v", u, 0, kv[:, u, 1])
        check_stored(c, "v", u, 20, one.expand(2, d))


def special_rows(d):
    r = [torch.zeros(d), torch.full((d,), 3.0), torch.full((d,), -7.5e-39)]
    for seed, spread in ((1, 1e-39), (2, 1e-30), (3, 1e30), (4, 2e37)):
        r.append(rows_bf16(seed, d).float() * spread)
    x = rows_bf16(9, d).float()
    for bad in (float("inf"), -float("inf"), float("nan")):
        y = x.clone()
        y[d - 3] = bad
        r.append(y)
    y = x.clone()
    y[5] = 2.0 ** 126
    r.append(y)
    y = x.clone()
    y[5] = 1.7e38                                     # one huge element
    r.append(y)
    # range 240 = 15 * 16: elements near and on the borders 8 (2 c + 1) - 120 between codes
    y = (torch.arange(d).float() % 16) * 16 + 8 - 120
    y = y.clamp(max=120)
    y[0], y[1] = -120.0, 120.0
    y[2], y[3], y[4], y[5] = 1e-30, -1e-30, 0.0, 2.0 ** -20
    y[6], y[7] = -2.0 ** -20, 16.0
    r.append(y)
    # borders of e4m3: halves between neighbouring codes, subnormals, the largest
    y = torch.cat([torch.tensor([448.0, 464.0 / 2, 17.0, 19.0, 2.0 ** -10, 2.0 ** -9 * 1.5, 2.0 ** -11]),
                   torch.linspace(-440, 440, d - 7)])
    r.append(y)
    r.append(torch.cat([torch.tensor([450.0]), torch.linspace(-1, 1, d - 1)]))   # just above 448
    r.append(torch.cat([torch.tensor([1e30]), torch.full((d - 1,), 1e-30)]))
    return torch.stack(r).to(torch.bfloat16)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("fmt", FMTS)
def test_write_special_rows(kc, fmt, d):
    x = special_rows(d).cuda()
    n = x.shape[0]
    c = make_cache(kc, fmt, [0], d, 16, n)
    c.write(x[None], x.flip(0)[None])
    check_stored(c, "k", 0, 0, x)
    check_stored(c, "v", 0, 0, x.flip(0))
    k, v = c.read(n_rows=n)
    if fmt == "bf16":
        assert torch.equal(k[0].view(torch.int16), x.view(torch.int16))
        return
    codes, par = co.quantise(f64(x), fmt)
    want = co.values(np.maximum(codes, 0), par, fmt)
    got = f64(k[0])
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    # three rows hold an infinity or NaN; int4 also gives up those that reach 2^126
    assert nan.all(1).sum() == (5 if fmt == "int4" else 3)
    tol = np.abs(want) * 2.0 ** -8 * (1 + 2.0 ** -14) + 2.0 ** -134
    assert np.all(np.abs(got - want)[~nan] <= tol[~nan])


@pytest.mark.parametrize("fmt", ["fp8", "int4"])
def test_read_back_is_the_rounded_value(kc, fmt):
    n = 3000
    c = make_cache(kc, fmt, [0, 0], 128, 64, n)
    k, v = rows_bf16(11, 2, n, 128, keys=True).cuda(), rows_bf16(12, 2, n, 128).cuda()
    c.write(k, v)
    kb, vb = c.read(n_rows=n)
    for side, src, got in (("k", k, kb), ("v", v, vb)):
        for u in range(2):
            codes, par = co.quantise(f64(src[u]), fmt)
            assert np.array_equal(f64(got[u]), co.bf16_round(co.values(codes, par, fmt)))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("fmt", FMTS)
def test_read_ranges(kc, fmt, d):
    """Packed and dense reads from given positions; rows that are not held, and
    outputs of other rows, stay as they were."""
    lens = [70, 0, 1, 33]
    c = make_cache(kc, fmt, [0] * 4, d, 32, 96)
    k, v = rows_bf16(13, 4, 70, d).cuda(), rows_bf16(14, 4, 70, d).cuda()
    c.write(k, v, counts=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    kd, vd = c.read(n_rows=80)
    starts = torch.tensor([10, 0, 1, 30], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 60, 60, 62, 70], dtype=torch.int64, device="cuda")
    ko, vo = (torch.full((70, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c.read(off, 70, starts=starts, k_out=ko, v_out=vo)
    c.check_status()
    for dense, packed, side in ((kd, ko, "k"), (vd, vo, "v")):
        for u, n in enumerate(lens):
            want = co.bf16_round(held_values(c, side, u, n))
            assert np.array_equal(f64(dense[u, :n]), want)
            assert torch.count_nonzero(dense[u, n:]) == 0
        assert torch.equal(packed[:60], dense[0, 10:70])
        assert torch.equal(packed[62:65], dense[3, 30:33])
        assert bool((packed[60:62] == 9).all()) and bool((packed[65:] == 9).all())


def test_read_feeds_the_packed_decoder(kc, kz):
    """Rows read back packed are what kvzip.decode_attention takes."""
    lens = [200, 3, 64]
    c = make_cache(kc, "int4", [0] * 3, 128, 64, 256)
    k, v = rows_bf16(15, 3, 200, 128).cuda(), rows_bf16(16, 3, 200, 128).cuda()
    c.write(k, v, counts=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    off = torch.tensor([0, 200, 203, 267], dtype=torch.int64, device="cuda")
    kp, vp = c.read(off, 267)
    q = rows_bf16(17, 3, 4, 128).cuda()
    a = kz.decode_attention(q, kp, vp, off)
    b = c.attend(q[:, :, None], out_dtype=torch.float32)[:, :, 0]
    assert torch.allclose(a, b, rtol=2e-2, atol=2e-2)      # k and v rounded to bf16 in between


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_past_the_pages_are_dropped(kc, kz, fmt):
    c = make_cache(kc, fmt, [30, 0], 128, 16, 32)          # 32 rows fit
    k = rows_bf16(18, 2, 10, 128).cuda()
    c.write(k, k)
    assert c.lens.tolist() == [32, 10]
    check_stored(c, "k", 0, 30, k[0, :2])
    check_stored(c, "v", 1, 0, k[1])
    with pytest.raises(kz.KvzipError) as e:
        c.check_status()
    assert e.value.status == kz.ERR_INVALID_ARG
    c.check_status()                                       # read and cleared


@pytest.mark.parametrize("fmt", FMTS)
def test_bad_lengths_and_pages_are_recorded(kc, kz, fmt):
    """Lengths, counts and page ids out of range touch nothing outside the pool."""
    c = make_cache(kc, fmt, [40, 40, -5, 1000], 128, 16, 64)
    c.page_table[0, 0] = -1
    c.page_table[1, 1] = c.n_pages
    q = rows_bf16(19, 4, 2, 1, 128).cuda()
    out = c.attend(q)
    k, _ = c.read(n_rows=40)
    assert torch.count_nonzero(out[2]) == 0
    assert torch.count_nonzero(k[0, :16]) == 0 and torch.count_nonzero(k[1, 16:32]) == 0
    with pytest.raises(kz.KvzipError):
        c.check_status()
    c.write(q[:, 0], q[:, 0], starts=torch.tensor([3, 17, -1, 70], dtype=torch.int32, device="cuda"),
            counts=torch.tensor([5, -1, 1, 1], dtype=torch.int32, device="cuda"))
    assert c.lens.tolist() == [4, 17, 1, 64]
    with pytest.raises(kz.KvzipError):
        c.check_status()


# ---------------------------------------------------------------- attention

def check_attention(c, q, out, lens, q_lens, scale=None, untouched=None):
    d, G = c.d, q.shape[1]
    scale = 1 / np.sqrt(d) if scale is None else scale
    half = torch.finfo(out.dtype).eps / 2
    tc = uses_tensor_memory(c.fmt, d, G, q.shape[2])
    quant = c.fmt != "bf16"
    w = 2.0 ** -11 if quant else (2.0 ** -8 if tc else 2.0 ** -16)
    got = f64(out)
    for u, (n, m) in enumerate(zip(lens, q_lens)):
        k, v = held_values(c, "k", u, n), held_values(c, "v", u, n)
        want, wt, reach = co.attention(f64(q[u]), k, v, m, scale)
        if c.fmt == "int4":                    # magnitudes of s c and z apart
            mags = []
            for side in "kv":
                codes, par = stored(c, side, u, 0, n)
                z = co.values(np.zeros_like(codes), par, "int4")
                mags.append(np.abs(co.values(codes, par, "int4") - z) + np.abs(z))
            _, wt, reach = co.attention(np.abs(f64(q[u])), mags[0], mags[1], m, scale)
            # weights are the true ones; bound sum p |v| by the largest row instead
            wt = np.broadcast_to(mags[1].max(0) if n else np.zeros(d), wt.shape)
        delta = d * 2.0 ** -24 * reach
        ww = w
        if tc and quant:
            delta = delta + 2.0 ** -38 * reach
        if tc and c.fmt == "int4":
            delta = delta + 2.0 ** -11 * reach
            ww = w + 2.0 ** -11
        tol = half * np.abs(want) + (ww + 2 * np.expm1(delta)[..., None] + 1e-5) * wt
        err = np.abs(got[u, :, :m] - want)
        assert np.all(np.isfinite(got[u, :, :m]))
        assert np.all(err <= tol), (u, n, m, float((err - tol).max()), float(err.max()))
        if untouched is not None:
            assert np.all(got[u, :, m:] == untouched)


def uses_tensor_memory(fmt, d, G, n_q):
    return G * n_q > (32 if d == 128 else 16) * (1 if fmt == "bf16" else 2)


def filled(kc, fmt, lens, d, page_rows, seed, capacity=None):
    c = make_cache(kc, fmt, [0] * len(lens), d, page_rows, capacity or max(max(lens), 1), seed=seed)
    n = max(max(lens), 1)
    k, v = rows_bf16(seed + 1, len(lens), n, d, keys=True), rows_bf16(seed + 2, len(lens), n, d)
    c.write(k.cuda(), v.cuda(), counts=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    return c


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 8, 16])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("fmt", FMTS)
def test_one_token(kc, fmt, d, G):
    lens = [700, 0, 1, 15, 16, 17, 64, 65, 129]
    c = filled(kc, fmt, lens, d, 16 << (G % 4), seed=G)
    q = rows_bf16(20 + G, len(lens), G, 1, d).cuda()
    for dt in (torch.bfloat16, torch.float32):
        check_attention(c, q, c.attend(q, out_dtype=dt), lens, [min(1, n) for n in lens])
    c.check_status()


@pytest.mark.parametrize("n_q", [2, 3, 9, 31, 64, 130])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("fmt", FMTS)
def test_chunk(kc, fmt, d, n_q):
    lens = [n_q, n_q + 1, n_q + 130, 517 + n_q]
    c = filled(kc, fmt, lens, d, 32, seed=n_q)
    G = {2: 4, 3: 5, 9: 1, 31: 8, 64: 2, 130: 3}[n_q]
    q = rows_bf16(40 + n_q, len(lens), G, n_q, d).cuda()
    check_attention(c, q, c.attend(q), lens, [n_q] * 4)
    check_attention(c, q, c.attend(q, scale=0.03, out_dtype=torch.float32), lens, [n_q] * 4,
                    scale=float(np.float32(0.03)))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,G,n_q", [(128, 4, 40), (256, 2, 40), (128, 1, 5), (128, 64, 3), (256, 7, 50)])
def test_ragged_chunks(kc, fmt, d, G, n_q):
    """Sequences with different new tokens (none, one, all); tokens that see
    nothing give zeros; rows past a unit's tokens stay as they were."""
    lens = [300, 0, n_q - 2, 90, n_q, 2]
    q_lens = [n_q, 0, n_q - 2, 1, n_q, 0]
    c = filled(kc, fmt, lens, d, 16, seed=3)
    q = rows_bf16(60, 6, G, n_q, d).cuda()
    out = torch.full((6, G, n_q, d), 7.0, dtype=torch.bfloat16, device="cuda")
    c.attend(q, q_lens=torch.tensor(q_lens, dtype=torch.int32, device="cuda"), out=out)
    check_attention(c, q, out, lens, q_lens, untouched=7.0)
    # more new tokens than rows: the first see nothing
    out = c.attend(q)
    for u, n in enumerate(lens):
        blind = max(0, n_q - n)
        assert torch.count_nonzero(out[u, :, :blind]) == 0
    c.check_status()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,G,n_q", [(128, 4, 8), (128, 4, 9), (128, 4, 16), (128, 5, 13),
                                     (128, 64, 1), (256, 4, 4), (256, 4, 8), (256, 3, 11), (256, 32, 1)])
def test_about_where_the_kernels_change(kc, fmt, d, G, n_q):
    """Several blocks of 16 query rows a unit, and the first sizes of the other kernel."""
    lens = [1500, 0, n_q, 3, 77, 130]
    q_lens = [n_q, 0, n_q, min(3, n_q), max(1, n_q - 3), n_q]
    c = filled(kc, fmt, lens, d, 32, seed=G + n_q)
    q = rows_bf16(180 + n_q, len(lens), G, n_q, d).cuda()
    out = torch.full(q.shape, 7.0, dtype=torch.float32, device="cuda")
    c.attend(q, q_lens=torch.tensor(q_lens, dtype=torch.int32, device="cuda"), out=out)
    check_attention(c, q, out, lens, q_lens, untouched=7.0)
    c.check_status()


@pytest.mark.parametrize("d,G,n_q", [(128, 4, 33), (256, 2, 1), (128, 5, 1), (256, 3, 70)])
@pytest.mark.parametrize("fmt", FMTS)
def test_attention_strides(kc, fmt, d, G, n_q):
    """Token-major q and out, as the projections around attention have them."""
    lens = [n_q + 77, n_q]
    c = filled(kc, fmt, lens, d, 64, seed=5)
    q = rows_bf16(70, n_q, 2, G, d).cuda().permute(1, 2, 0, 3)
    out = torch.empty(n_q, 2, G, d, dtype=torch.bfloat16, device="cuda").permute(1, 2, 0, 3)
    c.attend(q, out=out)
    check_attention(c, q, out, lens, [n_q] * 2)
    q1 = rows_bf16(71, d).cuda().expand(2, G, n_q, d)       # one query for all
    check_attention(c, q1, c.attend(q1), lens, [n_q] * 2)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,n_q", [(128, 1), (256, 1), (128, 70), (256, 70)])
def test_long_and_uneven_units(kc, fmt, d, n_q):
    """One long unit beside many short ones: items share CTAs and CTAs share items."""
    lens = [9000] + [n_q + i for i in range(20)] + [4001, 70]
    c = filled(kc, fmt, lens, d, 128, seed=7)
    q = rows_bf16(80, len(lens), 2, n_q, d).cuda()
    check_attention(c, q, c.attend(q), lens, [n_q] * len(lens))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n_q", [1, 40])
def test_magnitudes(kc, fmt, d, n_q):
    """Query and key rows of very different sizes, a dominating key, large logits."""
    lens = [600]
    c = make_cache(kc, fmt, [0], d, 64, 600)
    k, v = rows_bf16(90, 1, 600, d), rows_bf16(91, 1, 600, d)
    v = (v.float() * torch.logspace(-6, 3, 600).view(1, -1, 1)).to(torch.bfloat16)
    k[0, 5] *= 6.0
    c.write(k.cuda(), v.cuda())
    q = rows_bf16(92, 1, 3, n_q, d)
    q[0, 1] *= 2.0 ** -40
    q[0, 2] *= 4.0
    q = q.cuda()
    check_attention(c, q, c.attend(q, out_dtype=torch.float32), lens, [n_q])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n_q", [1, 40])
@pytest.mark.parametrize("stride", [1, 97])
def test_value_rows_far_apart(kc, fmt, d, n_q, stride):
    """Value rows from 2^-46 to 2^46, neighbours alike or far apart: the sum of the
    weights counts the small ones as well."""
    lens = [600]
    c = make_cache(kc, fmt, [0], d, 32, 600)
    k, v = rows_bf16(95, 1, 600, d), rows_bf16(96, 1, 600, d)
    exps = torch.linspace(-46, 46, 600)[(torch.arange(600) * stride) % 600]
    v = (v.float() * torch.exp2(exps).view(1, -1, 1)).to(torch.bfloat16)
    c.write(k.cuda(), v.cuda())
    q = rows_bf16(97, 1, 3, n_q, d).cuda()
    check_attention(c, q, c.attend(q, out_dtype=torch.float32), lens, [n_q])


@pytest.mark.parametrize("n_q", [1, 20])
@pytest.mark.parametrize("fmt", FMTS)
def test_non_finite_rows_reach_who_sees_them(kc, fmt, n_q):
    """A NaN in a seen row gives NaN; one in a page's rest, or of another unit, nothing."""
    c = filled(kc, fmt, [50, 50], 128, 64, seed=9)
    k, v = rows_bf16(93, 2, 1, 128).cuda(), rows_bf16(94, 2, 1, 128).cuda()
    v[0, 0, 3] = float("nan")
    c.write(k, v, starts=torch.tensor([10, 50], dtype=torch.int32, device="cuda"))
    c.lens.fill_(50)
    q = rows_bf16(95, 2, 4, n_q, 128).cuda()
    out = c.attend(q)
    assert bool(torch.isnan(out[0, :, :, 3]).all())
    if fmt == "bf16":
        assert bool(torch.isfinite(out[0, :, :, :3]).all())
    assert bool(torch.isfinite(out[1]).all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("G,n_q,bad", [(1, 3, 1), (4, 4, 3), (5, 33, 20), (2, 300, 0), (2, 300, 299), (4, 150, 77)])
def test_non_finite_rows_of_later_tokens(kc, fmt, d, G, n_q, bad):
    """A token whose own K and V rows are not finite: earlier tokens do not see them."""
    lens = [n_q + 41, n_q]
    c = filled(kc, fmt, lens, d, 32, seed=33)
    k, v = rows_bf16(98, 2, 1, d), rows_bf16(99, 2, 1, d)
    k[0, 0, 5] = float("nan")
    v[0, 0, 3] = float("inf")
    v[1, 0, d - 1] = float("nan")
    at = torch.tensor([n - n_q + bad for n in lens], dtype=torch.int32, device="cuda")
    c.write(k.cuda(), v.cuda(), starts=at)
    c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    q = rows_bf16(100, 2, G, n_q, d).cuda()
    out = c.attend(q)
    if bad:
        check_attention(c, q[:, :, :bad], out[:, :, :bad], at.tolist(), [bad, bad])
    assert not bool(torch.isfinite(out[0, :, bad:, 3]).any())
    assert not bool(torch.isfinite(out[1, :, bad:, d - 1]).any())


def test_captured_step_replays_with_growing_lengths(kc):
    """Append and attend in one CUDA graph: every replay adds a token."""
    for fmt in FMTS:
        c = filled(kc, fmt, [90, 33, 0], 128, 16, seed=11, capacity=160)
        k, v = (torch.empty(3, 1, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q = torch.empty(3, 4, 1, 128, dtype=torch.bfloat16, device="cuda")
        out = torch.empty_like(q)
        for t in (k, v, q):
            t.copy_(rows_bf16(1, *t.shape))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c.write(k, v)
            c.attend(q, out=out)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.write(k, v)
            c.attend(q, out=out)
        for step in range(3):
            for i, t in enumerate((k, v, q)):
                t.copy_(rows_bf16(100 + 3 * step + i, *t.shape))
            g.replay()
            lens = [92 + step, 35 + step, 2 + step]
            lens = [n for n in lens]
            assert c.lens.tolist() == lens
            check_attention(c, q, out, lens, [1] * 3)
            for u in range(3):
                check_stored(c, "k", u, lens[u] - 1, k[u])


def test_captured_behind_a_fork(kc):
    """Calls captured where two streams have joined: a launch has two predecessors."""
    for fmt in FMTS:
        c = filled(kc, fmt, [70, 9], 128, 16, seed=15, capacity=90)
        k, v = rows_bf16(140, 2, 1, 128).cuda(), rows_bf16(141, 2, 1, 128).cuda()
        q = rows_bf16(142, 2, 4, 1, 128).cuda()
        kk, vv, out = torch.empty_like(k), torch.empty_like(v), torch.empty_like(q)
        back = torch.zeros(2, 80, 128, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g):
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                kk.copy_(k)
            vv.copy_(v)
            main.wait_stream(side)
            c.write(kk, vv)
            side.wait_stream(main)
            c.attend(q, out=out)
            c.read(n_rows=80, k_out=back, v_out=torch.empty_like(back), stream=side)
            main.wait_stream(side)
        g.replay()
        g.replay()
        lens = [72, 11]
        assert c.lens.tolist() == lens
        check_attention(c, q, out, lens, [1, 1])
        assert np.array_equal(f64(back[0, :72]), held_values(c, "k", 0, 72)) or fmt == "int4"
        del g


@pytest.mark.parametrize("n_q", [1, 20])
@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_more_units_than_threads(kc, fmt, n_q):
    """A block finds its place among more items than it has threads."""
    g = torch.Generator().manual_seed(16)
    lens = torch.randint(0, 50, (700,), generator=g).tolist()
    lens[3], lens[650], lens[699] = 2500, 1300, 700
    c = filled(kc, fmt, lens, 128, 32, seed=16)
    q = rows_bf16(143, len(lens), 2, n_q, 128).cuda()
    q_lens = [min(n_q, n) for n in lens]
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    c.attend(q, q_lens=torch.tensor(q_lens, dtype=torch.int32, device="cuda"), out=out)
    c.check_status()
    some = [0, 1, 2, 3, 4, 255, 256, 257, 300, 639, 640, 649, 650, 651, 698, 699]
    for u in some:
        one = kc.PagedCache(c.fmt, c.k_pages, c.v_pages, c.k_params, c.v_params,
                            c.page_table[u:u + 1], c.lens[u:u + 1])
        check_attention(one, q[u:u + 1], out[u:u + 1], [lens[u]], [q_lens[u]], untouched=7.0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [128, 256])
def test_stalled_waits_end_and_are_recorded(kc, kz, fmt, d):
    """With the loads left out every wait runs out (10 ms here); the next call is right."""
    c = filled(kc, fmt, [900, 300], d, 32, seed=17)
    q = rows_bf16(144, 2, 4, 40, d).cuda()
    want = c.attend(q)
    c.check_status()
    kz.set_wait_timeout_ns(10_000_000)
    kz.set_test_stall(True)
    try:
        c.attend(q)
        status = kz.workspace_status(c.status)
    finally:
        kz.set_test_stall(False)
        kz.set_wait_timeout_ns(0)
    assert status == kz.ERR_TIMEOUT
    assert torch.equal(c.attend(q), want)
    c.check_status()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [128, 256])
def test_same_bits_where_blocks_cross_items(kc, fmt, d):
    """Many long items, several to a block: pages, tiles and parameters of one item come
    while the one before is still worked on."""
    g = torch.Generator().manual_seed(19)
    lens = torch.randint(310, 5000, (32,), generator=g).tolist()
    c = filled(kc, fmt, lens, d, 128, seed=19)
    q = rows_bf16(170, 32, 4, 301, d).cuda()
    ql = torch.tensor([301 - 7 * (u // 8) for u in range(32)], dtype=torch.int32, device="cuda")
    outs = [torch.zeros_like(q) for _ in range(30)]
    for o in outs:
        c.attend(q, q_lens=ql, out=o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs)
    for u in (0, 17, 31):
        one = kc.PagedCache(c.fmt, c.k_pages, c.v_pages, c.k_params, c.v_params,
                            c.page_table[u:u + 1], c.lens[u:u + 1])
        check_attention(one, q[u:u + 1], outs[0][u:u + 1], [lens[u]], [int(ql[u])], untouched=0.0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,n_q", [(128, 1), (128, 150), (256, 1), (256, 90)])
def test_calls_back_to_back(kc, fmt, d, n_q):
    """Calls that follow one another without a pause, through the same scratch memory:
    each gives the bits that it gives alone."""
    lens = [5000, 1200, 3333, 40]
    c = filled(kc, fmt, lens, d, 32, seed=18)
    qs = [rows_bf16(150 + i, 4, 4, n_q, d).cuda() for i in range(3)]
    k, v = (rows_bf16(160 + i, 4, 3, d).cuda() for i in range(2))
    start = torch.tensor([n - 3 for n in lens], dtype=torch.int32).cuda()
    want = []
    for i, q in enumerate(qs):
        c.write(k * (i + 1), v * (i + 1), starts=start)
        torch.cuda.synchronize()
        want.append(c.attend(q))
        torch.cuda.synchronize()
    news = [(k * (i + 1), v * (i + 1)) for i in range(3)]
    outs = [[torch.empty_like(q) for q in qs] for _ in range(40)]
    torch.cuda.synchronize()
    for step in outs:
        for q, o, (kn, vn) in zip(qs, step, news):
            c.write(kn, vn, starts=start)
            c.attend(q, out=o)
    torch.cuda.synchronize()
    for step in outs:
        for o, w in zip(step, want):
            assert torch.equal(o, w)


def test_two_captured_graphs_at_once(kc):
    """Two graphs of calls on the same cache, replayed on two streams together."""
    c = filled(kc, "fp8", [3000, 100], 128, 64, seed=12)
    qs = [rows_bf16(110 + i, 2, 4, n, 128).cuda() for i, n in enumerate((1, 2))]
    want = [c.attend(q) for q in qs]
    outs = [torch.zeros_like(q) for q in qs]
    graphs = []
    for q, o in zip(qs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.attend(q, out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_given_stream(kc):
    """Work on a stream that is not the current one, with memory made by the calls."""
    c = filled(kc, "int4", [2000, 1500], 128, 64, seed=13)
    q = rows_bf16(120, 2, 4, 3, 128).cuda()
    want = c.attend(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = c.attend(q, stream=s)
        junk = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")   # on the current stream
        k, v = c.read(n_rows=10, stream=s)
        del junk
    s.synchronize()
    assert torch.equal(got, want)
    assert torch.equal(k, c.read(n_rows=10)[0])


@pytest.mark.parametrize("fmt", FMTS)
def test_same_bits_every_time(kc, fmt):
    c = filled(kc, fmt, [5000, 70, 900], 128, 32, seed=14)
    for n_q in (1, 50):
        q = rows_bf16(130, 3, 4, n_q, 128).cuda()
        first = c.attend(q)
        for _ in range(3):
            assert torch.equal(c.attend(q), first)


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_past_32_bits(kc, fmt):
    """Rows at the far end of pools of more than 2^32 bytes."""
    d, page_rows = 256, 128
    row = {"bf16": 512, "fp8": 256, "int4": 128}[fmt]
    n_pages = (1 << 32) // (row * page_rows) + 40
    dt = torch.bfloat16 if fmt == "bf16" else torch.uint8
    width = d if fmt == "bf16" else row
    kp, vp = (torch.empty(n_pages, page_rows, width, dtype=dt, device="cuda") for _ in range(2))
    pk, pv = (None, None) if fmt == "bf16" else (
        torch.empty(n_pages, page_rows, dtype=torch.int32, device="cuda") for _ in range(2))
    table = torch.tensor([[n_pages - 1, 0, n_pages - 7], [3, n_pages - 2, 5]], dtype=torch.int32,
                         device="cuda")
    c = kc.PagedCache(fmt, kp, vp, pk, pv, table, torch.zeros(2, dtype=torch.int32, device="cuda"))
    k, v = rows_bf16(140, 2, 300, d).cuda(), rows_bf16(141, 2, 300, d).cuda()
    c.write(k, v)
    for u in range(2):
        check_stored(c, "k", u, 0, k[u])
        check_stored(c, "v", u, 0, v[u])
    kb, _ = c.read(n_rows=300)
    if fmt == "bf16":
        assert torch.equal(kb, k)
    for n_q in (1, 40):
        q = rows_bf16(142, 2, 2, n_q, d).cuda()
        check_attention(c, q, c.attend(q), [300, 300], [n_q] * 2)


def test_allocate_reserve_clear(kc):
    c = kc.PagedCache.allocate("fp8", 3, 128, 10, page_rows=16, max_pages=6)
    c.reserve([40, 0, 16])
    assert (c.page_table >= 0).sum(1).tolist() == [3, 0, 1]
    c.reserve(17)
    assert (c.page_table >= 0).sum(1).tolist() == [3, 2, 2]
    used = c.page_table[c.page_table >= 0].tolist()
    assert len(set(used)) == 7
    with pytest.raises(ValueError):
        c.reserve(16 * 6)                    # more pages than the pool has
    with pytest.raises(ValueError):
        c.reserve([16 * 7, 0, 0])            # more than max_pages
    assert (c.page_table >= 0).sum(1).tolist() == [3, 2, 2]
    c.clear()
    c.reserve([16 * 6, 16 * 4, 0])
    assert (c.page_table >= 0).sum(1).tolist() == [6, 4, 0]


def test_paged_cache_refuses(kc):
    c = filled(kc, "fp8", [20, 20], 128, 16, seed=15, capacity=64)
    q = rows_bf16(150, 2, 4, 1, 128).cuda()
    lens = c.lens.tolist()
    i32 = lambda n, dev="cuda": torch.zeros(n, dtype=torch.int32, device=dev)  # noqa: E731
    bad = [
        (TypeError, lambda: c.attend(q.float())), (ValueError, lambda: c.attend(q[:1])),
        (ValueError, lambda: c.attend(q[..., :64])), (ValueError, lambda: c.attend(q.cpu())),
        (ValueError, lambda: c.attend(q[:, :, 0])), (ValueError, lambda: c.attend(q, q_lens=i32(3))),
        (TypeError, lambda: c.attend(q, q_lens=i32(2).long())),
        (ValueError, lambda: c.attend(q, q_lens=i32(2, "cpu"))),
        (ValueError, lambda: c.attend(q, out=q[:, :1])), (ValueError, lambda: c.attend(q, out=q.half())),
        (ValueError, lambda: c.attend(q, out=q[:1, :1].expand(2, 4, 1, 128))),
        (ValueError, lambda: c.write(q[:, :, 0], q[:, :2, 0])),
        (ValueError, lambda: c.write(q[:1, :, 0], q[:1, :, 0])),
        (TypeError, lambda: c.write(q[:, :, 0].half(), q[:, :, 0].half())),
        (ValueError, lambda: c.write(q[:, :, 0], q[:, :, 0], starts=i32(1))),
        (ValueError, lambda: c.write(q[0, :, 0], q[0, :, 0], offsets=i32(3).long(), counts=i32(2))),
        (TypeError, lambda: c.write(q[0, :, 0], q[0, :, 0], offsets=i32(3))),
        (ValueError, lambda: c.read()), (ValueError, lambda: c.read(n_rows=3, k_out=q)),
        (ValueError, lambda: kc.PagedCache("fp8", c.k_pages, c.v_pages, None, None, c.page_table, c.lens)),
        (TypeError, lambda: kc.PagedCache("bf16", c.k_pages, c.v_pages, None, None, c.page_table, c.lens)),
        (ValueError, lambda: kc.PagedCache("fp8", c.k_pages, c.v_pages[:1], c.k_params, c.v_params,
                                           c.page_table, c.lens)),
    ]
    for err, call in bad:
        with pytest.raises(err):
            call()
    wide = torch.zeros(2, 4, 3, 130, dtype=torch.bfloat16, device="cuda")[..., 1:129]
    from attention_score_reduction_b200 import kvzip as kz
    with pytest.raises(kz.KvzipError):
        c.attend(wide)                       # rows not on 16-byte boundaries
    assert c.lens.tolist() == lens
    c.check_status()


@pytest.mark.parametrize("fmt", FMTS)
def test_compress_ask_and_answer(kc, fmt):
    """As a user runs it: a context is compressed, its kept rows go into the
    cache, a question is appended and attended, then tokens one by one."""
    from attention_score_reduction_b200 import pipeline, synth
    wl = synth.Workload("cache", L=1, H=4, G=4, d=128, n_c=900, m=300, r=(0.3,), hi_frac=0.01,
                        sinks=4, cfg_id=78)
    k_ctx, v = synth.context_kv(wl)
    chunks = [synth.chunk_qk(wl, i) for i in range(wl.n_chunks)]
    comp = pipeline.Compressor(wl.units, wl.n_c, wl.d, wl.G, max(q.shape[2] for q, _ in chunks))
    out = comp.compress(k_ctx.cuda(), v.cuda(), [(q.cuda(), s.cuda()) for q, s in chunks], r=0.3)
    comp.check_status()
    off = out.offsets.cpu().numpy()
    kept = np.diff(off)
    assert kept.min() != kept.max()
    n_q, steps = 23, 4
    c = kc.PagedCache.allocate(fmt, wl.units, wl.d, n_pages=120, page_rows=16, max_pages=60)
    c.reserve([int(n) + n_q + steps for n in kept])
    c.write(out.k, out.v, offsets=out.offsets)
    assert c.lens.tolist() == kept.tolist()
    kq, vq = rows_bf16(160, 4, n_q, 128).cuda(), rows_bf16(161, 4, n_q, 128).cuda()
    q = rows_bf16(162, 4, 4, n_q, 128).cuda()
    c.write(kq, vq)
    lens = [int(n) + n_q for n in kept]
    check_attention(c, q, c.attend(q), lens, [n_q] * 4)
    for u in range(4):
        check_stored(c, "k", u, 0, out.k[off[u]:off[u + 1]])
        check_stored(c, "v", u, int(kept[u]), vq[u])
    for step in range(steps):
        k1, v1 = rows_bf16(170 + step, 4, 1, 128).cuda(), rows_bf16(180 + step, 4, 1, 128).cuda()
        q1 = rows_bf16(190 + step, 4, 4, 1, 128).cuda()
        c.write(k1, v1)
        lens = [n + 1 for n in lens]
        check_attention(c, q1, c.attend(q1), lens, [1] * 4)
    assert c.lens.tolist() == lens
    c.check_status()
