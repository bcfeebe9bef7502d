"""Attention over the paged cache against its float64 definition, element by element with
the tolerances of tests/cache_check.py, which tests/test_cache_check.py shows to notice
wrong results of every kind."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co
from tests import cache_check as cc
from tests.test_gpu_cache import (FMTS, f64, filled, held_values, make_cache, rows_bf16, slots,
                                  uses_tensor_memory)

pytestmark = pytest.mark.gpu


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


def held(c, side, u, n):
    """Rows of a unit in float64 on the GPU, in the parts they are stored in."""
    s = torch.from_numpy(slots(c, u, 0, n)).cuda()
    pages = getattr(c, side + "_pages")
    raw = pages.view(-1, pages.shape[2])[s]
    if c.fmt == "bf16":
        return cc.Rows(raw.double())
    par = getattr(c, side + "_params").view(-1)[s].view(-1, 1)
    if c.fmt == "fp8":
        table = torch.from_numpy(co.e4m3_value(np.arange(256))).cuda()
        return cc.Rows(table[raw.long()] * par.view(torch.float32).double())
    sz = par.view(torch.bfloat16).double()
    codes = torch.stack((raw & 15, raw >> 4), 2).reshape(n, c.d).double()
    return cc.Rows(codes * sz[:, :1], sz[:, 1:].expand(n, c.d))


def check(c, q, out, lens, q_lens, alike=True, scale=None, units=None, common=0.0):
    scale = c.d ** -0.5 if scale is None else scale
    tc = uses_tensor_memory(c.fmt, c.d, q.shape[1], q.shape[2])
    half = torch.finfo(out.dtype).eps / 2
    for u in range(len(lens)) if units is None else units:
        n, m = lens[u], q_lens[u]
        want, tol = cc.attention(q[u, :, :m].double(), held(c, "k", u, n), held(c, "v", u, n), m, scale,
                                 c.fmt, tc, half)
        wrong = cc.close(out[u, :, :m].double(), want, tol, alike, common)
        assert wrong is None, (u, n, m, wrong)


@pytest.mark.parametrize("G,n_q", [(1, 1), (5, 1), (4, 4), (8, 7), (4, 40), (2, 130), (3, 301)])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("fmt", FMTS)
def test_numbers(kc, fmt, d, G, n_q):
    lens = [n_q + 1900, n_q + 700, n_q, n_q + 64, n_q + 1, n_q + 3333]
    c = filled(kc, fmt, lens, d, 64, seed=200 + n_q)
    q = rows_bf16(210 + n_q, len(lens), G, n_q, d).cuda()
    for dt in (torch.bfloat16, torch.float32):
        check(c, q, c.attend(q, out_dtype=dt), lens, [n_q] * len(lens))
    c.check_status()


def uneven_values(seed, units, n, d):
    """V rows whose size changes by powers of two from 64 rows to the next, and by another
    pattern within them."""
    v = rows_bf16(seed, units, n, d).float()
    j = torch.arange(n)
    e = ((j // 64) * 5 % 13 - 6) * 2 + (j * 7 % 3)
    return (v * torch.exp2(e.float()).view(1, n, 1)).to(torch.bfloat16)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [128, 256])
def test_each_tile_has_its_own_powers(kc, fmt, d):
    """Items of many tiles beside items of one to five, several to a block, and every output of
    every call: a tile that took another one's power of two would be far off."""
    g = torch.Generator().manual_seed(21)
    lens = torch.randint(400, 5000, (24,), generator=g).tolist()
    tile = 128 if d == 128 else 64
    lens += [tile * t - x for t in (1, 2, 3, 4, 5) for x in (0, 1, 13)] * 2
    order = torch.randperm(len(lens), generator=g).tolist()
    lens = [lens[i] for i in order]
    units, n_q, G = len(lens), 200, 3
    q_lens = [min(n_q - 9 * (u % 5), lens[u]) for u in range(units)]
    c = make_cache(kc, fmt, [0] * units, d, 128, max(lens), seed=22)
    k = rows_bf16(220, units, max(lens), d).cuda()
    v = uneven_values(221, units, max(lens), d).cuda()
    c.write(k, v, counts=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    q = rows_bf16(222, units, G, n_q, d).cuda()
    ql = torch.tensor(q_lens, dtype=torch.int32, device="cuda")
    outs = [torch.zeros_like(q) for _ in range(20)]
    for o in outs:
        c.attend(q, q_lens=ql, out=o)
    torch.cuda.synchronize()
    check(c, q, outs[0], lens, q_lens, alike=False)
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    c.check_status()


@pytest.mark.parametrize("fmt", FMTS)
def test_read_behind_a_fork(kc, fmt):
    """Rows read on a second stream of a captured graph are the stored rows, rounded once."""
    c = filled(kc, fmt, [70, 9], 128, 16, seed=23, capacity=90)
    k, v = rows_bf16(230, 2, 1, 128).cuda(), rows_bf16(231, 2, 1, 128).cuda()
    back = [torch.zeros(2, 80, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        c.write(k, v)
        side.wait_stream(main)
        c.read(n_rows=80, k_out=back[0], v_out=back[1], stream=side)
        main.wait_stream(side)
    g.replay()
    g.replay()
    assert c.lens.tolist() == [72, 11]
    for side_name, got in zip("kv", back):
        for u, n in enumerate((72, 11)):
            assert np.array_equal(f64(got[u, :n]), co.bf16_round(held_values(c, side_name, u, n)))
    del g


@pytest.mark.parametrize("sink,gap", [(s, g) for s in ("zero", "small", "alike") for g in (18, 25, 28, 33)] + [("zero", 60), ("zero", 80)])
@pytest.mark.parametrize("d,n_q", [(128, 1), (128, 40), (256, 1), (256, 40)])
@pytest.mark.parametrize("fmt", FMTS)
def test_a_sink_at_the_start_of_a_long_cache(kc, fmt, d, n_q, sink, gap):
    """One row takes nearly all the weight, 2^gap times another's, and adds little or nothing:
    the output is then the sum of the others, each far below fp16's normal numbers.  Once with
    the rows shared out to all blocks, once with so many units on the same pages that a block
    walks all rows of one."""
    n, G, m = 70000, 2, n_q
    one = make_cache(kc, fmt, [0], d, 128, n, seed=24)
    k, v = rows_bf16(240, 1, n, d), rows_bf16(241, 1, n, d)
    k[:, :, 0] = 0.0
    k[0, 0] = 0.0
    k[0, 0, 0] = gap / (8.0 * d ** -0.5 * 1.4427)
    if sink != "alike":
        v[0, 0] = 0.0 if sink == "zero" else v[0, 0] * 2.0 ** -7
    one.write(k.cuda(), v.cuda())
    q = rows_bf16(242, 1, G, n_q, d)
    q[..., 0] = 8.0
    q = q.cuda()
    out = one.attend(q, out_dtype=torch.float32)
    # few rows of 4-bit pages: s c and z are summed apart and nearly cancel here, so that
    # float32's rounding of either is no longer small beside the output
    alike = sink != "alike" and (fmt != "int4" or n_q > 1)
    # many: the sink's key is rounded to fp16 like any other, and its weight is in every sum
    common = 2.0 ** -11 * gap * np.log(2) if fmt == "int4" else 0.0
    check(one, q, out, [n], [m], alike=alike, common=common)
    units = 450
    c = kc.PagedCache(fmt, one.k_pages, one.v_pages, one.k_params, one.v_params,
                      one.page_table.repeat(units, 1), one.lens.repeat(units))
    out = c.attend(q.expand(units, -1, -1, -1), out_dtype=torch.float32)
    check(c, q.expand(units, -1, -1, -1), out, [n] * units, [m] * units, alike=alike, common=common,
          units=(0, 1, 211, 449))
    one.check_status()
    c.check_status()


@pytest.mark.parametrize("power", [60, 66, 67, 68, 70, 74, 90])
@pytest.mark.parametrize("d,n_q", [(128, 1), (128, 40), (256, 1), (256, 40)])
@pytest.mark.parametrize("fmt", ["fp8", "int4"])
def test_values_larger_than_the_products_hold(kc, fmt, d, n_q, power):
    """A V row of magnitude 2^power and a bit: with few query rows it is what it is, with many
    a row of NaN beyond 2^64, for the tokens that see it and in no way for the others."""
    lens, G = [300, 200 + n_q], 3
    c = make_cache(kc, fmt, [0, 0], d, 64, max(lens), seed=25)
    k, v = rows_bf16(250, 2, max(lens), d), rows_bf16(251, 2, max(lens), d)
    v[1] *= 2.0 ** -9
    at = 200 + n_q // 2                         # a token of the chunk, of unit 1
    v[1, at] = (v[1, at].float().clamp(-1, 1) * 2.0 ** power).to(torch.bfloat16)
    v[1, at, 7] = 1.0625 * 2.0 ** power
    c.write(k.cuda(), v.cuda(), counts=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    q = rows_bf16(252, 2, G, n_q, d).cuda()
    out = c.attend(q, out_dtype=torch.float32)
    check(c, q[:1], out[:1], lens[:1], [n_q])
    many = uses_tensor_memory(fmt, d, G, n_q)
    if many:
        first = n_q // 2
        head = kc.PagedCache(fmt, c.k_pages, c.v_pages, c.k_params, c.v_params, c.page_table[1:],
                             torch.tensor([at], dtype=torch.int32, device="cuda"))
        half = torch.finfo(torch.float32).eps / 2
        want, tol = cc.attention(q[1, :, :first].double(), held(head, "k", 0, at), held(head, "v", 0, at),
                                 first, d ** -0.5, fmt, True, half)
        assert cc.close(out[1, :, :first].double(), want, tol) is None
    if many and power >= 66:
        assert bool(torch.isnan(out[1, :, n_q // 2:]).all())
    else:
        want, tol = cc.attention(q[1].double(), held(c, "k", 1, lens[1]), held(c, "v", 1, lens[1]), n_q,
                                 d ** -0.5, fmt, many, torch.finfo(torch.float32).eps / 2)
        assert cc.close(out[1].double(), want, tol, alike=False) is None


def test_cleared_rows_are_cleared_for_every_lane(kc):
    """Few query rows over bf16 pages: lanes that find a row that is not finite clear it in
    shared memory, others multiply it.  Every call gives earlier tokens the same finite bits."""
    for d, G, n_q in ((128, 4, 8), (128, 1, 16), (256, 2, 8)):
        lens = [n_q + 16 * u for u in range(40)]
        c = filled(kc, "bf16", lens, d, 16, seed=26)
        kv = torch.full((40, 1, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        at = torch.tensor([n - 2 for n in lens], dtype=torch.int32, device="cuda")
        keep = c.lens.clone()
        c.write(rows_bf16(260, 40, 1, d).cuda(), kv, starts=at)
        c.lens.copy_(keep)
        q = rows_bf16(261, 40, G, n_q, d).cuda()
        outs = [c.attend(q) for _ in range(50)]
        m = n_q - 2
        head = kc.PagedCache("bf16", c.k_pages, c.v_pages, None, None, c.page_table, c.lens - 2)
        check(head, q[:, :, :m], outs[0][:, :, :m], [n - 2 for n in lens], [m] * 40)
        for o in outs:
            assert torch.equal(o[:, :, :m], outs[0][:, :, :m])
            assert bool(torch.isnan(o[:, :, m:]).all())


@pytest.mark.parametrize("codes", ["all", "one", "and a NaN scale"])
@pytest.mark.parametrize("d,G,n_q,bad", [(128, 2, 3, 1), (128, 4, 16, 9), (256, 2, 8, 5), (128, 3, 70, 30), (256, 2, 70, 69),
                                         (128, 2, 300, 299), (256, 1, 300, 40)])
def test_nan_codes_of_later_tokens(kc, d, G, n_q, bad, codes):
    """fp8 pages of another writer may hold e4m3's NaN codes.  Tokens that do not see such a
    row are as they would be without it, those that do are NaN."""
    lens = [n_q + 41, n_q, n_q + 700]
    c = filled(kc, "fp8", lens, d, 32, seed=27)
    at = [n - n_q + bad for n in lens]
    for u, pos in enumerate(at):
        s = int(slots(c, u, pos, 1)[0])
        for side in "kv":
            row = getattr(c, side + "_pages").view(-1, d)[s]
            if codes == "one":
                row[d - 3 - u] = 0xFF if u & 1 else 0x7F
            else:
                row.fill_(0x7F)
            if codes == "and a NaN scale":
                getattr(c, side + "_params").view(-1)[s] = 0x7FC00000
    q = rows_bf16(270, 3, G, n_q, d).cuda()
    out = c.attend(q)
    head = kc.PagedCache("fp8", c.k_pages, c.v_pages, c.k_params, c.v_params, c.page_table,
                         torch.tensor(at, dtype=torch.int32, device="cuda"))
    many = uses_tensor_memory("fp8", d, G, n_q)
    for u in range(3):
        want, tol = cc.attention(q[u, :, :bad].double(), held(head, "k", u, at[u]), held(head, "v", u, at[u]),
                                 bad, d ** -0.5, "fp8", many, torch.finfo(torch.bfloat16).eps / 2)
        assert cc.close(out[u, :, :bad].double(), want, tol) is None
    assert bool(torch.isnan(out[:, :, bad:]).all())
    c.check_status()


@pytest.mark.parametrize("d,n_q", [(128, 1), (256, 1), (128, 40), (256, 40)])
@pytest.mark.parametrize("fmt", FMTS)
def test_large_values_and_growing_logits(kc, fmt, d, n_q):
    """Values up to 2^96 (quantised pages and many rows: 2^62) under logits that grow from one
    row to the next by 2^29 in all: the sums stay finite wherever the weights' reference is."""
    n, G, units = 2000, 2, 450
    one = make_cache(kc, fmt, [0], d, 64, n, seed=28)
    k, v = rows_bf16(280, 1, n, d), rows_bf16(281, 1, n, d)
    k[0, :, 0] = (torch.linspace(0, 29, n) / (8.0 * d ** -0.5 * 1.4427)).to(torch.bfloat16)
    many = uses_tensor_memory(fmt, d, G, n_q)
    v = (0.5 + 0.5 * v.float().abs().clamp(max=1)) * 2.0 ** (62 if many and fmt != "bf16" else 96)
    v = v.to(torch.bfloat16)
    one.write(k.cuda(), v.cuda())
    c = kc.PagedCache(fmt, one.k_pages, one.v_pages, one.k_params, one.v_params,
                      one.page_table.repeat(units, 1), one.lens.repeat(units))
    q = rows_bf16(282, 1, G, n_q, d)
    q[..., 0] = 8.0
    q = q.cuda().expand(units, -1, -1, -1)
    out = c.attend(q, out_dtype=torch.float32)
    check(c, q, out, [n] * units, [n_q] * units, alike=False, units=(0, 1, 224, 449))


@pytest.mark.parametrize("d,G,n_q", [(128, 4, 1), (128, 2, 8), (128, 4, 40), (128, 2, 200), (256, 2, 1), (256, 2, 40)])
def test_logits_of_minus_infinity(kc, d, G, n_q):
    """bf16 keys of -infinity: such rows weigh nothing, and a token that sees no others has no
    softmax (NaN), unlike one that sees no rows at all (zeros)."""
    lens = [600, n_q + 700, 5000, n_q - 1]
    c = make_cache(kc, "bf16", [0] * 4, d, 64, max(lens), seed=29)
    k, v = rows_bf16(290, 4, max(lens), d), rows_bf16(291, 4, max(lens), d)
    inf = float("inf")
    k[0, :, 0] = -inf
    k[2, :, 0] = -inf
    k[1, :300:2, 0] = -inf
    k[1, 400:600, 0] = -inf                      # whole tiles of them
    c.write(k.cuda(), v.cuda(), counts=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    q = rows_bf16(292, 4, G, n_q, d)
    q[..., 0] = 1.0
    q = q.cuda()
    out = c.attend(q, out_dtype=torch.float32)
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(out[2]).all())
    some = torch.isfinite(k[1, :lens[1], 0]).cuda()
    kr, vr = (cc.Rows(held(c, side, 1, lens[1]).a[some]) for side in "kv")
    many = uses_tensor_memory("bf16", d, G, n_q)
    want, tol = cc.attention(q[1].double(), kr, vr, n_q, d ** -0.5, "bf16", many, 2.0 ** -24)
    assert cc.close(out[1].double(), want, tol) is None
    assert torch.count_nonzero(out[3, :, 0]) == 0


@pytest.mark.parametrize("d,G,n_q", [(128, 4, 1), (128, 4, 40), (128, 2, 200), (256, 2, 1), (256, 2, 40)])
@pytest.mark.parametrize("fmt", FMTS)
def test_rows_of_bad_pages_attend_as_zeros(kc, kz, fmt, d, G, n_q):
    """Pages outside the pool at the start, amid and at the end of a unit, the chunk's own among
    them, beside a unit without."""
    lens, page = [n_q + 900, n_q + 411], 32
    c = filled(kc, fmt, lens, d, page, seed=30)
    q = rows_bf16(300, 2, G, n_q, d).cuda()
    rows = [held(c, side, 0, lens[0]) for side in "kv"]
    bad = [0, 1, 7, 12, 13, 14, 15, (lens[0] - 1) // page]
    c.page_table[0, bad] = torch.tensor([-1, c.n_pages, 2 ** 31 - 1, -7, -1, -1, -1, c.n_pages + 5],
                                        dtype=torch.int32, device="cuda")
    out = c.attend(q, out_dtype=torch.float32)
    for r in rows:
        for p in bad:
            r.a[p * page:(p + 1) * page] = 0
        r.b = r.b.clone()
        for p in bad:
            r.b[p * page:(p + 1) * page] = 0
        r.value, r.parts = r.a + r.b, r.a.abs() + r.b.abs()
    want, tol = cc.attention(q[0].double(), rows[0], rows[1], n_q, d ** -0.5, fmt,
                             uses_tensor_memory(fmt, d, G, n_q), 2.0 ** -24)
    assert cc.close(out[0].double(), want, tol) is None
    check(c, q, out, lens, [n_q, n_q], units=(1,))
    with pytest.raises(kz.KvzipError):
        c.check_status()
    c.check_status()


@pytest.mark.parametrize("fmt", FMTS)
def test_calls_with_nothing_to_do(kc, fmt):
    c = filled(kc, fmt, [30, 7], 128, 16, seed=31, capacity=64)
    empty = torch.empty(2, 0, 128, dtype=torch.bfloat16, device="cuda")
    c.write(empty, empty)
    c.write(empty[0], empty[0], offsets=torch.zeros(3, dtype=torch.int64, device="cuda"))
    assert c.lens.tolist() == [30, 7]
    c.write(empty, empty, starts=torch.tensor([12, 5], dtype=torch.int32, device="cuda"))
    assert c.lens.tolist() == [12, 5]                 # an empty write at a position ends there
    k, v = c.read(n_rows=0)
    assert k.shape == v.shape == (2, 0, 128)
    assert c.attend(torch.empty(2, 3, 0, 128, dtype=torch.bfloat16, device="cuda")).shape == (2, 3, 0, 128)
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = rows_bf16(310, 2, 3, 20, 128).cuda()
    out = torch.full_like(q, 5.0)
    c.attend(q, q_lens=zero, out=out)
    assert bool((out == 5).all())
    c.lens.zero_()
    assert torch.count_nonzero(c.attend(q)) == 0 and torch.count_nonzero(c.attend(q[:, :, :1])) == 0
    c.check_status()
    none = kc.PagedCache.allocate(fmt, 0, 128, 4, page_rows=16)
    rows = torch.empty(0, 5, 128, dtype=torch.bfloat16, device="cuda")
    none.write(rows, rows)
    assert none.attend(torch.empty(0, 3, 4, 128, dtype=torch.bfloat16, device="cuda")).shape == (0, 3, 4, 128)
    assert none.read(n_rows=5)[0].shape == (0, 5, 128)
    none.check_status()


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("fmt", ["fp8", "int4"])
def test_weights_range_moves_all_the_way(kc, fmt, d):
    """Few rows: values of 2^96 first, which logits 2^250 larger then leave nothing of, and values
    of 2^-115 with those."""
    n, G, units = 2000, 2, 450
    one = make_cache(kc, fmt, [0], d, 64, n, seed=32)
    k, v = rows_bf16(320, 1, n, d), rows_bf16(321, 1, n, d).float()
    k[0, :, 0] = 0.0
    k[0, n // 2:, 0] = 250 / (8.0 * d ** -0.5 * 1.4427)
    v[0, :n // 2] *= 2.0 ** 94
    v[0, n // 2:] *= 2.0 ** -115
    one.write(k.cuda(), v.to(torch.bfloat16).cuda())
    c = kc.PagedCache(fmt, one.k_pages, one.v_pages, one.k_params, one.v_params,
                      one.page_table.repeat(units, 1), one.lens.repeat(units))
    q = rows_bf16(322, 1, G, 1, d)
    q[..., 0] = 8.0
    q = q.cuda().expand(units, -1, -1, -1)
    out = c.attend(q, out_dtype=torch.float32)
    check(c, q, out, [n] * units, [1] * units, alike=False, units=(0, 1, 224, 449))


def test_inputs_dropped_before_their_stream_has_used_them(kc):
    """Rows, queries and the cache itself may be temporaries of a call on another stream: their
    memory is not handed out again before that stream is done."""
    k, v = rows_bf16(330, 4, 600, 128).cuda(), rows_bf16(331, 4, 600, 128).cuda()
    q = rows_bf16(332, 4, 4, 40, 128).cuda()
    ref = kc.PagedCache.allocate("fp8", 4, 128, 60, page_rows=64)
    ref.reserve(600)
    ref.write(k, v)
    want = ref.attend(q)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        c = kc.PagedCache.allocate("fp8", 4, 128, 60, page_rows=64)
        c.reserve(600)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)               # the calls wait behind this
        kt, vt, qt = k.clone(), v.clone(), q.clone()
        s.wait_stream(torch.cuda.current_stream())
        c.write(kt, vt, stream=s)
        out = c.attend(qt, stream=s)
        shapes = [(t.shape, t.dtype) for t in (kt, vt, qt, c.k_pages, c.v_pages, c.k_params, c.page_table, c.lens)]
        del kt, vt, qt, c
        junk = [torch.full(sh, 113, dtype=dt, device="cuda") for sh, dt in shapes for _ in range(3)]
        s.synchronize()
        assert torch.equal(out, want)
        del junk
