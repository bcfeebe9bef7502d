"""Cases, plain forms and 64-bit definitions of the paged-cache operators:

write   rows of new K / V go into a paged cache (bf16, or quantised to 8 or 4
        bits as they are written); quantised rows are read back in the same pass
read    rows of a quantised cache back to bf16
attend  attention of a chunk of new tokens (or of one token) over the cache

A unit is one KV head of one sequence; every unit has its own length and list
of pages.  Cache formats (one row = one position of one unit, d elements):

bf16    the row itself
fp8     e4m3 codes and a float32 scale 2^e, e the smallest integer >= -126
        with max |x| <= 448 * 2^e (0 for a row of zeros)
int4    codes c in 0..15 and a bf16 pair (s, z), value s * c + z, with z the
        row's minimum, s = bf16((max - min) / 15), c = round((x - z) / s)
"""
import math
import random

import numpy as np
import torch

own = False

FORMATS = ("bf16", "fp8", "int4")


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step's K / V appended for 8 sequences of 8 KV heads: a call where latency counts
        dict(name="write_step_bf16", op="write", fmt="bf16", seqs=8, heads=8, d=128, page=64,
             n=1000, new=1, packed=False),
        # a question's 1027 tokens appended to a d = 256 cache (the 170K model's head size)
        dict(name="write_chunk_fp8_d256", op="write", fmt="fp8", seqs=1, heads=8, d=256, page=32,
             n=5000, new=1027, packed=False),
        # the kept rows of one layer after eviction (about 0.3 of 128K, ragged heads), quantised into pages
        dict(name="write_fill_int4", op="write", fmt="int4", seqs=1, heads=8, d=128, page=64,
             n=0, new=62000, packed=True),
        # a short ragged batch read back
        dict(name="read_batch_fp8", op="read", fmt="fp8", seqs=3, heads=8, d=128, page=16, n=2049),
        # a whole 128K layer read back
        dict(name="read_all_int4", op="read", fmt="int4", seqs=1, heads=8, d=128, page=128, n=131072),
        # one token over one layer's evicted 128K cache, bf16, heads of very different lengths
        dict(name="token_bf16", op="attend", fmt="bf16", seqs=1, heads=8, G=4, d=128, page=64,
             n=62000, new=1),
        # one token for each of 16 sequences, 4-bit cache, five query heads a KV head
        dict(name="token_batch_int4", op="attend", fmt="int4", seqs=16, heads=8, G=5, d=128, page=32,
             n=16411, new=1),
        # one token over a short d = 256 fp8 cache: a small call
        dict(name="token_short_fp8_d256", op="attend", fmt="fp8", seqs=1, heads=8, G=2, d=256, page=16,
             n=1500, new=1),
        # a question of 33 tokens over an evicted 120K layer
        dict(name="question_bf16", op="attend", fmt="bf16", seqs=1, heads=8, G=5, d=128, page=64,
             n=40000, new=33),
        # four sequences' questions of different lengths over 4-bit caches
        dict(name="questions_int4", op="attend", fmt="int4", seqs=4, heads=8, G=4, d=128, page=128,
             n=20011, new=301),
        # a 2048-token chunk over a whole 128K layer: the largest
        dict(name="chunk_bf16", op="attend", fmt="bf16", seqs=1, heads=8, G=4, d=128, page=128,
             n=131072, new=2048),
        # a 1024-token chunk over an fp8 d = 256 layer
        dict(name="chunk_fp8_d256", op="attend", fmt="fp8", seqs=1, heads=8, G=2, d=256, page=64,
             n=60000, new=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges: any format, head size and page size."""
    op = rng.choice(("write", "write", "read", "attend", "attend", "attend"))
    c = dict(op=op, fmt=rng.choice(FORMATS), d=rng.choice((128, 128, 256)),
             page=rng.choice((16, 32, 64, 128)), heads=rng.choice((1, 2, 4, 8)), seqs=_log(rng, 1, 16))
    units = c["seqs"] * c["heads"]
    rows = 8 * 131072 * 128 // c["d"] // units       # rows a unit so that the cache stays in range
    if op == "write":
        c["packed"] = rng.random() < 0.4
        c["n"] = 0 if c["packed"] else _log(rng, 1, max(2, min(20000, rows // 4)))
        c["new"] = _log(rng, 1, max(2, min(62000, rows // 4)))
    elif op == "read":
        if c["fmt"] == "bf16":
            c["fmt"] = "int4"
        c["n"] = _log(rng, 100, max(101, min(131072, rows)))
    else:
        c["G"] = rng.choice((1, 2, 4, 5, 8))
        c["new"] = 1 if rng.random() < 0.4 else _log(rng, 2, 2048)
        most = 8 * 131072 * 2048 * 4 * 128 // (units * c["new"] * c["G"] * c["d"])
        c["n"] = max(c["new"], _log(rng, 100, max(101, min(131072, rows, most))))
    return c


def _units(case):
    return case["seqs"] * case["heads"]


def _ragged(case):
    """Per unit: rows already held (or written, for a packed fill), between a
    twentieth of n and n as eviction leaves them, and the new tokens of its
    sequence.  Decided by the case alone, so that work() counts the same rows."""
    key = "/".join(f"{k}={case[k]}" for k in sorted(case) if k != "name")
    rng = random.Random(key)
    n, new = case["n"], case.get("new", 0)
    held, fresh = [], []
    for _ in range(case["seqs"]):
        m = new if case["seqs"] == 1 or new <= 1 else rng.randint((new + 1) // 2, new)
        for _ in range(case["heads"]):
            top = new if case.get("packed") else n
            share = 0.05 + 0.95 * rng.random()
            rows = max(min(top, 1), int(top * share))
            if case["op"] == "attend":
                rows = max(rows, m)                # the chunk's own rows are in the cache
            held.append(0 if case.get("packed") else rows)
            fresh.append(rows if case.get("packed") else m)
    if case["op"] in ("read", "attend"):
        held[-1] = n                               # one whole unit
    if case["op"] == "attend":
        fresh[case["heads"] - 1] = min(new, held[case["heads"] - 1])
    return held, fresh


def _row_bytes(case):
    d = case["d"]
    return {"bf16": 2 * d, "fp8": d + 4, "int4": d // 2 + 4}[case["fmt"]]


def work(case):
    held, fresh = _ragged(case)
    rb, d = _row_bytes(case), case["d"]
    if case["op"] == "write":
        rows = sum(fresh)
        back = 0 if case["fmt"] == "bf16" else 2 * rows * 2 * d
        return {"bytes": 2 * rows * (2 * d + rb) + back, "flops": 2 * rows * 4 * d}
    if case["op"] == "read":
        rows = sum(held)
        return {"bytes": 2 * rows * (rb + 2 * d), "flops": 2 * rows * 2 * d}
    tokens = sum(fresh)
    pairs = sum(m * (h - m) + m * (m + 1) // 2 for h, m in zip(held, fresh))
    return {"bytes": 2 * sum(held) * rb + 2 * tokens * case["G"] * d * 2,
            "flops": 4 * d * case["G"] * pairs}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(g, n, d, keys):
    """Rows as a cache meets them: keys with a few channels of large magnitude."""
    x = torch.randn(n, d, generator=g, device="cuda")
    if keys:
        x[:, ::37] *= 6.0
        x += 0.5 * torch.randn(1, d, generator=g, device="cuda")
    return x.to(torch.bfloat16)


def _inputs(case, seed):
    held, fresh = _ragged(case)
    units, d, page, fmt = _units(case), case["d"], case["page"], case["fmt"]
    g = _gen(seed)
    total = [h + (m if case["op"] == "write" else 0) for h, m in zip(held, fresh)]
    need = [(t + page - 1) // page for t in total]
    max_pages = max(1, max(need))
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((units, max_pages), -1, dtype=torch.int32, device="cuda")
    at = 0
    for u, c in enumerate(need):
        table[u, :c] = order[at:at + c]
        at += c
    width = {"bf16": d, "fp8": d, "int4": d // 2}[fmt]
    dtype = torch.bfloat16 if fmt == "bf16" else torch.uint8
    st = dict(fmt=fmt, d=d, page=page, table=table, host_lens=list(held),
              lens=torch.tensor(held, dtype=torch.int32, device="cuda"))
    for side in ("k", "v"):
        pages = torch.zeros(n_pages, page, width, dtype=dtype, device="cuda")
        params = None if fmt == "bf16" else torch.zeros(n_pages, page, dtype=torch.int32, device="cuda")
        if case["op"] != "write":
            for u, h in enumerate(held):
                slot = _slots(table[u], page, 0, h)
                codes, par = _pack(_rows(g, h, d, side == "k"), fmt)
                pages.view(-1, width)[slot] = codes
                if params is not None:
                    params.view(-1)[slot] = par
        st[side + "_pages"], st[side + "_params"] = pages, params
    if case["op"] == "write":
        st["host_fresh"] = fresh
        off = np.concatenate(([0], np.cumsum(fresh))).astype(np.int64)
        st["offsets"] = torch.from_numpy(off).cuda()
        st["starts"] = st["lens"].clone()
        if case["packed"]:
            st["k"] = _rows(g, int(off[-1]), d, True)
            st["v"] = _rows(g, int(off[-1]), d, False)
            st["counts"] = None
        else:
            new = max(fresh)
            st["k"] = _rows(g, units * new, d, True).view(units, new, d)
            st["v"] = _rows(g, units * new, d, False).view(units, new, d)
            st["counts"] = torch.tensor(fresh, dtype=torch.int32, device="cuda")
    elif case["op"] == "read":
        off = np.concatenate(([0], np.cumsum(held))).astype(np.int64)
        st["offsets"] = torch.from_numpy(off).cuda()
        st["total"] = int(off[-1])
    else:
        new = max(fresh)
        st["host_fresh"] = fresh
        st["counts"] = torch.tensor(fresh, dtype=torch.int32, device="cuda")
        st["q"] = torch.randn(units, case["G"], new, d, generator=g, device="cuda").to(torch.bfloat16)
        # tokens past a sequence's own are left as they were
        st["out"] = torch.zeros(units, case["G"], new, d, dtype=torch.bfloat16, device="cuda")
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["op"] = case["op"]
    if own:
        from attention_score_reduction_b200 import cache as kc
        st["cache"] = kc.PagedCache(st["fmt"], st["k_pages"], st["v_pages"], st["k_params"],
                                    st["v_params"], st["table"], st["lens"])
    return st


# -------------------------------------------------------------- plain forms

def _slots(table_row, page, first, n):
    """Flat row numbers in the pool of positions first .. first + n - 1."""
    pos = torch.arange(first, first + n, device="cuda")
    return table_row[pos // page].long() * page + pos % page


def _pack(x, fmt):
    """Codes and per-row parameters (int32 bits) of bf16 rows."""
    if fmt == "bf16":
        return x, None
    x = x.float()
    if fmt == "fp8":
        m, e = torch.frexp(x.abs().amax(1))
        e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
        scale = torch.where(m == 0, torch.ones_like(m), torch.ldexp(torch.ones_like(m), e))
        return (x / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale.view(torch.int32)
    lo, hi = x.amin(1), x.amax(1)
    s = ((hi - lo) / 15).to(torch.bfloat16)
    z = lo.to(torch.bfloat16)
    # in 64 bits: quotients next to a border between two codes
    t = (x.double() - z.double()[:, None]) / s.double()[:, None]
    c = torch.where(s[:, None] == 0, torch.zeros_like(t), t).round().clamp(0, 15).to(torch.uint8)
    par = torch.stack((s, z), 1).view(torch.int32).view(-1)
    return c[:, 0::2] | (c[:, 1::2] << 4), par


def _unpack(codes, par, fmt):
    """float32 values of stored rows."""
    if fmt == "bf16":
        return codes.float()
    if fmt == "fp8":
        return codes.view(torch.float8_e4m3fn).float() * par.view(torch.float32)[:, None]
    c = torch.stack((codes & 15, codes >> 4), 2).view(codes.shape[0], -1).float()
    sz = par.view(-1, 1).view(torch.bfloat16).float()
    return c * sz[:, :1] + sz[:, 1:]


def _stored(st, side, slot):
    pages, params = st[side + "_pages"], st[side + "_params"]
    codes = pages.view(-1, pages.shape[2])[slot]
    return _unpack(codes, None if params is None else params.view(-1)[slot], st["fmt"])


def _plain_write(st):
    back = {"k": [], "v": []}
    for u, (first, n) in enumerate(zip(st["host_lens"], st["host_fresh"])):
        slot = _slots(st["table"][u], st["page"], first, n)
        for side in ("k", "v"):
            if st["counts"] is None:
                at = sum(st["host_fresh"][:u])
                rows = st[side][at:at + n]
            else:
                rows = st[side][u, :n]
            codes, par = _pack(rows, st["fmt"])
            pages = st[side + "_pages"]
            pages.view(-1, pages.shape[2])[slot] = codes
            if par is not None:
                st[side + "_params"].view(-1)[slot] = par
                back[side].append(_unpack(codes, par, st["fmt"]).to(torch.bfloat16))
    lens = st["starts"] + (st["offsets"][1:] - st["offsets"][:-1]).to(torch.int32)
    if st["fmt"] == "bf16":
        return st["k_pages"], st["v_pages"], lens
    return torch.cat(back["k"]), torch.cat(back["v"]), lens


def _plain_read(st):
    out = []
    for side in ("k", "v"):
        out.append(torch.cat([_stored(st, side, _slots(st["table"][u], st["page"], 0, h))
                              .to(torch.bfloat16) for u, h in enumerate(st["host_lens"])]))
    return tuple(out)


def _plain_attend(st):
    q, out = st["q"], torch.zeros_like(st["out"])
    _, G, _, d = q.shape
    for u, (h, m) in enumerate(zip(st["host_lens"], st["host_fresh"])):
        slot = _slots(st["table"][u], st["page"], 0, h)
        k, v = _stored(st, "k", slot), _stored(st, "v", slot)
        j = torch.arange(h, device="cuda")
        step = max(1, (1 << 28) // (G * h))
        for i0 in range(0, m, step):
            i1 = min(m, i0 + step)
            x = (q[u, :, i0:i1].reshape(-1, d).float() @ k.t()) * (1.0 / math.sqrt(d))
            x = x.view(G, i1 - i0, h)
            last = h - m + torch.arange(i0, i1, device="cuda")
            x.masked_fill_(j[None, :] > last[:, None], float("-inf"))
            x = torch.exp(x - x.amax(2, keepdim=True))
            o = (x.view(-1, h) @ v) / x.view(-1, h).sum(1, keepdim=True)
            out[u, :, i0:i1] = o.view(G, i1 - i0, d).to(torch.bfloat16)
    return out


def run(st):
    if own:
        c = st["cache"]
        if st["op"] == "write":
            if st["counts"] is None:
                c.write(st["k"], st["v"], starts=st["starts"], offsets=st["offsets"])
            else:
                c.write(st["k"], st["v"], starts=st["starts"], counts=st["counts"])
            if st["fmt"] == "bf16":
                return c.k_pages, c.v_pages, c.lens
            total = sum(st["host_fresh"])
            k, v = c.read(st["offsets"], total, starts=st["starts"])
            return k, v, c.lens
        if st["op"] == "read":
            return c.read(st["offsets"], st["total"])
        return c.attend(st["q"], q_lens=st["counts"], out=st["out"])
    return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}[st["op"]](st)


# ------------------------------------------------- the definitions in 64 bits

def _e4m3_values():
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[b] = np.nan if (b & 127) == 127 else (-x if b & 128 else x)
    return torch.from_numpy(v).cuda()


def _quantised64(x, fmt):
    """What a row stands for once it was stored, float64, from the formulas."""
    x = x.double()
    if fmt == "bf16":
        return x
    if fmt == "fp8":
        top = x.abs().amax(1, keepdim=True)
        e = torch.ceil(torch.log2(torch.where(top == 0, torch.full_like(top, 448.0), top) / 448.0))
        e = torch.where(torch.exp2(e - 1) * 448.0 >= top, e - 1, e)       # log2 next to a whole number
        e = torch.where(torch.exp2(e) * 448.0 < top, e + 1, e).clamp(min=-126)
        e = torch.where(top == 0, torch.zeros_like(e), e)
        y = x / torch.exp2(e)
        _, p = torch.frexp(y)
        ulp = torch.exp2((p - 4).clamp(min=-9).double())
        return torch.round(y / ulp) * ulp * torch.exp2(e)
    lo, hi = x.amin(1, keepdim=True), x.amax(1, keepdim=True)
    s = ((hi - lo) / 15).to(torch.bfloat16).double()
    c = torch.where(s == 0, torch.zeros_like(x), torch.round((x - lo) / s)).clamp(0, 15)
    return s * c + lo


def _held64(st, side, u, n):
    pages, page = st[side + "_pages"], st["page"]
    k = (n + page - 1) // page
    raw = torch.cat([pages[p] for p in st["table"][u, :k].tolist()])[:n]
    if st["fmt"] == "bf16":
        return raw.double()
    par = torch.cat([st[side + "_params"][p] for p in st["table"][u, :k].tolist()])[:n]
    if st["fmt"] == "fp8":
        return _e4m3_values()[raw.long()] * par.view(torch.float32).double()[:, None]
    s = (par << 16).view(torch.float32).double()[:, None]
    z = (par & -65536).view(torch.float32).double()[:, None]
    c = torch.empty(n, 2 * raw.shape[1], dtype=torch.float64, device="cuda")
    c[:, 0::2] = (raw % 16).double()
    c[:, 1::2] = (raw // 16).double()
    return s * c + z


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "read":
        return tuple(torch.cat([_held64(st, side, u, h) for u, h in enumerate(st["host_lens"])])
                     for side in ("k", "v"))
    if case["op"] == "write":
        lens = torch.tensor([a + b for a, b in zip(st["host_lens"], st["host_fresh"])],
                            dtype=torch.int32, device="cuda")
        res = []
        for side in ("k", "v"):
            rows = [st[side][int(st["offsets"][u]):int(st["offsets"][u + 1])] if case["packed"]
                    else st[side][u, :n] for u, n in enumerate(st["host_fresh"])]
            vals = [_quantised64(r, st["fmt"]) for r in rows]
            if st["fmt"] != "bf16":
                res.append(torch.cat(vals))
                continue
            pages = st[side + "_pages"].double()
            for u, first in enumerate(st["host_lens"]):
                for t in range(vals[u].shape[0]) if vals[u].shape[0] <= 4 else ():
                    p = first + t
                    pages[int(st["table"][u, p // st["page"]]), p % st["page"]] = vals[u][t]
                if vals[u].shape[0] > 4:
                    pos = np.arange(first, first + vals[u].shape[0])
                    row = st["table"][u].cpu().numpy()
                    pages[torch.from_numpy(row[pos // st["page"]].astype(np.int64)).cuda(),
                          torch.from_numpy(pos % st["page"]).cuda()] = vals[u]
            res.append(pages)
        return res[0], res[1], lens
    q = st["q"].double()
    units, G, new, d = q.shape
    if work(case)["flops"] > 2e13:
        return None
    out = torch.zeros(units, G, new, d, dtype=torch.float64, device="cuda")
    for u in range(units):
        h, m = st["host_lens"][u], st["host_fresh"][u]
        k, v = _held64(st, "k", u, h), _held64(st, "v", u, h)
        block = max(1, (1 << 27) // (G * h))
        for a in range(0, m, block):
            b = min(m, a + block)
            seen = h - m + b                      # rows the block's last token sees
            s = torch.einsum("gid,jd->gij", q[u, :, a:b], k[:seen]) / math.sqrt(d)
            for i in range(a, b) if b - a <= 4 else ():
                s[:, i - a, h - m + i + 1:] = -math.inf
            if b - a > 4:
                i = torch.arange(a, b, device="cuda").view(1, -1, 1)
                jj = torch.arange(seen, device="cuda").view(1, 1, -1)
                s = torch.where(jj <= h - m + i, s, torch.full_like(s, -math.inf))
            lse = torch.logsumexp(s, 2, keepdim=True)
            out[u, :, a:b] = torch.einsum("gij,jd->gid", torch.exp(s - lse), v[:seen])
    return out
