"""The paged KV cache and the attention over it against plain fp64 forms.

Quantisation, write and read are compared bit for bit; attention by the tolerances that
paged_util.tolerances derives.
"""
import math

import pytest
import torch

import paged_util as P

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _cache(tam, n_pages, page, Hkv, d, dtype, layout="token", fill=None):
    """A cache whose pages are plain, head-major, or every other page of a shared tensor."""
    def one(x, t):
        if layout == "token":
            return t(n_pages, page, Hkv, d)
        if layout == "head":
            return t(n_pages, Hkv, page, d).transpose(1, 2)
        return t(n_pages, 2, page, Hkv, d)[:, x]
    if layout == "shared":
        both = torch.empty(n_pages, 2, page, Hkv, d, dtype=dtype, device="cuda")
        k, v = both[:, 0], both[:, 1]
    else:
        k, v = (one(x, lambda *s: torch.empty(*s, dtype=dtype, device="cuda")) for x in range(2))
    if dtype != E4M3:
        for t in (k, v):
            t.fill_(float("nan") if fill is None else fill)
        return tam.PagedKVCache(k, v)
    for t in (k, v):
        t.view(torch.uint8).fill_(0x7f)
    s = [torch.full((n_pages, Hkv, page), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    return tam.PagedKVCache(k, v, *s)


def _table(gen, lens, page, n_pages, extra=1):
    """Random distinct pages for every sequence; -1 behind its end."""
    need = [-(-n // page) for n in lens]
    assert sum(need) <= n_pages
    perm = torch.randperm(n_pages, generator=gen, device="cuda").tolist()
    rows, at, width = [], 0, max(max(need), 1) + extra
    for n in need:
        rows.append(perm[at:at + n] + [-1] * (width - n))
        at += n
    return torch.tensor(rows, dtype=torch.int32)


def _cu(n):
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    return cu


def _stored(cache, table, s, L):
    """fp64 values of the first L positions of sequence s ([L, Hkv, d] each), from the bits."""
    out = []
    ps = cache.page_size
    j = torch.arange(L, device="cuda")
    page = table.cuda()[s].long()[j // ps]
    for t, sc in ((cache.k_pages, cache.k_scale), (cache.v_pages, cache.v_scale)):
        if cache.dtype == E4M3:
            y = t.view(torch.uint8)[page, j % ps].view(E4M3).double()
            y = y * torch.exp2(sc.view(torch.uint8)[page, :, j % ps].double() - 127)[..., None]
        else:
            y = t[page, j % ps].double()
        out.append(y)
    return out


def _filled(tam, gen, lens, page, Hkv, d, dtype, layout="token", io=BF16, k_mul=1.0):
    """A cache that holds random tokens of every sequence (written by the library), NaN
    everywhere else."""
    n_pages = sum(-(-n // page) for n in lens) + 2
    cache = _cache(tam, n_pages, page, Hkv, d, dtype, layout)
    table = _table(gen, lens, page, n_pages)
    T = sum(lens)
    k, v = (_rand(gen, T, Hkv, d) * k_mul).to(io), _rand(gen, T, Hkv, d).to(io)
    tam.kv_cache_write(cache, tam.PagedBatch(table, _cu(lens), lens), k, v)
    return cache, table, k, v


# ------------------------------------------------------------------ write and read

SPECIAL = [0.0, -0.0, 1.0, 448.0, 449.0, 896.0, 0.875, 0.8750001, 2.0 ** -9, 2.0 ** -10,
           1.5 * 2.0 ** -10, 1e-30, -3e38, 3.3895e38, 57344.0, 1e-40, 17.0, 18.0, 19.0, -25.0,
           2.0 ** -107, 5e-39]


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_quantised_write_matches_the_definition_bit_for_bit(tam_lib, io, d):
    gen = _gen(d)
    page, Hkv, T = 16, 3, 211
    k = _rand(gen, T, Hkv, d) * torch.exp2(torch.randint(-40, 40, (T, Hkv, 1), generator=gen,
                                                         device="cuda").float())
    v = _rand(gen, T, Hkv, d)
    sp = torch.tensor(SPECIAL, device="cuda")
    for i in range(len(SPECIAL)):
        k[i, 0] = 0.0
        k[i, 0, (7 * i) % d] = sp[i]                       # alone in its row: its own maximum
        v[i, 1, :len(SPECIAL)] = sp.clamp(-448, 448)       # next to others
    k[30, 1, d - 1] = math.inf
    k[31, 2, 0] = -math.inf
    v[32, 0, 5] = math.nan
    k, v = k.to(io), v.to(io)
    cache = _cache(tam_lib, 20, page, Hkv, d, E4M3)
    table = _table(gen, [T], page, 20)
    batch = tam_lib.PagedBatch(table, [0, T], [T])
    tam_lib.kv_cache_write(cache, batch, k, v)
    j = torch.arange(T, device="cuda")
    pg = table.cuda()[0].long()[j // page]
    for x, t, s in ((k, cache.k_pages, cache.k_scale), (v, cache.v_pages, cache.v_scale)):
        y, e = P.quantise(x)
        assert torch.equal(s[pg, :, j % page].int(), e.int() + 127)
        got = t.view(torch.uint8)[pg, j % page]
        want = y.float().to(E4M3).view(torch.uint8)        # exact: y is an e4m3 value
        bad = (e == 128)[..., None]
        assert torch.equal(got.masked_fill(bad, 0), want.masked_fill(bad, 0))
        assert not got.masked_select(bad).any()
    # and back: the kept value times its scale, exactly, in bf16 and fp32; NaN rows as NaN
    for dt in (BF16, F32):
        ko, vo = tam_lib.kv_cache_read(cache, batch, dtype=dt)
        for x, o in ((k, ko), (v, vo)):
            y, e = P.quantise(x)
            want = torch.where((e == 128)[..., None], math.nan, y * torch.exp2(e.double())[..., None])
            assert torch.equal(o.double().nan_to_num(nan=1e300), want.nan_to_num(nan=1e300))


@pytest.mark.parametrize("dtype,io,layout,page,Hkv,d", [
    (BF16, BF16, "token", 16, 8, 128), (BF16, BF16, "head", 64, 2, 64),
    (F32, F32, "shared", 32, 1, 256), (F32, F32, "token", 128, 3, 64),
    (E4M3, BF16, "head", 256, 4, 128), (E4M3, F32, "shared", 16, 5, 256),
    (E4M3, BF16, "token", 64, 8, 64)])
def test_write_and_read_touch_the_named_rows_only(tam_lib, dtype, io, layout, page, Hkv, d):
    """Ragged batches with an empty sequence, a sequence without new tokens, new tokens that
    start inside a page, rows behind the last sequence; the rest of the cache keeps its bits."""
    gen = _gen(page + d)
    lens, new = [1, page + 1, 0, 5 * page, 3 * page - 1, 777], [1, 2, 0, 0, page + 3, 777]
    n_pages = sum(-(-n // page) for n in lens) + 3
    cache = _cache(tam_lib, n_pages, page, Hkv, d, dtype, layout)
    table = _table(gen, lens, page, n_pages)
    cu = _cu(new)
    T = cu[-1] + 9                                          # nine rows of no sequence
    k, v = _rand(gen, T, Hkv, d).to(io), _rand(gen, T, Hkv, d).to(io)
    want_k, want_v = cache.k_pages.clone().view(torch.uint8), cache.v_pages.clone().view(torch.uint8)
    ws = [None if t is None else t.clone() for t in (cache.k_scale, cache.v_scale)]
    places = []
    for s, n in enumerate(new):
        for i in range(n):
            p = lens[s] - n + i
            places.append((int(table[s, p // page]), p % page, cu[s] + i))
    pg, row, t = (torch.tensor(x, device="cuda") for x in zip(*places))
    for x, w, sc in ((k, want_k, ws[0]), (v, want_v, ws[1])):
        if dtype == E4M3:
            y, e = P.quantise(x[t])
            w[pg, row] = y.float().to(E4M3).view(torch.uint8)
            sc[pg, :, row] = (e + 127).to(torch.uint8)
        else:
            w[pg, row] = x[t].view(torch.uint8)
    batch = tam_lib.PagedBatch(table, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                               torch.tensor(lens, dtype=torch.int32, device="cuda"))
    tam_lib.kv_cache_write(cache, batch, k, v)
    assert torch.equal(cache.k_pages.view(torch.uint8), want_k)
    assert torch.equal(cache.v_pages.view(torch.uint8), want_v)
    if dtype == E4M3:
        assert torch.equal(cache.k_scale, ws[0]) and torch.equal(cache.v_scale, ws[1])
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, -7.0)
    tam_lib.kv_cache_read(cache, batch, out=(ko, vo))
    for x, o, rest in ((k, ko, 7.0), (v, vo, -7.0)):
        y = x[:cu[-1]].double()
        if dtype == E4M3:
            z, e = P.quantise(x[:cu[-1]])
            y = z * torch.exp2(e.double())[..., None]
        assert torch.equal(o[:cu[-1]].double(), y)
        assert bool((o[cu[-1]:] == rest).all())


def test_rows_before_the_sequence_and_unmapped_positions(tam_lib):
    """Negative positions are skipped by the write and read as zeros; positions without a page
    are reported, skipped and read as zeros."""
    gen = _gen(5)
    page, Hkv, d = 16, 2, 64
    k, v = _rand(gen, 40, Hkv, d).to(BF16), _rand(gen, 40, Hkv, d).to(BF16)
    cache = _cache(tam_lib, 4, page, Hkv, d, BF16, fill=3.0)
    # five rows, three tokens in the cache: rows 0 and 1 stand before the first position
    b = tam_lib.PagedBatch(torch.tensor([[2]]), [0, 5], [3])
    tam_lib.kv_cache_write(cache, b, k[:5], v[:5])
    assert torch.equal(cache.k_pages[2, :3], k[2:5]) and bool((cache.k_pages[2, 3:] == 3).all())
    ko, vo = tam_lib.kv_cache_read(cache, b)
    assert not ko[:2].any() and torch.equal(ko[2:], k[2:5]) and torch.equal(vo[2:], v[2:5])
    for bad in (-1, 4, 2 ** 31 - 1, -2 ** 31):
        cache.k_pages.fill_(3.0)
        b = tam_lib.PagedBatch(torch.tensor([[1, bad, 0]]), [0, 40], [40])
        with pytest.raises(tam_lib.TamError) as err:
            tam_lib.kv_cache_write(cache, b, k, v)
        assert err.value.code == tam_lib.TAM_ERR_PAGE
        assert torch.equal(cache.k_pages[1], k[:16]) and torch.equal(cache.k_pages[0, :8], k[32:])
        assert bool((cache.k_pages[0, 8:] == 3).all() and (cache.k_pages[2:] == 3).all())
        ko = torch.ones_like(k)
        with pytest.raises(tam_lib.TamError):
            tam_lib.kv_cache_read(cache, b, out=(ko, torch.empty_like(v)))
        assert not ko[16:32].any() and torch.equal(ko[:16], k[:16]) and torch.equal(ko[32:], k[32:])
    # a length behind the table's last column
    b = tam_lib.PagedBatch(torch.tensor([[1, 3]]), [0, 40], [40])
    with pytest.raises(tam_lib.TamError) as err:
        tam_lib.kv_cache_write(cache, b, k, v)
    assert err.value.code == tam_lib.TAM_ERR_PAGE
    assert torch.equal(cache.k_pages[3], k[16:32])


def test_write_and_read_at_offsets_past_32_bits(tam_lib):
    page, Hkv, d, n_pages = 256, 8, 128, 8300                # 2.18e9 elements per tensor
    cache = tam_lib.PagedKVCache.empty(n_pages, page, Hkv, d, dtype=E4M3)
    gen = _gen(9)
    k, v = _rand(gen, 300, Hkv, d).to(BF16), _rand(gen, 300, Hkv, d).to(BF16)
    b = tam_lib.PagedBatch(torch.tensor([[n_pages - 1, n_pages - 2]]), [0, 300], [300])
    tam_lib.kv_cache_write(cache, b, k, v)
    ko, vo = tam_lib.kv_cache_read(cache, b)
    for x, o in ((k, ko), (v, vo)):
        y, e = P.quantise(x)
        assert torch.equal(o.double(), y * torch.exp2(e.double())[..., None])
    q = _rand(gen, 300, 16, d).to(BF16)
    out, lse = tam_lib.paged_gqa_attention(q, cache, b, return_lse=True)
    _check(out, lse, q, ko, vo, [300], [300])


# ------------------------------------------------------------------ attention

def _check_seq(out, lse, q, k, v, n):
    """out [n, Hq, d], lse [Hq, n] against fp64 over k, v [L, Hkv, d]."""
    ro, rl, ab, size = P.attention(q, k, v, n)
    to, tl = P.tolerances(ro, rl, ab, size, q.shape[2], k.shape[0], q.dtype == BF16)
    assert torch.isfinite(out).all()
    err = ((out.double() - ro).abs() / to).max() if n else torch.zeros(())
    assert float(err) <= 1.0, f"out: {float(err):.3g} of the tolerance"
    none = rl == -math.inf
    assert torch.equal(lse == -math.inf, none)
    if not bool(none.all()):
        e = ((lse.double() - rl).abs() / tl)[~none].max()
        assert float(e) <= 1.0, f"lse: {float(e):.3g} of the tolerance"


def _check(out, lse, q, k, v, new, lens):
    """Packed out and flat lse against the packed k, v [sum(lens), Hkv, d]."""
    Hq, at, t = q.shape[1], 0, 0
    for n, L in zip(new, lens):
        _check_seq(out[t:t + n], lse[Hq * t:Hq * (t + n)].view(Hq, n), q[t:t + n],
                   k[at:at + L], v[at:at + L], n)
        at, t = at + L, t + n


ATTENTION = [
    # io, cache, Hq, Hkv, d, page, new tokens, lengths
    (BF16, BF16, 8, 2, 128, 16, [1, 1, 1], [1, 17, 700]),
    (BF16, BF16, 32, 8, 128, 64, [1], [4097]),
    (BF16, E4M3, 16, 4, 128, 32, [1, 1, 1, 1], [5, 2048, 33, 1000]),
    (BF16, E4M3, 16, 4, 64, 32, [5, 4, 1], [300, 4, 900]),
    (BF16, BF16, 4, 1, 64, 128, [300, 0, 1], [300, 50, 513]),
    (BF16, BF16, 32, 8, 128, 16, [200, 3, 64, 1], [1000, 3, 65, 129]),
    (BF16, E4M3, 32, 8, 128, 64, [129, 31], [2000, 31]),
    (BF16, BF16, 16, 8, 256, 32, [70, 1], [1111, 64]),
    (BF16, E4M3, 16, 8, 256, 16, [65, 2], [500, 222]),
    (BF16, BF16, 8, 8, 128, 256, [130, 1], [400, 1]),
    (BF16, BF16, 12, 2, 128, 16, [100, 1], [300, 77]),             # six heads per group
    (BF16, E4M3, 24, 1, 64, 16, [9, 1], [90, 260]),
    (BF16, BF16, 128, 1, 64, 64, [3, 40], [70, 200]),
    (BF16, E4M3, 8, 2, 64, 128, [1024], [1024]),
    (F32, F32, 4, 1, 64, 16, [1, 40], [513, 60]),
    (F32, E4M3, 8, 2, 128, 32, [33, 1], [100, 1500]),
    (F32, F32, 16, 8, 256, 64, [7], [200]),
    (F32, F32, 6, 2, 128, 16, [3, 0, 20], [3, 9, 300]),
    (F32, F32, 8, 2, 128, 32, [1, 1, 1], [1, 700, 45]),             # blocks of four rows
    (F32, E4M3, 7, 1, 64, 16, [1, 1], [333, 90]),
    (F32, F32, 2, 1, 256, 64, [4, 3, 1], [200, 3, 77]),
]


@pytest.mark.parametrize("io,dtype,Hq,Hkv,d,page,new,lens", ATTENTION)
def test_attention(tam_lib, io, dtype, Hq, Hkv, d, page, new, lens):
    """Everything behind the sequences' ends is NaN in the pages."""
    gen = _gen(Hq + d + page + sum(lens))
    cache, table, k, v = _filled(tam_lib, gen, lens, page, Hkv, d, dtype, io=io, k_mul=1.5)
    b_all = tam_lib.PagedBatch(table, _cu(lens), lens)
    k, v = tam_lib.kv_cache_read(cache, b_all, dtype=io)
    q = (1.5 * _rand(gen, sum(new), Hq, d)).to(io)
    batch = tam_lib.PagedBatch(table, _cu(new), lens)
    out, lse = tam_lib.paged_gqa_attention(q, cache, batch, return_lse=True)
    _check(out, lse, q, k, v, new, lens)
    # the same bits again; without lse, without the bound on the rows, into a given tensor
    again = torch.full_like(q, 9.0)
    tam_lib.paged_gqa_attention(q, cache, batch, out=again)
    assert torch.equal(out, again)


@pytest.mark.parametrize("io,dtype,d,max_rows", [(BF16, BF16, 128, None), (BF16, E4M3, 128, 1),
                                                 (BF16, BF16, 256, 1), (BF16, E4M3, 64, 500),
                                                 (F32, F32, 64, None)])
def test_attention_rows_without_keys_and_padding(tam_lib, io, dtype, d, max_rows):
    """More rows than keys (rows before the first position see none), an empty sequence with
    rows, rows behind the last sequence, a wrong bound on the rows."""
    gen = _gen(d)
    lens, new = [3, 0, 200], [40, 2, 30]
    cache, table, _, _ = _filled(tam_lib, gen, lens, 16, 2, d, dtype, io=io)
    k, v = tam_lib.kv_cache_read(cache, tam_lib.PagedBatch(table, _cu(lens), lens), dtype=io)
    T = sum(new) + 5
    q = _rand(gen, T, 8, d).to(io)
    q[sum(new):] = math.nan
    cu = torch.tensor(_cu(new), dtype=torch.int32, device="cuda")
    batch = tam_lib.PagedBatch(table, cu, lens, max_rows=max_rows)
    out = torch.full_like(q, 5.0)
    _, lse = tam_lib.paged_gqa_attention(q, cache, batch, return_lse=True, out=out)
    assert bool((out[sum(new):] == 5.0).all())
    assert not out[:37].any() and not out[40:42].any()
    at = 0
    for s, (n, L) in enumerate(zip(new, lens)):
        t0 = _cu(new)[s]
        m = min(n, L)                                   # the rows that have a position
        blk = lse[8 * t0:8 * (t0 + n)].view(8, n)
        assert bool((blk[:, :n - m] == -math.inf).all())
        _check_seq(out[t0 + n - m:t0 + n], blk[:, n - m:], q[t0 + n - m:t0 + n], k[at:at + L],
                   v[at:at + L], m)
        at += L


@pytest.mark.parametrize("io,dtype,d,n,L", [(BF16, BF16, 128, 1, 300), (BF16, BF16, 128, 200, 333),
                                            (BF16, BF16, 64, 300, 300), (BF16, BF16, 256, 90, 140),
                                            (BF16, E4M3, 128, 150, 290), (BF16, E4M3, 64, 9, 40),
                                            (BF16, E4M3, 256, 60, 99), (F32, F32, 64, 40, 70)])
def test_attention_ignores_what_a_row_does_not_see(tam_lib, io, dtype, d, n, L):
    """NaN and infinities in later tokens' K and V reach only the rows at and behind them."""
    gen = _gen(n + L)
    cache, table, k, v = _filled(tam_lib, gen, [L], 32, 2, d, dtype, io=io)
    q = _rand(gen, n, 8, d).to(io)
    batch = tam_lib.PagedBatch(table, [0, n], [L])
    clean, lse0 = tam_lib.paged_gqa_attention(q, cache, batch, return_lse=True)
    lse0 = lse0.view(8, n).clone()
    for bad in sorted({L - 1, L - max(1, n // 2), L - max(1, n - 1)}):
        for x, val in (("v", math.nan), ("v", math.inf), ("k", math.nan)):
            t = (cache.k_pages if x == "k" else cache.v_pages)
            sc = (cache.k_scale if x == "k" else cache.v_scale)
            pg, row = int(table[0, bad // 32]), bad % 32
            if dtype == E4M3:
                keep = sc[pg, :, row].clone()
                sc[pg, :, row] = 255
            else:
                keep = t[pg, row].clone()
                t[pg, row] = val
            out, lse = tam_lib.paged_gqa_attention(q, cache, batch, return_lse=True)
            i = bad - (L - n)                            # the first row that sees it
            assert torch.equal(out[:max(i, 0)], clean[:max(i, 0)])
            assert torch.equal(lse.view(8, n)[:, :max(i, 0)], lse0[:, :max(i, 0)])
            late = out[max(i, 0):].float()
            if dtype != E4M3 and val == math.inf:
                assert bool((late == math.inf).all())
            else:
                assert bool(late.isnan().all())
            if dtype == E4M3:
                sc[pg, :, row] = keep
            else:
                t[pg, row] = keep
    assert torch.equal(tam_lib.paged_gqa_attention(q, cache, batch), clean)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("n,G,d", [(1, 5, 64), (3, 4, 64), (5, 4, 64), (10, 3, 64), (1, 8, 128),
                                   (2, 5, 128), (6, 4, 128), (5, 6, 128), (7, 1, 256), (8, 2, 256)])
def test_attention_of_few_rows_by_their_number(tam_lib, dtype, n, G, d):
    """Every number of row tiles, beside a sequence that fills fewer; one value of a later V row
    that is not finite reaches its own column only, in the rows that see it."""
    gen = _gen(100 * n + G + d)
    new, lens, Hkv = [n, 1], [611, 170], 2
    cache, table, _, _ = _filled(tam_lib, gen, lens, 16, Hkv, d, dtype)
    q = (1.5 * _rand(gen, n + 1, G * Hkv, d)).to(BF16)
    batch = tam_lib.PagedBatch(table, _cu(new), lens)
    clean, lse = tam_lib.paged_gqa_attention(q, cache, batch, return_lse=True)
    k, v = tam_lib.kv_cache_read(cache, tam_lib.PagedBatch(table, _cu(lens), lens), dtype=BF16)
    _check(clean, lse, q, k, v, new, lens)
    for back, dim in ((1, 1), (max(1, n - 1), d // 2 + 3), (n + 40, d - 2)):
        at = lens[0] - back                              # seen from row n - back on
        page, row = int(table[0, at // 16]), at % 16
        keep = cache.v_pages[page, row, 1, dim].clone()
        cache.v_pages.view(torch.uint8 if dtype == E4M3 else BF16)[page, row, 1, dim] = (
            0x7f if dtype == E4M3 else math.inf)
        out = tam_lib.paged_gqa_attention(q, cache, batch)
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[max(n - back, 0):n, G:, dim] = True
        assert not bool(out[hit].isfinite().any())
        assert torch.equal(out[~hit], clean[~hit])
        cache.v_pages[page, row, 1, dim] = keep


@pytest.mark.parametrize("io,dtype,n,d", [(BF16, BF16, 1, 128), (BF16, BF16, 100, 128),
                                          (BF16, E4M3, 70, 128), (BF16, E4M3, 1, 64),
                                          (BF16, BF16, 80, 256), (F32, F32, 9, 64)])
def test_attention_reports_bad_pages_and_leaves_them_out(tam_lib, io, dtype, n, d):
    gen = _gen(n)
    L, page = 400, 16
    cache, table, _, _ = _filled(tam_lib, gen, [L], page, 2, d, dtype, io=io)
    q = _rand(gen, n, 4, d).to(io)
    keep = torch.ones(L, dtype=torch.bool, device="cuda")
    good = table.clone()
    for col, bad in ((1, -1), (7, cache.n_pages), (8, 2 ** 31 - 1), (12, -2 ** 31)):
        table[0, col] = bad
        keep[col * page:(col + 1) * page] = False
    batch = tam_lib.PagedBatch(table, [0, n], [L])
    out = torch.zeros_like(q)
    with pytest.raises(tam_lib.TamError) as err:
        tam_lib.paged_gqa_attention(q, cache, batch, out=out)
    assert err.value.code == tam_lib.TAM_ERR_PAGE
    k, v = tam_lib.kv_cache_read(cache, tam_lib.PagedBatch(good, [0, L], [L]), dtype=io)
    _, lse = tam_lib.paged_gqa_attention(q, cache, batch, out=out, return_lse=True, check=False)
    # the pages that are there, in order: the new tokens stand behind all that were dropped
    _check_seq(out, lse.view(4, n), q, k[keep], v[keep], n)


@pytest.mark.parametrize("io,n,d", [(BF16, 1, 128), (BF16, 5, 64), (BF16, 1, 256), (BF16, 90, 128),
                                    (BF16, 70, 64), (BF16, 40, 256), (F32, 3, 64)])
def test_quantised_attention_over_rows_of_very_different_sizes(tam_lib, io, n, d):
    """V rows between 2^-25 and 2^25, in runs and mixed, K and Q rows between 2^-30 and 2^30
    (their products kept at ordinary scores)."""
    gen = _gen(n + d)
    L, page, Hkv, Hq = 700, 16, 2, 8
    e = torch.randint(-25, 26, (L, Hkv, 1), generator=gen, device="cuda").float()
    e[100:300] = 3.0
    e[300:400, 0] = -20.0
    e[400:500, 1] = 20.0
    v = (_rand(gen, L, Hkv, d) * torch.exp2(e)).to(io)
    for size in (-30.0, 0.0, 30.0):
        k = (_rand(gen, L, Hkv, d) * 2.0 ** size).to(io)
        q = (_rand(gen, n, Hq, d) * 2.0 ** -size).to(io)
        cache = _cache(tam_lib, 50, page, Hkv, d, E4M3)
        table = _table(gen, [L], page, 50)
        tam_lib.kv_cache_write(cache, tam_lib.PagedBatch(table, [0, L], [L]), k, v)
        kk, vv = tam_lib.kv_cache_read(cache, tam_lib.PagedBatch(table, [0, L], [L]), dtype=io)
        out, lse = tam_lib.paged_gqa_attention(q, cache, tam_lib.PagedBatch(table, [0, n], [L]),
                                               return_lse=True)
        _check(out, lse, q, kk, vv, [n], [L])


def test_attention_layouts_give_the_same_bits(tam_lib):
    for dtype in (BF16, E4M3):
        for new, lens in (([1, 1], [300, 70]), ([90, 7], [300, 70])):
            got = []
            for layout in ("token", "head", "shared"):
                gen = _gen(77)
                cache, table, _, _ = _filled(tam_lib, gen, lens, 64, 4, 128, dtype, layout)
                q = _rand(gen, sum(new), 16, 128).to(BF16)
                got.append(tam_lib.paged_gqa_attention(q, cache, tam_lib.PagedBatch(
                    table, _cu(new), lens)))
            assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_attention_over_many_sequences(tam_lib):
    """More sequences than CTAs, most of them short; and more than one scan step of the plan."""
    gen = _gen(3)
    n_seq = 1500
    lens = [1 + (s * 37) % 90 for s in range(n_seq)]
    new = [1 + s % 2 if lens[s] > 1 else 1 for s in range(n_seq)]
    cache, table, _, _ = _filled(tam_lib, gen, lens, 16, 1, 64, BF16)
    k, v = tam_lib.kv_cache_read(cache, tam_lib.PagedBatch(table, _cu(lens), lens))
    q = _rand(gen, sum(new), 4, 64).to(BF16)
    for max_rows in (2, None):
        out, lse = tam_lib.paged_gqa_attention(
            q, cache, tam_lib.PagedBatch(table, torch.tensor(_cu(new), dtype=torch.int32,
                                                             device="cuda"), lens,
                                         max_rows=max_rows), return_lse=True)
        for s in range(0, n_seq, 97):
            t, a, n, L = _cu(new)[s], _cu(lens)[s], new[s], lens[s]
            _check_seq(out[t:t + n], lse[4 * t:4 * (t + n)].view(4, n), q[t:t + n], k[a:a + L],
                       v[a:a + L], n)


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(tam_lib, seed):
    """Random head layouts, page sizes and layouts, lengths from one token on, and bounds on the
    rows, right and wrong: write, read back, attention."""
    import random
    rng = random.Random(seed)
    gen = _gen(1000 + seed)
    Hkv, G = rng.choice([1, 2, 3, 8]), rng.choice([1, 2, 3, 4, 7, 8, 16])
    d, page = rng.choice([64, 128, 256]), rng.choice([16, 32, 64, 128, 256])
    io, dtype = rng.choice([(BF16, BF16), (BF16, E4M3), (BF16, BF16), (BF16, E4M3), (F32, F32),
                            (F32, E4M3)])
    n_seq = rng.choice([1, 2, 5, 17])
    top = rng.choice([1, 3, 40, 300])
    lens, new = [], []
    for _ in range(n_seq):
        n = rng.randint(0, top)
        new.append(n)
        lens.append(n + rng.choice([0, 0, 1, rng.randint(0, 900)]))
    if sum(new) == 0:
        new[0], lens[0] = 1, lens[0] + 1
    cache, table, _, _ = _filled(tam_lib, gen, lens, page, Hkv, d, dtype,
                                 rng.choice(["token", "head", "shared"]), io=io)
    k, v = tam_lib.kv_cache_read(cache, tam_lib.PagedBatch(table, _cu(lens), lens), dtype=io)
    q = (1.3 * _rand(gen, sum(new), Hkv * G, d)).to(io)
    cu = torch.tensor(_cu(new), dtype=torch.int32, device="cuda")
    for max_rows in (None, max(max(new), 1), rng.choice([1, 2, 500])):
        batch = tam_lib.PagedBatch(table, cu, lens, max_rows=max_rows)
        out, lse = tam_lib.paged_gqa_attention(q, cache, batch, return_lse=True)
        _check(out, lse, q, k, v, new, lens)


# ------------------------------------------------------------------ as they are used together

@pytest.mark.parametrize("dtype,d,Hq,Hkv", [(BF16, 128, 8, 2), (E4M3, 128, 32, 8), (BF16, 64, 4, 1),
                                            (E4M3, 256, 4, 2)])
def test_chunked_prefill_and_decoding_follow_the_dense_prefill(tam_lib, dtype, d, Hq, Hkv):
    """Two prompts go into the cache chunk by chunk and token by token; every step's attention
    is the dense prefill's of the whole sequences on the rows the cache holds."""
    gen = _gen(d + Hq)
    lens = [333, 150]
    cu = _cu(lens)
    k, v = _rand(gen, cu[-1], Hkv, d).to(BF16), _rand(gen, cu[-1], Hkv, d).to(BF16)
    q = _rand(gen, cu[-1], Hq, d).to(BF16)
    cache = _cache(tam_lib, 40, 16, Hkv, d, dtype)
    table = _table(gen, lens, 16, 40)
    outs, done = [[], []], [0, 0]
    for new in ([100, 0], [64, 150], [1, 0], [163, 0], [1, 0], [4, 0]):
        t = [torch.arange(cu[s] + done[s], cu[s] + done[s] + new[s], device="cuda") for s in (0, 1)]
        done = [done[s] + new[s] for s in (0, 1)]
        rows = torch.cat(t)
        batch = tam_lib.PagedBatch(table, _cu(new), done)
        tam_lib.kv_cache_write(cache, batch, k[rows], v[rows], check=False)
        o = tam_lib.paged_gqa_attention(q[rows], cache, batch)
        for s in (0, 1):
            outs[s].append(o[:new[0]] if s == 0 else o[new[0]:])
    assert done == lens
    kk, vv = tam_lib.kv_cache_read(cache, tam_lib.PagedBatch(table, cu, lens))
    if dtype == BF16:
        assert torch.equal(kk, k) and torch.equal(vv, v)
    dense, lse = tam_lib.dense_gqa_prefill_varlen(q, kk, vv, cu, return_lse=True)
    got = torch.cat([torch.cat(o) for o in outs])
    for s in (0, 1):
        a, b = cu[s], cu[s + 1]
        ro, rl, ab, size = P.attention(q[a:b], kk[a:b], vv[a:b], b - a)
        tol, _ = P.tolerances(ro, rl, ab, size, d, b - a, True)
        assert bool(((got[a:b].double() - ro).abs() <= tol).all())
        assert bool(((got[a:b].double() - dense[a:b].double()).abs() <= 2 * tol).all())


def test_decoding_step_captured_and_replayed(tam_lib):
    """A captured step follows the lengths, the tables and the rows that its tensors hold when
    it is replayed; two graphs with their own workspaces replay at the same time."""
    gen = _gen(12)
    page, Hq, Hkv, d, lens = 16, 8, 2, 128, [40, 301]
    pages = 60
    steps = 5
    graphs, states = [], []
    for dtype in (BF16, E4M3):
        cache, table, _, _ = _filled(tam_lib, gen, lens, page, Hkv, d, dtype)
        big = _cache(tam_lib, pages, page, Hkv, d, dtype)
        big.k_pages[:cache.n_pages].copy_(cache.k_pages)
        big.v_pages[:cache.n_pages].copy_(cache.v_pages)
        if dtype == E4M3:
            big.k_scale[:cache.n_pages].copy_(cache.k_scale)
            big.v_scale[:cache.n_pages].copy_(cache.v_scale)
        tab = torch.full((2, 24), -1, dtype=torch.int32, device="cuda")
        tab[:, :table.shape[1]] = table.cuda()
        kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
        batch = tam_lib.PagedBatch(tab, cu, kv_len, max_rows=1)
        ws = tam_lib.Workspace()
        ws.get(tam_lib.paged_attention_workspace(2, Hq, BF16, big, batch))
        q, k, v = (torch.zeros(2, h, d, dtype=BF16, device="cuda") for h in (Hq, Hkv, Hkv))
        out = torch.zeros_like(q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kv_len.add_(1)
            tam_lib.kv_cache_write(big, batch, k, v, workspace=ws, check=False)
            tam_lib.paged_gqa_attention(q, big, batch, out=out, workspace=ws, check=False)
        graphs.append(g)
        states.append((dtype, big, tab, kv_len, cu, batch, ws, q, k, v, out, cache.n_pages))
    streams = [torch.cuda.Stream() for _ in graphs]
    for step in range(steps):
        want = []
        for dtype, big, tab, kv_len, cu, batch, ws, q, k, v, out, used in states:
            now = [n + step + 1 for n in lens]
            for s in (0, 1):                       # a page for a position that starts one
                col = (now[s] - 1) // page
                if tab[s, col] < 0:
                    tab[s, col] = used + 2 * step + s
            for t in (q, k, v):
                t.copy_(_rand(gen, *t.shape))
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for dtype, big, tab, kv_len, cu, batch, ws, q, k, v, out, used in states:
            tam_lib.check_status(ws.buf)
            now = [n + step + 1 for n in lens]
            assert kv_len.tolist() == now
            for s in (0, 1):
                kk, vv = _stored(big, tab, s, now[s])
                if dtype == BF16:
                    assert torch.equal(kk[-1], k[s].double())
                ro, rl, ab, size = P.attention(q[s:s + 1], kk, vv, 1)
                tol, _ = P.tolerances(ro, rl, ab, size, d, now[s], True)
                assert bool(((out[s:s + 1].double() - ro).abs() <= tol).all())


def test_calls_on_a_given_stream_and_workspace(tam_lib):
    gen = _gen(8)
    cache, table, _, _ = _filled(tam_lib, gen, [500, 90], 32, 2, 128, BF16)
    q = _rand(gen, 60, 8, 128).to(BF16)
    batch = tam_lib.PagedBatch(table, [0, 40, 60], [500, 90])
    want = tam_lib.paged_gqa_attention(q, cache, batch)
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        st = torch.cuda.Stream()
        outs.append((st, tam_lib.paged_gqa_attention(q, cache, batch, stream=st, check=False)))
    ws = tam_lib.Workspace()
    with torch.cuda.stream(torch.cuda.Stream()):
        outs.append((None, tam_lib.paged_gqa_attention(q, cache, batch, workspace=ws)))
    torch.cuda.synchronize()
    for _, o in outs:
        assert torch.equal(o, want)


def test_calls_of_two_threads_on_one_stream(tam_lib):
    import threading
    gen = _gen(21)
    cases = []
    for dtype, n, L in ((BF16, 1, 900), (E4M3, 70, 300)):
        cache, table, _, _ = _filled(tam_lib, gen, [L, 40], 16, 2, 128, dtype)
        q = _rand(gen, n + 1, 8, 128).to(BF16)
        batch = tam_lib.PagedBatch(table, [0, n, n + 1], [L, 40])
        cases.append((q, cache, batch, tam_lib.paged_gqa_attention(q, cache, batch)))
    wrong = []

    def work(q, cache, batch, want):
        for i in range(200):
            got = tam_lib.paged_gqa_attention(q, cache, batch, check=i % 8 == 0)
            if not torch.equal(got, want):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_refusals_on_the_device(tam_lib):
    T = tam_lib
    cache = T.PagedKVCache.empty(4, 16, 2, 64)
    batch = T.PagedBatch(torch.tensor([[0, 1]]), [0, 3], [20])
    rows = torch.zeros(3, 2, 64, dtype=BF16, device="cuda")
    q = torch.zeros(3, 4, 64, dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        T.kv_cache_write(cache, batch, rows[:, :1], rows[:, :1])
    with pytest.raises(ValueError):
        T.kv_cache_write(cache, batch, rows, rows.float())
    with pytest.raises(ValueError):
        T.kv_cache_write(cache, batch, rows.cpu(), rows.cpu())
    with pytest.raises(T.TamError) as e:                         # fp32 rows, bf16 cache
        T.kv_cache_write(cache, batch, rows.float(), rows.float())
    assert e.value.code == T.TAM_ERR_UNSUPPORTED
    with pytest.raises(TypeError):
        T.kv_cache_write(cache, batch, rows.half(), rows.half())
    with pytest.raises(T.TamError):
        T.kv_cache_read(cache, batch, dtype=F32)
    with pytest.raises(TypeError):
        T.kv_cache_read(cache, batch, dtype=E4M3)
    with pytest.raises(ValueError):
        T.paged_gqa_attention(q[..., :32], cache, batch)
    with pytest.raises(T.TamError) as e:
        T.paged_gqa_attention(q[:, :3].contiguous(), cache, batch)
    assert e.value.code == T.TAM_ERR_INVALID_ARG
    with pytest.raises(T.TamError) as e:
        T.paged_gqa_attention(q.float(), cache, batch)
    assert e.value.code == T.TAM_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        T.paged_gqa_attention(q, cache, batch, out=q.float())
    with pytest.raises(ValueError):
        T.PagedKVCache(cache.k_pages, cache.v_pages[:, :, :1])
    with pytest.raises(ValueError):
        T.PagedKVCache(cache.k_pages.transpose(2, 3), cache.v_pages.transpose(2, 3))
    with pytest.raises(ValueError):
        T.PagedKVCache(cache.k_pages.to(E4M3), cache.v_pages.to(E4M3))
    with pytest.raises(TypeError):
        T.PagedKVCache(cache.k_pages.half(), cache.v_pages.half())
    with pytest.raises(ValueError):
        T.PagedBatch(torch.tensor([[0, 1]]), [0, 3, 4], [20])
    with pytest.raises(ValueError):
        T.PagedBatch(torch.tensor([[0, 1]]), [0, 3], [20], max_rows=0)
    with pytest.raises(ValueError):
        T.PagedBatch(torch.tensor([[0, 1]]), [1, 3], [20])
    for x in (dict(page_table=torch.tensor([[0, 2 ** 32]])), dict(kv_len=[2 ** 31])):
        with pytest.raises(ValueError):
            T.PagedBatch(**{**dict(page_table=torch.tensor([[0, 1]]), cu_rows=[0, 3], kv_len=[20]), **x})
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        T.kv_cache_read(cache, T.PagedBatch(torch.tensor([[0, 1]]), cu, [20]))
    # a capture without a workspace of its own, with one that is too small, or with a check
    ws = T.Workspace()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for kw in (dict(check=False), dict(check=False, workspace=ws), dict(workspace=ws)):
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            g.capture_begin()
            with pytest.raises(ValueError):
                T.kv_cache_write(cache, batch, rows, rows, **kw)
            g.capture_end()
    # cu_rows that go back: nothing out of range happens
    bad = T.PagedBatch(torch.tensor([[0, 1], [2, 3]]),
                       torch.tensor([0, 3, 1], dtype=torch.int32, device="cuda"), [20, 20])
    T.kv_cache_write(cache, bad, rows, rows, check=False)
    T.paged_gqa_attention(q, cache, bad, check=False)
    # no rows at all
    empty = T.PagedBatch(torch.tensor([[0, 1]]), [0, 0], [20])
    T.kv_cache_write(cache, empty, rows[:0], rows[:0])
    assert T.paged_gqa_attention(q[:0], cache, empty).shape == (0, 4, 64)
    assert T.kv_cache_read(cache, empty)[0].shape == (0, 2, 64)
    # uninitialised memory never shows: the first 20 tokens were not written
    cache.k_pages.zero_()
    cache.v_pages.zero_()
    assert not T.paged_gqa_attention(q, cache, batch).any()
