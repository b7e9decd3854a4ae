"""The attention over a paged cache at the ends of its range: zero rows, lengths past the page
table, and e4m3 scales that lie far apart, against plain fp64 forms."""
import math

import pytest
import torch

import paged_util as P
from test_gpu_paged import _cache, _check, _check_seq, _cu, _filled, _gen, _rand, _table

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn

# new tokens of one sequence, query heads, KV heads, head size: every kernel and its forms.
# Few rows of one and of several tiles; chunks of at most 128 rows, of more, and of d = 256
FEW = [(1, 8, 2, 128), (5, 8, 2, 64), (3, 4, 1, 256)]
CHUNKS = [(20, 8, 2, 128), (25, 8, 2, 64), (150, 8, 2, 128), (70, 8, 2, 64), (40, 4, 1, 256)]


def _quantised(tam, gen, k, v, page=16):
    """An e4m3 cache that holds the rows k, v [L, Hkv, d] as one sequence: (cache, table, and the
    kept values as fp32 rows)."""
    L, Hkv, d = k.shape
    n_pages = -(-L // page) + 2
    cache = _cache(tam, n_pages, page, Hkv, d, E4M3)
    table = _table(gen, [L], page, n_pages)
    batch = tam.PagedBatch(table, [0, L], [L])
    tam.kv_cache_write(cache, batch, k, v)
    kk, vv = tam.kv_cache_read(cache, batch, dtype=F32)
    return cache, table, kk, vv


def _attend(tam, q, cache, table, L):
    n, Hq = q.shape[:2]
    out, lse = tam.paged_gqa_attention(q, cache, tam.PagedBatch(table, [0, n], [L]), return_lse=True)
    return out, lse.view(Hq, n)


# ------------------------------------------------------------------ zero and tiny rows

@pytest.mark.parametrize("n,Hq,Hkv,d", FEW + CHUNKS)
@pytest.mark.parametrize("what", ["q", "k", "both", "some", "tiny"])
def test_zero_and_tiny_rows_of_q_and_k(tam_lib, n, Hq, Hkv, d, what):
    """A score of zero is a score: the rows are means of V, masked keys stay masked."""
    gen = _gen(n + d + len(what))
    L = n + 333
    k, v = _rand(gen, L, Hkv, d), _rand(gen, L, Hkv, d)
    q = _rand(gen, n, Hq, d)
    if what in ("k", "both"):
        k.zero_()
    if what in ("q", "both"):
        q.zero_()
    if what == "some":
        q[::3] = 0.0
        q[1::3] *= 1e-37
        k[L - n // 2 - 1:] = 0.0
        k[128:256] *= 1e-6
    if what == "tiny":
        q *= 1e-36
        k *= 1e-29
    cache, table, kk, vv = _quantised(tam_lib, gen, k.to(BF16), v.to(BF16))
    q = q.to(BF16)
    out, lse = _attend(tam_lib, q, cache, table, L)
    _check_seq(out, lse, q, kk, vv, n)


@pytest.mark.parametrize("n,Hq,Hkv,d", CHUNKS)
def test_tiny_queries_over_missing_tiles(tam_lib, n, Hq, Hkv, d):
    """Key tiles without a single page are left out, whatever the size of the query."""
    gen = _gen(n)
    L, page = n + 500, 16
    k, v = _rand(gen, L, Hkv, d).to(BF16), _rand(gen, L, Hkv, d).to(BF16)
    cache, table, kk, vv = _quantised(tam_lib, gen, k, v, page)
    keep = torch.ones(L, dtype=torch.bool, device="cuda")
    table[0, 8:16] = -1                                     # the keys 128 to 255
    keep[128:256] = False
    for size in (1.0, 2.0 ** -10, 2.0 ** -60, 0.0):
        q = (_rand(gen, n, Hq, d) * size).to(BF16)
        out, lse = tam_lib.paged_gqa_attention(q, cache, tam_lib.PagedBatch(table, [0, n], [L]),
                                               return_lse=True, check=False)
        _check_seq(out, lse.view(Hq, n), q, kk[keep], vv[keep], n)


# ------------------------------------------------------------------ lengths past the page table

@pytest.mark.parametrize("io,dtype", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
@pytest.mark.parametrize("n,Hq,Hkv,d", FEW + CHUNKS)
@pytest.mark.parametrize("page,cols", [(16, 5), (32, 7), (64, 3)])
def test_positions_past_the_table_are_left_out(tam_lib, io, dtype, n, Hq, Hkv, d, page, cols):
    """kv_len beyond the table's columns: reported, and every row sees the keys that the table
    has room for, up to its own position."""
    gen = _gen(n + d + page)
    cap = page * cols
    cache, table, _, _ = _filled(tam_lib, gen, [cap], page, Hkv, d, dtype, io=io)
    table = table[:, :cols].contiguous()
    k, v = tam_lib.kv_cache_read(cache, tam_lib.PagedBatch(table, [0, cap], [cap]), dtype=io)
    q = _rand(gen, n, Hq, d).to(io)
    for over in sorted({1, max(n // 2, 1), n, n + 300}):
        batch = tam_lib.PagedBatch(table, [0, n], [cap + over])
        with pytest.raises(tam_lib.TamError) as err:
            tam_lib.paged_gqa_attention(q, cache, batch)
        assert err.value.code == tam_lib.TAM_ERR_PAGE
        out, lse = tam_lib.paged_gqa_attention(q, cache, batch, return_lse=True, check=False)
        lse = lse.view(Hq, n)
        m = max(n - over, 0)                 # rows with a position in the table: the first m
        if m > cap:                          # and the first of these stand before position 0
            assert not out[:m - cap].any()
        a = max(m - cap, 0)
        if m > a:
            _check_seq(out[a:m], lse[:, a:m], q[a:m], k, v, m - a)
        for i in {m, (m + n - 1) // 2, n - 1}:
            if i >= m:
                _check_seq(out[i:i + 1], lse[:, i:i + 1], q[i:i + 1], k, v, 1)


# ------------------------------------------------------------------ scales that lie far apart

@pytest.mark.parametrize("n,Hq,Hkv,d", FEW + CHUNKS)
@pytest.mark.parametrize("x", ["k", "v"])
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 26, 2.0 ** 40, 2.0 ** 100])
def test_larger_later_tokens_have_no_effect_on_earlier_rows(tam_lib, n, Hq, Hkv, d, x, size):
    gen = _gen(n + d)
    L = n + 150
    k, v = _rand(gen, L, Hkv, d), _rand(gen, L, Hkv, d)
    q = _rand(gen, n, Hq, d).to(BF16)
    (k if x == "k" else v)[L - max(n // 2, 1)] *= size       # seen from row n - n // 2 on
    cache, table, kk, vv = _quantised(tam_lib, gen, k.to(BF16), v.to(BF16))
    out, lse = _attend(tam_lib, q, cache, table, L)
    m = n - max(n // 2, 1)
    if m:
        _check_seq(out[:m], lse[:, :m], q[:m], kk[:L - n + m], vv[:L - n + m], m)
    if x == "v":
        _check_seq(out, lse, q, kk, vv, n)


@pytest.mark.parametrize("n,Hq,Hkv,d", FEW + CHUNKS)
@pytest.mark.parametrize("size", [2.0 ** 26, 2.0 ** 60])
def test_keys_of_very_different_sizes(tam_lib, n, Hq, Hkv, d, size):
    """Large K rows in dimensions where Q is zero: the scores are those of the small ones."""
    gen = _gen(n + d)
    L = n + 700
    k, v = _rand(gen, L, Hkv, d), _rand(gen, L, Hkv, d)
    q = 2.0 * _rand(gen, n, Hq, d)
    q[..., d // 2:] = 0.0
    big = torch.arange(L, device="cuda") % 7 == 3
    k[big] *= size
    k[big, :, :d // 2] = 0.0
    cache, table, kk, vv = _quantised(tam_lib, gen, k.to(BF16), v.to(BF16))
    q = q.to(BF16)
    out, lse = _attend(tam_lib, q, cache, table, L)
    _check_seq(out, lse, q, kk, vv, n)


def _spans(gen, L, Hkv, d):
    """Sizes of V rows that change along the sequence."""
    one = torch.ones(L, 1, 1, device="cuda")
    runs = one.clone()
    runs[:L // 3] = 2.0 ** 60
    runs[L // 3:2 * L // 3] = 2.0 ** -60
    ends = one.clone()
    ends[: L // 2] = 2.0 ** 105
    ends[L // 2:] = 2.0 ** -95
    back = ends.flip(0)
    first = one.clone()
    first[0] = 2.0 ** 109
    mixed = torch.exp2(torch.randint(-95, 106, (L, Hkv, 1), generator=gen, device="cuda").float())
    zeros = one.clone()
    zeros[L // 4:L // 2] = 0.0
    zeros[::5] = 0.0
    zeros[-9:] = 0.0
    tail = 5000.0 * one
    tail[-200:] = 0.0
    return dict(runs=runs, ends=ends, back=back, first=first, mixed=mixed, zeros=zeros, tail=tail)


SPANS = ["runs", "ends", "back", "first", "mixed", "zeros", "tail"]


def _values_of_very_different_sizes(tam, n, Hq, Hkv, d, name, equal, L, n_seq=1):
    """V of one sign, so that its sums grow; with equal weights, or such that the rows see some
    keys much more than others.  Many sequences over the same pages: every one is whole in a
    CTA; one sequence is spread over all of them."""
    gen = _gen(n + d + len(name))
    v = (1.0 + _rand(gen, L, Hkv, d).abs()) * _spans(gen, L, Hkv, d)[name]
    k = _rand(gen, L, Hkv, d)
    q = ((0.0 if equal else 3.0) * _rand(gen, n, Hq, d)).to(BF16)
    cache, table, kk, vv = _quantised(tam, gen, k.to(BF16), v.to(BF16))
    batch = tam.PagedBatch(table.expand(n_seq, -1).contiguous(), [n * s for s in range(n_seq + 1)],
                           [L] * n_seq)
    out, lse = tam.paged_gqa_attention(q.repeat(n_seq, 1, 1), cache, batch, return_lse=True)
    out, lse = out.view(n_seq, n, Hq, d), lse.view(n_seq, Hq, n)
    for s in sorted({0, n_seq // 2, n_seq - 1}):
        _check_seq(out[s], lse[s], q, kk, vv, n)


@pytest.mark.parametrize("n,Hq,Hkv,d", CHUNKS)
@pytest.mark.parametrize("name", SPANS)
@pytest.mark.parametrize("equal", [False, True])
def test_values_of_very_different_sizes_in_chunks(tam_lib, n, Hq, Hkv, d, name, equal):
    _values_of_very_different_sizes(tam_lib, n, Hq, Hkv, d, name, equal, n + 2100)


@pytest.mark.parametrize("n,Hq,Hkv,d", CHUNKS)
@pytest.mark.parametrize("name", SPANS)
def test_sums_of_values_of_very_different_sizes_in_chunks(tam_lib, n, Hq, Hkv, d, name):
    _values_of_very_different_sizes(tam_lib, n, Hq, Hkv, d, name, True, n + 4096,
                                    8 * 148 // Hkv + 1)


@pytest.mark.parametrize("n,Hq,Hkv,d", FEW + [(8, 8, 2, 128)])
@pytest.mark.parametrize("name", SPANS)
@pytest.mark.parametrize("equal", [False, True])
def test_values_of_very_different_sizes_in_few_rows(tam_lib, n, Hq, Hkv, d, name, equal):
    _values_of_very_different_sizes(tam_lib, n, Hq, Hkv, d, name, equal, n + 16384)


@pytest.mark.parametrize("n,Hq,Hkv,d", FEW + [(8, 8, 2, 128)])
@pytest.mark.parametrize("name", SPANS)
def test_sums_of_values_of_very_different_sizes_in_few_rows(tam_lib, n, Hq, Hkv, d, name):
    _values_of_very_different_sizes(tam_lib, n, Hq, Hkv, d, name, True, n + 4096,
                                    8 * 148 * 3 // Hkv + 1)


@pytest.mark.parametrize("n,Hq,Hkv,d", FEW + CHUNKS)
@pytest.mark.parametrize("size", [2.0 ** 8, 2.0 ** 14, 2.0 ** 20, 2.0 ** 30, 2.0 ** 46])
@pytest.mark.parametrize("score", [-9.0, -15.0, -19.0, -22.0])
@pytest.mark.parametrize("far", [[3, 4, 13, 30], list(range(256, 384))], ids=["some", "tile"])
def test_small_probabilities_of_large_values(tam_lib, n, Hq, Hkv, d, size, score, far):
    """Keys of small probability whose V rows are much larger than the others': what they add is
    rounded as the rest is.  A tile of them comes after others, in the same CTA."""
    gen = _gen(n + d)
    L = n + far[-1] + 20
    n_seq = 1 if far[0] < 128 else 8 * 148 // Hkv + 1
    k, v = _rand(gen, L, Hkv, d), _rand(gen, L, Hkv, d)
    q = torch.zeros(n, Hq, d, device="cuda")
    q[..., 0] = 8.0
    k[..., 0] = 0.0
    far = torch.tensor(far, device="cuda")
    k[far, :, 0] = score * math.sqrt(d) / 8.0
    k[far, :, 1:] = 0.0
    v[far] *= size
    cache, table, kk, vv = _quantised(tam_lib, gen, k.to(BF16), v.to(BF16))
    q = q.to(BF16)
    batch = tam_lib.PagedBatch(table.expand(n_seq, -1).contiguous(),
                               [n * s for s in range(n_seq + 1)], [L] * n_seq)
    out, lse = tam_lib.paged_gqa_attention(q.repeat(n_seq, 1, 1), cache, batch, return_lse=True)
    for s in sorted({0, n_seq - 1}):
        _check_seq(out[n * s:n * (s + 1)], lse.view(n_seq, Hq, n)[s], q, kk, vv, n)


# ------------------------------------------------------------------ batches that overlap

@pytest.mark.parametrize("io,dtype,n", [(BF16, BF16, 1), (BF16, E4M3, 1), (BF16, E4M3, 40), (F32, F32, 3)])
def test_decreasing_row_offsets_are_reported(tam_lib, io, dtype, n):
    """On the device, where the host cannot see them: nothing is written, however many blocks the
    overlapping sequences would ask for."""
    gen = _gen(4)
    cache, table, _, _ = _filled(tam_lib, gen, [90], 16, 2, 64, dtype, io=io)
    T = 3 * n
    q = _rand(gen, T, 8, 64).to(io)
    for cu in ([0, T, n], [0, n, 0, T], [0] + [T, 0] * 2000, [0, n, 2 * n, -5, T]):
        batch = tam_lib.PagedBatch(table.expand(len(cu) - 1, -1).contiguous(),
                                   torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                   [90] * (len(cu) - 1), max_rows=n)
        out = torch.full_like(q, 4.0)
        with pytest.raises(tam_lib.TamError) as err:
            tam_lib.paged_gqa_attention(q, cache, batch, out=out)
        assert err.value.code == tam_lib.TAM_ERR_INVALID_ARG
        assert bool((out == 4.0).all())
    batch = tam_lib.PagedBatch(table, [0, T], [90])             # and the next call is right
    out, lse = tam_lib.paged_gqa_attention(q, cache, batch, return_lse=True)
    kk, vv = tam_lib.kv_cache_read(cache, tam_lib.PagedBatch(table, [0, 90], [90]), dtype=io)
    _check_seq(out, lse.view(8, T), q, kk, vv, T)


# ------------------------------------------------------------------ bounded waits

@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("n,Hq,Hkv,d", CHUNKS)
def test_forced_wait_timeout_is_reported(tam_lib, monkeypatch, dtype, n, Hq, Hkv, d):
    """A role that waits in vain: the others wind down, the call reports it, the next one works."""
    gen = _gen(n)
    L = n + 300
    cache, table, _, _ = _filled(tam_lib, gen, [L], 16, Hkv, d, dtype)
    q = _rand(gen, n, Hq, d).to(BF16)
    want = _attend(tam_lib, q, cache, table, L)
    monkeypatch.setenv("TAM_DEBUG_FORCE_TIMEOUT", "1")
    with pytest.raises(tam_lib.TamError) as err:
        _attend(tam_lib, q, cache, table, L)
    assert err.value.code == tam_lib.TAM_ERR_TIMEOUT
    monkeypatch.delenv("TAM_DEBUG_FORCE_TIMEOUT")
    got = _attend(tam_lib, q, cache, table, L)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ items computed again

@pytest.mark.parametrize("n,Hq,Hkv,d", FEW + CHUNKS)
def test_only_the_items_with_far_scales_change(tam_lib, n, Hq, Hkv, d):
    """One head of one of three sequences has V rows of very different sizes: the others keep their
    bits, rows behind the last sequence theirs, and a captured call follows its pages."""
    gen = _gen(n + d)
    lens = [n + 300, n + 41, n + 700]
    cache, table, _, _ = _filled(tam_lib, gen, lens, 16, Hkv, d, E4M3)
    T = 3 * n + 2
    q = _rand(gen, T, Hq, d).to(BF16)
    cu = torch.tensor(_cu([n] * 3), dtype=torch.int32, device="cuda")
    batch = tam_lib.PagedBatch(table, cu, lens, max_rows=n)
    ws = tam_lib.Workspace()
    ws.get(tam_lib.paged_attention_workspace(T, Hq, BF16, cache, batch))
    out = torch.full_like(q, 3.0)
    before, lse0 = tam_lib.paged_gqa_attention(q, cache, batch, out=out, return_lse=True)
    before, lse0 = before.clone(), lse0.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tam_lib.paged_gqa_attention(q, cache, batch, out=out, workspace=ws, check=False)
    scale = cache.v_scale.view(torch.uint8)
    kept = scale.clone()
    page, G = int(table[1, 1]), Hq // Hkv
    for step in range(3):
        scale.copy_(kept)
        if step != 1:
            scale[page, Hkv - 1, 3] -= 60           # the row 19 of the sequence 1
        out.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        tam_lib.check_status(ws.buf)
        again, lse = tam_lib.paged_gqa_attention(q, cache, batch, return_lse=True,
                                                 out=torch.full_like(q, 3.0))
        assert torch.equal(out, again) and bool((out[3 * n:] == 3.0).all())
        if step == 1:
            assert torch.equal(out, before) and torch.equal(lse[:Hq * 3 * n], lse0[:Hq * 3 * n])
            continue
        same = torch.ones_like(out, dtype=torch.bool)
        same[n:2 * n, Hq - G:] = False
        assert torch.equal(out[same], before[same])
        kk, vv = tam_lib.kv_cache_read(cache, tam_lib.PagedBatch(table, _cu(lens), lens), dtype=F32)
        for s in range(3):
            a, t = _cu(lens)[s], s * n
            _check_seq(out[t:t + n], lse[Hq * t:Hq * (t + n)].view(Hq, n), q[t:t + n],
                       kk[a:a + lens[s]], vv[a:a + lens[s]], n)


@pytest.mark.parametrize("n,Hq,Hkv,d", FEW + CHUNKS)
def test_far_scales_beside_missing_pages_and_a_table_too_short(tam_lib, n, Hq, Hkv, d):
    gen = _gen(n + 7 * d)
    page, cap = 16, 16 * 21
    k, v = _rand(gen, cap, Hkv, d), _rand(gen, cap, Hkv, d)
    v[::3] *= 2.0 ** 40
    k[5::7] *= 2.0 ** -40
    cache, table, kk, vv = _quantised(tam_lib, gen, k.to(BF16), v.to(BF16), page)
    table = table[:, :21].contiguous()
    keep = torch.ones(cap, dtype=torch.bool, device="cuda")
    for col, bad in ((0, -1), (6, cache.n_pages), (7, 2 ** 31 - 1)):
        table[0, col] = bad
        keep[col * page:(col + 1) * page] = False
    q = _rand(gen, n, Hq, d).to(BF16)
    for over in (0, n):                             # the rows at the table's end, or all behind it
        batch = tam_lib.PagedBatch(table, [0, n], [cap + over])
        out, lse = tam_lib.paged_gqa_attention(q, cache, batch, return_lse=True, check=False)
        lse = lse.view(Hq, n)
        if over == 0:
            _check_seq(out, lse, q, kk[keep], vv[keep], n)
        else:
            for i in {0, n // 2, n - 1}:
                _check_seq(out[i:i + 1], lse[:, i:i + 1], q[i:i + 1], kk[keep], vv[keep], 1)
