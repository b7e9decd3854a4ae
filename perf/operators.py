"""The paged KV cache and the attention over it: the cases that are measured.

Three operators, each in its plain form (elementary torch operations in fp32) and, with
``own = True``, as a user's program calls this package:

* ``write``      the K/V rows of new tokens into the pages of a cache, as they are (bf16,
                 fp32) or quantised to e4m3 with one power-of-two scale per token and KV head;
* ``read``       the tokens of every sequence back out of the pages, as packed rows;
* ``attention``  causal GQA attention of every sequence's newest tokens (one, a chunk, or a
                 whole prompt) over its pages, with the log-sum-exp.

A sequence's rows are its newest tokens: row t of its n rows stands at position
kv_len - n + t, and position p is kept in row p % page_size of the page
page_table[sequence, p // page_size].
"""
import math

import torch

own = False

HEADS = ((4, 1), (8, 2), (16, 4), (16, 8), (32, 8))
EXP_MIN, EXP_MAX, EXP_BIAS, E4M3_MAX = -100, 120, 127, 448.0


# ------------------------------------------------------------------ cases

def _case(name, op, cache, Hq, Hkv, d, page, n_seq, new_min, new_max, len_min, len_max):
    return {"name": name, "op": op, "cache": cache, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page,
            "n_seq": n_seq, "new_min": new_min, "new_max": new_max, "len_min": len_min,
            "len_max": len_max}


def listed():
    return [
        # one decoding step of 64 sequences: their new K/V rows, quantised as they are kept
        _case("write_decode_e4m3", "write", "e4m3", 32, 8, 128, 16, 64, 1, 1, 1, 2048),
        # the prompts of a packed 32K batch, ragged
        _case("write_prompts_e4m3", "write", "e4m3", 32, 8, 128, 64, 8, 1024, 7168, 1024, 7168),
        # two chunks of a head-dim-256 layer, kept in bf16
        _case("write_chunks_bf16", "write", "bf16", 16, 8, 256, 32, 2, 500, 777, 2000, 4000),
        # a quantised 32K batch read back into the packed rows that the prefill calls take
        _case("read_batch_e4m3", "read", "e4m3", 32, 8, 128, 64, 8, 1024, 7168, 1024, 7168),
        # one short fp32 sequence read back: the latency of a call
        _case("read_short_f32", "read", "f32", 4, 1, 64, 16, 1, 513, 513, 513, 513),
        # one token of one sequence over 4K: the latency of a decoding step
        _case("attn_decode_one_bf16", "attention", "bf16", 32, 8, 128, 16, 1, 1, 1, 4096, 4096),
        # one token of each of 64 ragged sequences
        _case("attn_decode_batch_bf16", "attention", "bf16", 32, 8, 128, 64, 64, 1, 1, 100, 8192),
        # one token of each of 32 long ragged sequences over a quantised cache
        _case("attn_decode_batch_e4m3", "attention", "e4m3", 16, 4, 128, 64, 32, 1, 1, 1000, 32768),
        # five drafted tokens of each of 16 sequences to be verified, head dim 64
        _case("attn_verify_e4m3", "attention", "e4m3", 16, 4, 64, 32, 16, 5, 5, 2900, 9001),
        # a chunk of a long prompt, head dim 256
        _case("attn_chunk_d256_bf16", "attention", "bf16", 16, 8, 256, 32, 1, 512, 512, 16384,
              16384),
        # a serving step that mixes decoding sequences with ragged chunks, quantised cache
        _case("attn_mixed_e4m3", "attention", "e4m3", 32, 8, 128, 16, 24, 1, 700, 700, 8191),
        # a large chunk of a 32K prompt
        _case("attn_prompt_bf16", "attention", "bf16", 32, 8, 128, 128, 1, 4096, 4096, 32768,
              32768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        Hq, Hkv = rng.choice(HEADS)
        op = rng.choice(("write", "read", "attention", "attention"))
        d, page = rng.choice((64, 128, 256)), rng.choice((16, 32, 64, 128))
        cache = rng.choice(("bf16", "e4m3", "bf16", "e4m3", "f32"))
        n_seq = _log(rng, 1, 64)
        if op == "read":
            len_max = _log(rng, 1, 32768)
            len_min = new_min = _log(rng, 1, len_max)
            new_max = len_max
        else:
            new_max = rng.choice((1, _log(rng, 1, 16), _log(rng, 1, 4096)))
            new_min = _log(rng, 1, new_max)
            len_max = _log(rng, new_max, 32768)
            len_min = _log(rng, new_min, len_max)
        c = _case("", op, cache, Hq, Hkv, d, page, n_seq, new_min, new_max, len_min, len_max)
        del c["name"]
        w = work(c)
        most_bytes = 8e8 if op == "attention" else 2e8
        most_flops = 2e10 if cache == "f32" else 5e11
        # the plain form's padded scores and keys stay well below the listed prompt's
        padded = n_seq * Hq * new_max * len_max + 4 * n_seq * len_max * Hkv * d
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops and padded <= 4e9:
            return c


def _lengths(case):
    """(new tokens, cached tokens with them) of every sequence; the cached tokens are
    spread over their range, ragged, and so are the new ones."""
    new, total = [], []
    for s in range(case["n_seq"]):
        f, g = (s * 0.6180339887 + 0.5) % 1.0, (s * 0.7548776662 + 0.75) % 1.0
        if case["n_seq"] == 1:
            f = g = 1.0
        lo, hi = case["new_min"], case["new_max"]
        n = min(hi, lo + int((hi - lo + 1) * f))
        if case["op"] == "read":
            m = n
        else:
            lo, hi = max(case["len_min"], n), max(case["len_max"], n)
            m = min(hi, lo + int((hi - lo + 1) * g))
        new.append(n)
        total.append(m)
    return new, total


_BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


def work(case):
    new, total = _lengths(case)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    # one K or V row of a KV head in the cache: its values, and a byte of scale where quantised
    row = d * _BYTES[case["cache"]] + (1 if case["cache"] == "e4m3" else 0)
    io = 4 if case["cache"] == "f32" else 2
    named = new if case["op"] == "write" else total         # the positions looked up
    index = 4 * sum(-(-m // case["page"]) for m in named) + 8 * case["n_seq"]
    T = sum(new)
    if case["op"] in ("write", "read"):
        return {"bytes": 2 * T * Hkv * (row + d * io) + index, "flops": 0}
    pairs = sum(n * m - n * (n - 1) // 2 for n, m in zip(new, total))
    # q and out once, every cached row once, the log-sum-exp
    moved = 2 * T * Hq * d * io + 2 * sum(total) * Hkv * row + 4 * T * Hq + index
    return {"bytes": moved, "flops": 4 * d * Hq * pairs}


# ------------------------------------------------------------------ inputs

def _pow2(e):
    """2^e in fp32, from the exponent field (e in [-126, 127])."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """e4m3 values and power-of-two scales (e8m0) of rows x[..., d]: the smallest exponent e
    in [EXP_MIN, EXP_MAX] with max |x| <= 448 * 2^e, the values rounded to nearest even."""
    x = x.float()
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(top == 0, torch.full_like(e, EXP_MIN), e).clamp(EXP_MIN, EXP_MAX)
    y = x * _pow2(-e).unsqueeze(-1)
    return (y.to(torch.float8_e4m3fn),
            (e + EXP_BIAS).to(torch.uint8).view(torch.float8_e8m0fnu))


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    Hq, Hkv, d, page, n_seq = (case[x] for x in ("Hq", "Hkv", "d", "page", "n_seq"))
    new, total = _lengths(case)
    io = torch.float32 if case["cache"] == "f32" else torch.bfloat16
    per_seq = [-(-m // page) for m in total]
    max_pages = max(per_seq)
    n_pages = sum(per_seq) + 3

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    # pages handed out in no order, as a pool that has served for a while does
    perm = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((n_seq, max_pages), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(per_seq):
        table[s, :n] = perm[at:at + n]
        at += n
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st = dict(case=dict(case), new=new, total=total, T=cu[-1], max_rows=max(new), table=table,
              cu=torch.tensor(cu, dtype=torch.int32, device=dev),
              kv_len=torch.tensor(total, dtype=torch.int32, device=dev), io=io)
    # keys with a few strong channels, as a trained layer's
    strong = 1.0 + 3.0 * (torch.rand(Hkv, d, generator=gen, device=dev) > 0.95).float()
    if case["op"] == "write":
        st["k"] = (randn(cu[-1], Hkv, d) * strong).to(io)
        st["v"] = randn(cu[-1], Hkv, d).to(io)
        keep = torch.float8_e4m3fn if case["cache"] == "e4m3" else io
        st["k_pages"] = torch.zeros(n_pages, page, Hkv, d, device=dev).to(keep)
        st["v_pages"] = torch.zeros(n_pages, page, Hkv, d, device=dev).to(keep)
        for x in ("k_scale", "v_scale"):
            st[x] = None if case["cache"] != "e4m3" else torch.full(
                (n_pages, Hkv, page), EXP_BIAS, dtype=torch.uint8,
                device=dev).view(torch.float8_e8m0fnu)
    else:
        for x, mul in (("k", strong), ("v", 1.0)):
            st[x + "_pages"] = torch.empty(
                n_pages, page, Hkv, d, device=dev,
                dtype=torch.float8_e4m3fn if case["cache"] == "e4m3" else io)
            st[x + "_scale"] = None if case["cache"] != "e4m3" else torch.empty(
                n_pages, Hkv, page, dtype=torch.uint8, device=dev)
            for a in range(0, n_pages, 4096):        # a slice at a time: bounded fp32 copies
                rows = randn(min(4096, n_pages - a), page, Hkv, d) * mul
                if case["cache"] == "e4m3":
                    y, e = _quantise(rows)
                    st[x + "_pages"][a:a + 4096] = y
                    st[x + "_scale"][a:a + 4096] = e.view(torch.uint8).transpose(1, 2)
                else:
                    st[x + "_pages"][a:a + 4096] = rows.to(io)
            if case["cache"] == "e4m3":
                st[x + "_scale"] = st[x + "_scale"].view(torch.float8_e8m0fnu)
    if case["op"] == "attention":
        st["q"] = (2.0 * randn(cu[-1], Hq, d)).to(io)
    if own:
        import top_attention_mass_b200 as tam
        st["kv"] = tam.PagedKVCache(st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"])
        st["batch"] = tam.PagedBatch(table, st["cu"], st["kv_len"], max_rows=max(new))
    return st


# ------------------------------------------------------------------ the operators

def _places(st):
    """(page, row in it, sequence, index among its rows) of every packed row."""
    cu, page = st["cu"].long(), st["case"]["page"]
    t = torch.arange(st["T"], device=cu.device)
    s = torch.searchsorted(cu[1:], t, right=True)
    i = t - cu[s]
    p = st["kv_len"].long()[s] - (cu[1:] - cu[:-1])[s] + i
    return st["table"].long()[s, p // page], p % page, s, i


def _values(st, x, page, row):
    """fp32 values of the rows (page, row) of the k or v pages, every KV head."""
    kept = st[x + "_pages"]
    if st["case"]["cache"] != "e4m3":
        return kept[page, row].float()
    y = kept.view(torch.uint8)[page, row].view(torch.float8_e4m3fn).float()
    e = st[x + "_scale"].view(torch.uint8)[page, :, row].int() - EXP_BIAS
    return y * _pow2(e).unsqueeze(-1)


def _write(st):
    page, row, _, _ = _places(st)
    for x in ("k", "v"):
        if st["case"]["cache"] == "e4m3":
            y, e = _quantise(st[x])
            st[x + "_pages"].view(torch.uint8)[page, row] = y.view(torch.uint8)
            st[x + "_scale"].view(torch.uint8)[page, :, row] = e.view(torch.uint8)
        else:
            st[x + "_pages"][page, row] = st[x]
    return [st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"]]


def _read(st):
    page, row, _, _ = _places(st)
    return [_values(st, x, page, row).to(st["io"]) for x in ("k", "v")]


def _attention(st):
    c = st["case"]
    Hq, Hkv, d, n_seq = c["Hq"], c["Hkv"], c["d"], c["n_seq"]
    G, Q, L = Hq // Hkv, st["max_rows"], st["table"].shape[1] * c["page"]
    dev = st["q"].device
    cu, kv_len = st["cu"].long(), st["kv_len"].long()
    n = cu[1:] - cu[:-1]
    # padded keys and values [n_seq, L, Hkv, d], zero behind a sequence's end
    j = torch.arange(L, device=dev)
    there = j[None] < kv_len[:, None]
    page = torch.where(there, st["table"].long()[:, j // c["page"]], 0)
    row = (j % c["page"]).expand(n_seq, L)
    k = _values(st, "k", page, row).masked_fill_(~there[:, :, None, None], 0.0)
    v = _values(st, "v", page, row).masked_fill_(~there[:, :, None, None], 0.0)
    # padded queries [n_seq, Hkv, Q * G, d]
    i = torch.arange(Q, device=dev)
    at = (cu[:-1, None] + i[None]).clamp(max=st["T"] - 1)
    q = st["q"].float()[at].view(n_seq, Q, Hkv, G, d).permute(0, 2, 1, 3, 4)
    q = q.reshape(n_seq, Hkv, Q * G, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(d))
    pos = (kv_len - n)[:, None] + i[None]                         # [n_seq, Q]
    hide = (j[None, None] > pos[:, :, None]) | ~there[:, None]    # [n_seq, Q, L]
    x.view(n_seq, Hkv, Q, G, L).masked_fill_(hide[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top).exp_()
    tot = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / tot
    lse = (top + tot.log()).view(n_seq, Hkv, Q, G)
    o = o.view(n_seq, Hkv, Q, G, d).permute(0, 2, 1, 3, 4).reshape(n_seq, Q, Hq, d)
    _, _, s, r = _places(st)
    h = torch.arange(Hq, device=dev)
    flat = torch.empty(Hq * st["T"], device=dev)
    where = Hq * cu[s][:, None] + h[None] * n[s][:, None] + r[:, None]
    flat[where] = lse.permute(0, 2, 1, 3).reshape(n_seq, Q, Hq)[s, r]
    return [o[s, r].to(st["io"]), flat]


def run(st):
    op = st["case"]["op"]
    if own:
        import top_attention_mass_b200 as tam
        if op == "write":
            tam.kv_cache_write(st["kv"], st["batch"], st["k"], st["v"], check=False)
            return [st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"]]
        if op == "read":
            return list(tam.kv_cache_read(st["kv"], st["batch"], st["T"], dtype=st["io"],
                                          check=False))
        return list(tam.paged_gqa_attention(st["q"], st["kv"], st["batch"], return_lse=True,
                                            check=False))
    return {"write": _write, "read": _read, "attention": _attention}[op](st)


# ------------------------------------------------------------------ 64-bit values

def _two_to(e):
    """2^e in fp64, from the exponent field, for whole e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3_values(y):
    """y (fp64, |y| <= 448) rounded to the nearest e4m3 value, ties to even."""
    _, e = torch.frexp(y)                       # y = m 2^e, 0.5 <= |m| < 1
    step = _two_to(torch.clamp(e - 1, min=-6) - 3)
    return torch.round(y / step) * step


def _row_exponent(top):
    """Smallest e in range with top <= 448 * 2^e, found by trying the neighbours of log2."""
    e = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / E4M3_MAX))
    e = torch.where(top > E4M3_MAX * _two_to(e), e + 1, e)
    e = torch.where(top <= E4M3_MAX * _two_to(e - 1), e - 1, e)
    return e.clamp(EXP_MIN, EXP_MAX)


def exact(case, seed):
    st = prepare(case, seed)
    page = case["page"]
    table, new, total = st["table"].tolist(), st["new"], st["total"]
    cu = st["cu"].tolist()

    def stored(x, s, lo, hi):
        """Positions [lo, hi) of sequence s in fp64, [hi - lo, Hkv, d]."""
        pages = torch.tensor(table[s][lo // page:-(-hi // page)], device="cuda")
        y = st[x + "_pages"].view(torch.uint8 if case["cache"] == "e4m3" else st["io"])[pages]
        if case["cache"] == "e4m3":
            e = st[x + "_scale"].view(torch.uint8)[pages].long() - 127
            y = y.view(torch.float8_e4m3fn).double() * _two_to(e).transpose(1, 2)[..., None]
        first = lo // page * page
        return y.double().flatten(0, 1)[lo - first:hi - first]

    if case["op"] == "write":
        outs = [st[x].double() for x in ("k_pages", "v_pages")]
        scales = [None if st[x] is None else st[x].double() for x in ("k_scale", "v_scale")]
        for s in range(case["n_seq"]):
            p = torch.arange(total[s] - new[s], total[s], device="cuda")
            pages = torch.tensor(table[s], device="cuda")[p // page]
            for out, scale, x in zip(outs, scales, ("k", "v")):
                r = st[x][cu[s]:cu[s + 1]].double()
                if scale is not None:
                    e = _row_exponent(r.abs().amax(-1))
                    r = _e4m3_values(r / _two_to(e)[..., None])
                    scale[pages, :, p % page] = _two_to(e)
                out[pages, p % page] = r
        return outs + scales
    if case["op"] == "read":
        return [torch.cat([stored(x, s, 0, total[s]) for s in range(case["n_seq"])])
                for x in ("k", "v")]
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    G = Hq // Hkv
    if work(case)["flops"] > 1.2e13:
        return None
    out, lse = [], []
    for s in range(case["n_seq"]):
        n, m = new[s], total[s]
        k, v = stored("k", s, 0, m), stored("v", s, 0, m)
        o = torch.empty(n, Hq, d, dtype=torch.float64, device="cuda")
        z = torch.empty(Hq, n, dtype=torch.float64, device="cuda")
        for h in range(Hq):
            for a in range(0, n, 1024):
                b = min(n, a + 1024)
                x = st["q"][cu[s] + a:cu[s] + b, h].double() @ k[:, h // G].T / math.sqrt(d)
                last = torch.arange(m - n + a, m - n + b, device="cuda")
                x.masked_fill_(torch.arange(m, device="cuda")[None] > last[:, None], -math.inf)
                z[h, a:b] = torch.logsumexp(x, -1)
                o[a:b, h] = torch.softmax(x, -1) @ v[:, h // G]
        out.append(o)
        lse.append(z.flatten())
    return [torch.cat(out), torch.cat(lse)]
