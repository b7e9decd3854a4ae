"""Plain fp64 forms of the paged KV cache's operators, for the tests."""
import math

import torch

EXP_MIN, EXP_MAX = -100, 120


def quantise(x):
    """(values, exponents) of e4m3 rows x[..., d] in fp64, by search over the exponents and
    the sorted list of every e4m3 value; a row with an infinity or NaN: zeros and exponent 128
    (the scale byte 255)."""
    x = x.double()
    bad = ~torch.isfinite(x).all(-1)
    top = torch.where(bad[..., None], torch.zeros_like(x), x).abs().amax(-1)
    es = torch.arange(EXP_MIN, EXP_MAX + 1, device=x.device)
    fits = top[..., None] <= 448.0 * torch.exp2(es.double())
    e = es[fits.int().argmax(-1)]
    e = torch.where(fits.any(-1), e, torch.full_like(e, EXP_MAX))
    y = x / torch.exp2(e.double())[..., None]
    # every non-negative e4m3 value, by its bits
    bits = torch.arange(127, device=x.device)
    ex, man = bits >> 3, bits & 7
    vals = torch.where(ex == 0, man.double() / 8 * 2.0 ** -6,
                       (1 + man.double() / 8) * torch.exp2((ex - 7).double()))
    a = torch.where(bad[..., None], torch.zeros_like(y), y.abs()).contiguous()
    hi = torch.searchsorted(vals, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - vals[lo], vals[hi] - a
    pick = torch.where(dl < dh, lo, torch.where(dh < dl, hi, torch.where(lo % 2 == 0, lo, hi)))
    pick = torch.where(a == vals[hi], hi, pick)
    z = torch.copysign(vals[pick], y)
    # 256 * 2^120 is beyond fp32: the largest exponent keeps at most 240
    z = torch.where((e == EXP_MAX)[..., None], z.clamp(-240.0, 240.0), z)
    z = torch.where(bad[..., None], torch.zeros_like(z), z)
    return z, torch.where(bad, torch.full_like(e, 128), e)


def attention(q, k, v, n):
    """fp64 attention of the n newest rows: q [n, Hq, d], k and v [L, Hkv, d] (row i at
    position L - n + i).  Returns out, lse [Hq, n], and for the tolerances the absolute sum
    sum_j p_j |v_j| [n, Hq, d] and the largest score's terms max_j sum_c |q_c k_c| scale [Hq, n]
    over the keys a row sees."""
    L, Hkv, d = k.shape
    Hq = q.shape[1]
    G = Hq // Hkv
    q, k, v = q.double(), k.double(), v.double()
    scale = 1 / math.sqrt(d)
    out, absum = torch.zeros(n, Hq, d, dtype=torch.float64, device=q.device), None
    absum = torch.zeros_like(out)
    lse = torch.full((Hq, n), -math.inf, dtype=torch.float64, device=q.device)
    size = torch.zeros_like(lse)
    pos = torch.arange(L - n, L, device=q.device)
    see = torch.arange(L, device=q.device)[None] <= pos[:, None]        # [n, L]
    some = pos >= 0
    if L == 0 or n == 0 or not bool(some.any()):
        return out, lse, absum, size
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        x = (q[:, h] @ kh.T * scale).masked_fill(~see, -math.inf)
        t = (q[:, h].abs() @ kh.abs().T * scale).masked_fill(~see, 0.0)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
        tot = p.sum(-1, keepdim=True)
        o = (p / tot)
        out[some, h] = (o @ vh)[some]
        absum[some, h] = (o @ vh.abs())[some]
        lse[h, some] = (m + tot.log())[some, 0]
        size[h, some] = t.amax(-1)[some]
    return out, lse, absum, size


def tolerances(out, lse, absum, size, d, keys, bf16):
    """Absolute tolerances of out and lse.

    A score is a sum of d products: fp32 accumulation is off by at most (d + 8) 2^-23 of the
    sum of their magnitudes (2^-24 per add for rounding, doubled for a tensor core that cuts
    its sums), the scale and the exponential add 2^-21 of the score's size and 2^-18.  That is
    the relative error of a probability, met twice in out (numerator, denominator); the sums
    over the keys add keys * 2^-24.  bf16: every probability is rounded to bf16 for the product
    with v (2^-8 of it), and so is out."""
    delta = size * (d + 16) * 2.0 ** -23 + 2.0 ** -18 + keys * 2.0 ** -24     # [Hq, n]
    rel = 2 * delta + (2.0 ** -8 if bf16 else 0.0)
    tol = absum * rel.T[..., None] + out.abs() * (2.0 ** -8 if bf16 else 2.0 ** -24) + 1e-30
    return tol, delta + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0, neginf=0)
