"""Plain 64-bit forms of the paged operators (numpy-style loops over sequences),
and the error bounds that their tests allow.

Bounds.  A BF16 rounding is off by at most 2^-8 of the value (half a step), an
FP32 one by 2^-24.

Norm and rotation: the sum of squares takes at most 8 + 5 additions a term, so
its relative error is below 14 * 2^-24 and the root's half of that; the inverse
root, the two products with it and the rotation's cosine, sine (2^-22 in all from
the reduced angle), products and sum add less than 2^-20.  Together the FP32
value is off by at most 2^-19 (|a| + |b|) for a pair (a, b).

Attention: a score is a sum of dim products in FP32, off by at most
ds = dim 2^-24 scale sum |q| |k|; a probability by 2 ds + 2^-18 (exponential, sums
of up to 2^17 terms taken in tiles, quotient) and, before it multiplies V, by one
BF16 rounding.  So |out - exact| <= 2^-8 |exact| + (2^-8 + 2^-18 + 2 ds) A with
A = sum p |v|; the logarithm of the sum is off by ds + 2^-17 + 2^-22 |lse|.
"""
import math

import torch


def norm_rotate(x, w, pos, freq, interleaved, eps):
    """(y, bound) of x [tokens, heads, dim] in FP64; bound for an FP32 result."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
    y, size = x.clone(), x.abs()
    if freq is not None:
        n = freq.numel()
        t = pos.double()[:, None, None] * freq
        if interleaved:
            a, b = slice(0, 2 * n, 2), slice(1, 2 * n, 2)
        else:
            a, b = slice(0, n), slice(n, 2 * n)
        y[..., a] = x[..., a] * t.cos() - x[..., b] * t.sin()
        y[..., b] = x[..., b] * t.cos() + x[..., a] * t.sin()
        both = x[..., a].abs() + x[..., b].abs()
        size[..., a], size[..., b] = both, both
    return y, 2.0 ** -19 * size


def close(got, want, bound, dtype):
    """Whether got (of `dtype`) is want within bound and one rounding to dtype."""
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    off = (got.double() - want).abs()
    return bool((off <= bound * (1 + 2.0 ** -8) + half * want.abs()).all())


def groups_of(sequences, group_start):
    """The group of every sequence, or None."""
    if group_start is None:
        return [None] * sequences
    return [next((g for g in range(len(group_start) - 1)
                  if group_start[g] <= b < group_start[g + 1]), None) for b in range(sequences)]


def attention(q, k_pages, v_pages, table, lens, q_lens, prefix_table, prefix_lens, group_start,
              scale):
    """(out, bound, lse, lse_bound) in FP64; lens, q_lens, prefix_lens and
    group_start are lists."""
    rows, heads, dim = q.shape
    kv_heads, page = k_pages.shape[2], k_pages.shape[1]
    n_seq = len(lens)
    chunk = rows // n_seq
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    lse = torch.full((rows, heads), -math.inf, dtype=torch.float64, device=q.device)
    lse_bound = torch.zeros_like(lse)
    group = groups_of(n_seq, group_start)

    def tokens(pages, row, n):
        ids = row[:-(-n // page)].long()
        return pages[ids].flatten(0, 1)[:n].double()

    for b in range(n_seq):
        fresh = chunk if q_lens is None else min(max(q_lens[b], 0), chunk)
        own = max(lens[b], 0)
        far = max(prefix_lens[group[b]], 0) if group[b] is not None else 0
        k, v = tokens(k_pages, table[b], own), tokens(v_pages, table[b], own)
        if far:
            k = torch.cat((tokens(k_pages, prefix_table[group[b]], far), k))
            v = torch.cat((tokens(v_pages, prefix_table[group[b]], far), v))
        for i in range(fresh):
            n = far + max(own - fresh + i + 1, 0)
            r = b * chunk + i
            if n == 0:
                continue
            qr = q[r].double().view(kv_heads, heads // kv_heads, dim)
            s = torch.einsum("hgd,nhd->hgn", qr, k[:n]) * scale
            ds = dim * 2.0 ** -24 * abs(scale) * torch.einsum("hgd,nhd->hgn", qr.abs(),
                                                              k[:n].abs()).amax(-1)
            p = torch.softmax(s, -1)
            o = torch.einsum("hgn,nhd->hgd", p, v[:n])
            size = torch.einsum("hgn,nhd->hgd", p, v[:n].abs())
            out[r] = o.reshape(heads, dim)
            bound[r] = ((2.0 ** -8 + 2.0 ** -18 + 2 * ds)[..., None] * size).reshape(heads, dim)
            lse[r] = torch.logsumexp(s, -1).reshape(heads)
            lse_bound[r] = (ds.reshape(heads) + 2.0 ** -17 + 2.0 ** -22 * lse[r].abs())
    return out, bound, lse, lse_bound
