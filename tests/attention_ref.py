"""Plain 64-bit implementations for the cache and attention tests, and the error
bounds their tolerances come from.  Shares no code with the library."""
import math

import torch

U_BF16 = 2.0 ** -8      # unit roundoff of bf16 (8 significant bits)
U_F16 = 2.0 ** -11      # of fp16 (11 bits)
U_F32 = 2.0 ** -24


def e4m3_values():
    """The 256 code values, by the format's definition."""
    out = torch.zeros(256, dtype=torch.float64)
    for c in range(256):
        field, low = (c >> 3) & 15, c & 7
        if field == 15 and low == 7:
            x = math.nan
        elif field == 0:
            x = low / 8 * 2.0 ** -6
        else:
            x = (1 + low / 8) * 2.0 ** (field - 7)
        out[c] = -x if c >= 128 else x
    return out


def row_exponent(row):
    """Smallest e in [-48, 48] with amax <= 448 * 2^e, by search."""
    amax = max([abs(x) for x in row if not math.isnan(x)] + [0.0])
    for e in range(-48, 48):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return 48


def quantise(rows):
    """(codes, exponent bytes) of float64 rows [n, d], by nearest value with ties
    to the even code, over a table of the values."""
    vals = e4m3_values()[:127]                    # the nonnegative finite ones, ascending
    codes = torch.zeros(rows.shape, dtype=torch.uint8)
    exps = torch.zeros(rows.shape[0], dtype=torch.uint8)
    for i, row in enumerate(rows.tolist()):
        e = row_exponent(row)
        exps[i] = e + 127
        x = torch.tensor(row, dtype=torch.float64) / 2.0 ** e
        a = x.abs().clamp(max=448.0)
        hi = torch.searchsorted(vals, a.nan_to_num(0.0)).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        dl, dh = (a - vals[lo]).abs(), (vals[hi] - a).abs()
        pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
        sign = torch.signbit(x).long() * 128
        codes[i] = torch.where(torch.isnan(x), torch.tensor(127), pick + sign).to(torch.uint8)
    return codes, exps


def cached_rows(cache, b, length, page_table, dtype=torch.float64):
    """Keys and values [length, heads, d] of request b from a (k, v, k_exp, v_exp)
    of CPU tensors."""
    ps = cache[0].shape[2]
    line = torch.arange(length)
    pages = page_table[b].long()[line // ps]
    out = []
    for x, e in ((cache[0], cache[2]), (cache[1], cache[3])):
        rows = x[pages, :, line % ps]
        if e is None:
            rows = rows.to(dtype)
        else:
            rows = e4m3_values()[rows.long()] * 2.0 ** (e[pages, :, line % ps].double() - 127)[..., None]
        out.append(rows)
    return out


def attend(q, k, v, seen, scale, weights_u, out_u):
    """q [t, hq, d], k and v [n, hk, d] in float64, seen bool [t, n] ->
    (out, lse, bound on |out error|, bound on |lse error|).

    The bound.  A logit z = scale * sum q k in fp32 has error at most
    dz = (d + 3) 2^-23 scale sum |q k| (one truncated or rounded add per product,
    and the factors' rounding), plus 2^-21 |z - max| for the base change and ex2.
    Weights move by a factor 1 +- 2 dz, are rounded by weights_u before the
    product with v, and n additions of w v each round or truncate by 2^-23.
    out_u is the output's rounding."""
    t, hq, d = q.shape
    n, hk, _ = k.shape
    g = hq // hk
    kk, vv = (x.repeat_interleave(g, dim=1) for x in (k, v))
    z = torch.einsum("thd,nhd->thn", q, kk.nan_to_num(0.0, 0.0, 0.0)) * scale
    mag = torch.einsum("thd,nhd->thn", q.abs(), kk.abs().nan_to_num(0.0, 0.0, 0.0)) * abs(scale)
    z = z.masked_fill(~seen[:, None, :], -math.inf)
    mag = mag.masked_fill(~seen[:, None, :], 0.0)
    lse = torch.logsumexp(z, -1)
    w = torch.exp(z - lse[..., None])
    w = torch.where(seen[:, None, :] & (z > -math.inf), w, torch.zeros(()).double())
    # only seen keys enter: unseen ones may hold anything
    anyone = seen.any(0)
    vz = torch.where(anyone[:, None, None], vv, torch.zeros(()).double())
    if torch.isfinite(vz).all():
        out = torch.einsum("thn,nhd->thd", w, vz)
    else:
        out = torch.zeros(t, hq, d, dtype=torch.float64)
        for i in range(t):
            vi = vv[seen[i]]
            out[i] = torch.einsum("hn,nhd->hd", w[i][:, seen[i]], vi)
    spread = torch.einsum("thn,nhd->thd", w, vz.abs().nan_to_num(0.0, 0.0, 0.0))
    dz = (d + 3) * 2.0 ** -23 * mag.amax(-1) + 2.0 ** -21 * 40 + 2.0 ** -22
    steps = (n + 64) * 2.0 ** -23
    bound = (2 * dz + weights_u + steps)[..., None] * 2 * spread + out_u * out.abs().nan_to_num(0.0) + 1e-30
    return out, lse, bound, 2 * dz + steps + 2.0 ** -22 * lse.abs().nan_to_num(0.0, 0.0, 0.0)


def chain_or_tree(t, ctx, words):
    """seen bool [t, ctx + t] of a chain (words None) or of int64 mask words [t, w]."""
    if words is None:
        return torch.arange(ctx + t)[None, :] <= (ctx + torch.arange(t))[:, None]
    seen = torch.ones((t, ctx + t), dtype=torch.bool)
    for i in range(t):
        for j in range(t):
            bit = j < 64 * words.shape[1] and (int(words[i, j // 64]) >> (j % 64)) & 1
            seen[i, ctx + j] = bool(bit)
    return seen


def check(name, got, want, bound):
    got = got.double().cpu()
    finite = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{name}: NaN places differ"
    inf = ~finite & ~torch.isnan(want)
    assert torch.equal(got[inf], want[inf]), f"{name}: infinities differ"
    over = ((got - want).abs() - bound)[finite]
    assert over.numel() == 0 or float(over.max()) <= 0.0, \
        f"{name}: error exceeds its bound by {float(over.max())}"
