"""Plain 64-bit implementations for the tests of the norms, the E4M3 block products and the
rotary positions, and the error bounds their tolerances come from.  Shares no code with the
library."""
import math

import torch

from attention_ref import U_BF16, U_F32, e4m3_values

HALF_STEP = {torch.bfloat16: U_BF16, torch.float32: U_F32}
TINY = 1e-37                      # values near fp32's underflow


def rows(n, cols, dtype, seed, spread=3.0):
    """Rows of unequal size with channels of unequal size."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, cols), generator=g)
    x *= torch.exp(torch.randn((n, 1), generator=g).clamp(-spread, spread))
    x *= torch.exp(0.5 * torch.randn((1, cols), generator=g))
    return x.to(dtype)


# ---- norms ------------------------------------------------------------------------------
# A row's sum of squares: at most 32 values per thread one after the other and ten steps over
# threads, all terms positive: 42 roundings relative to the sum, 21 after the root; the mean, eps,
# the root, w + offset and the two products add 7.
NORM = 32 * U_F32


def norm(x, w, offset, eps):
    """(rms(x) * (w + offset), 1 / root) of float64 rows."""
    r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    return x * r * (w + offset), r


def join(res, y, w_post, gate, act, branch, w_next, offset, eps):
    """(r', bound on |r' error| in fp32, out or None, bound on |out error| in fp32)."""
    h = y if w_post is None else norm(y, w_post, offset, eps)[0]
    if gate is not None:
        h = h * {"none": lambda t: t, "sigmoid": torch.sigmoid, "tanh": torch.tanh}[act](gate)
    r = res + branch * h
    # the norm, the gate (expf or tanhf 2 ulp, a sum, a division), two products, the sum
    dr = (NORM + 10 * U_F32) * (branch * h).abs() + U_F32 * r.abs() + TINY
    if w_next is None:
        return r, dr, None, None
    out, root = norm(r, w_next, offset, eps)
    # r' off by dr: the value itself, and the root by the norms' ratio (Cauchy-Schwarz)
    off = dr.square().sum(-1, keepdim=True).sqrt() / r.square().sum(-1, keepdim=True).sqrt().clamp(min=1e-300)
    return r, dr, out, (root * (w_next + offset)).abs() * dr * 1.01 + out.abs() * (off * 1.01 + NORM)


# ---- E4M3 blocks ------------------------------------------------------------------------
def encode(x):
    """Codes of float64 values, nearest, ties to the even code, saturating; NaN as 127."""
    vals = e4m3_values()[:127]
    a = x.abs().clamp(max=448.0).nan_to_num(0.0)
    hi = torch.searchsorted(vals, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = (a - vals[lo]).abs(), (vals[hi] - a).abs()
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    pick = pick + torch.signbit(x).long() * 128
    return torch.where(torch.isnan(x), torch.tensor(127), pick).to(torch.uint8)


def quantise_blocks(x):
    """(codes, scales) of fp32 rows by the definition: IEEE fp32 operations on the CPU."""
    n, cols = x.shape
    blocks = -(-cols // 128)
    codes = torch.zeros((n, cols), dtype=torch.uint8)
    scales = torch.ones((n, blocks), dtype=torch.float32)
    for b in range(blocks):
        part = x[:, b * 128:(b + 1) * 128].float()
        finite = torch.isfinite(part)
        amax = torch.where(finite, part.abs(), torch.zeros(())).amax(-1)
        some = amax > 0
        amax = amax.clamp(min=2.0 ** -100)
        scales[:, b] = torch.where(some, amax / 448.0, torch.ones(()))
        inv = torch.where(some, torch.tensor(448.0) / amax, torch.zeros(()))
        scaled = torch.where(finite, part, torch.tensor(math.nan)) * inv[:, None]
        codes[:, b * 128:(b + 1) * 128] = encode(scaled.double())
    return codes, scales


def same_codes(got, want):
    """Equal codes, where a NaN has no sign and a zero none."""
    got, want = got.cpu().long(), want.long()
    nan_g, nan_w = (got & 127) == 127, (want & 127) == 127
    zero = ((got & 127) == 0) & ((want & 127) == 0)
    return torch.equal(nan_g, nan_w) and bool(((got == want) | nan_g | zero).all())


def values(codes, scales):
    """What E4M3 blocks stand for, in 64 bits."""
    per = scales.double().repeat_interleave(128, 1)[:, :codes.shape[1]]
    return e4m3_values()[codes.long()] * per


def held_as_blocks(codes, scales, want, bound, name):
    """The blocks stand for `want` within a half step each and what the values may be off.  In a
    block the scale is off by as much as the largest value: the codes' own rounding hides it."""
    got = values(codes.cpu(), scales.cpu())
    per = scales.cpu().double().repeat_interleave(128, 1)[:, :codes.shape[1]]
    allowed = want.abs() * (2.0 ** -4 + 4 * U_F32) + per * 2.0 ** -10 + 1.1 * bound
    over = ((got - want).abs() - allowed).max()
    assert float(over) <= 0, f"{name}: off by {float(over)} more than a half step"


def weights(n_out, n_in, seed):
    """Codes [out, in] and scales of a linear layer's weights, blocks of unequal size."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (n_out, n_in), generator=g, dtype=torch.uint8)
    codes = torch.where((codes & 127) == 127, codes - 1, codes)
    scale = torch.exp(torch.randn((-(-n_out // 128), -(-n_in // 128)), generator=g)) * 2.0 ** -9
    return codes, scale


def product(x_q, x_scale, w_q, w_scale):
    """(y, bound on |y error| in fp32): every product of codes is exact; a block's sum of 128 and
    the sum over the blocks each lose at most 2^-23 of the summed magnitudes per addition (whether
    it rounds or truncates), the scales' product and its own two roundings more."""
    n_out, n_in = w_q.shape
    x = values(x_q, x_scale)
    w = e4m3_values()[w_q.long()]
    w = w * w_scale.double().repeat_interleave(128, 0)[:n_out].repeat_interleave(128, 1)[:, :n_in]
    size = x.abs() @ w.abs().T
    steps = 128 + 4 + -(-n_in // 128)
    return x @ w.T, steps * 2.0 ** -23 * size + TINY


# ---- rotary positions -------------------------------------------------------------------
def angles(positions, freq, axis):
    """Angles [n, pairs] in radians, from whole fractions of a turn: int64 positions [axes, n],
    int64 freq bits and axis."""
    out = torch.zeros((positions.shape[1], len(freq)), dtype=torch.float64)
    for j, (f, a) in enumerate(zip(freq.tolist(), axis.tolist())):
        if a >= positions.shape[0]:
            continue
        for i, p in enumerate(positions[a].tolist()):
            phase = (p * f) % 2 ** 64
            if phase >= 2 ** 63:
                phase -= 2 ** 64
            out[i, j] = phase * 2.0 ** -64 * math.tau
    return out


# Sines and cosines are within 0.8 of a place, then come the magnitude, the products and the sum:
# below ten roundings of |a| + |b| in all.
TURN = 10 * U_F32


def turn(x, angle, adjacent, magnitude=1.0):
    """(x turned, bound on its error in fp32) of float64 x [n, heads, d]."""
    half = angle.shape[1]
    first = torch.arange(half) * (2 if adjacent else 1)
    second = first + (1 if adjacent else half)
    c, s = (magnitude * f(angle)[:, None] for f in (torch.cos, torch.sin))
    a, b = x[..., first], x[..., second]
    out, bound = x.clone(), torch.zeros_like(x)
    out[..., first] = a * c - b * s
    out[..., second] = b * c + a * s
    bound[..., first] = bound[..., second] = TURN * abs(magnitude) * (a.abs() + b.abs())
    return out, bound
