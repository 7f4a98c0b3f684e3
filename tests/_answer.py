"""Plain 64-bit references of the block-scaled product, the head norms with rotation
and the token log probabilities (not collected by pytest)."""
import math

import torch

HALF = 2.0 ** -24              # half a step of fp32, relative
BLOCK = 128


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ----------------------------------------------------------------------------- product


def e4m3_nearest(v):
    """E4M3 value nearest to each f64 value, ties to even, saturating; NaN kept."""
    a = v.abs()
    step = torch.ldexp(torch.ones_like(a), torch.frexp(a)[1].clamp(min=-5) - 4)
    r = (torch.round(a / step) * step).clamp(max=448.0)
    return torch.where(v.isnan(), v, torch.copysign(r, v))


def scale_of(top):
    """fp32 scale of blocks with the largest magnitudes `top` (any float type)."""
    s = (top.float() * torch.tensor(1.0 / 448.0)).clamp(min=2.0 ** -126)
    s = torch.where(top.float() == 0, torch.zeros_like(s), s)
    return torch.where(top.isfinite(), s, torch.full_like(s, math.nan))


def quotients(v, s):
    """Codes' f64 values of v under fp32 scales s of the same shape."""
    return e4m3_nearest(v.double() / torch.where(s == 0, torch.ones_like(s), s).double())


def pad_to(x, rows, cols):
    return torch.nn.functional.pad(x, (0, -x.shape[1] % cols, 0, -x.shape[0] % rows))


def quantize_rows(x):
    """(f64 code values [rows, k], fp32 scales [rows, blocks])."""
    k = x.shape[1]
    b = pad_to(x, 1, BLOCK).unflatten(1, (-1, BLOCK))
    top = torch.where(b.isnan().any(-1), math.inf, b.abs().nan_to_num(0.0, math.inf).amax(-1).double())
    s = scale_of(top)
    return quotients(b, s.unsqueeze(-1).expand_as(b)).flatten(1)[:, :k], s


def quantize_weight(w):
    """(f64 code values [n, k], fp32 scales [n / 128, k / 128])."""
    n, k = w.shape
    b = pad_to(w, BLOCK, BLOCK)
    b = b.unflatten(1, (-1, BLOCK)).unflatten(0, (-1, BLOCK)).transpose(1, 2)      # [nb, kb, 128, 128]
    top = b.abs().flatten(2).amax(-1).double()
    s = scale_of(top)
    q = quotients(b, s[..., None, None].expand_as(b)).transpose(1, 2).flatten(0, 1).flatten(1)
    return q[:n, :k], s


def unpack(q, rows, cols):
    """uint8 codes [rows up to 16, cols up to 128] of packed ones."""
    rb, cb = -(-rows // 16), -(-cols // BLOCK)
    t = q.view(rb, cb, 2, 4, 16, 16)             # half, lane group, row, byte
    return t.permute(0, 4, 1, 3, 2, 5).reshape(rb * 16, cb * BLOCK)


def linear_ref(xq, xs, wq, ws, dtype):
    """(y, bound): the f64 product of f64 code values under their scales, and how far
    a result may be off: half a step of the output, and relative to the sum of
    magnitudes: 128 additions of a block, which may cut off a whole step of fp32 each
    (2^-23), as many as there are blocks and four products, half a step each.  On the way
    to bf16 also, for each eight neighbouring products, seven cut off at 2^-13 of the
    power of two of the largest, which neither their sum of magnitudes nor the product of both sides'
    largest is below."""
    rows, k = xq.shape
    n = wq.shape[0]
    y, mag, most = (torch.zeros(rows, n, dtype=torch.float64) for _ in range(3))
    grow = torch.arange(n) // BLOCK
    for b in range(xs.shape[1]):
        at = slice(b * BLOCK, (b + 1) * BLOCK)
        f = xs[:, b:b + 1].double() * ws[grow, b].double()
        xa, wa = xq[:, at], wq[:, at]
        y += f * (xa @ wa.T)
        xa, wa = xa.abs(), wa.abs()
        mag += f.abs() * (xa @ wa.T)
        eights = [pad_to(t, 1, 8).unflatten(1, (-1, 8)).amax(-1) for t in (xa, wa)]
        most += f.abs() * (eights[0] @ eights[1].T)
    bound = half_step(dtype) * y.abs() + (BLOCK * 2 + xs.shape[1] + 4) * HALF * mag
    if dtype == torch.bfloat16:
        bound = bound + 7 * 2.0 ** -13 * torch.minimum(mag, most)
    return y, bound


# ----------------------------------------------------------------------------- rotation


def turned(x, weight, positions, inv_freq, eps, interleaved, after):
    """(y, bound) of [rows, heads, head_dim] in f64.  The angle is the f64 product.
    Bound, before the output's rounding: relative to |a cos| + |b sin|, sines and cosines rounded to fp32
    (1), the product with the weight (1), the products and the sum (2), 1 / rms (3: the instruction's
    step of 2, and its correction's rounding), its product (1), and the mean of squares, whose 8 additions in a
    lane, 5 of lanes, division and eps, half of which reach the root (8); halves of a step each."""
    d, half = x.shape[2], inv_freq.numel()
    w = weight.double()
    n = x.double()
    n = n / torch.sqrt(n.square().mean(-1, keepdim=True) + eps)
    pre = n if after else n * w
    i = torch.arange(half)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    t = (positions.double()[:, None] * inv_freq.double())[:, None]
    a, b, c, s = pre[..., lo], pre[..., hi], torch.cos(t), torch.sin(t)
    y, mag = pre.clone(), pre.abs()
    y[..., lo], y[..., hi] = a * c - b * s, a * s + b * c
    mag[..., lo], mag[..., hi] = (a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs()
    if after:
        y, mag = y * w, mag * w.abs()
    return y, 16 * HALF * mag


# ----------------------------------------------------------------------------- log probabilities


def logprobs_ref(x, tokens, top):
    """f64 (logprob, entropy, top values, top tokens) and bounds of the first two.
    The sum's relative error: its additions (a thread's elements, 1/256 of the row, and 10 joins of 4 roundings), the exponentials
    (2^-22: their own step, and their argument's two roundings, weighted with |d| e^-|d| < 1/2);
    the log probability takes that and three roundings of the difference and the
    logarithm, which itself is good to 2 steps; the entropy that of both its sums, the second's terms up to log(vocab)."""
    rows, vocab = x.shape
    d = x.double()
    order = d.masked_fill(d.isnan(), -math.inf)
    most = order.amax(1)
    # from the maximum, not from the logarithm of the whole sum, which a maximum of 1e38 swallows
    lp = d - most.clamp(min=-1e300)[:, None]
    log_l = lp.exp().sum(1).log()
    lp = lp - log_l[:, None]
    p = lp.exp()
    h = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1)
    inside = (tokens >= 0) & (tokens < vocab)
    chosen = lp.gather(1, tokens.clamp(0, vocab - 1).long()[:, None])[:, 0]
    chosen = torch.where(inside, chosen, torch.full_like(chosen, -math.inf))
    empty = (d == -math.inf).all(1)
    chosen = torch.where(empty, torch.full_like(chosen, -math.inf), chosen)
    h = torch.where(empty, torch.zeros_like(h), h)
    ids = order.sort(dim=1, descending=True, stable=True).indices[:, :top]
    values = lp.gather(1, ids)
    values[empty] = -math.inf
    rel = (vocab / 256 + 40) * HALF + 2.0 ** -22
    log_v = math.log(vocab) + 1
    away = (d.gather(1, tokens.clamp(0, vocab - 1).long()[:, None])[:, 0] - most).abs().nan_to_num(0.0, 0.0, 0.0)
    b_lp = rel + 6 * HALF * (away + log_v)
    b_h = 2 * rel * log_v + 8 * HALF * log_v
    b_top = rel + 6 * HALF * ((values + log_l[:, None]).abs().nan_to_num(0.0, 0.0, 0.0) + log_v)
    return chosen, h, values, ids, b_lp, torch.full_like(h, b_h), b_top
