"""Plain forms of the rotary positions and of the paged 4-bit cache, for the tests: the
rotation in 64 bits, the cache's definition in the 32-bit steps that fix its codes, reading
it back and attention over it in 64 bits, on the CPU with elementary torch operations."""
import math

import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # eps / 2: a rounding's share


def rotate(x, positions, freqs, mscale=1.0, interleaved=False, inverse=False, dtype=torch.float64):
    """x [T, H, d] at positions [T]; sums and products in `dtype`, sines and cosines rounded to it."""
    rot = 2 * freqs.numel()
    a = positions.double()[:, None] * freqs
    c, s = (torch.cos(a) * mscale).to(dtype)[:, None], (torch.sin(a) * mscale).to(dtype)[:, None]
    s = -s if inverse else s
    x = x.to(dtype)
    y = x.clone()
    i0 = torch.arange(rot // 2) * 2 if interleaved else torch.arange(rot // 2)
    i1 = i0 + 1 if interleaved else i0 + rot // 2
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i1] * c + x[..., i0] * s
    return y


def quantize(x):
    """Codes uint8 [..., d] and fp16 params [..., d/64, 2] of fp32 x [..., d]."""
    g = x.float().unflatten(-1, (-1, 64))
    lo, hi = g.amin(-1), g.amax(-1)                  # both propagate NaN
    step, low = ((hi - lo) * torch.tensor(1 / 15)).half(), lo.half()   # fp32 product with fl(1/15)
    q = torch.round((g - low.float()[..., None]) / step.float()[..., None])
    q = torch.nan_to_num(q, nan=0.0, posinf=15.0, neginf=0.0).clamp(0, 15)
    q = torch.where(step[..., None] == 0, 0.0, q)
    return q.flatten(-2).to(torch.uint8), torch.stack((step, low), -1)


def regions(cache, page, d):
    """Views of a CPU cache [pages, H, bytes]: codes [pages, H, 2, page, d/2] and params
    [pages, H, 2, page, d/64, 2] (index 0 of the third axis: keys, 1: values)."""
    codes = cache[..., :page * d].unflatten(-1, (2, page, d // 2))
    return codes, cache[..., page * d:].view(torch.float16).unflatten(-1, (2, page, d // 64, 2))


def tokens(cache, page, d, table, n, dtype=torch.float64):
    """Values [n, H, d] of the first n tokens of a sequence with the given row of the block
    table: keys and values."""
    codes, params = regions(cache, page, d)
    j = torch.arange(n)
    ids, rows = table.long()[j // page], j % page
    out = []
    for x in (0, 1):
        b = codes[ids, :, x, rows]
        c = torch.stack((b & 15, b >> 4), -1).flatten(-2).to(dtype).unflatten(-1, (-1, 64))
        p = params[ids, :, x, rows].to(dtype)
        out.append((c * p[..., :1] + p[..., 1:]).flatten(-2))
    return out


def attend(q, k, v, causal=True, sm_scale=None):
    """q [n, Hq, d], k and v [len, Hkv, d] in 64 bits: out, lse, and for tolerances the largest
    sum over channels of |q k| sm_scale and sum over keys of p |v| per output."""
    n, Hq, d = q.shape
    length, Hkv = k.shape[0], k.shape[1]
    sm = 1 / math.sqrt(d) if sm_scale is None else sm_scale
    k, v = (x.repeat_interleave(Hq // Hkv, 1) for x in (k, v))
    if length == 0:
        z = torch.zeros((n, Hq), dtype=torch.float64)
        return torch.zeros_like(q), z - math.inf, z, torch.zeros_like(q)
    s = torch.einsum("ihd,jhd->ihj", q, k) * sm
    if causal:
        s = s.masked_fill((torch.arange(length)[None] > torch.arange(length - n, length)[:, None])[:, None],
                          -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    w = p / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total))[..., 0]
    big = torch.einsum("ihd,jhd->ihj", q.abs(), k.abs()).amax(-1) * sm
    # hidden keys have weight 0 and no part, whatever lies there
    pick = lambda x: torch.einsum("ihj,jhd->ihd", w, torch.nan_to_num(x, nan=0.0)) if causal else torch.einsum("ihj,jhd->ihd", w, x)  # noqa: E731
    return pick(v), lse, big, pick(v.abs())


def spans(cache, page, d, table, n):
    """|low| + 15 step of the first n tokens of a sequence, [n, H, d/64] of keys and of values: what
    the two terms that make up an element are at most."""
    _, params = regions(cache, page, d)
    j = torch.arange(n)
    ids, rows = table.long()[j // page], j % page
    p = [params[ids, :, x, rows].double() for x in (0, 1)]
    return [x[..., 1].abs() + 15 * x[..., 0] for x in p], p[1][..., 0]


def room(q, k, v, key_span, value_span, value_step, dtype, causal=True, sm_scale=None):
    """How far off, as a 2-norm over 64 channels, an output of `dtype` may be from its 64-bit value:
    that value [n, Hq, d], the limits [n, Hq, d/64], the log-sums and their limits [n, Hq].

    The limit is the output's own rounding, known exactly, joined by root of squares (they are
    independent) with what the attention's steps add, each to first order:
      - a score is off by 2^-18 A at the very worst, A = sm_scale sum |q| span, when about 20
        accumulations all err by their most in one direction; independent ones make 2^-18 A / 8, and
        twice that is allowed. Sums over n keys add n 2^-26, the exponential and what is left 2^-16.
        Errors d_j of the weights w_j move an output by sum w_j d_j (v_j - out), in the mean
        d sqrt(sum w_j^2 |v_j - out|^2);
      - a weight's two fp16 terms and the value's two terms: 2^-20 of sqrt(sum w_j^2 span_j^2);
      - the second fp16 term ends at 2^-28 of the group's largest step that any query sees, a key's
        code then counts up to 8 times: 2^-25 step sqrt(n) over the sum of exp(score - largest).
    The whole is allowed a tenth more, for norms over 64 channels of what was taken in the mean."""
    n, Hq, d = q.shape
    length, Hkv = k.shape[0], k.shape[1]
    sm = 1 / math.sqrt(d) if sm_scale is None else sm_scale
    q = q.double()
    k, v, key_span, value_span, value_step = (
        x.repeat_interleave(Hq // Hkv, 1) for x in (k, v, key_span, value_span, value_step))
    s = torch.einsum("ihd,jhd->ihj", q, k) * sm
    if causal:
        s = s.masked_fill((torch.arange(length)[None] > torch.arange(length - n, length)[:, None])[:, None],
                          -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    total = p.sum(-1)
    w = p / total[..., None]
    out = torch.einsum("ihj,jhd->ihd", w, v)
    size = sm * torch.einsum("ihg,jhg->ihj", q.abs().unflatten(-1, (-1, 64)).sum(-1), key_span).amax(-1)
    off = 2.0 ** -20 * size + length * 2.0 ** -26 + 2.0 ** -16
    w2 = w * w
    # sum_j w_j^2 |v_j - out|^2 over the group's channels
    mass = (torch.einsum("ihj,jhd->ihd", w2, v * v) - 2 * out * torch.einsum("ihj,jhd->ihd", w2, v)
            + out * out * w2.sum(-1, keepdim=True)).clamp(min=0).unflatten(-1, (-1, 64)).sum(-1)
    terms = 64 * torch.einsum("ihj,jhg->ihg", w2, value_span ** 2)
    largest = value_step.amax(0)[None]                   # [1, Hq, d/64]
    least = 8 * 2.0 ** -25 * largest * math.sqrt(length) / total[..., None]
    rounding = (out.to(dtype).double() - out).unflatten(-1, (-1, 64)).square().sum(-1)
    limit = 1.1 * ((rounding + off[..., None] ** 2 * mass + 2.0 ** -40 * terms).sqrt() + least)
    lse = top[..., 0] + torch.log(total)
    return out, limit, lse, off + 2.0 ** -20 + 2.0 ** -22 * lse.abs()


def misses(got, out, limit):
    """How many groups of 64 channels of `got` are further from `out` than `limit`, and by how much at most."""
    far = (got.double() - out).unflatten(-1, (-1, 64)).norm(dim=-1) / limit
    return int((~(far <= 1)).sum()), float(far.max())
