"""Timed cases of the rotary-position and 4-bit-cache operators.

Four operators that a program which serves a language model calls next to the quantized
attention of this package:

  rope     rotates queries and keys by their positions (`rope`), or back (`inverse`)
  append   rotates new queries and keys, quantizes keys and values to 4 bits and writes
           them into a paged cache (`kv4_append`)
  gather   reads tokens of the paged cache back as 16-bit tensors (`kv4_gather`), for the
           prefill attention of this package
  attend   attention of a few queries per sequence over the paged cache (`attn_kv4`)

Each case is one of them, or a run of them as a serving loop makes it. With `own` false a
pass computes the operators' formulas with elementary torch operations in 32 bits (angles
in 64); with `own` true it calls the package.

Rotation. Channel pairs (x0, x1) of the first `rot` channels of a head, pair i at position
p: c = cos(p f_i) m, s = sin(p f_i) m, y0 = x0 c - x1 s, y1 = x1 c + x0 s. Pairs are (i,
i + rot/2) in the half layout and (2i, 2i + 1) in the interleaved one; the inverse takes -s.

4-bit cache. Every token of a key or value head is cut into groups of 64 channels: with lo
and hi a group's least and greatest value, step = fp16((hi - lo) / 15), low = fp16(lo),
code = round((x - low) / step) clamped to 0..15 (0 where step is 0), and the group stands
for low + code * step. A page holds `page` tokens of one head: the key codes [page, d/2]
(channel 2i in the low half of byte i), the value codes, then (step, low) of the keys'
groups as fp16 [page, d/64, 2] and of the values'.
"""
import math

import torch

own = False

CARD = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------- cases


def listed():
    return [
        # one decode step's queries and keys of every sequence, at positions past 32768
        dict(name="rope step", op="rope", type="fp16", batch=8, new=1, hq=32, hkv=32, d=128, rot=128, pairs="half",
             scaling="none", inverse=False, start=32768),
        # the queries and keys of a whole causal prefill, context stretched by wavelength
        dict(name="rope prefill", op="rope", type="fp16", batch=4, new=4096, hq=32, hkv=32, d=128, rot=128, pairs="half",
             scaling="parts", inverse=False, start=0),
        # gradients of a rotation over part of the head, odd length, shared key heads
        dict(name="rope gradient", op="rope", type="bf16", batch=3, new=2731, hq=32, hkv=8, d=128, rot=64, pairs="interleaved",
             scaling="linear", inverse=True, start=0),
        # one new token for each of 64 sequences, from a fused projection, small pages
        dict(name="append step", op="append", type="fp16", nseq=64, lo=1, hi=8192, new=1, ragged=False, hq=32, hkv=8, d=128,
             page=16, rot=128, pairs="half", scaling="parts", mean=False),
        # a prefill chunk of ragged prompts, with the calibrated key mean taken off
        dict(name="append chunk", op="append", type="bf16", nseq=8, lo=1, hi=16384, new=4096, ragged=True, hq=32, hkv=8, d=128,
             page=64, rot=64, pairs="interleaved", scaling="none", mean=True),
        # one short prompt's first tokens, every head with keys of its own, d 64
        dict(name="append short", op="append", type="fp16", nseq=1, lo=130, hi=517, new=130, ragged=False, hq=2, hkv=2, d=64,
             page=32, rot=64, pairs="half", scaling="none", mean=True),
        # all cached keys of two 8192-token sequences for a chunk's prefill attention
        dict(name="gather chunk", op="gather", type="fp16", nseq=2, lo=8192, hi=8192, hkv=8, rep=4, d=128, page=64),
        # ragged short sequences, d 64, page 16
        dict(name="gather ragged", op="gather", type="bf16", nseq=48, lo=1, hi=700, hkv=6, rep=1, d=64, page=16),
        # a single stream early in its answer: latency
        dict(name="attend one", op="attend", type="fp16", nseq=1, lo=391, hi=391, new=1, ragged=False, hq=32, hkv=8, d=128,
             page=16, lse=False),
        # a server's step: 64 sequences of very different lengths, shared key heads
        dict(name="attend batch", op="attend", type="bf16", nseq=64, lo=1, hi=8192, new=1, ragged=False, hq=32, hkv=8, d=128,
             page=16, lse=False),
        # long contexts, every query head with keys of its own: the whole cache is 1.2 GB
        dict(name="attend long", op="attend", type="fp16", nseq=8, lo=32768, hi=32768, new=1, ragged=False, hq=32, hkv=32, d=128,
             page=128, lse=False),
        # append and attend together: up to five drafted tokens per sequence, d 64
        dict(name="step drafts", op="step", type="fp16", nseq=24, lo=5, hi=12000, new=5, ragged=True, hq=30, hkv=5, d=64,
             page=64, rot=64, pairs="half", scaling="none", mean=False, lse=True),
    ]


def _over(rng, lo, hi):
    """A whole number spread evenly over the logarithm of lo..hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "append", "gather", "attend", "attend", "step"))
    d = rng.choice((64, 128, 128))
    hkv = rng.choice((1, 2, 4, 5, 8, 32))
    hq = hkv * (1 if hkv == 32 else rng.choice((1, 3, 4, 6, 8)))
    case = dict(op=op, type=rng.choice(("fp16", "bf16")), hkv=hkv, d=d)
    rotary = dict(hq=hq, rot=rng.choice((d, d, d // 2)), pairs=rng.choice(("half", "half", "interleaved")),
                  scaling=rng.choice(("none", "linear", "parts")))
    if op == "rope":
        new = _over(rng, 1, 8192)
        case.update(rotary, batch=_over(rng, 1, max(1, 16384 // new)), new=new, inverse=rng.random() < 0.4,
                    start=rng.choice((0, 0, _over(rng, 1, 1000000))))
        return case
    page = rng.choice((16, 32, 64, 128, 256))
    hi = _over(rng, 1, 32768)
    # at most as many cached values as the longest listed case reads
    room = max(1, 8 * 32768 * 32 * 128 // (hi * hkv * d))
    case.update(nseq=_over(rng, 1, min(256, room)), lo=rng.choice((1, hi, max(1, hi // 2))), hi=hi, page=page)
    if op == "gather":
        case.update(rep=rng.choice((1, 1, 2, 4)))
        if case["nseq"] * hi * hkv * case["rep"] > 2 * 8192 * 32 * 4:
            case.update(nseq=max(1, 2 * 8192 * 32 * 4 // (hi * hkv * case["rep"])))
        return case
    if op == "append":
        new = _over(rng, 1, hi)
        case.update(rotary, new=new, ragged=rng.random() < 0.5, mean=rng.random() < 0.5)
        case.update(lo=min(hi, max(case["lo"], new)), nseq=max(1, min(case["nseq"], 16384 // new)))
        return case
    new = min(hi, rng.choice((1, 1, 1, 2, 4, 7)))
    # the keys are multiplied with every query that shares them
    room = max(1, int(room / max(1.0, new * hq / hkv / 4)))
    case.update(hq=hq, new=new, ragged=new > 1 and rng.random() < 0.5, lse=rng.random() < 0.5, lo=max(case["lo"], new),
                nseq=min(case["nseq"], room))
    if op == "step":
        case.update(rotary, mean=rng.random() < 0.5)
    return case


# ------------------------------------------------------------------------------ inputs


def _freqs(case):
    """Angle per position of each pair in 64 bits, and the factor on cos and sin."""
    rot, base = case["rot"], 10000.0
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=CARD) / rot)
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    if case["scaling"] == "parts":
        # pairs that turn often over the first 4096 positions keep their angle, pairs that
        # turn less than once are slowed by the factor, those between by parts of each
        factor, trained, fast, slow = 8.0, 4096.0, 32.0, 1.0
        pair = lambda turns: rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64, device=CARD) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _normal(g, shape, type_, scale=1.0):
    return (torch.randn(shape, generator=g, device=CARD, dtype=torch.float32) * scale).to(type_)


def _quantized(x):
    """Codes 0..15 (uint8) of float32 x [..., d] and fp16 (step, low) [..., d/64, 2]."""
    g = x.unflatten(-1, (-1, 64))
    lo, hi = g.amin(-1), g.amax(-1)
    step, low = ((hi - lo) / 15.0).to(torch.float16), lo.to(torch.float16)
    at = (g - low.float().unsqueeze(-1)) / step.float().unsqueeze(-1)
    code = torch.where(step.unsqueeze(-1) == 0, 0.0, torch.round(at).clamp(0, 15))
    return code.to(torch.uint8).flatten(-2), torch.stack((step, low), -1)


def _packed(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _regions(cache, page, d):
    """Views of a cache [pages, heads, bytes]: key codes, value codes, key and value (step, low)."""
    half, groups = page * d // 2, d // 64
    par = cache[..., 2 * half:].view(torch.float16).unflatten(-1, (2, page, groups, 2))
    return (cache[..., :half].unflatten(-1, (page, d // 2)), cache[..., half:2 * half].unflatten(-1, (page, d // 2)),
            par[:, :, 0], par[:, :, 1])


def _lengths(case, order):
    """Cached and new tokens of each sequence. Their numbers go by the case, so that outputs of
    every seed have the same shapes; which sequence has which goes by `order`."""
    n = case["nseq"]
    of = torch.Generator().manual_seed(n * 1000003 + case["hi"])
    lens = torch.randint(case["lo"], case["hi"] + 1, (n,), generator=of)
    lens[0] = case["hi"]
    new = torch.full((n,), case.get("new", 1), dtype=torch.int64)
    if case["op"] == "gather":
        new = lens.clone()
    elif case["ragged"]:
        new = torch.minimum(lens, torch.randint(0, case["new"] + 1, (n,), generator=of))
        new[0] = case["new"]
    return lens[order], new[order]


def prepare(case, seed):
    g = torch.Generator(device=CARD).manual_seed(seed)
    rnd = torch.Generator().manual_seed(seed)
    type_, op, d, hkv = TYPES[case["type"]], case["op"], case["d"], case["hkv"]
    s = dict(case=case, type=type_, op=op, d=d, hkv=hkv, hq=case.get("hq"))
    if "rot" in case:
        s["freqs"], s["mscale"] = _freqs(case)
        s["interleaved"] = case["pairs"] == "interleaved"
    if op == "rope":
        b, n = case["batch"], case["new"]
        s["q"] = _normal(g, (b, s["hq"], n, d), type_)
        s["k"] = _normal(g, (b, hkv, n, d), type_)
        first = torch.randint(0, case["start"] + 1, (b, 1), generator=rnd) + case["start"] // 2
        s["positions"] = (first + torch.arange(n)).to(torch.int32).to(CARD)
        return s

    page, nseq = case["page"], case["nseq"]
    lens, new = _lengths(case, torch.randperm(nseq, generator=rnd))
    pages = (lens + page - 1) // page
    s["page"], s["longest"] = page, int(lens.max())
    total_pages, width = int(pages.sum()) + 1, int(pages.max())
    order = torch.randperm(total_pages, generator=rnd)
    table = torch.zeros((nseq, width), dtype=torch.int32)
    used = torch.arange(width)[None] < pages[:, None]
    table[used] = order[:int(pages.sum())].to(torch.int32)
    s["table"], s["lens"] = table.to(CARD), lens.to(torch.int32).to(CARD)
    s["cache"] = torch.zeros((total_pages, hkv, page * (d + 8 * (d // 64))), dtype=torch.uint8, device=CARD)
    regions = _regions(s["cache"], page, d)
    offset = torch.randn((hkv, d), generator=g, device=CARD)
    some = max(1, (1 << 26) // (hkv * page * d))
    for p in range(0, total_pages, some):
        m = min(some, total_pages - p)
        for at, shift in ((0, offset[:, None]), (1, 0.0)):
            x = torch.randn((m, hkv, page, d), generator=g, device=CARD) + shift
            code, par = _quantized(x)
            regions[at][p:p + m] = _packed(code)
            regions[2 + at][p:p + m] = par

    s["rep"] = case.get("rep", 1)
    cu = torch.zeros(nseq + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(new, 0)
    s["cu"], s["total"], s["new"], s["nseq"] = cu.to(CARD), int(cu[-1]), case.get("new", 1), nseq
    if op in ("append", "step"):
        fused = _normal(g, (s["total"], s["hq"] + 2 * hkv, d), type_)
        s["q"], s["k"], s["v"] = fused[:, :s["hq"]], fused[:, s["hq"]:s["hq"] + hkv], fused[:, s["hq"] + hkv:]
        s["k"] += offset.to(type_)
        s["mean"] = offset if case["mean"] else None
    elif op == "attend":
        s["q"] = _normal(g, (s["total"], s["hq"], d), type_)
    if op in ("attend", "step"):
        s["lse"] = case["lse"]
    return s


# -------------------------------------------------------------------------- plain forms


def _rotated(x, angle, mscale, rot, interleaved, inverse=False):
    """x [..., d] in float32 rotated by angle [..., rot/2] (64 bits), unrounded."""
    c, t = (torch.cos(angle) * mscale).float(), (torch.sin(angle) * mscale).float()
    t = -t if inverse else t
    x = x.float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        return torch.cat((torch.stack((a * c - b * t, b * c + a * t), -1).flatten(-2), x[..., rot:]), -1)
    a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    return torch.cat((a * c - b * t, b * c + a * t, x[..., rot:]), -1)


def _places(s):
    """For every new token: its sequence, its position, its page and its row in the page."""
    token = torch.arange(s["total"], device=CARD)
    seq = torch.searchsorted(s["cu"][1:].long(), token, right=True)
    position = s["lens"].long()[seq] - (s["cu"].long()[seq + 1] - token)
    return seq, position, s["table"].long()[seq, position // s["page"]], position % s["page"]


def _values(codes, params):
    """float32 values [..., d] of packed codes [..., d/2] and (step, low) [..., d/64, 2]."""
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float().unflatten(-1, (-1, 64))
    return (code * params[..., 0:1].float() + params[..., 1:2].float()).flatten(-2)


def _appended(s):
    rot, mscale = s["case"]["rot"], s["mscale"]
    seq, position, page, row = _places(s)
    angle = (position.double()[:, None] * s["freqs"])[:, None]
    q = _rotated(s["q"], angle, mscale, rot, s["interleaved"]).to(s["type"])
    k = _rotated(s["k"], angle, mscale, rot, s["interleaved"])
    if s["mean"] is not None:
        k = k - s["mean"]
    regions = _regions(s["cache"], s["page"], s["d"])
    for at, x in ((0, k), (1, s["v"].float())):
        code, par = _quantized(x)
        regions[at][page, :, row] = _packed(code)
        regions[2 + at][page, :, row] = par
    return q


def _gathered(s, rep=1):
    seq, position, page, row = _places(s)
    kc, vc, kp, vp = _regions(s["cache"], s["page"], s["d"])
    k, v = _values(kc[page, :, row], kp[page, :, row]), _values(vc[page, :, row], vp[page, :, row])
    if rep > 1:
        k, v = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    return k.to(s["type"]), v.to(s["type"])


def _attended(s, q):
    """Softmax attention of the new tokens' queries over their sequences' cached tokens, the
    last of them the new ones: query i of n sees keys up to length - n + i."""
    n, width, group = s["nseq"], s["new"], s["hq"] // s["hkv"]
    position = torch.arange(s["longest"], device=CARD)
    kc, vc, kp, vp = _regions(s["cache"], s["page"], s["d"])
    page, row = s["table"].long()[:, position // s["page"]], (position % s["page"]).expand(n, -1)
    k = _values(kc[page, :, row], kp[page, :, row]).transpose(1, 2)      # [n, hkv, keys, d]
    v = _values(vc[page, :, row], vp[page, :, row]).transpose(1, 2)
    count = (s["cu"][1:] - s["cu"][:-1]).long()
    i = torch.arange(width, device=CARD)
    there = i[None] < count[:, None]                                     # [n, width]
    token = torch.where(there, s["cu"][:-1].long()[:, None] + i, 0)
    qs = q.float()[token].unflatten(2, (s["hkv"], group)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    score = (qs @ k.transpose(-1, -2)) * (1.0 / math.sqrt(s["d"]))       # [n, hkv, group*width, keys]
    last = s["lens"].long()[:, None] - count[:, None] + i
    seen = (position <= last[..., None])[:, None, None].expand(-1, 1, group, -1, -1).flatten(2, 3)
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total == 0, 1.0, total)
    back = lambda x: x.unflatten(2, (group, width)).permute(0, 3, 1, 2, 4).flatten(2, 3)[there]  # noqa: E731
    lse = back(top + torch.log(total))[..., 0]
    return back(out).to(s["type"]), lse


def run(state):
    s = state
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "rope":
        angle = (s["positions"].double()[..., None] * s["freqs"])[:, None]
        args = (angle, s["mscale"], s["case"]["rot"], s["interleaved"], s["case"]["inverse"])
        return {"q": _rotated(s["q"], *args).to(s["type"]), "k": _rotated(s["k"], *args).to(s["type"])}
    if op == "append":
        q = _appended(s)
        k, v = _gathered(s)
        return {"q": q, "k": k, "v": v}
    if op == "gather":
        k, v = _gathered(s, s["rep"])
        return {"k": k, "v": v}
    q = _appended(s) if op == "step" else s["q"]
    out, lse = _attended(s, q)
    got = {"out": out}
    if s["lse"]:
        got["lse"] = lse
    if op == "step":
        got["q"] = q
    return got


def _run_own(s):
    import quantized_attention_03_b200 as sage
    op = s["op"]
    if op == "rope":
        q, k = sage.rope(s["q"], s["k"], s["freqs"], s["positions"], mscale=s["mscale"], interleaved=s["interleaved"],
                         inverse=s["case"]["inverse"])
        return {"q": q, "k": k}
    where = (s["cache"], s["table"], s["lens"], s["cu"])
    if op == "gather":
        k, v = sage.kv4_gather(*where, s["total"], s["d"], dtype=s["type"], rep=s["rep"])
        return {"k": k, "v": v}
    q = s["q"]
    if op in ("append", "step"):
        q = sage.kv4_append(*where, s["k"], s["v"], q, s["freqs"], mscale=s["mscale"], interleaved=s["interleaved"],
                            k_mean=s["mean"])
    if op == "append":
        k, v = sage.kv4_gather(*where, s["total"], s["d"], dtype=s["type"])
        return {"q": q, "k": k, "v": v}
    got = {}
    if s["lse"]:
        got["lse"] = torch.empty((s["total"], s["hq"]), dtype=torch.float32, device=CARD)
    got["out"] = sage.attn_kv4(q, *where, max_q=s["new"], lse=got.get("lse"))
    if op == "step":
        got["q"] = q
    return got


# ---------------------------------------------------------------------------- the work


def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "rope":
        elements = case["batch"] * case["new"] * (case["hq"] + hkv) * d
        return {"bytes": 4.0 * elements + 4.0 * case["batch"] * case["new"], "flops": 3.0 * elements}
    lens, count = (x.double() for x in _lengths(case, torch.arange(case["nseq"])))
    held, new = float(lens.sum()), float(count.sum())
    token4 = hkv * 2 * (d / 2 + 4 * (d // 64))     # a token's codes, steps and lows, keys and values
    if case["op"] == "gather":
        return {"bytes": held * (token4 + 4.0 * hkv * case["rep"] * d), "flops": held * hkv * d * 4.0}
    if case["op"] == "append":     # reads q, k, v; writes q, the cache, and k, v as read back
        values = new * (2 * case["hq"] + 4 * hkv) * d
        return {"bytes": 2.0 * values + 2 * new * token4, "flops": 20.0 * new * hkv * d}
    pairs = float((count * (lens - (count - 1) / 2)).sum())
    size = held * token4 + 2.0 * new * 2 * case["hq"] * d
    if case["op"] == "step":
        size += new * (2.0 * (2 * hkv + 2 * case["hq"]) * d + token4)
    return {"bytes": size, "flops": 4.0 * pairs * case["hq"] * d}


# ---------------------------------------------------------------- the formulas in 64 bits


def _turn64(x, positions, s, inverse):
    """Rotation by complex numbers: x [tokens, heads, d] in 64 bits, positions [tokens]."""
    rot = s["case"]["rot"]
    z = torch.polar(torch.full((), s["mscale"], dtype=torch.float64, device=CARD), positions.double()[:, None] * s["freqs"])
    z = (z.conj() if inverse else z)[:, None]
    part = x.double()[..., :rot]
    part = part.unflatten(-1, (rot // 2, 2)) if s["interleaved"] else part.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(part.contiguous()) * z)
    turned = turned if s["interleaved"] else turned.transpose(-1, -2)
    return torch.cat((turned.flatten(-2), x.double()[..., rot:]), -1)


def _group64(x):
    """What the 4-bit groups of x [tokens, heads, d] stand for, in 64 bits."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 64, 64)
    lo = g.min(-1, keepdim=True).values
    step = ((g.max(-1, keepdim=True).values - lo) / 15).half().double()
    low = lo.half().double()
    code = torch.nan_to_num((g - low) / step, nan=0.0, posinf=0.0, neginf=0.0).round().clamp(0, 15)
    return (low + code * step).reshape(x.shape)


def _tokens64(s, i):
    """The cached keys and values of sequence i in 64 bits, [tokens, heads, d]."""
    n, page, d, hkv = int(s["lens"][i]), s["page"], s["d"], s["hkv"]
    raw = s["cache"][s["table"][i, :(n + page - 1) // page].long()]
    size, got = page * d // 2, []
    for at in (0, 1):
        byte = raw[:, :, at * size:(at + 1) * size].reshape(-1, hkv, page, d // 2)
        code = torch.empty(byte.shape[:-1] + (d,), dtype=torch.float64, device=CARD)
        code[..., 0::2], code[..., 1::2] = byte % 16, byte // 16
        groups = d // 64 * 4
        par = raw[:, :, 2 * size + at * page * groups:][:, :, :page * groups].contiguous().view(torch.float16)
        par = par.reshape(-1, hkv, page, d // 64, 2).double().repeat_interleave(64, 3)
        got.append((par[..., 1] + code * par[..., 0]).transpose(1, 2).reshape(-1, hkv, d)[:n])
    return got


def exact(case, seed):
    s = prepare(case, seed)
    op, d, hkv = s["op"], s["d"], s["hkv"]
    if op == "rope":
        b, n = case["batch"], case["new"]
        flat = lambda x: x.transpose(1, 2).flatten(0, 1)  # noqa: E731
        back = lambda x: x.unflatten(0, (b, n)).transpose(1, 2)  # noqa: E731
        at = s["positions"].flatten()
        return {x: back(_turn64(flat(s[x]), at, s, case["inverse"])) for x in ("q", "k")}
    starts, lens = s["cu"].tolist(), s["lens"].tolist()
    count = [b - a for a, b in zip(starts, starts[1:])]
    got = {}
    if op in ("append", "step"):
        at = torch.cat([torch.arange(m - c, m, device=CARD) for m, c in zip(lens, count)])
        got["q"] = _turn64(s["q"], at, s, False)
        k = _turn64(s["k"], at, s, False)
        k, v = _group64(k if s["mean"] is None else k - s["mean"].double()), _group64(s["v"].double())
        if op == "append":
            return dict(got, k=k, v=v)
    if op == "gather":
        parts = [_tokens64(s, i) for i in range(s["nseq"])]
        return {x: torch.cat([p[at] for p in parts]).repeat_interleave(s["rep"], 1) for at, x in ((0, "k"), (1, "v"))}
    q = (got["q"].to(s["type"]) if op == "step" else s["q"]).double()
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=CARD)
    group = s["hq"] // hkv
    for i in range(s["nseq"]):
        if not count[i]:
            continue
        a, b = starts[i], starts[i + 1]
        keys, values = _tokens64(s, i)
        if op == "step":
            keys[lens[i] - count[i]:], values[lens[i] - count[i]:] = k[a:b], v[a:b]
        hidden = torch.arange(lens[i], device=CARD)[None] > torch.arange(lens[i] - count[i], lens[i], device=CARD)[:, None]
        for h in range(s["hq"]):
            x = (q[a:b, h] @ keys[:, h // group].T / math.sqrt(d)).masked_fill(hidden, -math.inf)
            out[a:b, h] = torch.softmax(x, -1) @ values[:, h // group]
            lse[a:b, h] = torch.logsumexp(x, -1)
    got["out"] = out
    if s["lse"]:
        got["lse"] = lse
    return got
