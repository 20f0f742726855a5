"""The limits that the attention's tests hold outputs to (kv4_ref.room): mistakes planted in a plain
attention over the 4-bit cache have to pass them, exact results must not."""
import math

import pytest
import torch

import kv4_ref as ref

F16, BF16 = torch.float16, torch.bfloat16


def cached(n, H, d, g, scale=1.0):
    """Keys and values [n, H, d] as a 4-bit cache holds them, with their params."""
    out = []
    for x in (torch.randn((n, H, d), generator=g) + 0.5, torch.randn((n, H, d), generator=g) * scale):
        c, p = ref.quantize(x)
        c, p = c.double().unflatten(-1, (-1, 64)), p.double()
        out.append(((c * p[..., :1] + p[..., 1:]).flatten(-2), p[..., 1].abs() + 15 * p[..., 0], p))
    (k, key_span, _), (v, value_span, p) = out
    return k, v, key_span, value_span, p


def weights(q, k, sm):
    s = torch.einsum("ihd,jhd->ihj", q.double(), k.repeat_interleave(q.shape[1] // k.shape[1], 1)) * sm
    m = s.amax(-1, keepdim=True)
    return torch.exp(s - m)


CASES = [(90, 1, 128, 1.0), (700, 2, 64, 1.0), (1100, 1, 128, 1.0), (4097, 1, 128, 1.0), (300, 2, 64, 4.0)]


@pytest.mark.parametrize("n,H,d,sharp", CASES)
def test_the_limits_show_planted_mistakes(n, H, d, sharp):
    g = torch.Generator().manual_seed(n + d)
    k, v, key_span, value_span, p = cached(n, H, d, g)
    q = torch.randn((1, 4 * H, d), generator=g).to(F16)
    sm = sharp / math.sqrt(d)
    out, limit, _, _ = ref.room(q, k, v, key_span, value_span, p[..., 0], F16, True, sm)
    assert ref.misses(out.to(F16), out, limit)[0] == 0
    w = weights(q, k, sm)
    vv, step, mid = (x.repeat_interleave(4, 1) for x in (v, p[..., 0], p[..., 1] + 8 * p[..., 0]))
    code = ((vv.unflatten(-1, (-1, 64)) - mid[..., None]) / step[..., None]).round()
    total = w.sum(-1, keepdim=True)

    def result(weight, of=slice(None), bits=None):
        t = weight[..., None] * step[None].transpose(1, 2)     # [i, h, j, group]
        if bits is not None:
            t = torch.ldexp(torch.round(torch.ldexp(torch.frexp(t)[0], torch.tensor(bits))), torch.frexp(t)[1] - bits)
        a = torch.einsum("ihjg,jhgc->ihgc", t[:, :, of], code[of])
        b = torch.einsum("ihj,jhg->ihg", weight[..., of], mid[of])
        return ((a + b[..., None]).flatten(-2) / total).to(F16)

    # as the kernel has it (two terms of fp16), and what must be seen: one term alone (2^-11, but for
    # scores so sharp that they may be that far off themselves)
    assert ref.misses(result(w, bits=21), out, limit)[0] == 0
    assert sharp > 1 or ref.misses(result(w, bits=11), out, limit)[0] > 0
    # 16 keys forgotten, a half of the keys weighted 1% wrong, nothing written
    assert ref.misses(result(w, torch.arange(n) // 16 != n // 32), out, limit)[0] > 0
    half = torch.where(torch.arange(n) < n // 2, 1.01, 1.0).double()
    assert ref.misses(result(w * half), out, limit)[0] > 0
    assert ref.misses(torch.zeros_like(out), out, limit)[0] == limit.numel()


def test_the_limits_show_a_group_that_lost_its_bits_to_another():
    # the second group's values a millionth of the first's; one scale for both ends the weights'
    # products at 2^-28 of the first's step
    g = torch.Generator().manual_seed(3)
    scale = torch.cat((torch.full((64,), 100.0), torch.full((64,), 1e-4)))
    k, v, key_span, value_span, p = cached(700, 1, 128, g, scale)
    q = torch.randn((2, 4, 128), generator=g).to(BF16)
    args = (q, k, v, key_span, value_span, p[..., 0], BF16)
    out, limit, _, _ = ref.room(*args, causal=False)
    w = weights(q, k, 1 / math.sqrt(128))
    step, mid = p[:, 0, 1, 0], p[:, 0, 1, 1] + 8 * p[:, 0, 1, 0]
    code = ((v[:, 0, 64:] - mid[:, None]) / step[:, None]).round()
    quantum = 2.0 ** -27 * p[:, 0, 0, 0].max()
    t = torch.round(w * step / quantum) * quantum
    got = out.clone()
    got[..., 64:] = (torch.einsum("ihj,jc->ihc", t, code) + torch.einsum("ihj,j->ih", w, mid)[..., None]) / w.sum(-1, keepdim=True)
    assert ref.misses(out.to(BF16), out, limit)[0] == 0
    far = (got.to(BF16).double() - out).unflatten(-1, (-1, 64)).norm(dim=-1) / limit
    assert (far[..., 0] <= 1).all() and (far[..., 1] > 1).all()
