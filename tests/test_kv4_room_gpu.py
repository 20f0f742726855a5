"""Attention over the paged 4-bit cache held to the limits of kv4_ref.room: per row and 64 channels,
what the arithmetic allows (tests/test_kv4_room_cpu.py shows what those limits catch)."""
import math

import pytest
import torch

import kv4_ref as ref
import quantized_attention_03_b200 as sage
from test_rope_kv4_gpu import BF16, F16, World, ok

pytestmark = pytest.mark.gpu


def check(w, q, out, lse=None, causal=True, sm_scale=None):
    for s in range(len(w.lens)):
        a, b = int(w.cu[s]), int(w.cu[s + 1])
        if a == b:
            continue
        if w.lens[s] == 0:
            assert (out[a:b] == 0).all() and (lse is None or (lse[a:b] == -math.inf).all())
            continue
        k, v = w.tokens(s)
        (key_span, value_span), step = ref.spans(w.cache, w.page, w.d, w.table[s], w.lens[s])
        want, limit, wlse, llse = ref.room(q[a:b], k, v, key_span, value_span, step, out.dtype, causal, sm_scale)
        bad, far = ref.misses(out[a:b].cpu(), want, limit)
        assert bad == 0, f"sequence {s}: {bad} of {limit.numel()} groups off, up to {far:.3g} times the limit"
        if lse is not None:
            assert ((lse[a:b].cpu().double() - wlse).abs() <= llse).all(), s


def attend(w, q, max_q, **kw):
    lse = torch.empty((w.total, q.shape[1]), device="cuda")
    out = sage.attn_kv4(q.cuda(), w.cache.cuda(), *w.where(), max_q, lse=lse, **kw)
    ok()
    return out, lse


CASES = [
    # lens, news, Hq, Hkv, d, page, type, causal: rows of a key head from 1 to 40
    ([1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65], [1] * 11, 8, 8, 128, 16, F16, True),
    ([500, 1, 4097, 0, 260], [1, 1, 1, 1, 1], 8, 1, 128, 64, F16, True),
    ([500, 1, 4097, 96], [1, 0, 1, 1], 24, 8, 64, 32, F16, True),
    ([300, 3, 1030, 0, 77], [5, 3, 16, 0, 1], 6, 2, 128, 16, F16, True),
    ([300, 3, 1030, 2, 77], [5, 3, 16, 2, 1], 4, 1, 64, 256, BF16, True),
    ([300, 3, 1030, 0, 77], [5, 3, 16, 0, 1], 6, 2, 128, 16, F16, False),
    ([20000, 4999], [1, 1], 32, 4, 128, 64, F16, True),
    ([9000], [1], 4, 4, 64, 128, F16, True),
    ([640], [16], 40, 1, 64, 64, F16, True),
    ([900, 411], [2, 2], 16, 2, 128, 32, F16, True),
]


@pytest.mark.parametrize("lens,news,Hq,Hkv,d,page,dt,causal", CASES)
def test_attention(lens, news, Hq, Hkv, d, page, dt, causal):
    w = World(lens, news, Hkv, d, page, seed=31 + len(lens))
    w.fill(offset=0.5)
    q = torch.randn((w.total, Hq, d), generator=w.g).to(dt)
    check(w, q, *attend(w, q, max(news), causal=causal), causal=causal)


# query heads of a key head, drafted tokens, sequences: 16 rows in a pass and at least 148 segments
# of them, so that warps work alone; some sequences long, whose tiles several warps share
MANY = [(16, 1, 26), (8, 2, 26), (6, 5, 26), (4, 16, 10)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,new,nseq", MANY)
def test_sixteen_rows_of_many_segments(group, new, nseq, d):
    g = torch.Generator().manual_seed(group * new)
    lens = torch.randint(new, 700, (nseq,), generator=g).tolist()
    lens[3], lens[nseq - 1] = 5003, 2500
    w = World(lens, [new] * nseq, 8, d, 32, seed=33)
    w.fill()
    q = torch.randn((w.total, 8 * group, d), generator=w.g).to(F16)
    check(w, q, *attend(w, q, new))


@pytest.mark.parametrize("d", [64, 128])
def test_few_drafts_among_sequences_of_many(d):
    # row blocks of 16, 30 rows at most: sequences with 6, 12, .. 30 rows, and none
    g = torch.Generator().manual_seed(d)
    lens = torch.randint(5, 1500, (30,), generator=g).tolist()
    news = [i % 6 for i in range(30)]
    w = World(lens, news, 8, d, 16, seed=34)
    w.fill()
    q = torch.randn((w.total, 48, d), generator=w.g).to(F16)
    check(w, q, *attend(w, q, 5))


@pytest.mark.parametrize("Hq,Hkv,news", [(8, 2, [1, 1, 1, 1]), (4, 4, [1, 0, 16, 3])])
def test_most_queries_left_to_the_call(Hq, Hkv, news):
    w = World([900, 40, 333, 5], news, Hkv, 128, 32, seed=35)
    w.fill()
    q = torch.randn((w.total, Hq, 128), generator=w.g).to(F16)
    check(w, q, *attend(w, q, None))


@pytest.mark.parametrize("ratio", [1e3, 1e6, 1e8])
@pytest.mark.parametrize("Hq", [2, 8, 16])
def test_groups_of_channels_of_very_different_size(Hq, ratio):
    # values of one half of the channels `ratio` times smaller than those of the other
    w = World([700, 90, 2100], [1, 1, 1], 2, 128, 32, seed=36)
    for s, n in enumerate(w.lens):
        k, v = (torch.randn((n, 2, 128), generator=w.g) for _ in range(2))
        v[:, 0, :64] *= 1e3 / ratio
        v[:, 0, 64:] *= 1e3
        v[:, 1, :64] *= 1e3
        v[:, 1, 64:] *= 1e3 / ratio
        w.put(s, torch.arange(n), k, v)
    q = torch.randn((3, Hq, 128), generator=w.g).to(BF16)
    check(w, q, *attend(w, q, 1))


@pytest.mark.parametrize("d", [64, 128])
def test_tokens_of_very_different_size(d):
    w = World([1100, 333], [2, 2], 2, d, 64, seed=37)
    for s, n in enumerate(w.lens):
        size = 10.0 ** torch.randint(-4, 3, (n, 1, 1), generator=w.g)
        w.put(s, torch.arange(n), torch.randn((n, 2, d), generator=w.g), torch.randn((n, 2, d), generator=w.g) * size)
    q = torch.randn((w.total, 8, d), generator=w.g).to(BF16)
    check(w, q, *attend(w, q, 2))


@pytest.mark.parametrize("d,Hq", [(64, 8), (128, 2), (128, 32)])
def test_sharp_scores_and_queries_of_very_different_size(d, Hq):
    w = World([2100, 333], [2, 2], 2, d, 64, seed=38)
    w.fill(offset=1.0)
    q = torch.randn((w.total, Hq, d), generator=w.g) * 10.0 ** torch.randint(-3, 2, (w.total, Hq, 1), generator=w.g)
    q = q.to(F16)
    check(w, q, *attend(w, q, 2, sm_scale=0.5), sm_scale=0.5)


@pytest.mark.parametrize("nseq,Hq,new", [(3, 4, 1), (3, 32, 5), (90, 4, 1), (90, 16, 3), (90, 32, 5)])
def test_the_output_over_the_queries(nseq, Hq, new):
    # a row is read by the one segment that writes it, in CTAs and in warps that work alone
    g = torch.Generator().manual_seed(nseq + Hq)
    lens = torch.randint(new, 300, (nseq,), generator=g).tolist()
    lens[0] = 3000
    w = World(lens, [new] * nseq, 2, 128, 16, seed=39)
    w.fill()
    q = torch.randn((w.total, Hq, 128), generator=w.g).to(F16).cuda()
    cache, where = w.cache.cuda(), w.where()
    want = sage.attn_kv4(q, cache, *where, new)
    for _ in range(5):
        x = q.clone()
        assert sage.attn_kv4(x, cache, *where, new, out=x) is x
        assert torch.equal(x, want)
    ok()
