"""Rotary positions and the paged 4-bit cache on the GPU, against 64-bit plain forms.

Tolerances. A rounding to the output's type is off by at most half a step, 2^-11 (fp16) or
2^-8 (bf16) of the value. The rotation's 32-bit steps add at most 4 2^-24 (|x0| + |x1|) m: a
sine or cosine rounded once, a product, a sum. Codes and params are defined in 32-bit steps
and have to be equal. Attention's steps: a score is a sum over d channels in at most 20
accumulations; codes enter as fp16 subnormals, whose products are aligned with up to 10 leading
zeros, so each is good to 2^-24 + 10 / 4 bits of the terms' absolute sum and the score to less
than 2^-18 of it; probabilities follow their scores, and carry 2^-21 of their own (two fp16 terms, the
exponential); summing n keys in 32 bits adds at most 2^-23 per 16 keys.
"""
import math

import pytest
import torch

import kv4_ref as ref
import quantized_attention_03_b200 as sage

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
TINY = {F16: 2.0 ** -25, BF16: 0.0}       # half a step of the subnormals


def ok():
    code = sage.sage_get_device_status()
    assert code == sage.SAGE_OK, sage.status_string(code)


def near(got, want, slack, what=""):
    """|got - want| within the rounding of got's type and `slack` (a tensor or number)."""
    got64, limit = got.cpu().double(), slack + HALF(got.dtype) * want.abs() + TINY.get(got.dtype, 0.0)
    off = (got64 - want).abs()
    bad = ~(off <= limit * (1 + 2.0 ** -7))
    bad &= ~(got64.isnan() & want.isnan())
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / limit)[bad].max()):.3g} times"


def HALF(dtype):
    return ref.HALF_STEP.get(dtype, 2.0 ** -24)


# ------------------------------------------------------------------------------ rope


ROPE = [
    # B, Hq, Hk, N, d, rot, interleaved, inverse, type
    (1, 1, 0, 1, 64, 64, False, False, F16),
    (2, 4, 2, 33, 128, 128, False, False, F16),
    (1, 3, 3, 700, 128, 64, True, False, BF16),
    (3, 32, 8, 257, 128, 128, True, True, F16),
    (2, 5, 1, 129, 64, 16, False, True, BF16),
    (1, 2, 2, 5, 128, 112, False, False, F16),
]


@pytest.mark.parametrize("B,Hq,Hk,N,d,rot,inter,inv,dt", ROPE)
def test_rope(B, Hq, Hk, N, d, rot, inter, inv, dt):
    g = torch.Generator().manual_seed(B * N + rot)
    q = torch.randn((B, Hq, N, d), generator=g).to(dt)
    k = torch.randn((B, Hk, N, d), generator=g).to(dt) if Hk else None
    pos = torch.randint(0, 1 << 20, (B, N), generator=g, dtype=torch.int32)
    freqs, m = sage.rope_freqs(rot, scaling="parts", factor=8.0, original_len=4096)
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    qo, ko = sage.rope(dev(q), dev(k), freqs, pos.cuda(), m, inter, inv)
    ok()
    for x, y in ((q, qo), (k, ko)):
        if x is None:
            assert y is None
            continue
        flat = x.transpose(1, 2).flatten(0, 1)
        want = ref.rotate(flat, pos.flatten(), freqs.cpu(), m, inter, inv)
        want = want.unflatten(0, (B, N)).transpose(1, 2)
        near(y, want, 4 * 2.0 ** -24 * 2 * m * x.double().abs().amax())
        assert torch.equal(y.cpu()[..., rot:], x[..., rot:])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 48)])
def test_rope_is_the_defined_arithmetic(d, rot, inter):
    # sines and cosines rounded once to fp32, then products and sums each rounded: bit for bit
    g = torch.Generator().manual_seed(rot)
    x = torch.randn((640, 5, d), generator=g).to(F16)
    pos = torch.randint(0, 100000, (640,), generator=g, dtype=torch.int32)
    freqs, m = sage.rope_freqs(rot, scaling="parts", factor=8.0, original_len=4096)
    got, _ = sage.rope(x.cuda(), None, freqs, pos.cuda(), m, inter)
    ok()
    assert torch.equal(got.cpu(), ref.rotate(x, pos, freqs.cpu(), m, inter, dtype=torch.float32).to(F16))


def test_rope_views_in_place_and_packed():
    T, Hq, Hk, d = 77, 6, 2, 128
    fused = torch.randn((T, Hq + 2 * Hk, d), device="cuda").to(F16)
    q, k = fused[:, :Hq], fused[:, Hq:Hq + Hk]
    freqs, m = sage.rope_freqs(d)
    pos = torch.randint(0, 5000, (T,), dtype=torch.int32, device="cuda")
    want_q, want_k = sage.rope(q.contiguous(), k.contiguous(), freqs, pos)
    v = fused[:, Hq + Hk:].clone()
    got_q, got_k = sage.rope(q, k, freqs, pos)
    assert torch.equal(got_q, want_q) and torch.equal(got_k, want_k)
    r = sage.rope(q, k, freqs, pos, q_out=q, k_out=k)       # in place, inside the projection
    assert r[0] is q and torch.equal(q, want_q) and torch.equal(k, want_k)
    assert torch.equal(fused[:, Hq + Hk:], v)
    # dense and packed agree; positions default to 0 .. N-1, one row of them serves all
    x = torch.randn((3, 4, 50, d), device="cuda").to(BF16)
    a, _ = sage.rope(x, None, freqs)
    b, _ = sage.rope(x, None, freqs, torch.arange(50, dtype=torch.int32, device="cuda"))
    c, _ = sage.rope(x[1].transpose(0, 1), None, freqs)
    assert torch.equal(a, b) and torch.equal(a[1].transpose(0, 1), c)
    ok()


@pytest.mark.parametrize("inter", [False, True])
def test_rope_inverse_is_the_gradient(inter):
    # <R x, y> = <x, R^T y>, with the formula's R, and differences along a direction
    T, H, d = 9, 3, 64
    g = torch.Generator().manual_seed(4)
    x, y = (torch.randn((T, H, d), generator=g, dtype=torch.float64) for _ in range(2))
    pos = torch.arange(T, dtype=torch.int32) * 1000
    freqs, m = sage.rope_freqs(32, scaling="parts", factor=4.0, original_len=2048)
    xr = x.clone().requires_grad_()
    ref.rotate(xr, pos, freqs.cpu(), m, inter).backward(y)
    grad, _ = sage.rope(y.to(F16).cuda(), None, freqs, pos.cuda(), m, inter, True)
    near(grad, ref.rotate(y.to(F16), pos, freqs.cpu(), m, inter, True), 2.0 ** -20 * y.abs().amax())
    near(grad, xr.grad, 2.0 ** -10 * m * 2 * y.abs().amax())   # y itself was rounded
    h = 2.0 ** -3
    step = lambda s: ref.rotate((x + s * h * y), pos, freqs.cpu(), m, inter)  # noqa: E731
    along = ((step(1) - step(-1)) / (2 * h) * y).sum()
    assert abs(float((xr.grad * y).sum() - along)) < 1e-9 * float(along.abs() + 1)
    ok()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("inter,inv,rot", [(False, False, 128), (True, True, 64)])
def test_rope_in_autograd(packed, inter, inv, rot):
    g = torch.Generator().manual_seed(rot + packed)
    rnd = lambda *shape: torch.randn(shape, generator=g).to(F16).cuda()  # noqa: E731
    shape = (lambda h: (40, h, 128)) if packed else (lambda h: (2, h, 20, 128))
    q, k = rnd(*shape(6)).requires_grad_(), rnd(*shape(2)).requires_grad_()
    gq, gk = rnd(*shape(6)), rnd(*shape(2))
    pos = torch.randint(0, 9000, (40,) if packed else (2, 20), generator=g, dtype=torch.int32).cuda()
    freqs, m = sage.rope_freqs(rot, scaling="parts", factor=8.0, original_len=512)
    how = (freqs, pos, m, inter)
    plain = sage.rope(q.detach(), k.detach(), *how, inv)
    back = sage.rope(gq, gk, *how, not inv)
    assert not plain[0].requires_grad and not plain[1].requires_grad
    out = sage.rope(q, k, *how, inv)
    assert out[0].requires_grad and out[1].requires_grad
    assert torch.equal(out[0], plain[0]) and torch.equal(out[1], plain[1])
    got = torch.autograd.grad(out, (q, k), (gq, gk), retain_graph=True)
    assert torch.equal(got[0], back[0]) and torch.equal(got[1], back[1])
    # one of the two results used, and one of the two inputs differentiated
    assert torch.equal(torch.autograd.grad(out[0], q, gq, retain_graph=True)[0], back[0])
    assert torch.equal(torch.autograd.grad(out[1], k, gk, retain_graph=True)[0], back[1])
    assert torch.autograd.grad(out[1], q, gk, allow_unused=True)[0] is None
    qo, ko = sage.rope(q.detach(), k, *how, inv)
    assert not qo.requires_grad and torch.equal(qo, plain[0])
    assert torch.equal(torch.autograd.grad(ko, k, gk)[0], back[1])
    qo, ko = sage.rope(q, None, *how, inv)
    assert ko is None and torch.equal(torch.autograd.grad(qo, q, gq)[0], back[0])
    with torch.no_grad():
        assert not sage.rope(q, k, *how, inv)[0].requires_grad
    ok()


def test_rope_gradients_in_any_layout_and_of_views():
    # an expanded gradient (of a sum), a transposed one, one off its alignment; a key head that
    # all query heads share, and projections of one buffer
    g = torch.Generator().manual_seed(5)
    fused = torch.randn((24, 8, 64), generator=g).to(F16).cuda().requires_grad_()
    pos = torch.arange(24, dtype=torch.int32).cuda()
    freqs, _ = sage.rope_freqs(64)
    one = fused[:, 6:7]
    q, k = sage.rope(fused[:, :6], one.expand(24, 6, 64), freqs, pos)
    want = lambda y: sage.rope(y.clone(memory_format=torch.contiguous_format), None, freqs, pos, inverse=True)[0]  # noqa: E731
    ones = torch.ones((24, 6, 64), dtype=F16, device="cuda")
    grad, = torch.autograd.grad(q.sum() + k.sum(), fused, retain_graph=True)
    assert torch.equal(grad[:, :6], want(ones)) and (grad[:, 7] == 0).all()
    near(grad[:, 6], want(ones).double().sum(1).cpu(), 6 * 2.0 ** -10 * 6)
    odd = torch.randn(24 * 6 * 64 + 1, generator=g).to(F16).cuda()[1:].view(24, 6, 64)
    turned = torch.randn((64, 6, 24), generator=g).to(F16).cuda().permute(2, 1, 0)
    for y in (odd, turned):
        grad, = torch.autograd.grad(q, fused, y, retain_graph=True)
        assert torch.equal(grad[:, :6], want(y))
    ok()


def test_rope_gradient_twice_on_a_stream_and_after_its_inputs_changed():
    g = torch.Generator().manual_seed(6)
    x, y = (torch.randn((12, 2, 64), generator=g).to(F16).cuda() for _ in range(2))
    freqs, m = sage.rope_freqs(64, scaling="parts", factor=4.0, original_len=2048)
    pos = torch.arange(12, dtype=torch.int32).cuda()
    x.requires_grad_()
    # the gradient is linear in y: its gradient towards y is the rotation itself
    y.requires_grad_()
    out, _ = sage.rope(x, None, freqs, pos, m)
    grad, = torch.autograd.grad(out, x, y, create_graph=True)
    again, = torch.autograd.grad(grad, y, x.detach())
    assert torch.equal(again, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        leaf = x.detach().requires_grad_()
        there, _ = sage.rope(leaf, None, freqs, pos, m, stream=stream)
        got, = torch.autograd.grad(there, leaf, y.detach())
        torch.cuda.synchronize()
        assert torch.equal(there, out) and torch.equal(got, grad)
    # positions that were moved on since are noticed, as autograd does
    pos.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(out, x, y)
    ok()


def test_autograd_sees_that_outputs_are_written_over():
    # each output once where a product has saved it: its gradient cannot be had any more
    w = World([9, 30], [1, 1], 2, 64, 16, seed=19)
    w.fill()
    cache, where = w.cache.cuda(), w.where()
    freqs, _ = sage.rope_freqs(64)
    q, k = (torch.randn((2, h, 64), generator=w.g).to(F16).cuda() for h in (4, 2))
    pos = torch.arange(2, dtype=torch.int32).cuda()
    lse = torch.zeros((2, 4), device="cuda")
    for name, out, call in (
            ("q_out", q, lambda x: sage.rope(x, None, freqs, pos, q_out=x)),
            ("k_out", k, lambda x: sage.rope(q, x, freqs, pos, k_out=x)),
            ("append", q, lambda x: sage.kv4_append(cache, *where, k, k, x, freqs, q_out=x)),
            ("gather k", k, lambda x: sage.kv4_gather(cache, *where, 2, 64, k_out=x)),
            ("gather v", k, lambda x: sage.kv4_gather(cache, *where, 2, 64, v_out=x)),
            ("attention", q, lambda x: sage.attn_kv4(q, cache, *where, 1, out=x)),
            ("lse", lse, lambda x: sage.attn_kv4(q, cache, *where, 1, lse=x))):
        saved = out.clone()
        leaf = torch.ones_like(saved, requires_grad=True)
        product = leaf * saved
        call(saved)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            product.sum().backward()
        with torch.inference_mode():                    # tensors without versions
            call(out.clone())
    ok()


def test_rope_gradient_in_a_captured_graph():
    g = torch.Generator().manual_seed(7)
    x, y = (torch.randn((33, 4, 128), generator=g).to(BF16).cuda() for _ in range(2))
    freqs, _ = sage.rope_freqs(128)
    pos = torch.arange(33, dtype=torch.int32).cuda()

    def step():
        leaf = x.detach().requires_grad_()
        out, _ = sage.rope(leaf, None, freqs, pos)
        return out, torch.autograd.grad(out, leaf, y)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, grad = step()
    for _ in range(2):
        x.copy_(torch.randn(x.shape, generator=g))
        y.copy_(torch.randn(y.shape, generator=g))
        graph.replay()
        assert torch.equal(out, sage.rope(x, None, freqs, pos)[0])
        assert torch.equal(grad, sage.rope(y, None, freqs, pos, inverse=True)[0])
    ok()


def test_rope_far_positions():
    # 2^30 turns the fastest pair 1.7e8 times; a 32-bit angle would be off by 64
    d = 64
    pos = torch.tensor([0, 1, 1 << 24, (1 << 30) + 7, 2 ** 31 - 1], dtype=torch.int32)
    x = torch.randn((5, 2, d), generator=torch.Generator().manual_seed(2)).to(F16)
    freqs, _ = sage.rope_freqs(d)
    got, _ = sage.rope(x.cuda(), None, freqs, pos.cuda())
    near(got, ref.rotate(x, pos, freqs.cpu()), 4 * 2.0 ** -24 * 2 * x.double().abs().amax())
    ok()


# ------------------------------------------------------------------- cache: a small world


class World:
    """Sequences with their lengths and numbers of new tokens, a cache whose bytes are all 0xFF
    (params NaN) until written, and pages in random order."""

    def __init__(self, lens, news, Hkv, d, page, seed=0, spare=2, extra_width=1):
        g = torch.Generator().manual_seed(seed)
        self.g, self.lens, self.news, self.d, self.page, self.Hkv = g, lens, news, d, page, Hkv
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=g).tolist()
        width = max(need + [1]) + extra_width
        self.table = torch.full((len(lens), width), -1, dtype=torch.int32)
        for s, n in enumerate(need):
            self.table[s, :n] = torch.tensor(order[:n], dtype=torch.int32)
            order = order[n:]
        self.cache = torch.full((self.pages, Hkv, sage.sage_kv4_page_bytes(page, d)), 255, dtype=torch.uint8)
        self.cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
        self.cu[1:] = torch.cumsum(torch.tensor(news), 0)
        self.total = int(self.cu[-1])

    def where(self, cu=True):
        return [x.cuda() for x in (self.table, torch.tensor(self.lens, dtype=torch.int32))] + [
            self.cu.cuda() if cu else None]

    def positions(self):
        return torch.cat([torch.arange(n - c, n) for n, c in zip(self.lens, self.news)] + [torch.arange(0)])

    def put(self, s, positions, k, v):
        """Quantizes k, v [n, H, d] (fp32) into the CPU cache at positions of sequence s."""
        codes, params = ref.regions(self.cache, self.page, self.d)
        ids, rows = self.table[s].long()[positions // self.page], positions % self.page
        for x, y in ((0, k), (1, v)):
            c, p = ref.quantize(y)
            codes[ids, :, x, rows] = c[..., 0::2] | (c[..., 1::2] << 4)
            params[ids, :, x, rows] = p

    def fill(self, scale=1.0, offset=0.0):
        """Random tokens everywhere a sequence has some."""
        for s, n in enumerate(self.lens):
            if n:
                k, v = (torch.randn((n, self.Hkv, self.d), generator=self.g) * scale for _ in range(2))
                self.put(s, torch.arange(n), k + offset, v)

    def tokens(self, s, n=None, dtype=torch.float64):
        return ref.tokens(self.cache, self.page, self.d, self.table[s], self.lens[s] if n is None else n, dtype)


WORLDS = [
    # lens, news, Hq, Hkv, d, page, type
    ([1], [1], 1, 1, 64, 16, F16),
    ([16, 17, 31, 33, 1, 300], [1, 1, 1, 1, 1, 1], 8, 2, 128, 16, BF16),
    ([130, 64, 5], [130, 3, 0], 6, 6, 128, 64, F16),
    ([257, 256, 0, 700], [257, 255, 0, 1], 4, 1, 64, 256, F16),
    ([40, 41], [13, 41], 3, 3, 64, 32, BF16),
    ([1100, 900, 3], [1100, 20, 3], 10, 5, 128, 128, BF16),
]


@pytest.mark.parametrize("rotary", ["none", "half", "part", "inter"])
@pytest.mark.parametrize("lens,news,Hq,Hkv,d,page,dt", WORLDS)
def test_append_writes_the_defined_bytes(lens, news, Hq, Hkv, d, page, dt, rotary):
    w = World(lens, news, Hkv, d, page, seed=len(lens) + d)
    fused = torch.randn((w.total + 3, Hq + 2 * Hkv, d), generator=w.g)
    fused[..., Hq:, 3] += 5.0
    fused[0, Hq] = 0.25                                # a constant key: step 0
    fused = fused.to(dt)
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    mean = torch.randn((Hkv, d), generator=w.g) if rotary in ("half", "inter") else None
    freqs, m, inter = None, 1.0, rotary == "inter"
    if rotary != "none":
        freqs, m = sage.rope_freqs(d if rotary == "half" else d // 2, scaling="parts", factor=4.0, original_len=512)
    cache = w.cache.cuda()
    f = fused.cuda()
    qo = torch.full((w.total + 3, Hq, d), 7.0, dtype=dt, device="cuda")
    table, kv_lens, cu = w.where()
    # three rows of padding behind the last sequence: not read, not written
    sage.kv4_append(cache, table, kv_lens, cu, f[:, Hq:Hq + Hkv], f[:, Hq + Hkv:], f[:, :Hq], freqs, m, inter,
                    None if mean is None else mean.cuda(), qo)
    ok()
    pos, T = w.positions(), w.total
    k32, q64 = k[:T].float(), q[:T].double()
    if freqs is not None:
        k32 = ref.rotate(k[:T], pos, freqs.cpu(), m, inter, dtype=torch.float32)
        q64 = ref.rotate(q[:T], pos, freqs.cpu(), m, inter)
    if mean is not None:
        k32 = k32 - mean
    for s in range(len(lens)):
        a, b = int(w.cu[s]), int(w.cu[s + 1])
        w.put(s, pos[a:b], k32[a:b], v[a:b].float())
    assert torch.equal(cache.cpu(), w.cache)           # untouched bytes are still 0xFF
    near(qo[:T], q64, 4 * 2.0 ** -24 * 2 * m * q.double().abs().amax(), "q")
    assert (qo[T:] == 7.0).all()


@pytest.mark.parametrize("rep", [1, 3])
@pytest.mark.parametrize("lens,news,Hq,Hkv,d,page,dt", WORLDS)
def test_gather(lens, news, Hq, Hkv, d, page, dt, rep):
    w = World(lens, news, Hkv, d, page, seed=7)
    w.fill(scale=3.0, offset=1.0)
    table, kv_lens, cu = w.where()
    for all_tokens in (False, True):
        if all_tokens:
            cu = torch.cumsum(torch.tensor([0] + lens), 0).to(torch.int32).cuda()
        T = int(cu[-1])
        ko, vo = (torch.full((T + 2, Hkv * rep, d), 9.0, dtype=dt, device="cuda") for _ in range(2))
        sage.kv4_gather(w.cache.cuda(), table, kv_lens, cu, T + 2, d, dt, rep, ko, vo)
        ok()
        for x, out in ((0, ko), (1, vo)):
            want = torch.cat([w.tokens(s)[x][n - (n if all_tokens else c):] for s, (n, c) in enumerate(zip(lens, news))])
            near(out[:T], want.repeat_interleave(rep, 1), 2.0 ** -24 * want.repeat_interleave(rep, 1).abs())
            assert (out[T:] == 9.0).all()


def test_append_rotates_queries_in_place():
    w = World([30, 900], [30, 700], 2, 64, 32, seed=1)
    fused = torch.randn((w.total, 8, 64), generator=w.g).to(BF16).cuda()
    freqs, m = sage.rope_freqs(64)
    where = w.where()
    a, b = w.cache.cuda(), w.cache.cuda()
    want = sage.kv4_append(a, *where, fused[:, 4:6], fused[:, 6:], fused[:, :4], freqs, m)
    kv = fused[:, 4:].clone()
    got = sage.kv4_append(b, *where, fused[:, 4:6], fused[:, 6:], fused[:, :4], freqs, m, q_out=fused[:, :4])
    ok()
    assert torch.equal(got, want) and torch.equal(fused[:, :4], want)
    assert torch.equal(a, b) and torch.equal(fused[:, 4:], kv)


# ------------------------------------------------------------------------- attention


def check_attn(w, q, out, lse, causal=True, sm_scale=None):
    Hq, keys = q.shape[1], max(w.lens)
    for s in range(len(w.lens)):
        a, b = int(w.cu[s]), int(w.cu[s + 1])
        if a == b:
            continue
        k, v = w.tokens(s)
        want, wlse, big, mass = ref.attend(q[a:b].double(), k, v, causal, sm_scale)
        # the key terms' and value terms' own sizes: |low| + 15 step bounds both
        kb, vb = (x.abs().amax() if x.numel() else torch.zeros(()) for x in (k, v))
        err = 2.0 ** -18 * (q[a:b].double().abs().sum(-1) * 2 * kb * (sm_scale or 1 / math.sqrt(w.d)) + 1)
        slack = ((2 * err + 2.0 ** -20 + keys / 16 * 2.0 ** -23) * 2 * vb)[..., None]
        near(out[a:b], want, slack, f"sequence {s}")
        if lse is not None:
            got = lse[a:b].cpu().double()
            dead = wlse == -math.inf
            assert (got[dead] == -math.inf).all()
            assert ((got - wlse)[~dead].abs() <= (err + 2.0 ** -20 + 2.0 ** -22 * wlse.abs())[~dead]).all()


ATTN = [
    # lens, news, Hq, Hkv, d, page, type, causal
    ([1], [1], 1, 1, 64, 16, F16, True),
    ([1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65], [1] * 11, 8, 8, 128, 16, F16, True),
    ([500, 1, 4097, 0, 260], [1, 1, 1, 1, 1], 8, 1, 128, 64, BF16, True),
    ([500, 1, 4097, 96], [1, 0, 1, 1], 24, 8, 64, 32, F16, True),
    ([300, 4, 1030, 9, 77], [3, 4, 2, 0, 1], 4, 2, 128, 128, F16, True),
    ([300, 3, 1030, 2, 77], [5, 7, 16, 2, 1], 4, 1, 64, 256, BF16, True),
    ([300, 3, 1030, 0, 77], [5, 7, 16, 2, 1], 6, 2, 128, 16, F16, True),
    ([300, 3, 1030, 0, 77], [5, 7, 16, 2, 1], 6, 2, 128, 16, F16, False),
    ([5000, 4999], [1, 1], 32, 4, 128, 64, F16, True),
    ([640], [16], 40, 1, 64, 64, F16, True),
]


@pytest.mark.parametrize("lens,news,Hq,Hkv,d,page,dt,causal", ATTN)
def test_attention(lens, news, Hq, Hkv, d, page, dt, causal):
    w = World(lens, news, Hkv, d, page, seed=11 + len(lens))
    w.fill(scale=1.0, offset=0.5)
    q = torch.randn((w.total + 1, Hq, d), generator=w.g).to(dt)
    table, kv_lens, cu = w.where()
    out = torch.full((w.total + 1, Hq, d), 5.0, dtype=dt, device="cuda")
    lse = torch.full((w.total + 1, Hq), 5.0, device="cuda")
    got = sage.attn_kv4(q.cuda(), w.cache.cuda(), table, kv_lens, cu, max(news), causal, out=out, lse=lse)
    ok()
    assert got is out and (out[w.total:] == 5.0).all() and (lse[w.total:] == 5.0).all()
    check_attn(w, q[:w.total], out, lse, causal)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,new", [(4, 1), (8, 1), (4, 5)])
def test_attention_of_many_segments(group, new, d):
    # from 148 (sequence, key head, row block) on, warps work alone; rows 4, 8 and 20 of a key head
    g = torch.Generator().manual_seed(group + new)
    lens = torch.randint(0, 900, (26,), generator=g).tolist()
    news = [min(n, int(x)) for n, x in zip(lens, torch.randint(new > 1 and 0 or 1, new + 1, (26,), generator=g))]
    w = World(lens, news, 8, d, 32, seed=13)
    w.fill()
    q = torch.randn((w.total, 8 * group, d), generator=w.g).to(F16)
    lse = torch.empty((w.total, 8 * group), device="cuda")
    out = sage.attn_kv4(q.cuda(), w.cache.cuda(), *w.where(), new, lse=lse)
    ok()
    check_attn(w, q, out, lse)


def test_attention_over_shared_pages():
    # three sequences that begin with the same pages (a common prompt) and end in their own
    w = World([100, 90, 64], [1, 1, 1], 2, 64, 32, seed=14)
    w.fill()
    w.table[1, :2] = w.table[0, :2]
    w.table[2, :2] = w.table[0, :2]
    q = torch.randn((3, 4, 64), generator=w.g).to(F16)
    out = sage.attn_kv4(q.cuda(), w.cache.cuda(), *w.where(), 1)
    ok()
    check_attn(w, q, out, None)


def test_two_calls_at_once():
    # the same cache read by two streams at a time, a workspace each
    w = World([2000, 900, 1500, 40] * 8, [1] * 32, 8, 128, 16, seed=15)
    w.fill()
    qs = [torch.randn((32, h, 128), generator=w.g).to(F16).cuda() for h in (32, 64)]
    cache, where = w.cache.cuda(), w.where()
    want = [sage.attn_kv4(q, cache, *where, 1) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(sage.attn_kv4(qs[i], cache, *where, 1))
    torch.cuda.synchronize()
    ok()
    for i in (0, 1):
        assert all(torch.equal(x, want[i]) for x in got[i])


@pytest.mark.parametrize("d", [64, 128])
def test_attention_sharp_scores_and_value_scales(d):
    # a large softmax scale (few keys carry the weight), values whose size differs by 10^6
    # between tokens, rows of queries of very different sizes
    lens, Hkv, Hq, page = [2100, 333], 2, 8, 64
    w = World(lens, [2, 2], Hkv, d, page, seed=5)
    for s, n in enumerate(lens):
        size = 10.0 ** torch.randint(-4, 3, (n, 1, 1), generator=w.g)
        w.put(s, torch.arange(n), torch.randn((n, Hkv, d), generator=w.g),
              torch.randn((n, Hkv, d), generator=w.g) * size)
    q = torch.randn((w.total, Hq, d), generator=w.g) * 10.0 ** torch.randint(-3, 2, (w.total, Hq, 1), generator=w.g)
    q = q.to(F16)
    table, kv_lens, cu = w.where()
    lse = torch.empty((w.total, Hq), device="cuda")
    out = sage.attn_kv4(q.cuda(), w.cache.cuda(), table, kv_lens, cu, 2, True, 0.5, lse=lse)
    ok()
    check_attn(w, q, out, lse, True, 0.5)


def test_attention_values_of_one_small_size():
    # values near 1e-4: products with the probabilities far below fp16's normal range
    w = World([700, 90], [1, 1], 2, 128, 32, seed=6)
    w.fill(scale=1e-4)
    q = torch.randn((2, 8, 128), generator=w.g).to(BF16)
    table, kv_lens, cu = w.where()
    out = sage.attn_kv4(q.cuda(), w.cache.cuda(), table, kv_lens, cu, 1)
    ok()
    check_attn(w, q, out, None)


def test_uniform_queries_without_cu_seqlens_and_strided_queries():
    lens, n, Hq, Hkv, d = [50, 7, 200], 2, 6, 3, 64
    w = World(lens, [n] * 3, Hkv, d, 16, seed=3)
    w.fill()
    fused = torch.randn((w.total, Hq + 4, d), generator=w.g).to(F16).cuda()
    q = fused[:, 2:2 + Hq]
    table, kv_lens, cu = w.where()
    a = sage.attn_kv4(q, w.cache.cuda(), table, kv_lens)
    b = sage.attn_kv4(q.contiguous(), w.cache.cuda(), table, kv_lens, cu, n)
    assert torch.equal(a, b)
    ok()
    check_attn(w, q.cpu(), a, None)


def test_hidden_places_do_not_reach_the_result():
    # a drafted token whose value is NaN and whose key is infinite: earlier queries of the
    # sequence do not see it, later ones do; the tail of the last page is NaN throughout
    lens, news, Hq, Hkv, d, page = [70, 20], [4, 1], 4, 2, 128, 64
    w = World(lens, news, Hkv, d, page, seed=9)
    w.fill()
    bad = torch.full((1, Hkv, d), math.nan)
    w.put(0, torch.tensor([68]), bad * math.inf, bad)
    q = torch.randn((w.total, Hq, d), generator=w.g).to(F16)
    table, kv_lens, cu = w.where()
    out = sage.attn_kv4(q.cuda(), w.cache.cuda(), table, kv_lens, cu, 4).cpu()
    ok()
    assert out[2:4].isnan().all()                       # queries at 68 and 69 see it
    for i in (0, 1):
        k, v = (x[:67 + i] for x in w.tokens(0))
        want, _, _, _ = ref.attend(q[i:i + 1].double(), k, v)
        near(out[i:i + 1], want, 2.0 ** -15 * v.abs().amax())
    assert out[4].isfinite().all()


@pytest.mark.parametrize("Hq", [2, 4, 16, 32])
def test_zero_queries_at_a_scale_that_underflows(Hq):
    # logits of 0 over the keys that a query sees, and none over the hidden ones: every visible
    # key counts alike
    w = World([70, 3, 20], [4, 5, 1], 2, 128, 16, seed=16)
    w.fill()
    q = torch.randn((w.total, Hq, 128), generator=w.g).to(F16)
    q[:3] = 0.0
    q[6] = 0.0
    lse = torch.empty((w.total, Hq), device="cuda")
    out = sage.attn_kv4(q.cuda(), w.cache.cuda(), *w.where(), 5, sm_scale=1e-30, lse=lse)
    ok()
    check_attn(w, q, out, lse, sm_scale=1e-30)


def test_non_finite_inputs_stay_in_their_group():
    w = World([20], [20], 2, 128, 32)
    k = torch.randn((20, 2, 128), generator=w.g).to(F16)
    v = k.clone()
    k[3, 1, 70], k[4, 0, 5], v[5, 1, 0] = math.nan, math.inf, -math.inf
    table, kv_lens, cu = w.where()
    cache = w.cache.cuda()
    sage.kv4_append(cache, table, kv_lens, cu, k.cuda(), v.cuda())
    ko, vo = sage.kv4_gather(cache, table, kv_lens, cu, 20, 128)
    ok()
    want_k, want_v = torch.ones(20, 2, 2, dtype=torch.bool), torch.ones(20, 2, 2, dtype=torch.bool)
    want_k[3, 1, 1] = want_k[4, 0, 0] = want_v[5, 1, 0] = False
    for got, want in ((ko, want_k), (vo, want_v)):
        finite = got.isfinite().cpu().unflatten(-1, (2, 64))
        assert finite[want].all()
        assert not finite[~want].all(-1).any()


# ------------------------------------------------------------- use, state, capture, errors


def test_same_bits_again_and_on_another_stream():
    w = World([3000, 17, 900, 2500], [2, 1, 2, 2], 4, 128, 16, seed=2)
    w.fill()
    q = torch.randn((w.total, 16, 128), generator=w.g).to(F16).cuda()
    table, kv_lens, cu = w.where()
    cache = w.cache.cuda()
    ws = torch.full((sage.sage_attn_kv4_workspace_size(16, 4, 2, 128),), 255, dtype=torch.uint8, device="cuda")
    first = sage.attn_kv4(q, cache, table, kv_lens, cu, 2, workspace=ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(side):
            again = sage.attn_kv4(q, cache, table, kv_lens, cu, 2, workspace=ws)
        side.synchronize()
        assert torch.equal(first, again)
    explicit = sage.attn_kv4(q, cache, table, kv_lens, cu, 2, stream=side)
    side.synchronize()
    assert torch.equal(first, explicit)
    ok()


def test_what_a_call_allocates_belongs_to_its_stream():
    # a workspace is free again when the call returns: memory of another stream could be handed
    # out to that stream while the kernel still uses it
    def owner(ptr):
        return [x["stream"] for x in torch.cuda.memory_snapshot()
                if x["address"] <= ptr < x["address"] + x["total_size"]]

    w = World([500, 40], [1, 1], 2, 64, 16, seed=17)
    w.fill()
    q, kv = (torch.randn((2, h, 64), generator=w.g).to(F16).cuda() for h in (4, 2))
    cache, spare, where = w.cache.cuda(), w.cache.cuda(), w.where()
    freqs = torch.tensor([2.0 ** -i for i in range(32)], dtype=torch.float64).cuda()
    want = sage.attn_kv4(q, cache, *where, 1)
    torch.cuda.synchronize()
    for s in (torch.cuda.Stream(), torch.cuda.default_stream()):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [*sage.rope(q, kv, freqs=freqs, stream=s), sage.attn_kv4(q, cache, *where, 1, stream=s),
                   *sage.kv4_gather(cache, *where, 2, 64, stream=s),
                   sage.kv4_append(spare, *where, kv, kv, q=q, freqs=freqs, stream=s)]
            assert all(owner(x.data_ptr()) == [s.cuda_stream] for x in got)
            s.synchronize()
            assert torch.equal(got[2].cpu(), want.cpu())
            t = torch.cuda.Stream(priority=-1)         # for the workspace alone
            sage.attn_kv4(q, cache, *where, 1, out=got[2], stream=t)
            need = sage.sage_attn_kv4_workspace_size(4, 2, 1, 64)
            assert sum(x["total_size"] for x in torch.cuda.memory_snapshot() if x["stream"] == t.cuda_stream) >= need
            t.synchronize()
    ok()


def test_the_c_calls_by_address():
    # the entry points of sage.h as they are, which the tensor calls make for their tensors
    d, Hq, Hkv, page, dt = 64, 4, 2, 16, sage.SAGE_BF16
    w = World([70, 5, 33], [2, 1, 2], Hkv, d, page, seed=18)
    w.fill()
    fused = torch.randn((w.total, Hq + 2 * Hkv, d), generator=w.g).to(BF16).cuda()
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    freqs, m = sage.rope_freqs(d, scaling="linear", factor=2.0)
    table, kv_lens, cu = w.where()
    seqs = (len(w.lens), w.total)
    sizes = (page, w.pages, table.shape[1])
    row = fused.shape[1] * d
    pos = w.positions().to(torch.int32).cuda()

    rq, rk = torch.empty_like(q), torch.empty_like(k)
    one = [0, d, row]
    sage.sage_rope(q, rq, k, rk, pos, freqs, dt, 1, w.total, Hq, Hkv, d, d, 0,
                   one + [0, d, Hq * d] + one + [0, d, Hkv * d], m, 0)
    want = sage.rope(q, k, freqs, pos, m)
    assert torch.equal(rq, want[0]) and torch.equal(rk, want[1])

    a, b = w.cache.cuda(), w.cache.cuda()
    qo = torch.empty_like(q)
    sage.sage_kv4_append(a, table, kv_lens, cu, k, v, q, qo, freqs, None, dt, *seqs, Hq, Hkv, d, *sizes, d,
                         [row, d] * 3 + [Hq * d, d], m, 0)
    assert torch.equal(qo, sage.kv4_append(b, table, kv_lens, cu, k, v, q, freqs, m)) and torch.equal(a, b)
    assert torch.equal(qo, rq)

    ko, vo = (torch.empty((w.total, Hkv * 2, d), dtype=BF16, device="cuda") for _ in range(2))
    sage.sage_kv4_gather(a, table, kv_lens, cu, ko, vo, dt, *seqs, Hkv, 2, d, *sizes)
    want = sage.kv4_gather(a, table, kv_lens, cu, w.total, d, BF16, 2)
    assert torch.equal(ko, want[0]) and torch.equal(vo, want[1])

    out, lse = torch.empty_like(qo), torch.empty((w.total, Hq), device="cuda")
    ws = torch.empty(sage.sage_attn_kv4_workspace_size(Hq, Hkv, 2, d), dtype=torch.uint8, device="cuda")
    sage.sage_attn_kv4(qo, a, table, kv_lens, cu, out, lse, dt, *seqs, 2, Hq, Hkv, d, *sizes, True, 0.0, None, ws,
                       ws.numel())
    ok()
    w.cache = a.cpu()
    check_attn(w, qo.cpu(), out, lse)
    assert torch.equal(out, sage.attn_kv4(qo, a, table, kv_lens, cu, 2))


def test_memory_that_is_not_there_is_torchs_error():
    # 140 TB of outputs: refused by the allocator before anything runs
    w = World([4], [4], 2, 64, 16)
    with pytest.raises(torch.OutOfMemoryError):
        sage.kv4_gather(w.cache.cuda(), *w.where(), 2 ** 31 - 1, 64, rep=256)
    ok()


def test_a_serving_loop_in_a_graph():
    """Prompt by append, gather and the package's own prefill attention; then decode steps,
    each an append and an attention captured once and replayed with new lengths."""
    d, Hq, Hkv, page, dt = 64, 4, 2, 16, F16
    prompts, steps = [37, 5, 90], 20
    lens = [p + steps for p in prompts]
    w = World(lens, prompts, Hkv, d, page, seed=8)
    freqs, m = sage.rope_freqs(d)
    table = w.table.cuda()
    cache = w.cache.cuda()
    kv_lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    cu = torch.cumsum(torch.tensor([0] + prompts), 0).to(torch.int32).cuda()
    T = sum(prompts)
    mean = torch.randn((Hkv, d), generator=w.g)
    fused = torch.randn((T, Hq + 2 * Hkv, d), generator=w.g)
    fused[:, Hq:Hq + Hkv] += mean
    fused = fused.to(dt).cuda()
    split = lambda x: (x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:])  # noqa: E731
    q, k, v = split(fused)
    qr = sage.kv4_append(cache, table, kv_lens, cu, k, v, q, freqs, m, k_mean=mean.cuda())
    kg, vg = sage.kv4_gather(cache, table, kv_lens, cu, T, d, rep=Hq // Hkv)
    out = sage.sageattn_varlen_kv(qr, kg, vg, cu, cu, max(prompts), max(prompts), causal=True)
    ok()

    def state():
        w.cache = cache.cpu()
        w.lens = kv_lens.tolist()

    state()
    for s, n in enumerate(prompts):                     # 8-bit attention over the 4-bit cache
        a = int(cu[s])
        kk, vv = w.tokens(s)
        want, _, _, _ = ref.attend(qr[a:a + n].cpu().double(), kk, vv)
        got = out[a:a + n].cpu().double()
        assert float((got * want).sum() / (got.norm() * want.norm())) > 0.999

    new = torch.zeros((3, Hq + 2 * Hkv, d), dtype=dt, device="cuda")
    ws = torch.empty(sage.sage_attn_kv4_workspace_size(Hq, Hkv, 1, d), dtype=torch.uint8, device="cuda")
    hold = {}

    def step():
        q, k, v = split(new)
        kv_lens.add_(1)
        hold["q"] = sage.kv4_append(cache, table, kv_lens, None, k, v, q, freqs, m, k_mean=mean.cuda())
        hold["out"] = sage.attn_kv4(hold["q"], cache, table, kv_lens, None, workspace=ws)

    mean = mean.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                       # warm-up; then the lengths go back
        step()
        kv_lens.sub_(1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    kv_lens.copy_(torch.tensor(prompts, dtype=torch.int32))
    w.cu = torch.arange(4, dtype=torch.int32)
    for i in range(steps):
        new.copy_(torch.randn(new.shape, generator=w.g).to(dt))
        graph.replay()
        ok()
        state()
        assert w.lens == [p + i + 1 for p in prompts]
        q, k, v = (x.cpu() for x in split(new))
        pos = torch.tensor(w.lens) - 1
        k32 = ref.rotate(k, pos, freqs.cpu(), m, dtype=torch.float32) - mean.cpu()
        for s in range(3):
            ids = int(w.table[s, pos[s] // page])
            codes, params = ref.regions(w.cache, page, d)
            for x, y in ((0, k32[s]), (1, v[s].float())):
                c, p = ref.quantize(y)
                assert torch.equal(codes[ids, :, x, pos[s] % page], c[..., 0::2] | (c[..., 1::2] << 4))
                assert torch.equal(params[ids, :, x, pos[s] % page], p)
        near(hold["q"], ref.rotate(q, pos, freqs.cpu(), m), 2.0 ** -21 * q.double().abs().amax())
        check_attn(w, hold["q"].cpu(), hold["out"], None)


def test_bad_tables_and_lengths_are_reported_and_touch_nothing_else():
    # checked before every access, so nothing here reads or writes outside the buffers
    lens, news, Hkv, Hq, d, page = [40, 20, 33], [1, 1, 1], 2, 4, 64, 16
    w = World(lens, news, Hkv, d, page, seed=12)
    w.fill()
    q = torch.randn((3, Hq, d), generator=w.g).to(F16).cuda()
    kv = torch.randn((3, Hkv, d), generator=w.g).to(F16).cuda()
    good = w.where()
    want = sage.attn_kv4(q, w.cache.cuda(), *good, 1)
    ok()

    def run(table, kv_lens, cu, code, others):
        for op in ("append", "gather", "attend"):
            cache = w.cache.cuda()
            if op == "append":
                sage.kv4_append(cache, table, kv_lens, cu, kv, kv)
            elif op == "gather":
                sage.kv4_gather(cache, table, kv_lens, cu, 3, d)
            else:
                out = sage.attn_kv4(q, cache, table, kv_lens, cu, 1)
                assert torch.equal(out[others], want[others])
            assert sage.sage_get_device_status() == code, op
            ok()

    table, kv_lens, cu = good
    for wrong in (-1, w.pages, 2 ** 30):
        t = table.clone()
        t[1, 1] = wrong                                 # token 19 of sequence 1 lies there
        run(t, kv_lens, cu, sage.SAGE_ERR_BAD_PAGE, [0, 2])
    for wrong in (-1, table.shape[1] * page + 1, 2 ** 31 - 1):
        n = kv_lens.clone()
        n[1] = wrong
        run(table, n, cu, sage.SAGE_ERR_BAD_SEQLENS, [0, 2])
    for wrong in ([0, 1, 0, 3], [0, -1, 2, 3], [0, 1, 2, 900]):
        c = torch.tensor(wrong, dtype=torch.int32, device="cuda")
        run(table, kv_lens, c, sage.SAGE_ERR_BAD_SEQLENS, [0] if wrong[1] == 1 else [])
    # more queries than max_q; more new tokens than the sequence holds
    c = torch.tensor([0, 1, 3, 3], dtype=torch.int32, device="cuda")
    out = sage.attn_kv4(q, w.cache.cuda(), table, kv_lens, c, 1)
    assert sage.sage_get_device_status() == sage.SAGE_ERR_BAD_SEQLENS and torch.equal(out[0], want[0])
    n = kv_lens.clone()
    n[1] = 1
    sage.kv4_append(w.cache.cuda(), table, n, c, kv, kv)
    assert sage.sage_get_device_status() == sage.SAGE_ERR_BAD_SEQLENS
    ok()


def test_many_short_sequences():
    # more sequences than a CTA has threads: the list of work is summed in rounds
    n, Hq, Hkv, d, page = 700, 4, 2, 64, 16
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 40, (n,), generator=g).tolist()
    news = [min(x, int(c)) for x, c in zip(lens, torch.randint(0, 3, (n,), generator=g))]
    w = World(lens, news, Hkv, d, page, seed=4)
    w.fill()
    fused = torch.randn((w.total, Hq + 2 * Hkv, d), generator=g).to(F16).cuda()
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    table, kv_lens, cu = w.where()
    cache = w.cache.cuda()
    sage.kv4_append(cache, table, kv_lens, cu, k, v)
    ko, vo = sage.kv4_gather(cache, table, kv_lens, cu, w.total, d)
    out = sage.attn_kv4(q, cache, table, kv_lens, cu, 2)
    ok()
    pos = w.positions()
    for s in range(n):
        a, b = int(w.cu[s]), int(w.cu[s + 1])
        w.put(s, pos[a:b], k[a:b].cpu().float(), v[a:b].cpu().float())
    assert torch.equal(cache.cpu(), w.cache)
    check_attn(w, q.cpu(), out, None)
    for s in range(0, n, 50):
        a, b = int(w.cu[s]), int(w.cu[s + 1])
        for x, got in ((0, ko), (1, vo)):
            want = w.tokens(s)[x][lens[s] - (b - a):]
            near(got[a:b], want, 2.0 ** -24 * want.abs())


def test_pages_past_four_gigabytes():
    # page numbers times page bytes past 2^32: only the pages in use are ever written
    Hkv, d, page, Hq = 8, 128, 256, 8
    pages = (5 << 30) // (Hkv * sage.sage_kv4_page_bytes(page, d))
    cache = sage.kv4_cache(pages, Hkv, page, d)
    n = 300
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((n, Hkv, d), generator=g).to(F16) for _ in range(2))
    q = torch.randn((1, Hq, d), generator=g).to(F16)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32)
    kv_lens = torch.tensor([n], dtype=torch.int32).cuda()
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    sage.kv4_append(cache, table.cuda(), kv_lens, cu, k.cuda(), v.cuda())
    ko, vo = sage.kv4_gather(cache, table.cuda(), kv_lens, cu, n, d)
    out = sage.attn_kv4(q.cuda(), cache, table.cuda(), kv_lens)
    ok()
    small = World([n], [n], Hkv, d, page)
    small.put(0, torch.arange(n), k.float(), v.float())
    kk, vv = small.tokens(0)
    near(ko, kk, 2.0 ** -24 * kk.abs())
    near(vo, vv, 2.0 ** -24 * vv.abs())
    want, _, _, _ = ref.attend(q.double(), kk, vv)
    near(out, want, 2.0 ** -13 * vv.abs().amax())


def test_the_longest_sequence():
    # 2^31 - 1 tokens, all on one page: equal weights over values of which the first 64 of 256
    # are 0 and the others 1. A lane adds 2^31 / (1776 warps 8 lanes) = 151 000 terms, each sum
    # off by at most 2^-24 of itself a term; two such sums make the result
    w = World([256], [1], 1, 64, 256)
    v = (torch.arange(256) >= 64).float()[:, None, None].expand(256, 1, 64)
    w.put(0, torch.arange(256), torch.zeros(256, 1, 64), v)
    n = 2 ** 31 - 1
    table = torch.full((1, 2 ** 23), int(w.table[0, 0]), dtype=torch.int32, device="cuda")
    kv_lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    q = torch.randn((1, 1, 64), generator=w.g).to(F16).cuda()
    out = sage.attn_kv4(q, w.cache.cuda(), table, kv_lens)
    _, last = sage.kv4_gather(w.cache.cuda(), table, kv_lens, None, 1, 64)
    ok()
    assert (last == 1).all()
    want = torch.full((1, 1, 64), 1 - 64 * 2 ** 23 / n, dtype=torch.float64)
    near(out, want, 2 * 151_000 * 2.0 ** -24)


@pytest.mark.parametrize("d,page,Hkv,rep", [(128, 64, 2, 4), (64, 16, 3, 1)])
def test_prefill_over_the_cache_is_attention_over_what_it_stands_for(d, page, Hkv, rep):
    # a chunk of new tokens over cached ones: the package's attention has the same bits over
    # gathered keys and values as over the cache's values worked out on the CPU (code times step
    # is exact in 32 bits, the sum with low and the fp16 result are each rounded once)
    lens, news = [300, 45, 129], [200, 45, 1]
    w = World(lens, news, Hkv, d, page, seed=21)
    w.fill(offset=0.5)
    table, kv_lens, cu = w.where()
    cu_all = torch.cumsum(torch.tensor([0] + lens), 0).to(torch.int32).cuda()
    total = sum(lens)
    kg, vg = sage.kv4_gather(w.cache.cuda(), table, kv_lens, cu_all, total, d, rep=rep)
    parts = [w.tokens(s, dtype=torch.float32) for s in range(len(lens))]
    want = [torch.cat([p[x] for p in parts]).to(F16).repeat_interleave(rep, 1) for x in (0, 1)]
    assert torch.equal(kg.cpu(), want[0]) and torch.equal(vg.cpu(), want[1])
    q = torch.randn((w.total, Hkv * rep, d), generator=w.g).to(F16).cuda()
    got = sage.sageattn_varlen_kv(q, kg, vg, cu, cu_all, max(news), max(lens), causal=True)
    same = sage.sageattn_varlen_kv(q, want[0].cuda(), want[1].cuda(), cu, cu_all, max(news), max(lens), causal=True)
    ok()
    assert torch.equal(got, same)
    for s, n in enumerate(news):                        # and near the 64-bit attention over it
        a = int(w.cu[s])
        exact, _, _, _ = ref.attend(q[a:a + n].cpu().double(), *(x.double().repeat_interleave(rep, 1) for x in parts[s]))
        off = got[a:a + n].cpu().double() - exact
        assert float(off.norm() / exact.norm()) < 0.02
