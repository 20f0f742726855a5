"""Rotary positions and the 4-bit cache without a GPU: the angles' formulas, and every refusal
of the C entry points and of the wrappers, all of which happen before any CUDA call."""
import ctypes
import math
import sys

import pytest
import torch

import quantized_attention_03_b200 as sage

FAKE, MIS = 0x10000, 0x10008      # 16-byte aligned, and not; never dereferenced


@pytest.fixture(scope="module")
def lib():
    from quantized_attention_03_b200 import build
    build.build()
    return sage.lib()


# ---------------------------------------------------------------------------- angles


@pytest.mark.parametrize("rot,base", [(16, 10000.0), (64, 10000.0), (128, 500000.0), (2, 100.0)])
def test_plain_and_linear_freqs(lib, rot, base):
    f, m = sage.rope_freqs(rot, base, device="cpu")
    assert m == 1.0 and f.shape == (rot // 2,)
    for i in range(rot // 2):
        assert f[i].item() == pytest.approx(math.exp(-2 * i / rot * math.log(base)), rel=1e-14)
    g, m = sage.rope_freqs(rot, base, "linear", 4.0, device="cpu")
    assert m == 1.0 and torch.equal(g, f / 4)


def test_base_scaling_keeps_the_fastest_pair_and_divides_the_slowest(lib):
    f, _ = sage.rope_freqs(128, device="cpu")
    g, m = sage.rope_freqs(128, scaling="base", factor=8.0, device="cpu")
    assert m == 1.0 and g[0] == f[0]
    assert g[-1].item() == pytest.approx(f[-1].item() / 8, rel=1e-12)
    assert bool((g[1:] < f[1:]).all())


def test_parts_scaling(lib):
    f, _ = sage.rope_freqs(128, device="cpu")
    g, m = sage.rope_freqs(128, scaling="parts", factor=16.0, original_len=4096, device="cpu")
    assert m == pytest.approx(0.1 * math.log(16) + 1, rel=1e-15)
    turns = 4096 * f / (2 * math.pi)
    share = (1 - g / f) / (1 - 1 / 16)                # 0: kept, 1: divided by the factor
    assert bool((share[turns > 33] < 0.03).all()) and bool((share[turns < 0.95] > 0.97).all())
    assert bool((share.diff() >= -1e-12).all())
    mid = (turns < 25) & (turns > 1.5)
    assert bool((share[mid] > 0.02).all()) and bool((share[mid] < 0.99).all())
    same, m = sage.rope_freqs(128, scaling="parts", factor=1.0, original_len=4096, device="cpu")
    assert m == 1.0 and torch.allclose(same, f, rtol=1e-15, atol=0)


def test_freqs_refusals(lib):
    out = (ctypes.c_double * 64)()

    def go(freqs=out, rot=128, base=1e4, scaling=0, factor=2.0, orig=4096.0, fast=32.0, slow=1.0):
        return lib.sage_rope_freqs(freqs, None, rot, base, scaling, factor, orig, fast, slow)

    bad = sage.SAGE_ERR_INVALID_ARG
    assert go() == sage.SAGE_OK
    assert go(freqs=None) == bad and go(rot=0) == bad and go(rot=7) == bad and go(rot=-2) == bad
    assert go(base=1.0) == bad and go(base=math.nan) == bad
    assert go(scaling=4) == bad and go(scaling=-1) == bad
    assert go(scaling=1, factor=0.5) == bad and go(scaling=2, rot=2) == bad
    assert go(scaling=3, orig=0.0) == bad and go(scaling=3, fast=1.0) == bad
    assert go(scaling=3, slow=0.0) == bad
    with pytest.raises(ValueError):
        sage.rope_freqs(64, scaling="other", device="cpu")
    with pytest.raises(sage.SageError):
        sage.rope_freqs(0, device="cpu")


# -------------------------------------------------------------------- C entry points


def _rope(lib, q=FAKE, qo=FAKE, k=FAKE, ko=FAKE, freqs=FAKE, dtype=0, B=1, N=4, Hq=2, Hk=2, d=128, rot=128,
          strides=None, flags=0):
    s = None if strides is None else (ctypes.c_int64 * 12)(*strides)
    return lib.sage_rope(q, qo, k, ko, None, freqs, dtype, B, N, Hq, Hk, d, rot, 0, s, 1.0, flags, None)


def test_rope_refusals(lib):
    bad, uns, mis = sage.SAGE_ERR_INVALID_ARG, sage.SAGE_ERR_UNSUPPORTED, sage.SAGE_ERR_MISALIGNED
    assert _rope(lib, q=0) == bad and _rope(lib, qo=0) == bad and _rope(lib, k=0) == bad and _rope(lib, ko=0) == bad
    assert _rope(lib, freqs=0) == bad and _rope(lib, dtype=2) == bad and _rope(lib, B=-1) == bad
    assert _rope(lib, rot=0) == bad and _rope(lib, rot=144) == bad and _rope(lib, rot=-16) == bad
    assert _rope(lib, rot=24) == uns and _rope(lib, d=96, rot=32) == uns and _rope(lib, Hq=70000) == uns
    assert _rope(lib, B=65536, N=65536) == uns
    assert _rope(lib, flags=4) == bad
    assert _rope(lib, q=MIS) == mis and _rope(lib, ko=MIS) == mis
    assert _rope(lib, strides=[512, 256, 130] + [512, 256, 128] * 3) == mis
    assert _rope(lib, B=0) == sage.SAGE_OK and _rope(lib, N=0, q=0) == sage.SAGE_OK
    assert _rope(lib, Hq=0, Hk=0) == sage.SAGE_OK


def _append(lib, cache=FAKE, table=FAKE, lens=FAKE, cu=FAKE, k=FAKE, v=FAKE, q=FAKE, qo=FAKE, freqs=FAKE, mean=None,
            dtype=0, nseq=2, total=4, Hq=4, Hkv=2, d=128, page=16, pages=8, width=4, rot=128, strides=None, flags=0):
    s = None if strides is None else (ctypes.c_int64 * 8)(*strides)
    return lib.sage_kv4_append(cache, table, lens, cu, k, v, q, qo, freqs, mean, dtype, nseq, total, Hq, Hkv, d, page,
                               pages, width, rot, s, 1.0, flags, None)


def test_append_refusals(lib):
    bad, uns, mis = sage.SAGE_ERR_INVALID_ARG, sage.SAGE_ERR_UNSUPPORTED, sage.SAGE_ERR_MISALIGNED
    for name in ("cache", "table", "lens", "k", "v", "qo", "freqs"):
        assert _append(lib, **{name: 0}) == bad, name
    for name in ("dtype", "nseq", "total", "Hkv", "pages", "width", "Hq"):
        assert _append(lib, **{name: -1}) == bad, name
    for page in (0, 8, 24, 512, -16):
        assert _append(lib, page=page) == uns, page
    assert _append(lib, d=96) == uns and _append(lib, rot=40) == uns and _append(lib, rot=256) == bad
    assert _append(lib, flags=sage.SAGE_ROPE_INVERSE) == bad
    assert _append(lib, cu=0, total=5) == bad          # 5 rows do not divide into 2 sequences
    for name in ("cache", "k", "v", "q", "qo", "mean"):
        assert _append(lib, **{name: MIS}) == mis, name
    assert _append(lib, strides=[256, 128, 256, 132, 512, 128, 512, 128]) == mis
    assert _append(lib, nseq=0) == sage.SAGE_OK and _append(lib, total=0, cache=0) == sage.SAGE_OK


def _gather(lib, cache=FAKE, table=FAKE, lens=FAKE, cu=FAKE, ko=FAKE, vo=FAKE, dtype=0, nseq=2, total=4, Hkv=2, rep=1,
            d=128, page=16, pages=8, width=4):
    return lib.sage_kv4_gather(cache, table, lens, cu, ko, vo, dtype, nseq, total, Hkv, rep, d, page, pages, width, None)


def test_gather_refusals(lib):
    bad, uns, mis = sage.SAGE_ERR_INVALID_ARG, sage.SAGE_ERR_UNSUPPORTED, sage.SAGE_ERR_MISALIGNED
    for name in ("cache", "table", "lens", "ko", "vo", "rep"):
        assert _gather(lib, **{name: 0}) == bad, name
    assert _gather(lib, dtype=5) == bad and _gather(lib, page=17) == uns and _gather(lib, d=80) == uns
    for name in ("cache", "ko", "vo"):
        assert _gather(lib, **{name: MIS}) == mis, name
    assert _gather(lib, total=0, ko=0) == sage.SAGE_OK


@pytest.mark.parametrize("Hkv,rep", [(8, 1 << 24), (2, 1 << 30), (1, 65536), (65535, 2), (4, 2 ** 31 - 1)])
def test_gather_refuses_more_heads_than_the_other_calls(lib, Hkv, rep):
    # heads of the outputs, as everywhere at most 65535: products of them stay within 32 bits
    assert _gather(lib, Hkv=Hkv, rep=rep) == sage.SAGE_ERR_UNSUPPORTED
    assert _gather(lib, Hkv=Hkv, rep=rep, total=0) == sage.SAGE_ERR_UNSUPPORTED
    cache, table, lens, cu = _cpu_sequences(Hkv=min(Hkv, 8))
    with pytest.raises(sage.SageError):
        sage.kv4_gather(cache, table, lens, cu, 2, 64, rep=max(rep, 65536))


def _attn(lib, q=FAKE, cache=FAKE, table=FAKE, lens=FAKE, cu=FAKE, out=FAKE, lse=None, dtype=0, nseq=2, total=4,
          max_q=2, Hq=4, Hkv=2, d=128, page=16, pages=8, width=4, strides=None, ws=FAKE, ws_bytes=1 << 30):
    s = None if strides is None else (ctypes.c_int64 * 2)(*strides)
    return lib.sage_attn_kv4(q, cache, table, lens, cu, out, lse, dtype, nseq, total, max_q, Hq, Hkv, d, page, pages,
                             width, 1, 0.0, s, ws, ws_bytes, None)


def test_attn_refusals(lib):
    bad, uns, mis = sage.SAGE_ERR_INVALID_ARG, sage.SAGE_ERR_UNSUPPORTED, sage.SAGE_ERR_MISALIGNED
    for name in ("q", "cache", "table", "lens", "out", "ws", "max_q", "pages"):
        assert _attn(lib, **{name: 0}) == bad, name
    assert _attn(lib, Hq=5) == bad and _attn(lib, Hkv=0) == bad and _attn(lib, max_q=-1) == bad
    assert _attn(lib, max_q=17) == uns and _attn(lib, page=12) == uns and _attn(lib, d=32) == uns
    assert _attn(lib, cu=0, max_q=1) == bad            # 4 rows of 2 sequences: two queries each
    for name in ("q", "cache", "out", "ws"):
        assert _attn(lib, **{name: MIS}) == mis, name
    assert _attn(lib, strides=[512, 100]) == mis
    need = lib.sage_attn_kv4_workspace_size(4, 2, 2, 128)
    assert need > 0 and _attn(lib, ws_bytes=need - 1) == sage.SAGE_ERR_WORKSPACE
    assert _attn(lib, total=0, q=0) == sage.SAGE_OK and _attn(lib, nseq=0) == sage.SAGE_OK


def test_sizes(lib):
    assert sage.sage_kv4_page_bytes(16, 64) == 16 * 64 // 2 * 2 + 16 * 4 * 2
    assert sage.sage_kv4_page_bytes(256, 128) == 256 * (128 + 16)
    for page, d in ((15, 64), (512, 64), (16, 96), (0, 128), (-16, 64)):
        assert sage.sage_kv4_page_bytes(page, d) == 0
    size = sage.sage_attn_kv4_workspace_size
    assert size(32, 8, 1, 128) > 0 and size(32, 8, 17, 128) == 0 and size(32, 5, 1, 128) == 0
    assert size(0, 0, 1, 128) == 0 and size(8, 8, 1, 96) == 0


# -------------------------------------------------------------------------- wrappers


def _cpu_sequences(nseq=2, width=2, pages=4, Hkv=2, d=64, page=16):
    cache = sage.kv4_cache(pages, Hkv, page, d, device="cpu")
    table = torch.zeros((nseq, width), dtype=torch.int32)
    return cache, table, torch.ones(nseq, dtype=torch.int32), torch.arange(nseq + 1, dtype=torch.int32)


def test_wrappers_refuse_wrong_tensors_before_the_library(lib):
    cache, table, lens, cu = _cpu_sequences()
    f, _ = sage.rope_freqs(64, device="cpu")
    k = torch.zeros((2, 2, 64), dtype=torch.float16)
    q = torch.zeros((2, 4, 64), dtype=torch.float16)
    wrong = [
        lambda: sage.kv4_append(cache, table, lens, cu, k[:, :1], k, q, f),
        lambda: sage.kv4_append(cache, table, lens, cu, k, k.bfloat16(), q, f),
        lambda: sage.kv4_append(cache, table, lens, cu, k.float(), k.float(), None, f),
        lambda: sage.kv4_append(cache, table, lens, cu, k, k, q[:1], f),
        lambda: sage.kv4_append(cache, table, lens, cu, k, k, q, f.float()),
        lambda: sage.kv4_append(cache, table.long(), lens, cu, k, k, q, f),
        lambda: sage.kv4_append(cache, table, lens, cu[:-1], k, k, q, f),
        lambda: sage.kv4_append(cache, table[:1], lens, cu, k, k, q, f),
        lambda: sage.kv4_append(cache, table, lens, cu, k, k, q, f, k_mean=torch.zeros(2, 32)),
        lambda: sage.kv4_append(cache[..., :-9], table, lens, cu, k, k, q, f),
        lambda: sage.kv4_append(cache, table, lens, cu, k, k, q, f, q_out=q.bfloat16()),
        lambda: sage.kv4_gather(cache, table, lens, cu, 2, 128),
        lambda: sage.kv4_gather(cache, table, lens, cu, 2, 64, dtype=torch.float32),
        lambda: sage.kv4_gather(cache, table, lens, cu, 2, 64, k_out=torch.zeros((2, 4, 64), dtype=torch.float16)),
        lambda: sage.attn_kv4(q, cache, table, lens, cu, 1, out=q.transpose(0, 1)),
        lambda: sage.attn_kv4(q, cache, table, lens, cu, 1, lse=torch.zeros(2, 4).double()),
        lambda: sage.attn_kv4(q.float(), cache, table, lens, cu, 1),
        lambda: sage.attn_kv4(torch.zeros((2, 4, 128), dtype=torch.float16), cache, table, lens, cu, 1),
        lambda: sage.rope(q, k[:1], f),
        lambda: sage.rope(q, k, f, torch.zeros(2, dtype=torch.int64)),
        lambda: sage.rope(q, k, f, torch.zeros(3, dtype=torch.int32)),
        lambda: sage.rope(q[0], None, f),
        lambda: sage.rope(q.transpose(1, 2), None, f),
        lambda: sage.kv4_cache(4, 2, 20, 64, device="cpu"),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(i)


def test_outputs_that_overlap_are_refused(lib):
    cache, table, lens, cu = _cpu_sequences()
    f, _ = sage.rope_freqs(32, device="cpu")
    buf = torch.zeros(4096, dtype=torch.float16)
    at = lambda shape, stride, start=0: buf.as_strided(shape, stride, start)  # noqa: E731
    q, k = at((2, 4, 64), (512, 64, 1)), at((2, 2, 64), (512, 64, 1), 256)     # of one projection
    other = torch.zeros((2, 4, 64), dtype=torch.float16)
    wrong = [
        lambda: sage.rope(q, None, f, q_out=other[:, :1].expand(2, 4, 64)),        # one place for all heads
        lambda: sage.rope(q, None, f, q_out=at((2, 4, 64), (256, 64, 1), 2048)[:1].expand(2, 4, 64)),
        lambda: sage.rope(q, None, f, q_out=at((2, 4, 64), (256, 64, 1))),         # q's address, other strides
        lambda: sage.rope(q, None, f, q_out=at((2, 4, 64), (64, 128, 1))),
        lambda: sage.rope(q, None, f, q_out=at((2, 4, 64), (512, 64, 1), 64)),     # one head further
        lambda: sage.rope(q, None, f, q_out=at((2, 4, 64), (512, 64, 1), 512)),    # one token further
        lambda: sage.rope(q, None, f, q_out=at((2, 4, 64), (512, 64, 1), 8)),      # 8 channels further
        lambda: sage.rope(other, None, f, q_out=at((2, 4, 64), (32, 64, 1))),      # heads in one another
        lambda: sage.rope(q[:, :2], k, f, q_out=k),
        lambda: sage.rope(q[:, :2], k, f, k_out=q[:, :2]),
        lambda: sage.rope(q, k, f, q_out=other, k_out=other[:, 2:]),
        lambda: sage.rope(other[None], None, f, q_out=other.as_strided((1, 2, 4, 64), (512, 64, 128, 1))),
        lambda: sage.kv4_append(cache, table, lens, cu, k, k, q, f, q_out=at((2, 4, 64), (256, 64, 1))),
        lambda: sage.kv4_append(cache, table, lens, cu, k, k, q, f, q_out=other[:, :1].expand(2, 4, 64)),
        lambda: sage.kv4_append(cache, table, lens, cu, k, k, q, f, q_out=at((2, 4, 64), (512, 64, 1), 128)),
        lambda: sage.kv4_append(cache, table, lens, cu, k, other[:, :2], q, f, q_out=other),
        lambda: sage.kv4_gather(cache, table, lens, cu, 2, 64, k_out=at((2, 2, 64), (128, 64, 1)),
                                v_out=at((2, 2, 64), (128, 64, 1), 64)),
        lambda: sage.attn_kv4(q, cache, table, lens, cu, 1, out=at((2, 4, 64), (256, 64, 1))),
        lambda: sage.attn_kv4(at((2, 4, 64), (256, 64, 1)), cache, table, lens, cu, 1,
                              out=at((2, 4, 64), (256, 64, 1), 64)),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises(ValueError, match="apart"):
            call()
            raise AssertionError(i)
    # in place, side by side in one buffer, and places of dimensions of one: past these checks,
    # to the refusal of CPU tensors
    fine = [
        lambda: sage.rope(q, k, f, q_out=q, k_out=k),
        lambda: sage.rope(q, k, f, q_out=at((2, 4, 64), (512, 64, 1), 2048), k_out=at((2, 2, 64), (512, 64, 1), 2304)),
        lambda: sage.rope(q[:, :2], k, f, q_out=at((2, 2, 64), (512, 64, 1), 128), k_out=at((2, 2, 64), (512, 64, 1), 384)),
        lambda: sage.rope(q[:1], None, f, q_out=at((1, 4, 64), (8, 64, 1))),
        lambda: sage.rope(other[:, :1].expand(2, 4, 64), None, f),
        lambda: sage.kv4_append(cache, table, lens, cu, k, at((2, 2, 64), (512, 64, 1), 384), q, f, q_out=q),
        lambda: sage.kv4_gather(cache, table, lens, cu, 2, 64, k_out=at((2, 2, 64), (128, 64, 1)),
                                v_out=at((2, 2, 64), (128, 64, 1), 256)),
        lambda: sage.attn_kv4(other, cache, table, lens, cu, 1, out=other),
    ]
    for call in fine:
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_c_calls_refuse_outputs_over_their_input(lib):
    bad = sage.SAGE_ERR_INVALID_ARG
    dense = [1024, 512, 128]
    # q_out = q and k_out = k at 0x10000: other strides, and none for several places
    assert _rope(lib, strides=dense + [1024, 128, 256] + dense * 2) == bad
    assert _rope(lib, strides=dense * 3 + [1024, 128, 256]) == bad
    assert _rope(lib, qo=FAKE + 65536, strides=dense + [1024, 0, 128] + dense * 2) == bad
    assert _rope(lib, ko=FAKE + 65536, strides=dense * 3 + [1024, 512, 0]) == bad
    assert _append(lib, strides=[256, 128, 256, 128, 512, 128, 1024, 128]) == bad
    assert _append(lib, qo=FAKE + 65536, strides=[256, 128, 256, 128, 512, 128, 512, 0]) == bad


def test_tensors_of_the_cpu_are_refused(lib):
    cache, table, lens, cu = _cpu_sequences()
    f, _ = sage.rope_freqs(64, device="cpu")
    k = torch.zeros((2, 2, 64), dtype=torch.float16)
    for call in (lambda: sage.rope(k, None, f), lambda: sage.kv4_append(cache, table, lens, cu, k, k, None, f),
                 lambda: sage.kv4_gather(cache, table, lens, cu, 2, 64),
                 lambda: sage.attn_kv4(k, cache, table, lens, cu, 1)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    with pytest.raises(ValueError, match="is a tensor"):
        sage.rope([1.0], None, f)


def test_missing_binding_fails_loudly(lib, monkeypatch):
    monkeypatch.setattr(sage, "_calls", None)
    monkeypatch.delattr(sage, "_binding", raising=False)
    monkeypatch.setitem(sys.modules, "quantized_attention_03_b200._binding", None)
    with pytest.raises(RuntimeError, match="_binding.so"):
        sage.rope(torch.zeros((1, 1, 64), dtype=torch.float16), None, torch.zeros(32, dtype=torch.float64))


def test_fp16_calls_refuse_what_the_cache_calls_give_in_bf16(lib):
    # the attention and quantization calls pass addresses on: bf16, or a strided view (a
    # projection rotated in place), would be read as contiguous fp16
    half = lambda *shape: torch.zeros(shape, dtype=torch.float16)  # noqa: E731
    cu = torch.tensor([0, 4], dtype=torch.int32)
    q, k = half(4, 4, 64), half(4, 4, 64)
    dq, dk = half(1, 4, 4, 64), half(1, 4, 8, 64)
    codes, scales = torch.zeros((1, 4, 4, 64), dtype=torch.int8), torch.zeros((1, 4, 1))
    b, view = torch.bfloat16, half(4, 8, 64)[:, :4]
    wrong = [
        lambda: sage.sageattn_varlen_kv(q.to(b), k, k, cu, cu, 4, 4),
        lambda: sage.sageattn_varlen_kv(q, k.to(b), k.to(b), cu, cu, 4, 4),
        lambda: sage.sageattn_varlen_kv(q, k, k.to(b), cu, cu, 4, 4),
        lambda: sage.sageattn_varlen_kv(view, k, k, cu, cu, 4, 4),
        lambda: sage.sageattn_varlen_kv(q, k, k, cu, cu, 4, 4, out=q.to(b)),
        lambda: sage.sageattn_varlen_kv(q, half(4, 2, 64), half(4, 2, 64), cu, cu, 4, 4),      # heads not repeated
        lambda: sage.sageattn_varlen_kv(q, k, k[:3], cu, cu, 4, 4),
        lambda: sage.sageattn_varlen(q.to(b), k.to(b), k.to(b), cu, 4),
        lambda: sage.sageattn_varlen(q, half(3, 4, 64), half(3, 4, 64), cu, 4),
        lambda: sage.sageattn_varlen(q, k, k, cu, 4, out=q[:3]),
        lambda: sage.sageattn(dq.to(b), dk, dk),
        lambda: sage.sageattn(dq, dk, dk.to(b)),
        lambda: sage.sageattn(dq.transpose(1, 2), dk, dk),
        lambda: sage.sageattn(dq, dk[:, :2].contiguous(), dk[:, :2].contiguous()),
        lambda: sage.quant_qk(dq.to(b), dk.to(b)),
        lambda: sage.quant_qk_varlen(q, k.to(b), cu, 4),
        lambda: sage.quant_v_fp8(dk.to(b)),
        lambda: sage.quant_v_fp8_varlen(k.to(b), cu, 4),
        lambda: sage.attn_quantized(codes, scales, codes, scales, dq.to(b), None),
        lambda: sage.attn_decode(codes, scales, codes, scales, dq.to(b)),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(i)


def test_rope_takes_no_gradient_for_what_has_none(lib):
    f, _ = sage.rope_freqs(64, device="cpu")
    x = torch.zeros((2, 2, 64), dtype=torch.float16)
    leaf = x.clone().requires_grad_()
    for call in (lambda: sage.rope(leaf, None, f, q_out=x), lambda: sage.rope(x, leaf, f, k_out=x.clone()),
                 lambda: sage.rope(x, None, f, q_out=leaf), lambda: sage.rope(x, None, f.clone().requires_grad_())):
        with pytest.raises(ValueError, match="no gradient"):
            call()
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):
        sage.rope(leaf, None, f, q_out=x)
    with pytest.raises(ValueError, match="CUDA device"):
        sage.rope(leaf, leaf, f)


def test_a_binding_for_another_torch_is_built_again_and_not_used(lib, monkeypatch):
    from quantized_attention_03_b200 import build
    assert not build._binding_stale()
    sage._bound()
    monkeypatch.setattr(build, "binding_for", lambda: "another python and torch")
    assert build._binding_stale()
    monkeypatch.setattr(sage, "_calls", None)
    with pytest.raises(RuntimeError, match="is built for"):
        sage.rope(torch.zeros((1, 1, 64), dtype=torch.float16), None, torch.zeros(32, dtype=torch.float64))


def test_the_library_is_built_without_the_binding(lib, monkeypatch, tmp_path):
    from quantized_attention_03_b200 import build
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    real = build.subprocess.run

    def no_headers(cmd, **kw):
        if cmd[0] == "g++":
            cmd = ["false"]
        return real(cmd, **kw)

    monkeypatch.setattr(build.subprocess, "run", no_headers)
    with pytest.warns(UserWarning, match="no Python extension"):
        assert build.build() == build.LIB
    assert not (tmp_path / "_binding.so").exists()
    monkeypatch.setitem(sys.modules, "torch", None)     # nor is torch needed for it
    with pytest.warns(UserWarning, match="no Python extension"):
        assert build.build() == build.LIB


def test_fp16_calls_take_the_same_memory_in_another_shape(lib, monkeypatch):
    # what the kernels read and write is there, whatever the tensors' shapes say beyond it
    half = lambda *shape: torch.zeros(shape, dtype=torch.float16)  # noqa: E731
    cu = torch.tensor([0, 4], dtype=torch.int32)
    made = []
    monkeypatch.setattr(sage, "_call", lambda name, *args: made.append(name))
    monkeypatch.setattr(sage, "_stream", lambda s: 0)
    q, dq, dk = half(4, 4, 64), half(2, 4, 4, 64), half(2, 4, 8, 64)
    sage.sageattn(dq, dk, dk.view(8, 8, 64), out=half(8, 4, 64))
    sage.sageattn(dq, half(1, 8, 8, 64), dk)
    sage.sageattn_varlen(q, half(9, 4, 64), half(9, 4, 64), cu, 4, out=half(6, 4, 64))
    sage.sageattn_varlen_kv(q, half(9, 4, 64), half(12, 4, 64), cu, cu, 4, 4, out=half(4, 256))
    sage.quant_qk(dq, half(1, 8, 8, 64))
    sage.quant_qk_varlen(q, half(9, 4, 64), cu, 4)
    assert len(made) == 6
