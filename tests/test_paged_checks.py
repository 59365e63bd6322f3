"""Refusals of the rotary and paged-cache entry points (CPU): return codes of the
C ABI in their documented order, before any device work, and the binding's
TypeError and ValueError; the frequencies against their formulas."""
import ctypes
import math
import os

import pytest
import torch

import exact_tiled_attention_14_gb300 as fa

FAKE = 0x10000   # 256-byte aligned, never dereferenced (errors are returned first)
NAN, INF = float("nan"), float("inf")
OK, SHAPE, WIDTH, DTYPE = fa.FA_OK, fa.FA_ERR_SHAPE, fa.FA_ERR_UNSUPPORTED_D, fa.FA_ERR_DTYPE
ALIGN, SCALE, NULL = fa.FA_ERR_ALIGN, fa.FA_ERR_SCALE, fa.FA_ERR_NULLPTR


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(fa.LIB_PATH):
        fa.build()
    return fa.load_library()


ROT = dict(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE, B=2, H=6, Hk=3, N=10, d=64, strides=[64] * 12,
           freqs=FAKE, rot=32, mscale=1.0, interleaved=0, inverse=0, positions=None, seqlens=None,
           dtype=fa.FA_BF16)


@pytest.mark.parametrize("args,code", [
    (dict(B=-1), SHAPE), (dict(H=-1), SHAPE), (dict(Hk=-1), SHAPE), (dict(N=-1), SHAPE),
    (dict(d=0), SHAPE), (dict(B=1 << 16, N=(1 << 14) + 1), SHAPE), (dict(H=1 << 30), SHAPE),
    (dict(d=96), WIDTH), (dict(rot=0), SHAPE), (dict(rot=24), SHAPE), (dict(rot=80), SHAPE),
    (dict(rot=-16), SHAPE), (dict(positions=FAKE, seqlens=FAKE), SHAPE), (dict(dtype=2), DTYPE),
    (dict(mscale=0.0), SCALE), (dict(mscale=NAN), SCALE), (dict(mscale=INF), SCALE),
    (dict(B=0, q=None), OK), (dict(N=0, strides=None), OK), (dict(H=0, Hk=0, q=None, k=None), OK),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(k_out=None), NULL), (dict(freqs=None), NULL),
    (dict(strides=None), NULL), (dict(q=FAKE + 8), ALIGN), (dict(k_out=FAKE + 2), ALIGN),
    (dict(freqs=FAKE + 8), ALIGN), (dict(positions=FAKE + 2), ALIGN), (dict(seqlens=FAKE + 1), ALIGN),
    (dict(strides=[64] * 11 + [60]), ALIGN), (dict(strides=[4] + [64] * 11), ALIGN),
])
def test_rotary(args, code):
    assert fa.fa_rotary(**{**ROT, **args}) == code


POOL = dict(k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, v_scale=FAKE, B=2, Hk=3, d=64, pages=9,
            page_size=32, page_table=FAKE, pages_per_seq=4, seqlens=FAKE, dtype=fa.FA_FP16,
            cache_dtype=fa.FA_INT8)
PAGED = [
    (dict(B=-1), SHAPE), (dict(Hk=-1), SHAPE), (dict(d=0), SHAPE), (dict(pages=0), SHAPE),
    (dict(pages_per_seq=0), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=24), SHAPE),
    (dict(page_size=144), SHAPE), (dict(page_size=-16), SHAPE), (dict(pages=1 << 26), SHAPE),
    (dict(pages_per_seq=1 << 26), SHAPE), (dict(d=96), WIDTH), (dict(cache_dtype=2), DTYPE),
    (dict(cache_dtype=-1), DTYPE), (dict(dtype=2), DTYPE),
    (dict(B=0, k_cache=None), OK), (dict(k_cache=None), NULL), (dict(v_scale=None), NULL),
    (dict(page_table=None), NULL), (dict(seqlens=None), NULL), (dict(k_cache=FAKE + 8), ALIGN),
    (dict(v_scale=FAKE + 2), ALIGN), (dict(page_table=FAKE + 2), ALIGN),
    (dict(seqlens=FAKE + 2), ALIGN),
]
APPEND = dict(POOL, k=FAKE, v=FAKE, T=5, strides=[64] * 6, counts=FAKE, freqs=FAKE, rot=32, mscale=1.0,
              interleaved=0, positions=FAKE)


@pytest.mark.parametrize("args,code", PAGED + [
    (dict(T=-1), SHAPE), (dict(B=1 << 10, T=(1 << 20) + 1), SHAPE), (dict(rot=8), SHAPE),
    (dict(rot=80), SHAPE), (dict(mscale=-1.0), SCALE), (dict(mscale=NAN), SCALE),
    (dict(T=0, k=None), OK), (dict(Hk=0, k=None), OK), (dict(k=None), NULL), (dict(strides=None), NULL),
    (dict(v=FAKE + 8), ALIGN), (dict(counts=FAKE + 1), ALIGN), (dict(positions=FAKE + 2), ALIGN),
    (dict(freqs=FAKE + 8), ALIGN), (dict(strides=[64] * 5 + [4]), ALIGN),
    (dict(pages=1 << 25, Hk=1 << 10), SHAPE),
])
def test_append(args, code):
    assert fa.fa_cache_append(**{**APPEND, **args}) == code


READ = dict(POOL, k=FAKE, v=FAKE, N=100)


@pytest.mark.parametrize("args,code", PAGED + [
    (dict(N=-1), SHAPE), (dict(N=(1 << 30) + 1), SHAPE), (dict(B=32768), SHAPE), (dict(N=0, k=None), OK),
    (dict(v=None), NULL), (dict(k=FAKE + 4), ALIGN),
])
def test_read(args, code):
    assert fa.fa_cache_read(**{**READ, **args}) == code


DEC = dict(POOL, q=FAKE, o=FAKE, lse=FAKE, H=6, Nq=4, window=0, sinks=0, scale=0.1, workspace=FAKE,
           workspace_bytes=1 << 40)


@pytest.mark.parametrize("args,code", PAGED + [
    (dict(H=-6), SHAPE), (dict(H=7), SHAPE), (dict(Hk=0), SHAPE), (dict(H=0), SHAPE), (dict(Nq=0), SHAPE),
    (dict(Nq=17), SHAPE), (dict(window=-1), SHAPE), (dict(sinks=-1), SHAPE), (dict(scale=0.0), SCALE),
    (dict(scale=INF), SCALE), (dict(H=0, Hk=0, q=None), OK), (dict(q=None), NULL), (dict(o=None), NULL),
    (dict(lse=None), NULL), (dict(q=FAKE + 8), ALIGN), (dict(o=FAKE + 8), ALIGN), (dict(lse=FAKE + 2), ALIGN),
    (dict(B=1 << 17, H=1 << 13, Hk=1 << 13), SHAPE),           # rows
])
def test_decode(args, code):
    assert fa.fa_decode_paged(**{**DEC, **args}) == code


@pytest.mark.parametrize("B,Hk,G,Nq,d,per_seq,ok", [
    # units times (tiles of a capacity + 1) stay below 2^31: up to 16 rows a key/value head tiles
    # of 32 keys at d = 128 and of 64 at 64, for more rows units of 128 and tiles of 128 keys
    (1 << 10, 1 << 10, 1, 1, 128, 2047, False), (1 << 10, 1 << 10, 1, 1, 128, 2046, True),
    (1 << 10, 1 << 10, 1, 1, 64, 4094, False), (1 << 10, 1 << 10, 1, 1, 64, 4092, True),
    (1 << 10, 1 << 9, 1, 16, 128, 4095, False), (1 << 10, 1 << 9, 1, 16, 128, 4094, True),
    (1 << 10, 1 << 8, 2, 16, 128, 32764, False), (1 << 10, 1 << 8, 2, 16, 64, 32760, True),
    (1 << 10, 1 << 7, 9, 16, 64, 32764, False), (1 << 10, 1 << 7, 9, 16, 128, 32760, True),
])
def test_units_times_tiles(lib, B, Hk, G, Nq, d, per_seq, ok):
    if ok and torch.cuda.is_available():
        pytest.skip("a GPU is present")
    H = Hk * G
    a = dict(DEC, B=B, H=H, Hk=Hk, Nq=Nq, d=d, pages=3, page_size=32, pages_per_seq=per_seq)
    assert fa.fa_decode_paged(**a) == (fa.FA_ERR_DEVICE if ok else SHAPE)
    out = ctypes.c_size_t(0)
    assert lib.fa_decode_paged_workspace_size(B, H, Hk, Nq, d, 32, per_seq, ctypes.byref(out)) == \
        (fa.FA_ERR_DEVICE if ok else SHAPE)


def test_workspace_size_refusals(lib):
    out = ctypes.c_size_t(7)
    size = lib.fa_decode_paged_workspace_size
    assert size(1, 2, 1, 4, 64, 32, 4, None) == NULL
    for args, code in (((1, 2, 0, 4, 64, 32, 4), SHAPE), ((1, 2, 1, 17, 64, 32, 4), SHAPE),
                       ((1, 2, 1, 4, 32, 32, 4), WIDTH), ((1, 2, 1, 4, 64, 20, 4), SHAPE),
                       ((0, 2, 1, 4, 64, 32, 4), OK)):
        assert size(*args, ctypes.byref(out)) == code
    assert out.value == 0


def test_a_valid_call_needs_the_device():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert fa.fa_rotary(**ROT) == fa.FA_ERR_DEVICE
    assert fa.fa_rotary(**{**ROT, "Hk": 0, "k": None, "k_out": None}) == fa.FA_ERR_DEVICE
    assert fa.fa_cache_append(**APPEND) == fa.FA_ERR_DEVICE
    assert fa.fa_cache_append(**{**APPEND, "freqs": None, "rot": 0, "mscale": 0.0}) == fa.FA_ERR_DEVICE
    assert fa.fa_cache_read(**READ) == fa.FA_ERR_DEVICE
    assert fa.fa_decode_paged(**DEC) == fa.FA_ERR_DEVICE


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_rotary():
    q, k, f = t(1, 4, 8, 64), t(1, 2, 8, 64), fa.rotary_frequencies(32)
    for call in (fa.rotary_forward, fa.rotary_backward, fa.rotary_embedding):
        with pytest.raises(TypeError):
            call(q, k.half(), f)
        with pytest.raises(TypeError):
            call(q.float(), k.float(), f)
        for a, b in ((q[0], k), (q, t(2, 2, 8, 64)), (q, t(1, 2, 9, 64)), (q, t(1, 2, 8, 128)), (q, k)):
            with pytest.raises(ValueError):     # the last: host tensors
                call(a, b, f)


def test_rotary_embedding_is_differentiable_once(monkeypatch):
    """As the attention wrappers: a second differentiation raises."""
    monkeypatch.setattr(fa, "rotary_forward", lambda q, k, *a, **kw: ((3.0 * q).detach(), None))
    monkeypatch.setattr(fa, "rotary_backward", lambda q, k, *a, **kw: ((3.0 * q).detach(), None))
    q = torch.ones(1, 1, 5, 8, requires_grad=True)
    y, none = fa.rotary_embedding(q, None, fa.rotary_frequencies(16))
    assert none is None
    (g,) = torch.autograd.grad((y ** 2).sum(), q, create_graph=True)
    assert torch.equal(g, torch.full_like(g, 18.0))
    with pytest.raises(RuntimeError, match="once_differentiable"):
        ((g ** 2).sum() + (q ** 2).sum()).backward()


def test_binding_cache():
    with pytest.raises(ValueError):
        fa.make_paged_cache(4, 2, 24, 64, device="cpu")
    with pytest.raises(TypeError):
        fa.make_paged_cache(4, 2, 32, 64, dtype=torch.uint8, device="cpu")
    cache = fa.make_paged_cache(4, 2, 32, 64, device="cpu")
    assert cache.k.dtype == torch.float8_e4m3fn and cache.k.shape == (4, 2, 32, 64)
    assert cache.v_scale.shape == (4, 2)
    table, lens = t(1, 2, dtype=torch.int32), t(1, dtype=torch.int32)
    k, q = t(1, 2, 3, 64), t(1, 4, 3, 64)
    calls = [lambda c, tb, n: fa.cache_append(k, k, c, tb, n), lambda c, tb, n: fa.cache_read(c, tb, n),
             lambda c, tb, n: fa.attention_decode_paged(q, c, tb, n)]
    for call in calls:
        with pytest.raises(ValueError):
            call(cache, table, lens)                                      # host tensors
        with pytest.raises(TypeError):
            call(cache._replace(k=cache.k.view(torch.uint8)), table, lens)
        with pytest.raises(TypeError):
            call(cache._replace(v=cache.v.view(torch.int8)), table, lens)
    with pytest.raises(TypeError):
        fa.cache_append(k, k.half(), cache, table, lens)
    with pytest.raises(ValueError):
        fa.cache_append(k, t(1, 2, 4, 64), cache, table, lens)
    with pytest.raises(TypeError):
        fa.cache_read(cache, table, lens, dtype=torch.float32)


@pytest.mark.parametrize("rot", [16, 48, 128])
def test_frequencies(rot):
    """Against the formulas in exact steps: turns in units of 2^-64, off by the
    rounding of the angle in float64 (2^-50 of it covers power and quotient)."""
    def turns(f):
        return [x % 2 ** 64 / 2 ** 64 for x in f.tolist()]

    def close(f, angles):
        for a, b in zip(turns(f), angles):
            assert abs(a - b / (2 * math.pi)) <= 2.0 ** -48 * b + 2.0 ** -64
        assert f.dtype == torch.int64 and f.shape == (rot // 2,)
    w = [10000.0 ** (-2 * j / rot) for j in range(rot // 2)]
    close(fa.rotary_frequencies(rot), w)
    close(fa.rotary_frequencies(rot, 500.0), [500.0 ** (-2 * j / rot) for j in range(rot // 2)])
    close(fa.rotary_frequencies(rot, scaling="linear", factor=4.0), [x / 4 for x in w])
    b = fa.rotary_frequencies(rot, scaling="base", factor=8.0)
    assert turns(b)[0] == turns(fa.rotary_frequencies(rot))[0]
    assert turns(b)[-1] == pytest.approx(w[-1] / 8 / (2 * math.pi), rel=1e-12)
    parts = turns(fa.rotary_frequencies(rot, scaling="parts", factor=16.0, original_length=4096))
    for a, x in zip(parts, w):
        n, a = 4096 * x / (2 * math.pi), a * 2 * math.pi
        if n >= 32:
            assert a == pytest.approx(x, rel=1e-12)
        elif n <= 1:
            assert a == pytest.approx(x / 16, rel=1e-12)
        else:
            assert x / 16 < a < x
    # more than half a turn a position: the number wraps as the kernels' does
    assert 0.5 < turns(fa.rotary_frequencies(rot, scaling="linear", factor=0.2))[0] < 1.0
    for bad in (dict(rot=8), dict(rot=24), dict(rot=rot, scaling="other"), dict(rot=rot, base=-1.0),
                dict(rot=rot, scaling="parts"), dict(rot=rot, scaling="linear", factor=0.0)):
        with pytest.raises(ValueError):
            fa.rotary_frequencies(**bad)
