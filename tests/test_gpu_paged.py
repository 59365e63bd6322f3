"""The paged 8-bit cache: appending (fa_cache_append), reading back
(fa_cache_read) and decoding over it (fa_decode_paged), each against its
definition in float64, and a serving run of all of them together."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_14_gb300 as fa
import paged_common as pc
from gpu_common import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def status_ok():
    torch.cuda.synchronize()
    code, word = fa.fa_status()
    assert code == fa.FA_OK, f"device status {word:#x}"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def deal(B, per, pages, seed):
    """A page table of distinct pages."""
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(pages, generator=g)[:B * per].view(B, per).int().cuda()


def clone(cache):
    return fa.PagedCache(*(x.clone() for x in cache))


# ---------------------------------------------------------------- append

def check_append(before, after, k, v, table, lens, counts, code, w=None, mscale=1.0, inter=False,
                 positions=None):
    """The cache after an append against the definition: scales, new codes, the
    earlier codes of pages whose scale rose, and everything else untouched."""
    B, Hk, T, d = k.shape
    pages, _, page, _ = before.k.shape
    table = table.cpu().numpy()
    for name, x in (("k", k), ("v", v)):
        x = x.double().cpu().numpy()
        r = np.zeros_like(x)
        old, new = pc.numpy_codes(getattr(before, name)), pc.numpy_codes(getattr(after, name))
        old_bits, new_bits = (getattr(c, name).view(torch.uint8).cpu().numpy() for c in (before, after))
        s0, s1 = (getattr(c, name + "_scale").double().cpu().numpy() for c in (before, after))
        left = np.ones((pages, Hk, page), dtype=bool)          # slots not yet accounted for
        scale_left = np.ones((pages, Hk), dtype=bool)
        for b in range(B):
            c = max(0, min(T, counts[b]))
            first = max(lens[b], 0) - c
            slots = first + np.arange(c)
            if name == "k" and w is not None:
                pos = slots if positions is None else positions[b, :c]
                x[b, :, :c], r[b, :, :c] = pc.rotate(x[b, :, :c], pos, w, mscale, inter)
            slots_ok = (slots >= 0) & (slots < table.shape[1] * page)
            for n in sorted(set((slots[slots_ok] // page).tolist())):
                p = int(table[b, n])
                if not 0 <= p < pages:
                    continue
                mine = slots_ok & (slots // page == n)
                tok, row = np.flatnonzero(mine), slots[mine] - n * page
                val, err = x[b][:, tok], r[b][:, tok]             # [Hk, m, d]
                keep = np.arange(row[0])
                for h in range(Hk):
                    scale_left[p, h] = False
                    left[p, h, row] = False
                    top, e = np.abs(val[h]).max(), err[h].max()
                    s, before_s = s1[p, h], (s0[p, h] if len(keep) else 0.0)
                    if not np.isfinite(val[h]).all() or np.isnan(before_s):
                        assert np.isnan(s), (name, p, h)
                        left[p, h, keep] = False                   # their codes stay
                        assert (old_bits[p, h, keep] == new_bits[p, h, keep]).all()
                        continue
                    if s == before_s:
                        low = 2.0 ** -100
                        need = top / (448 if code == "e4m3" else 127)
                        assert need <= max(s, low) * (1 + 2.0 ** -22) + e
                        assert (old_bits[p, h, keep] == new_bits[p, h, keep]).all()
                    else:
                        assert s > before_s
                        if code == "e4m3":
                            assert np.frexp(s)[0] == 0.5 and top - e <= 448 * s
                            assert s == 2.0 ** -100 or top + e > 224 * s
                        elif s != 2.0 ** -100:
                            assert abs(s - top / 127) <= (e + 2.0 ** -23 * top) / 127
                        f = old[p, h, keep] * (before_s / s)
                        off = np.abs(new[p, h, keep] - f)
                        assert (off <= pc.half_code(f, code) + np.abs(f) * 2.0 ** -21).all(), (name, p, h)
                    left[p, h, keep] = False
                    y = val[h] / s
                    off = np.abs(new[p, h, row] - y)
                    tol = pc.half_code(np.abs(y) + err[h] / s, code) + err[h] / s + np.abs(y) * 2.0 ** -22
                    assert (off <= tol).all(), (name, b, n, h, np.max(off - tol))
        assert (old_bits[left] == new_bits[left]).all(), f"{name}: slots that no token goes to"
        same = getattr(before, name + "_scale") == getattr(after, name + "_scale")
        assert same.cpu().numpy()[scale_left].all(), f"{name}: scales of pages without tokens"


APPEND = [
    # B, Hk, T, page, per, d, code, dtype, rot, interleaved, lens (after), counts, std
    (1, 1, 1, 16, 1, 64, "e4m3", "bf16", 64, False, [1], None, 1.0),
    (2, 3, 1, 32, 3, 64, "int8", "fp16", 32, True, [33, 96], None, 1.0),
    (3, 2, 5, 16, 4, 128, "e4m3", "fp16", 128, False, [5, 18, 64], None, 1.0),
    (3, 2, 40, 48, 3, 64, "int8", "bf16", 48, False, [144, 41, 40], [40, 7, 0], 1.0),
    (2, 9, 100, 64, 5, 128, "e4m3", "bf16", 96, True, [300, 130], [100, 99], 2.0),
    (2, 1, 257, 128, 4, 128, "int8", "fp16", 0, False, [400, 257], None, 0.01),
    (1, 2, 30, 16, 2, 64, "e4m3", "bf16", 16, False, [40], None, 1.0),          # past the capacity
    (2, 2, 30, 80, 2, 128, "int8", "bf16", 128, True, [12, -4], None, 1.0),     # before slot 0
    (70, 2, 3, 16, 2, 64, "e4m3", "fp16", 64, False, [3 + 29 * b % 30 for b in range(70)], None, 30.0),
    (2, 2, 20, 16, 3, 64, "e4m3", "bf16", 64, False, [30, 20], [25, -3], 1e-36),  # least scales
    (3, 5, 8, 16, 3, 128, "int8", "bf16", 112, True, [20, 8, 48], [8, 3, 5], 4.0),  # a warp's most
    (3, 5, 9, 16, 3, 64, "e4m3", "fp16", 32, False, [20, 9, 48], [9, 3, 5], 4.0),
    (2, 3, 300, 128, 3, 128, "e4m3", "bf16", 128, False, [384, 310], [300, 299], 1.0),
]


@pytest.mark.parametrize("case", APPEND, ids=["-".join(map(str, c[:10])) for c in APPEND])
@pytest.mark.parametrize("own_positions", [False, True])
def test_append(case, own_positions):
    B, Hk, T, page, per, d, code, dtype, rot, inter, lens, counts, std = case
    pages = B * per + 2
    cache = pc.random_cache(pages, Hk, page, d, code, seed=T, spread=2.0)
    table = deal(B, per, pages, seed=T + 1)
    kv = pc.normal((B, T, 2 * Hk, d), dtype, T + 2, std).cuda()
    k, v = kv[:, :, :Hk].transpose(1, 2), kv[:, :, Hk:].transpose(1, 2)
    if T >= 3:
        v = v.contiguous()
        v[:, 0, 1] = 0                                # a row of zeros
    freqs = fa.rotary_frequencies(rot, device="cuda") if rot else None
    g = torch.Generator().manual_seed(T + 3)
    pos = torch.randint(0, 1 << 18, (B, T), generator=g, dtype=torch.int32) if own_positions else None
    before = clone(cache)
    fa.cache_append(k, v, cache, table, ints(lens), counts=None if counts is None else ints(counts),
                    freqs=freqs, positions=None if pos is None else pos.cuda(), interleaved=inter,
                    mscale=1.25 if rot else 1.0)
    status_ok()
    w = pc.frequencies(rot) if rot else None
    check_append(before, cache, k, v, table, lens, [T] * B if counts is None else counts, code, w,
                 1.25, inter, None if pos is None else pos.numpy())
    # the same append again changes nothing: the scales have what they need
    again = clone(cache)
    fa.cache_append(k, v, again, table, ints(lens), counts=None if counts is None else ints(counts),
                    freqs=freqs, positions=None if pos is None else pos.cuda(), interleaved=inter,
                    mscale=1.25 if rot else 1.0)
    status_ok()
    assert all(torch.equal(a.view(torch.uint8) if a.element_size() == 1 else a,
                           b.view(torch.uint8) if b.element_size() == 1 else b)
               for a, b in zip(cache, again))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_append_token_by_token(code):
    """A page that fills one token at a time, magnitudes growing, each step from
    the cache that the last one left."""
    B, Hk, page, d = 2, 2, 32, 64
    cache = fa.make_paged_cache(5, Hk, page, d, pc.CODE_DT[code])
    table = ints([[3, 1], [0, 4]])
    for i in range(40):
        k, v = (pc.normal((B, Hk, 1, d), "bf16", 7 * i + x, 1.0 + i / 8).cuda() for x in (0, 1))
        before, lens = clone(cache), [i + 1, i + 3]
        fa.cache_append(k, v, cache, table, ints(lens))
        check_append(before, cache, k, v, table, lens, [1, 1], code)
    status_ok()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_append_leaves_bad_pages_and_nonfinite(code):
    """Table entries outside the pool are skipped, also around its ends; a NaN or
    an infinity makes its page's scale NaN for that head, until the page starts
    again."""
    B, Hk, T, page, d = 5, 2, 20, 16, 64
    cache = pc.random_cache(4, Hk, page, d, code, seed=1)
    table = ints([[-1, 2], [4, 0], [2 ** 31 - 1, -2 ** 31], [1, 3], [-7, 99]])
    k, v = pc.normal((B, Hk, T, d), "bf16", 2).cuda(), pc.normal((B, Hk, T, d), "bf16", 3).cuda()
    k[3, 0, 3, 5] = float("nan")
    v[3, 1, 19, 63] = float("-inf")
    lens = [T] * B
    before = clone(cache)
    fa.cache_append(k, v, cache, table, ints(lens))
    status_ok()
    check_append(before, cache, k, v, table, lens, lens, code)
    ks, vs = cache.k_scale.cpu(), cache.v_scale.cpu()
    assert torch.isnan(ks[1, 0]) and torch.isfinite(ks[1, 1]) and torch.isnan(vs[3, 1])
    # a finite token behind it leaves the NaN, a new start clears it
    one = pc.normal((1, Hk, 1, d), "bf16", 4).cuda()
    row = ints([[1, 3]])
    fa.cache_append(one, one, cache, row, ints([9]))
    assert torch.isnan(cache.k_scale[1, 0])
    fa.cache_append(one, one, cache, row, ints([1]))
    status_ok()
    assert torch.isfinite(cache.k_scale[1]).all()


@pytest.mark.parametrize("T", [1, 40])
def test_append_in_a_graph(T):
    """A captured append reads lengths and counts when it is replayed: the steps of
    a decoding loop by one graph, as by eager calls."""
    B, Hk, page, per, d = 3, 2, 32, 6, 64
    caches = [fa.make_paged_cache(B * per, Hk, page, d) for _ in range(2)]
    table, f = deal(B, per, B * per, seed=30), fa.rotary_frequencies(64, device="cuda")
    k, v = (torch.zeros(B, Hk, T, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n, c = ints([0] * B), ints([0] * B)
    fa.cache_append(k, v, caches[1], table, n, counts=c, freqs=f)         # writes nothing
    assert not any(x.view(torch.uint8).any() if x.element_size() == 1 else x.any() for x in caches[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.cache_append(k, v, caches[1], table, n, counts=c, freqs=f)
    for step in range(4):
        k.copy_(pc.normal((B, Hk, T, d), "bf16", 40 + step).cuda())
        v.copy_(pc.normal((B, Hk, T, d), "bf16", 50 + step).cuda())
        c.copy_(ints([T, max(T - step, 1), 0]))
        n.add_(c)
        fa.cache_append(k, v, caches[0], table, n, counts=c, freqs=f)
        g.replay()
    status_ok()
    assert all(torch.equal(a.view(torch.uint8) if a.element_size() == 1 else a,
                           b.view(torch.uint8) if b.element_size() == 1 else b) for a, b in zip(*caches))


# ---------------------------------------------------------------- read

@pytest.mark.parametrize("B,Hk,page,per,d,code,dtype,lens,length", [
    (1, 1, 16, 1, 64, "e4m3", "bf16", [1], None), (3, 2, 48, 3, 128, "int8", "fp16", [144, 0, 50], None),
    (2, 3, 32, 40, 64, "e4m3", "fp16", [1279, 9999], 1300), (2, 5, 128, 4, 128, "int8", "bf16", [-3, 500], 77),
])
def test_read(B, Hk, page, per, d, code, dtype, lens, length):
    pages = B * per + 1
    cache = pc.random_cache(pages, Hk, page, d, code, seed=B, spread=3.0)
    table = deal(B, per, pages, seed=2)
    if per > 2:
        table[0, 1], table[-1, 0] = -1, pages                      # pages outside the pool
    k, v = fa.cache_read(cache, table, ints(lens), length=length, dtype=pc.DT[dtype])
    status_ok()
    N = per * page if length is None else length
    assert k.shape == v.shape == (B, Hk, N, d)
    t = table.cpu().numpy()
    for got, codes, scales in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        want = torch.zeros(B, Hk, N, d)
        val = codes.float().cpu() * scales.cpu()[..., None, None]
        for b in range(B):
            for n in range(min(N, max(lens[b], 0), per * page)):
                p = int(t[b, n // page])
                if 0 <= p < pages:
                    want[b, :, n] = val[p, :, n % page]
        assert torch.equal(got.cpu(), want.to(pc.DT[dtype]))       # one product, rounded once more
    out = (torch.empty_like(k), torch.empty_like(v))
    assert fa.cache_read(cache, table, ints(lens), length=length, dtype=pc.DT[dtype], out=out)[0] is out[0]
    assert torch.equal(out[0], k) and torch.equal(out[1], v)


# ---------------------------------------------------------------- decoding

@pytest.mark.parametrize("d", [64, 128])
def test_read_into_any_aligned_buffer(d):
    """Outputs that begin at a multiple of 16 bytes, of 32 or not."""
    cache = pc.random_cache(5, 2, 48, d, "e4m3", seed=3)
    table, lens = ints([[4, 1], [0, 2]]), ints([70, 33])
    want = fa.cache_read(cache, table, lens, length=77)
    n = want[0].numel()
    for offsets in ((0, 8), (8, 16), (24, 8)):
        whole = [torch.full((n + 32,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        out = [x[o:o + n].view(2, 2, 77, d) for x, o in zip(whole, offsets)]
        fa.cache_read(cache, table, lens, length=77, out=out)
        status_ok()
        for x, y, z, o in zip(out, want, whole, offsets):
            assert torch.equal(x, y)
            assert (z[:o] == 7).all() and (z[o + n:] == 7).all()


DECODE = [
    # B, H, Hk, Nq, page, per, d, code, dtype, window, sinks, lens
    (1, 1, 1, 1, 16, 1, 64, "e4m3", "bf16", None, 0, [1]),
    (1, 1, 1, 1, 16, 1, 128, "int8", "fp16", None, 0, [0]),
    (1, 8, 2, 1, 64, 16, 128, "e4m3", "bf16", None, 0, [1000]),
    (2, 4, 4, 3, 32, 20, 64, "int8", "fp16", None, 0, [640, 333]),
    (3, 6, 2, 16, 48, 20, 128, "e4m3", "fp16", 300, 5, [900, 7, 0]),          # rows before key 0
    (2, 16, 1, 16, 16, 60, 64, "int8", "bf16", 700, 16, [950, 801]),          # 256 rows
    (1, 24, 1, 2, 80, 9, 128, "int8", "bf16", None, 0, [700]),                # 48 rows
    (5, 2, 2, 3, 128, 4, 64, "e4m3", "bf16", 17, 130, [500, 499, 131, 146, 2]),
    (2, 3, 3, 2, 32, 11, 128, "int8", "fp16", 1, 0, [333, 40]),
    (40, 12, 1, 1, 32, 16, 128, "e4m3", "fp16", 200, 4, [11 * b % 501 for b in range(40)]),
    (1, 2, 1, 8, 64, 80, 128, "e4m3", "bf16", 4000, 1, [4999]),
    (300, 2, 2, 1, 16, 9, 64, "int8", "bf16", 64, 2, [(7 * b) % 131 for b in range(300)]),
    (2, 40, 8, 4, 96, 30, 64, "e4m3", "fp16", None, 0, [2880, 2001]),
    (3, 5, 5, 5, 112, 5, 64, "int8", "bf16", 2 ** 31 - 1, 7, [560, 3, -9]),
    # rows a key/value head: 9, 16 (one warp's most), 17 to 128 (one unit), 144
    (2, 9, 1, 1, 16, 40, 128, "int8", "bf16", None, 0, [640, 77]),
    (3, 4, 1, 4, 64, 12, 64, "e4m3", "fp16", 90, 2, [768, 5, 300]),
    (2, 17, 1, 1, 128, 6, 128, "e4m3", "bf16", None, 0, [768, 129]),
    (4, 12, 2, 6, 16, 20, 64, "int8", "fp16", 40, 130, [320, 190, 4, 0]),
    (1, 8, 1, 16, 48, 60, 128, "e4m3", "bf16", None, 0, [2880]),
    (2, 9, 1, 16, 32, 30, 64, "e4m3", "bf16", 500, 3, [960, 10]),
    (1, 9, 1, 16, 80, 12, 128, "int8", "fp16", None, 0, [950]),
    (70, 20, 1, 1, 32, 5, 128, "int8", "bf16", None, 0, [13 * b % 161 for b in range(70)]),
]


def masks_of(table, pages, page, Nq, lens, win, sinks):
    cap = table.shape[1] * page
    t = table.cpu().numpy()
    ok = np.repeat((t >= 0) & (t < pages), page, axis=1)
    win = cap + 99 if win is None else win
    return [pc.window_mask(Nq, cap, max(0, min(n, cap)), "bottom_right", win, sinks) & ok[b]
            for b, n in enumerate(lens)]


def run_decode(q, cache, table, lens, **kw):
    o, lse = fa.attention_decode_paged(q, cache, table, ints(lens), **kw)
    status_ok()
    return {"o": o, "lse": lse}


@pytest.mark.parametrize("case", DECODE, ids=["-".join(map(str, c[:11])) for c in DECODE])
def test_decode_against_definition(case):
    B, H, Hk, Nq, page, per, d, code, dtype, win, sinks, lens = case
    pages = B * per + 2
    cache = pc.random_cache(pages, Hk, page, d, code, seed=H, spread=2.0)
    table = deal(B, per, pages, seed=H + 1)
    q = pc.normal((B, H, Nq, d), dtype, H + 2).cuda()
    got = run_decode(q, cache, table, lens, window=win, sinks=sinks)
    k, v = pc.values(cache, table, lens)
    masks = masks_of(table, pages, page, Nq, lens, win, sinks)
    pc.check(got, *pc.reference(q, k, v, masks, pc.scale_of(d), dtype), "decode")
    # again, into the caller's buffers: bit for bit
    ws = fa.make_paged_workspace(q, cache, table)
    out, lse = torch.full_like(q, float("nan")), torch.full((B, H, Nq), float("nan"), device="cuda")
    fa.attention_decode_paged(q, cache, table, ints(lens), window=win, sinks=sinks, out=out, lse=lse,
                              workspace=ws)
    status_ok()
    assert torch.equal(out, got["o"]) and torch.equal(lse, got["lse"])


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H", [4, 8, 24])     # 8, 16 and 48 rows a key/value head
def test_unseen_slots_may_hold_anything(code, d, H):
    """NaN codes and NaN or infinite scales in slots and pages that nobody sees,
    table entries that name no page, and tokens that do not see the last page."""
    B, Hk, Nq, page, per = 3, 2, 4, 16, 12
    pages = B * per + 3
    cache = pc.random_cache(pages, Hk, page, d, code, seed=3)
    table = deal(B, per, pages, seed=4)
    lens, win, sinks = [150, 97, 20], 50, 3
    q = pc.normal((B, H, Nq, d), "bf16", 5).cuda()
    k, v = pc.values(cache, table, lens)
    masks = masks_of(table, pages, page, Nq, lens, win, sinks)
    bad = clone(cache)
    bits = [x.view(torch.uint8) for x in (bad.k, bad.v)]
    for b in range(B):
        seen = masks[b].any(0)
        for n in range(per):
            rows = ~seen[n * page:(n + 1) * page]
            p = int(table[b, n])
            for x in bits:
                x[p, :, torch.from_numpy(rows).cuda()] = 0x7f if code == "e4m3" else 0x80
            if rows.all():
                bad.k_scale[p], bad.v_scale[p] = float("nan"), (float("inf"), 1e38, -1e30)[n % 3]
    free = [p for p in range(pages) if p not in set(table.flatten().tolist())]
    for x in bits:
        x[free] = 0x7f
    bad.k_scale[free] = bad.v_scale[free] = float("nan")
    got = run_decode(q, bad, table, lens, window=win, sinks=sinks)
    val, tol = pc.reference(q, k, v, masks, pc.scale_of(d), "bf16")
    pc.check(got, val, tol, "unseen")
    # pages behind the sequences and before the window are not named at all
    gone = table.clone()
    for b in range(B):
        for n in range(per):
            if not masks[b].any(0)[n * page:(n + 1) * page].any():
                gone[b, n] = (-1, pages, 2 ** 31 - 1, -2 ** 31)[n % 4]
    again = run_decode(q, cache, gone, lens, window=win, sinks=sinks)
    assert torch.equal(again["o"], got["o"]) and torch.equal(again["lse"], got["lse"])
    # a missing page inside the window: its keys are not seen
    hole = table.clone()
    hole[0, 7] = -1
    m2 = masks_of(hole, pages, page, Nq, lens, win, sinks)
    pc.check(run_decode(q, cache, hole, lens, window=win, sinks=sinks),
             *pc.reference(q, k, v, m2, pc.scale_of(d), "bf16"), "hole")


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("H", [2, 4, 20])     # 6, 12 and 60 rows
def test_a_scale_that_is_not_finite_reaches_only_who_sees_it(page, H):
    """The last page's scale is NaN (its only token was): the tokens before it
    do not see the page and keep their results, the last one gets NaN."""
    B, Hk, Nq, d = 1, 1, 3, 128
    for which in ("k_scale", "v_scale"):
        cache = pc.random_cache(6, Hk, page, d, "e4m3", seed=6)
        table = ints([[4, 2, 0, 5]])
        lens = [3 * page + 1]
        q = pc.normal((B, H, Nq, d), "fp16", 7).cuda()
        ref = run_decode(q, cache, table, lens)
        getattr(cache, which)[5, 0] = float("nan")
        got = run_decode(q, cache, table, lens)
        assert torch.equal(got["o"][:, :, :2], ref["o"][:, :, :2])
        assert torch.equal(got["lse"][:, :, :2], ref["lse"][:, :, :2])
        assert torch.isnan(got["o"][:, :, 2]).all()


@pytest.mark.parametrize("T", [1, 3, 12])
@pytest.mark.parametrize("H", [1, 2, 10])     # 4 to 150 rows
@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_a_spoilt_token_reaches_only_who_sees_its_page(code, H, T):
    """The last append begins a page with a token that is not finite: the tokens
    before that page keep their results, the others get NaN."""
    d, page, Nq, lens = 128, 16, T + 3, 32 + T    # the append's first token begins a page
    q = pc.normal((1, H, Nq, d), "bf16", 31).cuda()
    table, results = ints([[3, 0, 2]]), []
    for spoilt in (0.0, float("nan"), float("inf")):
        cache = fa.make_paged_cache(4, 1, page, d, pc.CODE_DT[code])
        k, v = pc.normal((1, 1, lens, d), "bf16", 32).cuda(), pc.normal((1, 1, lens, d), "bf16", 33).cuda()
        fa.cache_append(k[:, :, :-T], v[:, :, :-T], cache, table, ints([lens - T]))
        v[0, 0, -T, 5] += spoilt
        fa.cache_append(k[:, :, -T:], v[:, :, -T:], cache, table, ints([lens]))
        results.append(run_decode(q, cache, table, [lens]))
    for bad in results[1:]:
        assert torch.equal(bad["o"][:, :, :3], results[0]["o"][:, :, :3])
        assert torch.equal(bad["lse"], results[0]["lse"])
        assert torch.isnan(bad["o"][:, :, 3:]).all()


@pytest.mark.parametrize("G,Nq,page,d,code", [(25, 4, 16, 128, "int8"), (25, 4, 64, 128, "e4m3"),
                                              (14, 4, 16, 128, "int8"), (25, 4, 16, 64, "e4m3"),
                                              (1, 4, 16, 128, "int8"), (4, 4, 64, 64, "e4m3")])
def test_many_runs_of_short_units(G, Nq, page, d, code):
    """Units of one to seven tiles, several to a run: every run gives the same bits."""
    B, Hk, per = 60, 4, 912 // page
    cache = pc.random_cache(B * per + 1, Hk, page, d, code, seed=2)
    table = deal(B, per, B * per + 1, seed=3)
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, per * page + 1, (B,), generator=g, dtype=torch.int32).cuda()
    q = pc.normal((B, Hk * G, Nq, d), "fp16", 5).cuda()
    ws = fa.make_paged_workspace(q, cache, table)
    want = fa.attention_decode_paged(q, cache, table, lens, workspace=ws)
    differ = torch.zeros(400, dtype=torch.bool, device="cuda")
    for i in range(400):
        o, lse = fa.attention_decode_paged(q, cache, table, lens, workspace=ws)
        differ[i] = (o != want[0]).any() | (lse != want[1]).any()
    status_ok()
    assert not differ.any()


@pytest.mark.parametrize("heads", [1, 4, 12])   # 4, 16 and 48 rows
def test_nonfinite_scores(heads):
    """A NaN or +inf score gives NaN, one of -inf weighs nothing."""
    cache = pc.random_cache(4, 1, 32, 64, "int8", seed=8)
    cache.k.view(torch.uint8)[:] = 0
    cache.k[1, 0, 3, 0] = 1                    # key 35's first element
    table, lens = ints([[0, 1]]), [40]
    q = torch.zeros(1, 4 * heads, 1, 64, dtype=torch.float16, device="cuda")
    cache.k_scale[1] = float("inf")            # 0 * inf is NaN: every score of the page is
    assert torch.isnan(run_decode(q, cache, table, lens)["o"]).all()
    cache.k_scale[1] = 3e38
    q[0, 0, 0, 0], q[0, 1, 0, 0], q[0, 2, 0, 0] = 6e4, -6e4, float("nan")
    q = q[:, :4].repeat(1, heads, 1, 1)
    got = run_decode(q, cache, table, lens)
    for x in got.values():
        assert torch.equal(x[:, :4].repeat(1, heads, *[1] * (x.dim() - 2)).nan_to_num(7e4), x.nan_to_num(7e4))
    assert torch.isnan(got["o"][0, 0]).all() and torch.isnan(got["lse"][0, 0]).all()
    assert torch.isnan(got["o"][0, 2]).all()
    _, v = pc.values(cache, table, lens)
    for h, keys in ((1, [j for j in range(40) if j != 35]), (3, range(40))):
        want = v[0, 0][list(keys)].mean(0)
        tol = (2.0 ** -10 + 2.0 ** -17) * np.abs(v[0, 0][:40]).mean(0) + 2.0 ** -11 * np.abs(want) + 2.0 ** -19
        assert (np.abs(got["o"][0, h, 0].double().cpu().numpy() - want) <= tol).all()
        assert abs(got["lse"][0, h, 0].item() - np.log(len(list(keys)))) <= 2.0 ** -17


@pytest.mark.parametrize("G", [1, 2, 5])
def test_wide_ranges(G):
    """Queries of extreme magnitude and pages of very different scales: large
    values in pages of no weight, the weight in pages of small ones."""
    B, H, Hk, Nq, page, d = 1, 8 * G, 1, 1, 32, 128
    cache = pc.random_cache(8, Hk, page, d, "e4m3", seed=9)
    table, lens = ints([[7, 6, 5, 4, 3, 2, 1, 0]]), [250]
    cache.v_scale[7:] = 2.0 ** 60 / 448
    cache.v_scale[3] = 2.0 ** -40
    q = pc.normal((B, H, Nq, d), "bf16", 10)
    q = (q.float() * torch.exp2(torch.tensor([-120.0, -60, -20, 0, 0, 2, 2, 3] * G))[None, :, None, None]).bfloat16().cuda()
    for ks in (1.0, 1e-30):
        cache.k_scale[:] = ks / 100
        scale = pc.scale_of(d) / ks
        got = run_decode(q, cache, table, lens, scale=scale)
        k, v = pc.values(cache, table, lens)
        pc.check(got, *pc.reference(q, k, v, masks_of(table, 8, page, Nq, lens, None, 0), scale, "bf16"), "wide")


def test_pool_beyond_two_gigabytes():
    """Rows past 2^31 bytes of the pool, written, read and attended."""
    Hk, page, d = 8, 128, 128
    pages = 2 ** 31 // (Hk * page * d) + 40
    cache = fa.make_paged_cache(pages, Hk, page, d)
    table = ints([[pages - 1, 0, pages - 30], [5, pages - 2, pages - 17]])
    lens, T = [300, 384], 384
    k, v = pc.normal((2, Hk, T, d), "bf16", 11).cuda(), pc.normal((2, Hk, T, d), "bf16", 12).cuda()
    fa.cache_append(k, v, cache, table, ints(lens), counts=ints(lens))
    rk, rv = fa.cache_read(cache, table, ints(lens))
    status_ok()
    for b, n in enumerate(lens):
        for x, y in ((rk, k), (rv, v)):
            # a code's half step relative to its value, 2^-4, or the smallest codes'
            e = (x[b, :, :n].float() - y[b, :, :n].float()).abs()
            assert (e <= y[b, :, :n].float().abs() * (2.0 ** -4 + 2.0 ** -8) + 2.0 ** -16).all()
            assert not x[b, :, n:].any()
    q = pc.normal((2, Hk, 2, d), "bf16", 13).cuda()
    got = run_decode(q, cache, table, lens)
    small = fa.PagedCache(*(x[table.flatten().long()] if x.element_size() > 1 else
                            x.view(torch.uint8)[table.flatten().long()].view(x.dtype) for x in cache))
    t2 = ints([[0, 1, 2], [3, 4, 5]])
    ref = run_decode(q, small, t2, lens)
    assert torch.equal(got["o"], ref["o"]) and torch.equal(got["lse"], ref["lse"])
    kk, vv = pc.values(small, t2, lens)
    pc.check(got, *pc.reference(q, kk, vv, masks_of(t2, 6, page, 2, lens, None, 0), pc.scale_of(d), "bf16"), "far")


@pytest.mark.parametrize("H", [8, 24, 64])
def test_two_graphs_and_streams(H):
    """Two captured calls with workspaces of their own replayed together on two
    streams, and a call on a stream that is not current."""
    B, Hk, Nq, page, per, d = 4, 2, 1, 32, 40, 128
    pages = B * per
    cache = pc.random_cache(pages, Hk, page, d, "e4m3", seed=14)
    table, lens = deal(B, per, pages, seed=15), [1280, 700, 33, 1000]
    qs = [pc.normal((B, H, Nq, d), "bf16", s).cuda() for s in (16, 17)]
    refs = [run_decode(q, cache, table, lens) for q in qs]
    n = ints(lens)
    graphs, outs = [], []
    for q in qs:
        ws = fa.make_paged_workspace(q, cache, table)
        o, lse = torch.empty_like(q), torch.empty((B, H, Nq), device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fa.attention_decode_paged(q, cache, table, n, out=o, lse=lse, workspace=ws)
        graphs.append((g, ws))
        outs.append((o, lse))
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(5):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    status_ok()
    for (o, lse), ref in zip(outs, refs):
        assert torch.equal(o, ref["o"]) and torch.equal(lse, ref["lse"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = fa.attention_decode_paged(qs[0], cache, table, n, stream=side)
    side.synchronize()
    assert torch.equal(o, refs[0]["o"]) and torch.equal(lse, refs[0]["lse"])
    status_ok()


def test_refusals_on_the_device():
    cache = fa.make_paged_cache(6, 2, 16, 64)
    table, lens = ints([[0, 1], [2, 3]]), ints([20, 20])
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16, device="cuda")
    ok = fa.attention_decode_paged(q, cache, table, lens)
    assert ok[0].shape == q.shape
    tables = [table.long(), table[0], table.t(), table.cpu()]
    lengths = [lens.long(), lens[:1], lens.cpu(), table]
    for c, tb, n in ([(cache, x, lens) for x in tables] + [(cache, table, x) for x in lengths] +
                     [(cache._replace(k=cache.k.transpose(2, 3)), table, lens),
                      (cache._replace(v=cache.v[:5]), table, lens),
                      (cache._replace(k_scale=cache.k_scale.double()), table, lens),
                      (cache._replace(v_scale=cache.v_scale[:, :1]), table, lens)]):
        for call in (lambda: fa.attention_decode_paged(q, c, tb, n), lambda: fa.cache_read(c, tb, n),
                     lambda: fa.cache_append(k, k, c, tb, n)):
            with pytest.raises(ValueError):
                call()
    one = ints([1, 1])
    for kw in (dict(window=0), dict(sinks=-1), dict(out=q.half()), dict(lse=torch.zeros(2, 4, device="cuda")),
               dict(workspace=torch.zeros(9)), dict(q=q[:, :3].contiguous()), dict(q=q[:1]),
               dict(q=q.transpose(1, 2))):
        with pytest.raises(ValueError):
            fa.attention_decode_paged(**dict(dict(q=q, cache=cache, page_table=table, seqlens=one), **kw))
    for kw in (dict(workspace=torch.zeros(9, dtype=torch.uint8, device="cuda")),
               dict(q=q.expand(2, 4, 17, 64).contiguous())):
        with pytest.raises(fa.FaError):
            fa.attention_decode_paged(**dict(dict(q=q, cache=cache, page_table=table, seqlens=one), **kw))
    for kw in (dict(counts=one.long()), dict(positions=one), dict(k=k[:, :1], v=k[:, :1]),
               dict(k=k.transpose(2, 3), v=k.transpose(2, 3)), dict(freqs=fa.rotary_frequencies(32)),
               dict(freqs=fa.rotary_frequencies(128, device="cuda"))):
        with pytest.raises(ValueError):
            fa.cache_append(**dict(dict(k=k, v=k, cache=cache, page_table=table, seqlens=one), **kw))
    with pytest.raises(ValueError):
        fa.cache_read(cache, table, lens, length=-1)
    with pytest.raises(ValueError):
        fa.cache_read(cache, table, lens, out=(q, q))
    status_ok()


# ---------------------------------------------------------------- a run of them

@pytest.mark.parametrize("code,interleaved", [("e4m3", False), ("int8", True)])
def test_serving_run(code, interleaved):
    """A padded batch of prompts, then a chunk, then single tokens: rotation,
    append, the chunk's attention over the cache read back, decoding over the
    pages; each attention against float64 on what the cache holds, and the cache
    against the rotated keys that went in."""
    B, H, Hk, d, page, per, rot = 3, 6, 2, 64, 32, 12, 48
    cache = fa.make_paged_cache(B * per + 1, Hk, page, d, pc.CODE_DT[code])
    table = deal(B, per, B * per + 1, seed=20)
    freqs, w = fa.rotary_frequencies(rot, device="cuda"), pc.frequencies(rot)
    turn = dict(interleaved=interleaved)
    lens, scale = np.zeros(B, dtype=int), pc.scale_of(d)
    kept = [np.zeros((B, Hk, per * page, d)) for _ in range(2)]     # what went in
    for step, counts in enumerate([[70, 33, 101], [64, 64, 64]] + [[1, 1, 1]] * 6):
        T = max(counts)
        qkv = pc.normal((B, T, H + 2 * Hk, d), "bf16", 100 + step).cuda()
        q, k, v = (x.transpose(1, 2) for x in qkv.split((H, Hk, Hk), 2))
        before, lens = clone(cache), lens + np.array(counts)
        n, c = ints(lens.tolist()), ints(counts)
        fa.cache_append(k, v, cache, table, n, counts=c, freqs=freqs, **turn)
        check_append(before, cache, k, v, table, lens.tolist(), counts, code, w, 1.0, interleaved)
        for b in range(B):
            at = slice(lens[b] - counts[b], lens[b])
            pos = np.arange(at.start, at.stop)
            kept[0][b, :, at] = pc.rotate(k[b, :, :counts[b]].double().cpu().numpy(), pos, w, 1.0, interleaved)[0]
            kept[1][b, :, at] = v[b, :, :counts[b]].double().cpu().numpy()
        held = pc.values(cache, table, lens)
        if step == 0:
            # prompts: their own keys, padded queries rotated from position 0
            rq, rk = fa.rotary_forward(q, k, freqs, **turn)
            assert torch.isfinite(fa.attention_forward_window(rq, rk, v.contiguous(), 4096, causal="upper_left",
                                                              seqlens_k=c)[0]).all()
        elif T > 1:
            rq, _ = fa.rotary_forward(q, None, freqs, seqlens=n, **turn)
            ck, cv = fa.cache_read(cache, table, n)
            o, lse = fa.attention_forward_window(rq, ck, cv, 100, 4, causal="bottom_right", seqlens_k=n)
            status_ok()
            got = {"o": o, "lse": lse}
            masks = masks_of(table, B * per + 1, page, T, lens.tolist(), 100, 4)
            val, tol = pc.wc.reference(rq.cpu(), ck.cpu(), cv.cpu(), masks, scale, "bf16")
            pc.check(got, val, tol, f"chunk {step}")
        else:
            rq, _ = fa.rotary_forward(q, None, freqs, seqlens=n, **turn)
            got = run_decode(rq, cache, table, lens.tolist(), window=100, sinks=4)
            masks = masks_of(table, B * per + 1, page, T, lens.tolist(), 100, 4)
            pc.check(got, *pc.reference(rq, *held, masks, scale, "bf16"), f"token {step}")
    # the cache holds what went in: at most every raise of a scale rounded once more
    for x, y in zip(held, kept):
        for b in range(B):
            rms = np.sqrt(np.mean((x[b, :, :lens[b]] - y[b, :, :lens[b]]) ** 2))
            # a code's rounding is off by at most 2^-4 of the value (e4m3), or half of top / 127
            # with top under 8 standard deviations (int8); eight raises at most
            assert rms <= (2.0 ** -4 if code == "e4m3" else 8 * 4.0 / 127) * 1.0
    status_ok()
