"""Decoding over pages whose scales differ widely (fa_decode_paged), against the
definition in float64.

Bounds.  u = eps / 2 is half a step of the 16-bit type.  A score is a sum of d
products of exact numbers in float32, off by at most e = 128 * 2^-23 * scale *
sum |q||k|.  A weight p_j times the scale vs_j of its values' page is rounded
to half precision: 2^-11 relative (11 significant bits: steps of 2^-10 from 1 on,
half of one is off by 2^-11 of 1 at most), or half of the smallest step, 2^-25,
in the unit of O, and by no more than itself.  While the scales so far are within
2^4 of one another each is 2^2 units or more, and the half step at most 2^-27
vs_j.  Once they are not, a row's unit is at most 2^-6 of the power of two next to
2^-8 of its largest p_j vs_j, or what it was while they were, 2^-2 of its
scales then: 2^-27 max (p vs) a code covers both.  Weights are relative to a
reference that only rises and that the row's sum is at least 1 times, so for
codes b and values v = vs b
    |dO| <= (2^-11 + 2 e + 2^-17 + s) A + u |O| + t,   A = sum_j p_j |v_j|,
    t = sum min(p_j, 2^-27) |v_j| + 2^-27 max_j (p_j vs_j) sum |b_j|  over the keys
the row sees, s = n / 16 * 2^-23 the sums of n keys, 16 a product, and 2^-17 the
exponential, the factors of merging and the division.  |dLSE| <= e + 2^-17 + s
+ 2^-21 |LSE|.  fp16 results add half of their smallest step, 2^-25.
"""
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


def decode(q, cache, table, lens, **kw):
    o, lse = fa.attention_decode_paged(q, cache, table, ints(lens), **kw)
    status_ok()
    return o.double().cpu().numpy(), lse.double().cpu().numpy()


def sequence(cache, pages, n):
    """k, v, v's codes and v's scales of the first n slots of the pages, float64
    [Hk, n, d] and [Hk, n]."""
    out = []
    for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        code = pc.numpy_codes(x[pages] if x.dtype == torch.int8 else
                              x.view(torch.uint8)[pages].view(x.dtype))
        scale = s[pages].double().cpu().numpy()
        out.append((np.moveaxis(code, 1, 0).reshape(code.shape[1], -1, code.shape[3])[:, :n],
                    np.repeat(scale.T, code.shape[2], 1)[:, :n]))
    (ka, ks), (b, vs) = out
    with np.errstate(invalid="ignore"):
        return ka * ks[..., None], b * vs[..., None], np.abs(b), np.abs(vs)


def check(got, q, cache, table, lens, b, window=None, sinks=0, scale=None, rows=None):
    """O and LSE of sequence b (of its tokens `rows`) within their bounds."""
    o, lse = got
    H, Nq, d = q.shape[1:]
    n, Hk = lens[b], cache.k.shape[1]
    scale = pc.scale_of(d) if scale is None else scale
    u = pc.wc.half_step("bf16" if q.dtype == torch.bfloat16 else "fp16")
    tiny = 0.0 if q.dtype == torch.bfloat16 else 2.0 ** -25
    page = cache.k.shape[2]
    k, v, codes, vs = sequence(cache, table[b, :-(-n // page)].long(), n)
    mask = pc.window_mask(Nq, n, n, "bottom_right", n + 99 if window is None else window, sinks)
    qd = q[b].double().cpu().numpy()
    for i in range(Nq) if rows is None else rows:
        m = mask[i]
        sums = m.sum() / 16 * 2.0 ** -23
        for hk in range(Hk):
            kk, vv = k[hk][m], v[hk][m]
            for h in range(hk * (H // Hk), (hk + 1) * (H // Hk)):
                s = scale * (kk @ qd[h, i])
                e = 128 * 2.0 ** -23 * scale * (np.abs(kk) @ np.abs(qd[h, i])).max()
                mx = s.max()
                p = np.exp(s - mx)
                l = p.sum()
                p = p / l
                ref, size = p @ vv, p @ np.abs(vv)
                t = (np.minimum(p, 2.0 ** -27) @ np.abs(vv)
                     + 2.0 ** -27 * (p * vs[hk][m]).max() * codes[hk][m].sum(0))
                tol = (2.0 ** -11 + 2 * e + 2.0 ** -17 + sums) * size + u * np.abs(ref) + t + tiny
                err = np.abs(o[b, h, i] - ref)
                assert (err <= tol).all(), (f"token {i} head {h}: off {np.max(err - tol):.3e} more than "
                                            f"the bound, |O| {np.abs(ref).max():.3e}, "
                                            f"worst {np.max(err / tol):.3g} of it")
                want = mx + np.log(l)
                assert abs(lse[b, h, i] - want) <= e + 2.0 ** -17 + sums + 2.0 ** -21 * abs(want)


@pytest.mark.parametrize("bits", [4, 8, 16, 20, 26, 40, 90])
@pytest.mark.parametrize("H", [4, 8, 24])      # 8, 16 and 48 rows a key/value head
@pytest.mark.parametrize("d,code,page", [(64, "int8", 16), (64, "e4m3", 128), (128, "e4m3", 16),
                                         (128, "int8", 128)])
def test_a_large_scale_beside_ordinary_ones(d, code, page, H, bits):
    """One page's values are 2^bits times the others': the last one, which only
    the last token sees, or one at the window's start, which only the first sees.
    Each token's result is as exact as its own keys allow."""
    for large, window in ((3, None), (1, page + 1), (0, None)):
        cache = pc.random_cache(5, 1, page, d, code, seed=bits)
        table, lens = ints([[4, 2, 0, 3]]), [3 * page + 1]
        cache.v_scale[int(table[0, large])] *= 2.0 ** bits
        q = pc.normal((1, H, 2, d), "bf16", 1).cuda()
        check(decode(q, cache, table, lens, window=window), q, cache, table, lens, 0, window)


@pytest.mark.parametrize("bits", [8, 16, 20, 30, 40])
@pytest.mark.parametrize("H", [4, 8, 24])
@pytest.mark.parametrize("d,code", [(64, "e4m3"), (128, "int8"), (128, "e4m3")])
def test_large_values_of_no_weight(d, code, H, bits):
    """A page of values 2^bits times the others' whose scores are 28 (d = 128) or
    40 below them, anywhere in the sequence: the weight is on the small pages."""
    for large in (0, 1, 4, 8):
        cache = pc.random_cache(10, 1, 16, d, code, seed=bits + 1)
        table, lens = ints([[7, 2, 5, 0, 3, 6, 8, 1, 9]]), [16 * 9 - 3]
        p = int(table[0, large])
        cache.v_scale[p] *= 2.0 ** bits
        cache.k.view(torch.uint8)[:, :, :, 0] = 0
        cache.k.view(torch.uint8)[p] = 0
        cache.k[p, 0, :, 0] = torch.tensor(-80.0, device="cuda").to(cache.k.dtype)
        cache.k_scale[p] = 0.5
        q = pc.normal((1, H, 2, d), "bf16", 2)
        q[..., 0] = 8.0
        q = q.cuda()
        check(decode(q, cache, table, lens), q, cache, table, lens, 0)


@pytest.mark.parametrize("ratio", [1.5, 8.0, 60.0, 1000.0])
@pytest.mark.parametrize("G,Hk", [(4, 8), (16, 8), (32, 4)])
def test_many_light_keys(G, Hk, ratio):
    """A key 14 above 32768 others and without values of its own, behind a page
    of larger ones, in one run: the result is what the light keys add up to."""
    d, page, n = 128, 128, 32768 + 256
    warps = 12 if G <= 8 else 10 if G <= 16 else 1
    B = torch.cuda.get_device_properties(0).multi_processor_count * warps // Hk
    cache = pc.random_cache(10, Hk, page, d, "e4m3", seed=3, spread=0.0)
    per = n // page
    table = ints([[8, 9] + [i % 8 for i in range(per - 2)]]).expand(B, per).contiguous()
    cache.v_scale[8] *= ratio
    cache.k.view(torch.uint8)[:, :, :, 0] = 0
    cache.k.view(torch.uint8)[9, :, 5] = 0
    cache.v.copy_(cache.v.float().abs())           # the light keys' values add up
    cache.v.view(torch.uint8)[9, :, 5] = 0
    cache.k[9, :, 5, 0] = torch.tensor(160.0, device="cuda").to(cache.k.dtype)   # 1.6 * 9 q
    q = pc.normal((1, Hk * G, 1, d), "fp16", 4)
    q[..., 0] = 14 / 1.6 / pc.scale_of(d)
    q = q.expand(B, -1, -1, -1).contiguous().cuda()
    got = decode(q, cache, table, [n] * B)
    check(got, q, cache, table, [n] * B, B // 2)
    check(got, q, cache, table, [n] * B, 0)


@pytest.mark.parametrize("H", [3, 10, 30])     # 12, 40 and 120 rows
@pytest.mark.parametrize("page,d,code", [(16, 128, "e4m3"), (48, 64, "int8"), (128, 128, "int8")])
def test_scales_that_rise_and_fall(page, d, code, H):
    """Pages 2^-20 to 2^20 times the usual scale in random order, under a window
    of 40 keys behind sequences of every length."""
    per = 8
    lens = [7 * i % (per * page + 1) for i in range(30)]
    lens = [n for n in lens if n >= 4]
    B = len(lens)
    cache = pc.random_cache(per * B, 1, page, d, code, seed=5, spread=20.0)
    cache.k_scale[:] = 0.01
    table = torch.randperm(per * B, generator=torch.Generator().manual_seed(6)).view(B, per).int().cuda()
    q = pc.normal((B, H, 4, d), "bf16", 7).cuda()
    got = decode(q, cache, table, lens, window=40, sinks=2)
    for b in range(B):
        check(got, q, cache, table, lens, b, window=40, sinks=2)


@pytest.mark.parametrize("size", [2.0 ** 117, 2.0 ** -100])
@pytest.mark.parametrize("H", [4, 12, 40])
@pytest.mark.parametrize("n", [300, 30000])
def test_values_near_the_ends_of_the_range(n, H, size):
    """Values of up to 2^126, or of 2^-91, whether a unit lies in one run or is cut
    into parts: results stay in range, and as exact as usual ones."""
    page, d = 48, 64
    per = -(-n // page)
    for B, code in ((1, "e4m3"), (600, "e4m3"), (1, "int8")):
        pages = 20 if B > 1 else per
        cache = pc.random_cache(pages, 1, page, d, code, seed=8, spread=0.5)
        cache.v.copy_(cache.v.float().abs())
        cache.v_scale.copy_((cache.v_scale * 100).log2().round().exp2() * (size / 2))
        table = ints([[i % pages for i in range(per)]] * B)
        lens = [n - b % 3 for b in range(B)]
        q = pc.normal((B, H, 1, d), "bf16", 9).cuda()
        got = decode(q, cache, table, lens)
        assert np.isfinite(got[0]).all() and np.isfinite(got[1]).all()
        for b in sorted({0, B // 2, B - 1}):
            check(got, q, cache, table, lens, b)


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("H", [2, 5, 20])      # 6, 15 and 60 rows
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_keys_of_a_scale_that_is_not_finite(bad, H, page):
    """Whatever the sign of its products, such a page gives NaN to the tokens that see
    it (here the last, and the first in a window that the second does not reach back
    to), and nothing to the others."""
    d = 64
    cache = pc.random_cache(6, 1, page, d, "int8", seed=10)
    table, lens = ints([[4, 2, 0, 5]]), [3 * page + 1]
    q = pc.normal((1, H, 3, d), "bf16", 11).abs().cuda()
    cache.k.copy_(cache.k.float().abs())
    for large, window, seen, other in ((3, None, [2], [0, 1]), (1, page, [0], [1, 2])):
        ref = fa.attention_decode_paged(q, cache, table, ints(lens), window=window)
        for sign in (1, -1):
            spoilt = fa.PagedCache(*(x.clone() for x in cache))
            spoilt.k_scale[int(table[0, large])] = bad
            spoilt.k[int(table[0, large])] *= sign
            o, lse = fa.attention_decode_paged(q, spoilt, table, ints(lens), window=window)
            status_ok()
            assert torch.isnan(o[:, :, seen]).all() and torch.isnan(lse[:, :, seen]).all()
            assert torch.equal(o[:, :, other], ref[0][:, :, other])
            assert torch.equal(lse[:, :, other], ref[1][:, :, other])


@pytest.mark.parametrize("H", [4, 12, 40])
@pytest.mark.parametrize("bits", [120, 60, -60])
def test_queries_and_keys_of_opposite_size(bits, H):
    """Queries of 2^bits and keys of 2^-bits, whose products are of usual size."""
    for d, code in ((64, "int8"), (128, "e4m3")):
        cache = pc.random_cache(7, 1, 48, d, code, seed=12)
        cache.k_scale.mul_(2.0 ** (-bits / 2)).mul_(2.0 ** (-bits / 2))
        table, lens = ints([[4, 2, 0, 5, 6]]), [230]
        q = (pc.normal((1, H, 2, d), "bf16", 13).float() * 2.0 ** (bits / 2) * 2.0 ** (bits / 2)).bfloat16().cuda()
        check(decode(q, cache, table, lens), q, cache, table, lens, 0)
    # keys of 0 score 0, whatever their scale
    cache.k.view(torch.uint8).zero_()
    cache.k_scale.fill_(2.0 ** 40)
    check(decode(q, cache, table, lens), q, cache, table, lens, 0)


@pytest.mark.parametrize("B,Hk,G,Nq,page,per,d,code", [
    (8, 8, 8, 8, 128, 6, 64, "int8"), (150, 1, 17, 1, 16, 9, 128, "e4m3"), (40, 4, 8, 16, 32, 13, 128, "int8"),
    (300, 2, 9, 2, 48, 3, 64, "e4m3"), (7, 5, 33, 3, 80, 21, 128, "e4m3"),
])
def test_every_run_of_many_rows_gives_the_same_bits(B, Hk, G, Nq, page, per, d, code):
    """Codes are turned out of slots that the next copies write: a copy that came
    before all lanes have their codes would change some run's result.  Other work on
    a second stream moves the copies."""
    cache = pc.random_cache(B * per, Hk, page, d, code, seed=14)
    table = torch.randperm(B * per, generator=torch.Generator().manual_seed(15)).view(B, per).int().cuda()
    lens = torch.randint(0, per * page + 1, (B,), generator=torch.Generator().manual_seed(16),
                         dtype=torch.int32).cuda()
    q = pc.normal((B, Hk * G, Nq, d), "fp16", 17).cuda()
    ws = fa.make_paged_workspace(q, cache, table)
    want = fa.attention_decode_paged(q, cache, table, lens, workspace=ws)
    side, noise = torch.cuda.Stream(), torch.zeros(1 << 24, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    differ = torch.zeros(300, dtype=torch.bool, device="cuda")
    for i in range(300):
        if i % 3 == 0:
            with torch.cuda.stream(side):
                noise.add_(1.0)
        o, lse = fa.attention_decode_paged(q, cache, table, lens, workspace=ws)
        differ[i] = (o != want[0]).any() | (lse != want[1]).any()
    status_ok()
    assert not differ.any()


@pytest.mark.parametrize("H", [4, 8, 40])
def test_a_head_of_extreme_queries_costs_the_others_nothing(H):
    """Keys of 2^33, queries of 2^-38, and one head of 2^110, whose scores leave
    float32's range: the other heads' results are as usual."""
    for d, code in ((64, "int8"), (128, "e4m3")):
        cache = pc.random_cache(7, 1, 48, d, code, seed=18)
        cache.k_scale.mul_(2.0 ** 38)
        table, lens = ints([[4, 2, 0, 5, 6]]), [230]
        q = pc.normal((1, H, 2, d), "bf16", 19).float() * 2.0 ** -38
        q[:, 1] *= 2.0 ** 74
        q[:, 1] *= 2.0 ** 74
        q = q.bfloat16().cuda()
        rest = [h for h in range(H) if h != 1]
        o, lse = decode(q, cache, table, lens)
        check((o[:, rest], lse[:, rest]), q[:, rest].contiguous(), cache, table, lens, 0)
