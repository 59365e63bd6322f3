"""What a paged cache holds of what went in: every quantisation's half step and no
more, over appends of any length, and long appends of int8 codes."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_14_gb300 as fa
import paged_common as pc
from gpu_common import require_gpu
from test_gpu_paged import check_append, clone, deal, ints, status_ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("sizes", [[1] * 45, [70, 1, 1, 1, 20, 1, 1, 9, 1], [3, 8, 9, 2] * 5])
def test_held_values_are_off_by_their_roundings(sizes, code):
    """A token is rounded when it is written, by half a step next to its value (or of
    the smallest codes), and once more each time its page's scale rises, by half a
    code (int8) or half of the smallest step, 2^-10 of the scale (e4m3: the others
    are shifts): the bound is their sum, 0.05 % above it for the products' roundings."""
    B, Hk, page, d, per = 2, 2, 32, 64, 4
    cache = fa.make_paged_cache(B * per + 1, Hk, page, d, pc.CODE_DT[code])
    table = deal(B, per, B * per + 1, seed=40)
    went = np.zeros((2, B, Hk, per * page, d))
    bound = np.zeros_like(went)
    lens = 0
    scales = np.zeros((2, B, Hk, per))
    for step, T in enumerate(sizes):
        kv = [pc.normal((B, Hk, T, d), "bf16", 50 + 2 * step + x, 1.0 + step / 16) for x in (0, 1)]
        lens += T
        fa.cache_append(kv[0].cuda(), kv[1].cuda(), cache, table, ints([lens] * B))
        now = np.stack([s[table.long()].transpose(1, 2).double().cpu().numpy()
                        for s in (cache.k_scale, cache.v_scale)])           # [2, B, Hk, per]
        rose = np.repeat(now > scales, page, 3)
        s = np.repeat(now, page, 3)
        old = np.arange(per * page) < lens - T
        bound += (rose & old)[..., None] * s[..., None] * (0.5 if code == "int8" else 2.0 ** -10)
        at = slice(lens - T, lens)
        for x in (0, 1):
            went[x, :, :, at] = kv[x].double().numpy()
            y = np.abs(went[x, :, :, at]) / s[x, :, :, at, None]
            bound[x, :, :, at] = pc.half_code(y, code) * s[x, :, :, at, None]
        scales = now
    status_ok()
    held = pc.values(cache, table, [lens] * B)
    for x in (0, 1):
        off = np.abs(held[x] - went[x])[:, :, :lens]
        assert (off <= bound[x][:, :, :lens] * 1.0005).all(), np.max(off / bound[x][:, :, :lens])
        assert off.max() > 0


@pytest.mark.parametrize("dtype,d,page,rot,inter", [("bf16", 128, 64, 128, False), ("fp16", 64, 48, 32, True)])
def test_long_appends_of_int8(dtype, d, page, rot, inter):
    """Prompts of 1500 and 3000 tokens, rotated, behind partly filled pages."""
    B, Hk, T, per = 2, 3, 3000, -(-3100 // page)
    cache = pc.random_cache(B * per + 1, Hk, page, d, "int8", seed=41, spread=2.0)
    table = deal(B, per, B * per + 1, seed=42)
    kv = pc.normal((B, T, 2 * Hk, d), dtype, 43, 2.0).cuda()
    k, v = kv[:, :, :Hk].transpose(1, 2), kv[:, :, Hk:].transpose(1, 2)
    lens, counts, before = [3033, 1501], [3000, 1500], clone(cache)
    fa.cache_append(k, v, cache, table, ints(lens), counts=ints(counts),
                    freqs=fa.rotary_frequencies(rot, device="cuda"), interleaved=inter)
    status_ok()
    check_append(before, cache, k, v, table, lens, counts, "int8", pc.frequencies(rot), 1.0, inter)


def test_read_into_one_tensor_twice_is_refused():
    cache = pc.random_cache(4, 2, 16, 64, "int8", seed=44)
    table, lens = ints([[0, 1], [2, 3]]), ints([20, 30])
    whole = torch.zeros(2 * 2 * 2 * 32 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    n = 2 * 2 * 32 * 64
    a, b, c = (whole[o:o + n].view(2, 2, 32, 64) for o in (0, n, n - 8))
    for out in ((a, a), (a, c), (c, b)):
        with pytest.raises(ValueError):
            fa.cache_read(cache, table, lens, out=out)
    want = fa.cache_read(cache, table, lens)
    assert all(torch.equal(x, y) for x, y in zip(fa.cache_read(cache, table, lens, out=(b, a)), want))
    status_ok()
