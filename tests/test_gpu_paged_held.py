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


@pytest.mark.parametrize("H,Nq", [(4, 1), (8, 3), (24, 2)])     # 2, 12 and 24 rows a key/value head
def test_a_captured_decoding_loop(H, Nq):
    """Append and decoding captured once: replays read lengths, counts and the page
    table of their time, as eager calls do, down to empty sequences."""
    B, Hk, page, per, d = 5, 2, 16, 40, 64
    caches = [fa.make_paged_cache(2 * B * per, Hk, page, d) for _ in range(2)]
    tables = [deal(B, per, B * per, seed=60) + x for x in (0, B * per)]
    table = tables[0].clone()
    k, v = (torch.zeros(B, Hk, Nq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, n = torch.zeros(B, H, Nq, d, dtype=torch.bfloat16, device="cuda"), ints([0] * B)
    ws = fa.make_paged_workspace(q, caches[1], table)
    out, lse = torch.empty_like(q), torch.empty(B, H, Nq, device="cuda")

    def step(cache, **kw):
        fa.cache_append(k, v, cache, table, n)
        return fa.attention_decode_paged(q, cache, table, n, window=300, sinks=2, **kw)
    step(caches[1], out=out, lse=lse, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(caches[1], out=out, lse=lse, workspace=ws)
    for i, lens in enumerate(([Nq] * B, [600, 17, 0, 33, 640], [640, 1, 16, 0, 0], [0] * B, [5, 300, 301, 640, 2])):
        for x, t in enumerate((k, v, q)):
            t.copy_(pc.normal(tuple(t.shape), "bf16", 70 + 3 * i + x).cuda())
        n.copy_(ints(lens))
        table.copy_(tables[i % 2])
        want = step(caches[0])
        g.replay()
        status_ok()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), i
        assert (lse[[b for b, m in enumerate(lens) if m == 0]] == float("-inf")).all()


def test_many_short_sequences():
    """A sequence's result beside 2999 others and alone: each is rounded to bf16 (2^-8
    of its value), and its weights to 11 bits (2^-11 of at most the largest value); LSE
    adds up to 48 weights in another order (48 * 2^-24 and the logarithm's own)."""
    B, Hk, page, per, d = 3000, 1, 16, 3, 64
    cache = pc.random_cache(50, Hk, page, d, "int8", seed=61)
    g = torch.Generator().manual_seed(62)
    table = torch.randint(0, 50, (B, per), generator=g, dtype=torch.int32).cuda()
    lens = torch.randint(0, per * page + 1, (B,), generator=g, dtype=torch.int32).cuda()
    q = pc.normal((B, 20, 1, d), "bf16", 63).cuda()
    vmax = (cache.v.float().abs().amax((1, 2, 3)) * cache.v_scale[:, 0]).max()
    for heads in (2, 10, 20):
        o, lse = fa.attention_decode_paged(q[:, :heads].contiguous(), cache, table, lens)
        status_ok()
        some = list(range(0, B, 499)) + [B - 1]           # alone: whole units in other places
        for b in some:
            x, y = fa.attention_decode_paged(q[b:b + 1, :heads].contiguous(), cache, table[b:b + 1].contiguous(),
                                             lens[b:b + 1])
            assert ((o[b] - x[0]).abs().float() <= 2.0 ** -7 * x[0].abs().float() + 2.0 ** -10 * vmax).all()
            assert torch.equal(lse[b].isinf(), y[0].isinf())
            assert (lse[b] - y[0]).nan_to_num(0.0, 0.0, 0.0).abs().max() <= 2.0 ** -15
    status_ok()
