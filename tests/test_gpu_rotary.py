"""Rotary positions (fa_rotary) against the float64 rotation: layouts, parts of
the head, far positions, strides, in place, the gradient, graphs and streams."""
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


def expect(x, pos, w, dtype, mscale=1.0, interleaved=False, sign=1.0):
    """Reference and bound of x [B, heads, N, d] at pos [B, N]."""
    y, r = pc.rotate(x.double().cpu().numpy(), pos[:, None, :], w, mscale, interleaved, sign)
    tol = r + (pc.wc.half_step(dtype) * (np.abs(y) + r) + 2.0 ** -25) * (r > 0)
    return y, tol


def compare(got, ref, what):
    y, tol = ref
    x = got.detach().double().cpu().numpy()
    err = np.abs(x - y)
    assert np.all(err <= tol), f"{what}: {int((err > tol).sum())} out, worst {np.max(err - tol):.3e}"


CASES = [
    # B, H, Hk, N, d, rot, interleaved, dtype, positions, mscale
    (1, 1, 1, 1, 64, 64, False, "bf16", "start", 1.0),
    (1, 1, 0, 1, 128, 16, True, "fp16", "start", 1.0),
    (2, 3, 1, 33, 64, 32, False, "fp16", "positions", 1.0),
    (2, 3, 1, 33, 64, 48, True, "bf16", "positions", 1.3),
    (3, 8, 2, 5, 128, 128, False, "bf16", "seqlens", 1.0),
    (3, 5, 5, 7, 128, 96, True, "fp16", "seqlens", 0.7),
    (1, 40, 8, 300, 128, 128, False, "bf16", "start", 1.0),
    (2, 2, 2, 2500, 64, 64, True, "bf16", "start", 1.0),
    (4, 70, 3, 200, 64, 16, False, "fp16", "positions", 1.0),
]


def inputs(case, seed=0):
    B, H, Hk, N, d, rot, inter, dtype, at, mscale = case
    q = pc.normal((B, H, N, d), dtype, seed, std=3.0).cuda()
    k = pc.normal((B, Hk, N, d), dtype, seed + 1).cuda() if Hk else None
    g = torch.Generator().manual_seed(seed + 2)
    pos = torch.arange(N).expand(B, N)
    kw = dict(mscale=mscale, interleaved=inter)
    if at == "positions":
        pos = torch.randint(-5, 1 << 20, (B, N), generator=g, dtype=torch.int32)
        kw["positions"] = pos.cuda()
    if at == "seqlens":
        lens = torch.randint(0, 1 << 20, (B,), generator=g, dtype=torch.int32)
        lens[0] = N // 2                              # rows before the sequence's start
        kw["seqlens"] = lens.cuda()
        pos = lens[:, None] - N + torch.arange(N)
    return q, k, fa.rotary_frequencies(rot, device="cuda"), pc.frequencies(rot), pos.numpy(), kw


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_forward_and_backward(case):
    B, H, Hk, N, d, rot, inter, dtype, at, mscale = case
    q, k, freqs, w, pos, kw = inputs(case)
    for call, sign in ((fa.rotary_forward, 1.0), (fa.rotary_backward, -1.0)):
        yq, yk = call(q, k, freqs, **kw)
        status_ok()
        compare(yq, expect(q, pos, w, dtype, mscale, inter, sign), f"q {sign}")
        assert torch.equal(yq[..., rot:], q[..., rot:]) and yq.is_contiguous()
        if k is None:
            assert yk is None
        else:
            compare(yk, expect(k, pos, w, dtype, mscale, inter, sign), f"k {sign}")
            # one head's result does not depend on the others
            assert torch.equal(yk, call(k, None, freqs, **kw)[0])


@pytest.mark.parametrize("pos", [1, 2 ** 20 + 1, 2 ** 31 - 1, -2 ** 31])
def test_far_positions(pos):
    """The angle keeps its fraction of a turn at any position: the result is the
    rotation by pos times the given frequency (in its units of 2^-64) exactly."""
    f = fa.rotary_frequencies(64, device="cuda")
    q = pc.normal((1, 2, 1, 64), "fp16", 3).cuda()
    y, _ = fa.rotary_forward(q, None, f, positions=torch.tensor([[pos]], dtype=torch.int32, device="cuda"))
    status_ok()
    turns = np.array([(pos * (x % 2 ** 64) % 2 ** 64) / 2 ** 64 for x in f.tolist()])
    ref = expect(q, np.array([[1]]), 2 * np.pi * turns, "fp16")
    compare(y, ref, f"position {pos}")


def test_strided_in_place_and_broadcast():
    """Slices of a fused projection's output, results in the caller's layout, in
    place, and an input that all heads share: as from contiguous copies."""
    B, H, Hk, N, d = 2, 6, 2, 37, 128
    qkv = pc.normal((B, N, H + 2 * Hk, d), "bf16", 5).cuda()
    q, k = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hk].transpose(1, 2)
    f = fa.rotary_frequencies(64, device="cuda")
    rq, rk = fa.rotary_forward(q.contiguous(), k.contiguous(), f)
    sq, sk = fa.rotary_forward(q, k, f)
    assert sq.is_contiguous() and torch.equal(sq, rq) and torch.equal(sk, rk)
    out = (torch.empty_like(q.transpose(1, 2).contiguous()).transpose(1, 2),
           torch.empty((B, N, 3, Hk, d), dtype=q.dtype, device="cuda")[:, :, 1].transpose(1, 2))
    assert fa.rotary_forward(q, k, f, out=out)[1] is out[1]
    assert torch.equal(out[0], rq) and torch.equal(out[1], rk)
    v = qkv[:, :, H + Hk:].clone()
    fa.rotary_forward(q, k, f, out=(q, k))
    assert torch.equal(q, rq) and torch.equal(k, rk) and torch.equal(qkv[:, :, H + Hk:], v)
    one = pc.normal((B, 1, N, d), "bf16", 6).cuda().expand(B, H, N, d)
    assert torch.equal(fa.rotary_forward(one, None, f)[0], fa.rotary_forward(one.contiguous(), None, f)[0])
    # a packed batch: tokens of all sequences in a row, positions given
    packed = pc.normal((N, H, d), "bf16", 7).cuda()
    pos = torch.randint(0, 9999, (1, N), dtype=torch.int32, device="cuda")
    a = fa.rotary_forward(packed.transpose(0, 1)[None], None, f, positions=pos)[0]
    b = fa.rotary_forward(packed.transpose(0, 1)[None].contiguous(), None, f, positions=pos)[0]
    assert torch.equal(a, b)
    status_ok()


def test_refusals_on_the_device():
    f = fa.rotary_frequencies(64, device="cuda")
    x = torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16, device="cuda")
    ints = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    bad = [dict(q=x.transpose(2, 3)), dict(positions=ints, seqlens=ints[:, 0].contiguous()),
           dict(positions=ints.long()), dict(positions=ints[:1]), dict(seqlens=ints[:, 0]),
           dict(freqs=f.cpu()), dict(freqs=f.int()), dict(freqs=f[:5]),
           dict(freqs=fa.rotary_frequencies(128, device="cuda")), dict(out=(x, x)),
           dict(out=(x[:1].expand(2, 2, 8, 64), None)), dict(out=(x.half(), None)),
           dict(out=(x[:, :1].expand(2, 2, 8, 64), None))]
    for a in bad:
        a = dict(dict(q=x, k=None, freqs=f), **a)
        with pytest.raises(ValueError):
            fa.rotary_forward(**a)
    with pytest.raises(fa.FaError) as e:                       # rows at no multiple of 16 bytes
        fa.rotary_forward(torch.zeros(2, 2, 8, 68, dtype=torch.bfloat16, device="cuda")[..., :64], None, f)
    assert e.value.code == fa.FA_ERR_ALIGN
    with pytest.raises(fa.FaError) as e:
        fa.rotary_forward(x, None, f, mscale=0.0)
    assert e.value.code == fa.FA_ERR_SCALE
    assert fa.rotary_forward(x[:, :, :0], None, f)[0].shape == (2, 2, 0, 64)
    status_ok()


@pytest.mark.parametrize("inter", [False, True])
def test_gradient(inter):
    """Autograd's gradient against the formula's and against differences (the
    operator is linear, so a difference of results is its derivative, off by
    the results' rounding); a broadcast input's gradient is the sum."""
    B, H, Hk, N, d, rot = 2, 4, 2, 19, 64, 48
    f, w = fa.rotary_frequencies(rot, device="cuda"), pc.frequencies(rot)
    lens = torch.tensor([100, 5000], dtype=torch.int32, device="cuda")
    q = pc.normal((B, H, N, d), "fp16", 8).cuda().requires_grad_()
    k = pc.normal((B, 1, N, d), "fp16", 9).cuda().requires_grad_()
    gq, gk = pc.normal((B, H, N, d), "fp16", 10).cuda(), pc.normal((B, Hk, N, d), "fp16", 11).cuda()
    kw = dict(seqlens=lens, mscale=1.2, interleaved=inter)
    yq, yk = fa.rotary_embedding(q, k.expand(B, Hk, N, d), f, **kw)
    torch.autograd.backward((yq, yk), (gq, gk))
    status_ok()
    pos = (lens[:, None].cpu() - N + torch.arange(N)).numpy()
    compare(q.grad, expect(gq, pos, w, "fp16", 1.2, inter, -1.0), "dq")
    ref, tol = expect(gk, pos, w, "fp16", 1.2, inter, -1.0)
    total = ref.sum(1, keepdims=True)
    compare(k.grad, (total, tol.sum(1, keepdims=True) + 2.0 ** -11 * np.abs(total) + 2.0 ** -24), "dk")
    # d sum(yq * gq) along a direction, in float64 from two results
    e = pc.normal((B, H, N, d), "fp16", 12).cuda()
    with torch.no_grad():
        a = fa.rotary_forward(q, None, f, **kw)[0].double()
        b = fa.rotary_forward((q.detach() + e), None, f, **kw)[0].double()
        step = (q.detach() + e).double() - q.detach().double()
        lhs = ((b - a) * gq.double()).sum().item()
        rhs = (q.grad.double() * step).sum().item()
        size = ((a.abs() + b.abs()) * gq.double().abs()).sum().item() \
            + (q.grad.double() * step).abs().sum().item()
    assert abs(lhs - rhs) <= 2.0 ** -10 * size       # 2^-11 of each rounded result, twice for r
    # no gradient asked of k, or no k
    q2 = q.detach().clone().requires_grad_()
    fa.rotary_embedding(q2, None, f, **kw)[0].backward(gq)
    assert torch.equal(q2.grad, q.grad)


def test_graph_and_stream():
    q, k, f, w, pos, kw = inputs(CASES[4])
    ref = fa.rotary_forward(q, k, f, **kw)
    out = (torch.empty_like(q), torch.empty_like(k))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fa.rotary_forward(q, k, f, out=out, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(ref, out))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.rotary_forward(q, k, f, out=out, **kw)
    q.mul_(-1)
    g.replay()
    status_ok()
    assert torch.equal(out[0], -ref[0]) and torch.equal(out[1], ref[1])
