"""Outputs of the rotation that overlap its inputs or each other: told from index
sets on the CPU, refused on the GPU."""
import random

import pytest
import torch

import exact_tiled_attention_14_gb300 as fa


def elements(t):
    base = torch.arange(t.untyped_storage().size() // t.element_size(), dtype=torch.int32)
    return set(base.as_strided(t.shape, t.stride(), t.storage_offset()).flatten().tolist())


def views(rng, d=8):
    """Two views of one buffer, as slices of a fused projection's output or not."""
    B, N, T = rng.randint(1, 3), rng.randint(1, 4), rng.randint(2, 7)
    x = torch.zeros(B * N * T * d + 64, dtype=torch.int16)
    fused = x[:B * N * T * d].view(B, N, T, d) if rng.random() < 0.5 else \
        x[:B * N * T * d].view(B, T, N, d).transpose(1, 2)
    out = []
    for _ in range(2):
        h = rng.randint(0, T - 1)
        y = fused[rng.randint(0, B - 1):, :rng.randint(1, N), h:rng.randint(h + 1, T)].transpose(1, 2)
        out.append(y if rng.random() < 0.8 else y[:, :1].expand_as(y))
    return out


def test_shared_elements_are_found():
    """All of them where the strides agree; no others elsewhere."""
    rng = random.Random(1)
    found = 0
    for _ in range(4000):
        a, b = views(rng)
        got, want = fa._overlap(a, b), bool(elements(a) & elements(b))
        agree = all(s == t for m, n, s, t in zip(a.shape, b.shape, a.stride(), b.stride()) if m > 1 and n > 1)
        assert got == fa._overlap(b, a)
        assert got == want or (want and not agree), (a.shape, a.stride(), b.shape, b.stride())
        found += got
    assert 500 < found < 3500


def test_other_strides():
    x = torch.zeros(4 * 6 * 5 * 8, dtype=torch.int16)
    a, b = x.view(4, 6, 5, 8), x.view(4, 5, 6, 8).transpose(1, 2)
    assert fa._overlap(a, b)                                     # both fill the buffer
    assert not fa._overlap(a[:2], b[2:])
    assert not fa._overlap(a[:0], b)


@pytest.mark.gpu
def test_refusals_and_what_stays_allowed():
    B, H, N, d = 2, 4, 9, 64
    f = fa.rotary_frequencies(64, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    qkv = torch.randn(B, N, 3 * H, d, generator=g, device="cuda").bfloat16()
    q, k, v = (x.transpose(1, 2) for x in qkv.split(H, 2))
    want = fa.rotary_forward(q, k, f)
    for out in ((k, q), (q, q), (v, v), (k, v),
                (qkv[:, :, 1:H + 1].transpose(1, 2), v)):
        with pytest.raises(ValueError):
            fa.rotary_forward(q, k, f, out=out)
    square = torch.randn(1, 8, 8, d, generator=g, device="cuda").half()
    with pytest.raises(ValueError):                              # in place, but transposed
        fa.rotary_forward(square, None, f, out=(square.transpose(1, 2), None))
    out = fa.rotary_forward(q, None, f, out=(v, None))           # beside the inputs
    assert torch.equal(out[0], want[0])
    fa.rotary_forward(q, k, f, out=(q, k))                       # in place
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    torch.cuda.synchronize()
    assert fa.fa_status()[0] == fa.FA_OK
