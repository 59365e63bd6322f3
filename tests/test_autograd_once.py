"""The autograd wrappers' gradients are first-order only: the kernels leave no
graph behind, so a second differentiation raises instead of leaving the terms
through the attention out of a sum.  (CPU: the entry points are replaced by
functions that, like the kernels, fill new tensors.)"""
import pytest
import torch

import exact_tiled_attention_14_gb300 as fa


def fake_forward(q, *_args, **_kw):
    return (3.0 * q).detach(), q.detach().sum(-1)


def fake_backward(q, k, v, _o, _lse, do, *_args, **_kw):
    return (3.0 * do).detach(), torch.zeros_like(k), torch.zeros_like(v)


CU = torch.tensor([0, 5], dtype=torch.int32)
CALLS = [
    ("attention_forward", "attention_backward", lambda q: fa.flash_attention(q, q, q)),
    ("attention_forward_kv", "attention_backward_kv", lambda q: fa.flash_attention_kv(q, q, q)),
    ("attention_forward_varlen", "attention_backward_varlen",
     lambda q: fa.flash_attention_varlen(q, q, q, CU, CU, 5, 5)),
    ("attention_forward_window", "attention_backward_window",
     lambda q: fa.flash_attention_window(q, q, q, 4)),
]


@pytest.mark.parametrize("fwd,bwd,call", CALLS, ids=[c[1] for c in CALLS])
def test_second_differentiation_raises(monkeypatch, fwd, bwd, call):
    monkeypatch.setattr(fa, fwd, fake_forward)
    monkeypatch.setattr(fa, bwd, fake_backward)
    q = torch.ones(1, 1, 5, 4, requires_grad=True)
    o, _ = call(q)
    (g,) = torch.autograd.grad((o ** 2).sum(), q, create_graph=True)
    assert torch.equal(g, torch.full_like(g, 18.0))
    # d/dq of this has a term through g that the wrapper cannot give
    with pytest.raises(RuntimeError, match="once_differentiable"):
        ((g ** 2).sum() + (q ** 2).sum()).backward()
