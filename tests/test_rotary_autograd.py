"""rotary_embedding's backward pass rotates what is asked for and nothing else.
(CPU: the entry points are replaced by functions that count their tensors.)"""
import pytest
import torch

import exact_tiled_attention_14_gb300 as fa


@pytest.fixture
def calls(monkeypatch):
    seen = []

    def forward(q, k, *_args, **_kw):
        return (3.0 * q).detach(), None if k is None else (5.0 * k).detach()

    def backward(dq, dk, *args, **_kw):
        seen.append((dq.shape, None if dk is None else dk.shape, args[1:]))
        factor = {4: 3.0, 2: 5.0}                 # by the number of heads
        return tuple(None if g is None else factor[g.shape[1]] * g for g in (dq, dk))
    monkeypatch.setattr(fa, "rotary_forward", forward)
    monkeypatch.setattr(fa, "rotary_backward", backward)
    return seen


def leaves(q_grad, k_grad):
    return (torch.ones(1, 4, 5, 16, requires_grad=q_grad), torch.ones(1, 2, 5, 16, requires_grad=k_grad),
            fa.rotary_frequencies(16))


@pytest.mark.parametrize("q_grad,k_grad", [(True, True), (True, False), (False, True)])
def test_only_the_inputs_that_ask(calls, q_grad, k_grad):
    q, k, f = leaves(q_grad, k_grad)
    lens = torch.tensor([7], dtype=torch.int32)
    yq, yk = fa.rotary_embedding(q, k, f, seqlens=lens, mscale=1.5, interleaved=True)
    (yq.sum() + yk.sum()).backward()
    want = [x.shape for x, g in ((q, q_grad), (k, k_grad)) if g] + [None]
    assert len(calls) == 1 and list(calls[0][:2]) == want[:2]
    assert calls[0][2][0] is None and calls[0][2][1] is lens and calls[0][2][2:] == (1.5, True)
    assert (q.grad is None) == (not q_grad) and (k.grad is None) == (not k_grad)
    assert not q_grad or torch.equal(q.grad, torch.full_like(q, 3.0))
    assert not k_grad or torch.equal(k.grad, torch.full_like(k, 5.0))


@pytest.mark.parametrize("used", [0, 1])
def test_an_unused_result_has_a_gradient_of_zeros(calls, used):
    q, k, f = leaves(True, True)
    y = fa.rotary_embedding(q, k, f)
    grads = torch.autograd.grad(y[used].sum(), (q, k))
    assert len(calls) == 1 and calls[0][:2] == ((q, k)[used].shape, None)
    assert torch.equal(grads[used], torch.full_like((q, k)[used], (3.0, 5.0)[used]))
    assert torch.equal(grads[1 - used], torch.zeros_like((q, k)[1 - used]))


def test_nothing_is_rotated_for_results_that_nobody_uses(calls):
    q, k, f = leaves(False, True)
    yq, _ = fa.rotary_embedding(q, k, f)
    assert torch.equal(torch.autograd.grad(yq.sum(), k)[0], torch.zeros_like(k))
    assert calls == []
