"""Autograd of attention() and attention_packed() on the CPU, their kernels' calls replaced by stand-ins of the same shapes."""
import pytest
import torch

import exact_attention_32_gb300 as fa
from exact_attention_32_gb300 import _binding


def stand_ins(packed, monkeypatch, backward):
    """(q, a call of attention of q over itself) with these gradients; the forward gives q."""
    def forward(q, k, v, *a, **kw):
        return q.clone(), q.new_zeros(1)

    for name in ("forward", "forward_packed"):
        monkeypatch.setattr(_binding, name, forward)
    for name in ("backward", "backward_packed"):
        monkeypatch.setattr(_binding, name, backward)
    monkeypatch.setattr(_binding, "packed_plan", lambda cu, T, causal: _binding.PackedPlan(torch.zeros(1), T, 1, causal))
    q = torch.randn(*((4, 1, 64) if packed else (1, 1, 4, 64)), requires_grad=True)
    return q, lambda: fa.attention_packed(q, q, q, torch.tensor([0, 4])) if packed else fa.attention(q, q, q)


@pytest.mark.parametrize("packed", [False, True])
def test_a_second_derivative_is_refused(packed, monkeypatch):
    # the kernels' gradients are constants to autograd: a loss that holds them beside other terms would lose its derivative
    # through them without a word
    q, out = stand_ins(packed, monkeypatch, lambda q, k, v, o, lse, dout, *a, **kw: (dout.clone(), dout.clone(), dout.clone()))
    once, = torch.autograd.grad(out().sum(), q)
    assert (once == 3).all()  # (q's, k's and v's)
    g, = torch.autograd.grad(out().sum(), q, create_graph=True)
    assert (g == 3).all()
    with pytest.raises(RuntimeError, match="second derivative"):
        (g.sum() + (q * q).sum()).backward()


@pytest.mark.parametrize("packed", [False, True])
def test_an_output_gradient_that_lies_off_sixteen_bytes(packed, monkeypatch):
    # as behind a concatenation of flattened tensors: its gradient is a contiguous view at any offset, and the kernels take 16 bytes
    seen = []

    def backward(q, k, v, o, lse, dout, *a, **kw):
        seen.append((dout.data_ptr() % 16, dout.is_contiguous()))
        return dout.clone(), dout.clone(), dout.clone()

    q, out = stand_ins(packed, monkeypatch, backward)
    weight = torch.arange(3 + q.numel(), dtype=torch.float32)
    (torch.cat([torch.zeros(3), out().flatten()]) * weight).sum().backward()
    assert seen == [(0, True)] and torch.equal(q.grad.flatten(), 3 * weight[3:])


def test_offsets_that_change_before_the_backward(monkeypatch):
    # a step's offsets in one buffer, overwritten with the next ones before this one's backward: the plan holds what it was made from
    monkeypatch.setattr(_binding, "packed_plan", lambda cu, T, causal: _binding.PackedPlan(torch.zeros(1), T, cu.shape[0] - 1, causal))
    monkeypatch.setattr(_binding, "forward_packed", lambda q, k, v, cu, **kw: (q.clone(), q.new_zeros(1)))
    seen = []

    def backward(q, k, v, o, lse, dout, cu, plan, **kw):
        seen.append((cu.shape[0], plan[1:]))
        return dout.clone(), dout.clone(), dout.clone()

    monkeypatch.setattr(_binding, "backward_packed", backward)
    q, cu = torch.randn(4, 1, 64, requires_grad=True), torch.tensor([0, 3, 4])
    o = fa.attention_packed(q, q, q, cu, causal=True)
    cu.copy_(torch.tensor([0, 1, 4]))
    o.sum().backward()
    assert (q.grad == 3).all() and seen == [(3, (4, 2, True))]
