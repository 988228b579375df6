"""The reference that the gate's gradients are held to (no GPU): it agrees with differentiating the
step, and it sees each term of each gradient go missing."""
import math

import pytest
import torch

from gate_reference import F, GateGradients, gate_inputs


def step(h, kv, wq, wk, on, eps=1e-6):
    T, hc, d = h.shape
    k, v = kv[:, :hc * d].reshape(T, hc, d), kv[:, hc * d:].reshape(T, 1, d)
    nh = h / torch.sqrt((h * h).mean(2, keepdim=True) + eps)
    nk = k / torch.sqrt((k * k).mean(2, keepdim=True) + eps)
    x = (nh * wq * nk * wk).sum(2, keepdim=True) / math.sqrt(d)
    return h + torch.sigmoid(torch.copysign(x.abs().clamp_min(1e-6).sqrt(), x)) * on * v


SHAPES = [(7, 1, 256), (9, 5, 2816), (12, 4, 5120), (7, 1, 20_736)]


@pytest.mark.parametrize("T,hc,d", SHAPES)
def test_terms_add_up_to_the_derivative(T, hc, d):
    h, kv, _, wq, wk, dy, on = gate_inputs(T, hc, d, T)
    leaves = [t.to(F).requires_grad_() for t in (h, kv, wq, wk)]
    want = torch.autograd.grad(step(*leaves, on), leaves, dy.to(F))
    g = GateGradients(h, kv, on, wq, wk, dy)
    for a, b in ((g.dh, want[0]), (torch.cat([g.dk.reshape(T, -1), g.dv], 1), want[1]), (g.dwq, want[2]),
                 (g.dwk, want[3])):
        assert (a - b).abs().max() <= 1e-9 * b.abs().max()


@pytest.mark.parametrize("T,hc,d", SHAPES)
def test_a_missing_term_is_seen(T, hc, d):
    h, kv, _, wq, wk, dy, on = gate_inputs(T, hc, d, T)
    g = GateGradients(h, kv, on, wq, wk, dy)

    def misses(dh=g.dh, dk=g.dk, dv=g.dv):
        return g.misses(dh.bfloat16(), torch.cat([dk.reshape(T, hc * d), dv], 1).bfloat16())

    assert misses() == []
    assert misses(dh=g.dy) == ["dh"]
    assert misses(dh=g.dh - g.first["dh"]) == ["dh"]
    assert misses(dh=g.dh - g.second["dh"]) == ["dh"]
    assert misses(dh=g.dh - g.dy) == ["dh"]
    assert misses(dk=torch.zeros_like(g.dk)) == ["dk"]
    assert misses(dk=g.first["dk"]) == ["dk"]
    assert misses(dk=g.second["dk"]) == ["dk"]
    assert misses(dk=g.dk * 1.02) == ["dk"]
    assert misses(dv=torch.zeros_like(g.dv)) == ["dv"]
    assert misses(dv=g.dv * 1.02) == ["dv"]
    # and in every branch by itself
    for b in range(hc):
        only = torch.zeros(1, hc, 1, dtype=F)
        only[:, b] = 1
        assert misses(dk=g.dk * (1 - only)) == ["dk"] and misses(dh=g.dh - only * (g.dh - g.dy)) == ["dh"]
