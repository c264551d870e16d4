"""Gradient of renormalised sigmoid weights where every chosen score is next to fp32's smallest numbers.

u = 2^-24. A score of at least 3.5e-39 is within 2^-150 of its rounded value, 3.4 u, beyond the 6 u of the
formula; the quotient of a score and their sum is within 6 + 6 + 2 * 3.4 + 8 + 2 u = 29 u of its value, and
the gradient, two such terms of at most M = scale max|d_w| + max|d_scores|, within 64 u (2 M), as
elsewhere. No gradient is infinite: a score's own, (d_w - mean) / sum, is near the largest number here.
"""
import pytest
import torch

import sparse_moe_layer_route_gb300 as M

U = 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(9, 16, 2), (40, 40, 1), (33, 256, 8)])
@pytest.mark.parametrize("with_scores", [False, True])
def test_gradient_of_low_sigmoids(T, E, k, with_scores):
    g = torch.Generator().manual_seed(E)
    l = (-88.4 + 2.4 * torch.rand(T, E, generator=g)).cuda()
    l[1] = -88.5
    cfg = M.GateConfig.make(T, E, k, score=M.SCORE_SIGMOID, scale=2.5)
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    M.route_logits(cfg, l, None, idx, w)
    d_w = (8 * torch.randn(T, k, generator=g)).cuda()
    d_s = torch.randn(T, E, generator=g).cuda() if with_scores else None
    out = torch.full((T, E), float("nan"), device="cuda")
    M.route_logits_backward(cfg, l, idx, d_w, d_s, out)
    x = l.double().requires_grad_(True)
    s = torch.sigmoid(x)
    sel = s.gather(1, idx.long())
    w64 = 2.5 * sel / sel.sum(-1, keepdim=True)
    loss = (w64 * d_w).sum() + ((s * d_s).sum() if with_scores else 0)
    want = torch.autograd.grad(loss, x)[0]
    most = 2 * 2.5 * d_w.abs().amax(-1, keepdim=True) + (d_s.abs().amax(-1, keepdim=True)
                                                         if with_scores else 0)
    assert ((out - want).abs() <= 64 * U * most).all()
    assert ((w - w64).abs() <= 40 * U * w64).all()
