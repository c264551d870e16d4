"""The example layer: routing from logits, dispatch, 8-bit experts and combine together, and the
router's training step."""
import pytest
import torch

import sparse_moe_layer_route_gb300 as M
from examples.int8_layer import Int8MoeLayer


def codes64(x):
    s = x.abs().amax(-1, keepdim=True) / 127
    return torch.nan_to_num(x / s).round(), s


def expert64(q, s, mats, names, e):
    gate, up, down = (mats[n] for n in names)
    a = (q @ gate[0][e].double().T) * s * gate[1][e].double()
    b = (q @ up[0][e].double().T) * s * up[1][e].double()
    qh, sh = codes64(a * torch.sigmoid(a) * b)
    return (qh @ down[0][e].double().T) * sh * down[1][e].double()


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [1, 3, 64, 300])
def test_layer_output(tokens):
    """Against 64 bits on the layer's own routing: codes that move by one (half-way values) give
    5e-3 of the norm, as for the experts alone, and the combine rounds once to bf16, 2^-8."""
    layer = Int8MoeLayer(tokens, seed=tokens)
    x = torch.randn(tokens, layer.cfg.d, device="cuda").bfloat16()
    out = layer.forward(x)
    assert M.device_status(layer.ws) == 0 and M.device_status(layer.ws8) == 0
    assert abs(layer.topk_w.sum(-1) - 2.5).max() < 1e-5
    mats = dict(zip(("gate", "up", "down", "sh_gate", "sh_up", "sh_down"), layer.weights._tensors))
    q, s = codes64(x.double())
    want = expert64(q, s, mats, ("sh_gate", "sh_up", "sh_down"), 0)
    for e in range(layer.cfg.E):
        t, j = torch.nonzero(layer.idx == e, as_tuple=True)
        if t.numel():
            y = expert64(q[t], s[t], mats, ("gate", "up", "down"), e)
            want.index_add_(0, t, y * layer.topk_w[t, j].double()[:, None])
    off = out.double() - want
    assert off.norm() <= (5e-3 + 2.0 ** -8) * want.norm()


@pytest.mark.gpu
def test_training_step_lowers_the_loss():
    layer = Int8MoeLayer(256, seed=1)
    x = torch.randn(256, layer.cfg.d, device="cuda").bfloat16()
    target = torch.randn(256, layer.cfg.d, device="cuda")
    losses = []
    for _ in range(10):
        out = layer.forward(x).float()
        losses.append((out - target).square().mean().item())
        layer.W_router -= 50.0 * layer.router_gradient(x, (out - target) * (2.0 / out.numel()))
    assert losses[-1] < losses[0]
    assert M.device_status(layer.ws) == 0 and M.device_status(layer.ws8) == 0
