"""Routing of as many tokens as the configuration's limits admit (T * top_k < 2^31)."""
import pytest
import torch

import sparse_moe_layer_route_gb300 as M


@pytest.mark.gpu
def test_tokens_up_to_the_limit():
    """One expert and logits of 0: its sigmoid is 1/2, its renormalised weight 1, the gradient of the score
    1/4; all exact."""
    T = 2 ** 31 - 1
    cfg = M.GateConfig.make(T, 1, 1, score=M.SCORE_SIGMOID, dtype=M.DTYPE_BF16)
    logits = torch.zeros(T, 1, dtype=torch.bfloat16, device="cuda")
    idx = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
    w = torch.zeros(T, 1, device="cuda")
    M.route_logits(cfg, logits, None, idx, w)
    assert idx.min() == 0 and idx.max() == 0 and w.min() == 1 and w.max() == 1
    w.fill_(3.0)                                    # gradients now: of the weights, which has none,
    d = torch.full((T, 1), float("nan"), dtype=torch.bfloat16, device="cuda")
    M.route_logits_backward(cfg, logits, idx, w, None, d)
    assert d.min() == 0 and d.max() == 0
    M.route_logits_backward(cfg, logits, idx, None, w, d)   # and of the scores
    assert d.min() == 0.75 and d.max() == 0.75
