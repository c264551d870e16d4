"""Norms around a block on matrices of more than 2^31 elements, forward and backward: rows at both ends hold values, those
between them zeros, which add nothing to any sum, so the few rows' definition is the answer."""
import pytest
import torch

import norm_reference as R
import sparse_moe_layer_route_gb300 as M
from test_norm_gpu import BF16, F32, SEED, STEP

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d,pad", [(300001, 7200, 8), (300001, 7201, 0), (140001, 16384, 0)])
def test_past_2_to_the_31_elements(T, d, pad):
    g = torch.Generator().manual_seed(d)
    rows = torch.tensor([0, 1, 2, T // 2, T - 3, T - 2, T - 1])
    gate_rows, p = T // 3 + 1, 0.1

    def matrix(ld):
        m = torch.zeros(T, ld, dtype=BF16, device="cuda")[:, :d]
        m[rows.cuda()] = torch.randn(len(rows), d, generator=g).to(BF16).cuda()
        return m

    h, y, d_h_out, d_n = matrix(d + pad), matrix(d + pad), matrix(d), matrix(d)
    assert h.numel() > 2 ** 31
    w = {k: (1 + 0.3 * torch.randn(n, d, generator=g)).cuda().squeeze(0)
         for k, n in (("w_after", 1), ("gate", 3), ("w_before", 1))}
    cfg = M.ResidualNormConfig.make(T, d, after=M.NORM_RMS, before=M.NORM_LAYER, w_dtype=M.DTYPE_F32,
                                    gate_rows=gate_rows, eps=1e-5, alpha=0.75, beta=1.25, p_drop=p,
                                    ld_h=d + pad, ld_y=d + pad)
    rng = torch.tensor([SEED, STEP], device="cuda")
    c = dict(after=R.RMS, before=R.LAYER, alpha=cfg.alpha, beta=cfg.beta, eps=cfg.eps, gate_rows=1)
    m = torch.cat([R.factors(SEED, STEP, 1, d, p, row0=int(r)) for r in rows]).cuda()

    def some(v):
        return v[rows.cuda()].double()

    t = {"h": some(h), "y": some(y), "w_after": w["w_after"].double(), "b_after": None,
         "gate": w["gate"].double()[rows.cuda() // gate_rows], "w_before": w["w_before"].double(), "b_before": None}
    h_out, n = torch.empty(T, d, dtype=BF16, device="cuda"), torch.empty(T, d, dtype=BF16, device="cuda")
    M.residual_norm(cfg, h, y, h_out, n, **w, rng=rng)
    h64, n64, dh, dn = R.forward(c, t, m)
    R.assert_close("h_out", h_out[rows.cuda()], h64, dh)
    R.assert_close("n", n[rows.cuda()], n64, dn)
    assert (h_out[3:T // 2] == 0).all() and (n[T // 2 + 1:T - 3] == 0).all()
    del n
    # the gradient, in the place of the gradients that come in
    stream = h
    stream[rows.cuda()] = h_out[rows.cuda()]
    del h_out
    before = {"h_out": some(stream), "d_h_out": some(d_h_out), "d_n": some(d_n)}
    ws = torch.empty(M.residual_norm_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    sums = {k: torch.full(v.shape, float("nan"), dtype=F32, device="cuda") for k, v in w.items()}
    M.residual_norm_backward(cfg, stream, y, d_h_out, d_n, d_h_out, d_n, ws, **w, rng=rng,
                             **{"d_" + k: v for k, v in sums.items()})
    want, err = R.backward(c, {**t, **before}, m)
    R.assert_close("d_h", d_h_out[rows.cuda()], want["d_h"], err["d_h"])
    R.assert_close("d_y", d_n[rows.cuda()], want["d_y"], err["d_y"])
    assert (d_h_out[3:T // 2] == 0).all() and (d_n[T // 2 + 1:T - 3] == 0).all()
    for name in ("w_after", "w_before"):
        R.assert_close(name, sums[name], want["d_" + name], err["d_" + name])
    for i in range(3):
        mine = (rows // gate_rows == i).cuda()
        R.assert_close("gate", sums["gate"][i], want["d_gate"][mine].sum(0), err["d_gate"][mine].sum(0))
