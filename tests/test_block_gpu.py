"""The few-token layer, the norms around it and dropout together, as a model's blocks run them: decoding steps,
eagerly and as a graph, and a training step."""
import pytest
import torch

import few_reference as F
import norm_reference as R
import sparse_moe_layer_route_gb300 as M

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
CODE = {F32: M.DTYPE_F32, BF16: M.DTYPE_BF16}
SHAPE = dict(d=576, E=12, k=3, f=320, S=1)


class Decoder:
    """Three blocks of T tokens: a norm, the layer, a norm of its output, a gate per channel, the residual.
    One workspace and one row of buffers serve all blocks; h is updated in place."""

    def __init__(self, T, stream, first_gate=1):
        g = torch.Generator().manual_seed(T)
        d, E, k, f, S = SHAPE.values()
        self.T, self.d, self.k, self.S, self.stream = T, d, k, S, stream
        self.p = [F.make(T, d, E, k, f, S, seed=10 + i) for i in range(3)]
        self.w = [M.make_weights(p["W_g"], p["bias"], p["W_gate"], p["W_up"], p["W_down"], p["Wsh_gate"],
                                 p["Wsh_up"], p["Wsh_down"], W_g_t=M.prepare_router(p["W_g"]))
                  for p in self.p]
        self.cfg = M.MoeConfig.make(T, d, E, k, f, n_shared=S, mode=M.ROUTE_BIAS_SELECT)
        kw = dict(h_dtype=CODE[stream], y_dtype=M.DTYPE_BF16, w_dtype=M.DTYPE_F32)
        self.enter = M.ResidualNormConfig.make(T, d, before=M.NORM_RMS, **kw)
        self.between = M.ResidualNormConfig.make(T, d, after=M.NORM_RMS, before=M.NORM_RMS, gate_rows=T,
                                                 alpha=0.5, **kw)
        self.leave = M.ResidualNormConfig.make(T, d, after=M.NORM_RMS, before=M.NORM_NONE, gate_rows=T,
                                               alpha=0.5, **kw)

        def param(*shape):
            return (0.3 * torch.randn(*shape, generator=g) + 1).cuda()

        self.norms = [dict(w_after=param(d), gate=param(1, d), w_before=param(d) if i < 2 else None)
                      for i in range(3)]
        self.w_first = param(d)
        self.ws = M.alloc_few_workspace(self.cfg)
        self.h = torch.zeros(T, d, dtype=stream, device="cuda")
        self.n = torch.zeros(T, d, dtype=BF16, device="cuda")
        self.y = torch.zeros(T, d, dtype=BF16, device="cuda")
        self.idx = [torch.zeros(T, k, dtype=torch.int32, device="cuda") for _ in range(3)]
        self.gates = [torch.zeros(T, k, device="cuda") for _ in range(3)]
        self.route = [M.make_route_out(i, w) for i, w in zip(self.idx, self.gates)]

    def run(self, look=lambda name, i: None):
        M.residual_norm(self.enter, self.h, None, None, self.n, w_before=self.w_first)
        look("enter", 0)
        for i in range(3):
            M.layer_forward_few(self.cfg, self.w[i], self.n, None, self.y, self.route[i], self.ws)
            look("layer", i)
            cfg = self.between if i < 2 else self.leave
            M.residual_norm(cfg, self.h, self.y, self.h, self.n if i < 2 else None, **self.norms[i])
            look("norm", i)


def inputs(T, dtype, seed):
    return torch.randn(T, SHAPE["d"], generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("stream", [F32, BF16])
@pytest.mark.parametrize("T", [1, 6, 16])
def test_decoding_steps(T, stream):
    """Each step of the blocks against 64 bits, from what the step before left."""
    m = Decoder(T, stream)
    m.h.copy_(inputs(T, stream, 1))
    before = {"h": m.h.clone()}

    def look(name, i):
        if name == "layer":
            idx, w, gap = F.choose({**m.p[i], "x": m.n}, m.k, F.BIAS)
            # logits are the same sums whatever else runs; a choice decided by less than 1e-6 is not looked at
            same = gap > 1e-6
            assert not same or torch.equal(m.idx[i].long(), idx)
            want, err = F.layer({**m.p[i], "x": m.n}, m.idx[i], m.gates[i], 0, m.S)
            F.assert_rounded(m.y, want, err)
            return
        cfg = m.enter if name == "enter" else m.between if i < 2 else m.leave
        p = dict(w_after=None, b_after=None, gate=None, w_before=m.w_first, b_before=None)
        if name == "norm":
            p.update(m.norms[i])
        c = dict(after=cfg.after, before=cfg.before, alpha=cfg.alpha, beta=cfg.beta, eps=cfg.eps,
                 gate_rows=cfg.gate_rows)
        t = {k: None if v is None else v.double() for k, v in p.items()}
        t.update(h=before["h"].double(), y=m.y.double() if name == "norm" else None)
        h, n, dh, dn = R.forward(c, t)
        if name == "norm":
            R.assert_close("h", m.h, h, dh)
        if n is not None:
            R.assert_close("n", m.n, n, dn)
        before["h"] = m.h.clone()

    m.run(look)
    assert M.device_status(m.ws) == 0


def test_a_graph_of_blocks():
    """All blocks in one graph, replayed with other inputs, are the eager calls bit for bit; two models' graphs
    on two streams, each with a workspace of its own, do not disturb one another."""
    models = [Decoder(5, F32), Decoder(16, BF16)]
    streams = [torch.cuda.Stream() for _ in models]
    graphs = []
    for m, s in zip(models, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            m.run()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            m.run()
        graphs.append(graph)
    for seed in (2, 3, 4):
        want = []
        for m in models:
            m.h.copy_(inputs(m.T, m.stream, seed))
            m.run()
            want.append((m.h.clone(), [i.clone() for i in m.idx]))
            m.h.copy_(inputs(m.T, m.stream, seed))
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for m, (h, idx) in zip(models, want):
            assert torch.equal(m.h, h)
            assert all(torch.equal(a, b) for a, b in zip(m.idx, idx))
            assert M.device_status(m.ws) == 0


@pytest.mark.parametrize("T,d", [(37, 96), (130, 257)])
def test_a_training_step(T, d):
    """x -> dropout -> h1; n1 = norm(h1); y = n1 W; h2 = h1 / 2 + gate * drop(norm(y)), n2 = norm(h2), and back
    through all of it, against automatic differentiation in 64 bits.

    Every step's result is off by its own bound and by what the steps before were off, which goes through the
    absolute values of its derivative: backward()'s bound is 500 U of the terms' sizes for d_h and d_y, so a
    call with the errors for gradients gives that as bound / (500 U). Its 500 U are for the step's sums; that
    values of the forward pass are off by some 50 U is less than them again, hence twice the bound."""
    g = torch.Generator().manual_seed(T)

    def rand(*shape, scale=1.0, mean=0.0):
        return (scale * torch.randn(*shape, generator=g) + mean).cuda()

    x, W, c_h, c_n = rand(T, d), rand(d, d, scale=d ** -0.5), rand(T, d), rand(T, d)
    w1, b1, w2, w3, gate = (rand(d, scale=0.3, mean=1.0), rand(d), rand(d, mean=1.0, scale=0.3),
                            rand(d, mean=1.0, scale=0.3), rand(-(-T // 20), d))
    rng = [torch.tensor([5, step], device="cuda") for step in (1, 2)]
    first = M.ResidualNormConfig.make(T, d, before=M.NORM_LAYER, h_dtype=M.DTYPE_F32, y_dtype=M.DTYPE_F32,
                                      w_dtype=M.DTYPE_F32)
    block = M.ResidualNormConfig.make(T, d, after=M.NORM_RMS, before=M.NORM_RMS, h_dtype=M.DTYPE_F32,
                                      y_dtype=M.DTYPE_F32, w_dtype=M.DTYPE_F32, gate_rows=20, alpha=0.5,
                                      p_drop=0.25)
    ws = torch.empty(max(M.residual_norm_workspace_size(first), M.residual_norm_workspace_size(block)),
                     dtype=torch.uint8, device="cuda")

    def new(*shape):
        return torch.full(shape, float("nan"), device="cuda")

    h1, n1, h2, n2 = (new(T, d) for _ in range(4))
    M.dropout(x, 0.1, rng[0], h1)
    M.residual_norm(first, h1, None, None, n1, w_before=w1, b_before=b1)
    y = (n1.double() @ W.double()).float()
    M.residual_norm(block, h1, y, h2, n2, w_after=w2, gate=gate, w_before=w3, rng=rng[1])
    got = {k: new(T, d) for k in ("d_h1", "d_y", "d_x")}
    got.update(w1=new(d), b1=new(d), w2=new(d), w3=new(d), gate=new(*gate.shape))
    M.residual_norm_backward(block, h2, y, c_h, c_n, got["d_h1"], got["d_y"], ws, w_after=w2, gate=gate,
                             w_before=w3, rng=rng[1], d_w_after=got["w2"], d_gate=got["gate"],
                             d_w_before=got["w3"])
    d_n1 = (got["d_y"].double() @ W.double().T).float()
    M.residual_norm_backward(first, h1, None, got["d_h1"], d_n1, got["d_h1"], None, ws, w_before=w1,
                             d_w_before=got["w1"], d_b_before=got["b1"])
    M.dropout(got["d_h1"], 0.1, rng[0], got["d_x"])

    # automatic differentiation, 64 bits
    m = [R.factors(5, step, T, d, p).cuda() for step, p in ((1, 0.1), (2, 0.25))]
    leaves = {k: v.double().requires_grad_() for k, v in
              dict(d_x=x, w1=w1, b1=b1, w2=w2, w3=w3, gate=gate).items()}
    W64, eps = W.double(), block.eps
    a1 = leaves["d_x"] * m[0]
    an1 = R.normed(R.LAYER, a1, eps)[0] * leaves["w1"] + leaves["b1"]
    ay = an1 @ W64
    au = R.normed(R.RMS, ay, eps)[0] * leaves["w2"] * m[1]
    a2 = 0.5 * a1 + leaves["gate"].repeat_interleave(20, 0)[:T] * au
    an2 = R.normed(R.RMS, a2, eps)[0] * leaves["w3"]
    ((a2 * c_h.double()).sum() + (an2 * c_n.double()).sum()).backward()

    # the bounds, step by step back
    def double(v):
        return None if v is None else v.detach().double()

    c2 = dict(after=R.RMS, before=R.RMS, alpha=0.5, beta=1.0, eps=eps, gate_rows=20)
    t2 = dict(h=double(a1), y=double(ay), h_out=double(a2), d_h_out=double(c_h), d_n=double(c_n),
              w_after=double(w2), b_after=None, gate=double(gate), w_before=double(w3), b_before=None)
    g2, e2 = R.backward(c2, t2, m[1])
    dn1 = g2["d_y"] @ W64.T
    en1 = e2["d_y"] @ W64.abs().T + 2 * R.U * dn1.abs()
    c1 = dict(after=R.NONE, before=R.LAYER, alpha=1.0, beta=1.0, eps=eps, gate_rows=0)
    t1 = dict(h=double(a1), y=None, h_out=double(a1), d_h_out=g2["d_h"], d_n=dn1, w_after=None, b_after=None,
              gate=None, w_before=double(w1), b_before=None)
    _, e1 = R.backward(c1, t1)
    _, through = R.backward(c1, {**t1, "d_h_out": e2["d_h"], "d_n": en1})
    steps = {"d_h": 500, "d_w_before": 700 + T / 100, "d_b_before": 700 + T / 100}
    through = {k: through[k] / (n * R.U) for k, n in steps.items()}
    err = {"d_x": m[0] * (e1["d_h"] + through["d_h"]), "w1": e1["d_w_before"] + through["d_w_before"],
           "b1": e1["d_b_before"] + through["d_b_before"], "w2": e2["d_w_after"], "w3": e2["d_w_before"],
           "gate": e2["d_gate"]}
    for name, leaf in leaves.items():
        R.assert_close(name, got[name], leaf.grad, 2 * err[name])
