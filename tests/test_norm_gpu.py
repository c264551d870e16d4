"""Norms around a block, gates and dropout, forward and backward, against 64 bits."""
import pytest
import torch

import norm_reference as R
import sparse_moe_layer_route_gb300 as M

pytestmark = pytest.mark.gpu

CODE = {torch.float32: M.DTYPE_F32, torch.bfloat16: M.DTYPE_BF16, torch.float16: M.DTYPE_F16}
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
SEED, STEP = -0x123456789ABCDEF, 0x7654321F00000005
PARAMS = ("w_after", "b_after", "gate", "w_before", "b_before")


def rows(g, T, d, dtype, pad, scale=1.0, mean=0.0):
    return (torch.randn(T, d + pad, generator=g) * scale + mean).to(dtype).cuda()[:, :d]


class Case:
    def __init__(self, T, d, after, before, h=BF16, y=BF16, w=F32, gate=0, bias=False, weight=True,
                 alpha=1.0, beta=1.0, p=0.0, pad_h=0, pad_y=0, mean=0.0, block=True, seed=0, eps=1e-5):
        g = torch.Generator().manual_seed(seed + T * 7 + d)
        self.T, self.d, self.p, self.h_type, self.y_type = T, d, p, h, y
        self.c = dict(after=after, before=before, alpha=alpha, beta=beta, eps=eps, gate_rows=gate)
        self.cfg = M.ResidualNormConfig.make(
            T, d, after=after, before=before, h_dtype=CODE[h], y_dtype=CODE[y], w_dtype=CODE[w],
            gate_rows=gate, eps=eps, alpha=alpha, beta=beta, p_drop=p, ld_h=d + pad_h if pad_h else 0,
            ld_y=d + pad_y if pad_y else 0)
        # 32-bit factors, as the configuration carries them
        self.c.update(alpha=self.cfg.alpha, beta=self.cfg.beta, eps=self.cfg.eps)
        self.h = rows(g, T, d, h, pad_h, 2.0, mean)
        self.y = rows(g, T, d, y, pad_y, 0.7, -mean) if block else None

        def param(there, *shape, mean=1.0):
            return (torch.randn(*shape, generator=g) * 0.3 + mean).to(w).cuda() if there else None

        self.w = {"w_after": param(weight and after, d), "b_after": param(bias and after, d, mean=0.1),
                  "gate": param(gate, -(-T // gate) if gate else 0, d, mean=0.5),
                  "w_before": param(weight and before, d), "b_before": param(bias and before, d, mean=0.1)}
        self.rng = torch.tensor([SEED, STEP], device="cuda") if p else None
        self.m = R.factors(SEED, STEP, T, d, p).cuda() if p else None
        self.d_h_out = rows(g, T, d, h, 0)
        self.d_n = rows(g, T, d, y, 0) if before else None

    def tensors(self):
        t = {name: None if v is None else v.double() for name, v in self.w.items()}
        return {**t, "h": self.h.double(), "y": None if self.y is None else self.y.double()}

    def run(self, **kw):
        h_out = torch.full((self.T, self.d), float("nan"), dtype=self.h_type, device="cuda")
        n = torch.full((self.T, self.d), float("nan"), dtype=self.y_type, device="cuda") \
            if self.c["before"] else None
        M.residual_norm(self.cfg, self.h, self.y, h_out, n, **self.w, rng=self.rng, **kw)
        return h_out, n

    def check_forward(self):
        h_out, n = self.run()
        h64, n64, dh, dn = R.forward(self.c, self.tensors(), self.m)
        R.assert_close("h_out", h_out, h64, dh)
        if n is not None:
            R.assert_close("n", n, n64, dn)
        return h_out

    def gradients(self, h_out, d_h_out, d_n, ws=None, **kw):
        def out(*shape, dtype=F32):
            return torch.full(shape, float("nan"), dtype=dtype, device="cuda")

        g = {"d_h": out(self.T, self.d, dtype=self.h_type),
             "d_y": None if self.y is None else out(self.T, self.d, dtype=self.y_type)}
        for name, v in self.w.items():
            g["d_" + name] = None if v is None else out(*v.shape)
        if ws is None:
            ws = torch.empty(M.residual_norm_workspace_size(self.cfg), dtype=torch.uint8, device="cuda")
            ws.fill_(255)                    # NaN wherever it is read before it is written
        M.residual_norm_backward(
            self.cfg, h_out, self.y, d_h_out, d_n, g["d_h"], g["d_y"], ws,
            **{k: v for k, v in self.w.items() if k != "b_before"}, rng=self.rng,
            **{"d_" + k: g["d_" + k] for k in PARAMS}, **kw)
        return g

    def check_backward(self, d_h_out, d_n):
        h_out = self.stream()
        g = self.gradients(h_out, d_h_out, d_n)
        t = {**self.tensors(), "h_out": h_out.double(),
             "d_h_out": None if d_h_out is None else d_h_out.double(),
             "d_n": None if d_n is None else d_n.double()}
        want, err = R.backward(self.c, t, self.m)
        for name, v in g.items():
            if v is None:
                continue
            if name not in want:             # no gradient reaches it
                assert (v == 0).all(), name
            else:
                R.assert_close(name, v, want[name], err[name])

    def stream(self):
        """h' in the stream's type, with the strides that the configuration says."""
        wide = torch.zeros(self.T, self.cfg.ld_h or self.d, dtype=self.h_type, device="cuda")
        wide[:, :self.d] = R.forward(self.c, self.tensors(), self.m)[0]
        return wide[:, :self.d]


KINDS = [(R.RMS, R.RMS), (R.NONE, R.RMS), (R.LAYER, R.LAYER), (R.RMS, R.NONE), (R.NONE, R.LAYER),
         (R.NONE, R.NONE)]
# every form of rows (one warp to clusters), its edges, odd ones
WIDTHS = [1, 7, 8, 255, 256, 257, 512, 513, 1024, 1027, 1536, 1537, 2048, 2049, 4096, 4100, 7168, 8192, 8200, 16384, 16385]


@pytest.mark.parametrize("after,before", KINDS)
@pytest.mark.parametrize("d", WIDTHS)
def test_widths(after, before, d):
    c = Case(5, d, after, before, gate=2, bias=True, alpha=0.75, beta=1.25, p=0.1)
    c.check_forward()
    c.check_backward(c.d_h_out, c.d_n)


@pytest.mark.parametrize("T,d", [(2, 32768), (3, 65536), (2, 40001)])
def test_rows_of_large_clusters(T, d):
    c = Case(T, d, R.LAYER, R.RMS, h=F32, y=F16, gate=1)
    c.check_forward()
    c.check_backward(c.d_h_out, c.d_n)


@pytest.mark.parametrize("h", [F32, BF16, F16])
@pytest.mark.parametrize("y", [F32, BF16, F16])
@pytest.mark.parametrize("w", [F32, BF16, F16])
def test_types(h, y, w):
    for d, pad in ((320, 0), (321, 3), (1536, 8)):
        c = Case(9, d, R.RMS, R.LAYER, h=h, y=y, w=w, gate=4, bias=True, pad_h=pad, pad_y=2 * pad)
        c.check_forward()
        c.check_backward(c.d_h_out, c.d_n)


@pytest.mark.parametrize("gate", [0, 1, 2, 7, 100, 701, 702, 703, 5000])
@pytest.mark.parametrize("T,d", [(1, 64), (702, 96), (702, 640), (702, 2304), (350, 8192)])
def test_rows_of_gates(T, d, gate):
    """Tokens of one row of gates in one CTA's run, or in several."""
    c = Case(T, d, R.RMS, R.RMS, gate=gate)
    c.check_forward()
    c.check_backward(c.d_h_out, c.d_n)


@pytest.mark.parametrize("T,d", [(1, 4096), (17, 4096), (3000, 1024), (3001, 1027), (20000, 48), (612, 8192)])
def test_numbers_of_tokens(T, d):
    c = Case(T, d, R.LAYER, R.RMS, h=F32, gate=max(1, T // 3), bias=True, p=0.25)
    c.check_forward()
    c.check_backward(c.d_h_out, c.d_n)


@pytest.mark.parametrize("d", [96, 2000, 7168])
def test_parts_that_are_not_there(d):
    for kw in (dict(after=R.NONE, before=R.RMS, block=False, alpha=0.5),
               dict(after=R.RMS, before=R.RMS, weight=False),
               dict(after=R.LAYER, before=R.LAYER, weight=False, bias=True),
               dict(after=R.NONE, before=R.NONE), dict(after=R.NONE, before=R.NONE, gate=3, p=0.5)):
        c = Case(11, d, **kw)
        c.check_forward()
        c.check_backward(c.d_h_out, c.d_n)
    c = Case(11, d, R.RMS, R.RMS, gate=4, bias=True)
    c.check_backward(None, c.d_n)
    c.check_backward(c.d_h_out, None)
    # only the next input, only the stream
    h_out, n = c.run()
    only = torch.empty_like(n)
    M.residual_norm(c.cfg, c.h, c.y, None, only, **c.w)
    assert torch.equal(only, n)


@pytest.mark.parametrize("d", [200, 1300, 5000])
def test_gradients_that_are_not_wanted(d):
    c = Case(300, d, R.RMS, R.LAYER, gate=77, bias=True, p=0.1)
    h_out = c.stream()
    full = c.gradients(h_out, c.d_h_out, c.d_n)
    for wanted in PARAMS + (None,):
        keep = {k: v for k, v in c.w.items()}
        ws = torch.empty(M.residual_norm_workspace_size(c.cfg), dtype=torch.uint8, device="cuda")
        d_h, d_y = torch.empty_like(c.d_h_out), torch.empty_like(c.d_n)
        grads = {} if wanted is None else {"d_" + wanted: torch.empty_like(full["d_" + wanted])}
        M.residual_norm_backward(c.cfg, h_out, c.y, c.d_h_out, c.d_n, d_h, d_y, ws,
                                 **{k: v for k, v in keep.items() if k != "b_before"}, rng=c.rng, **grads)
        assert torch.equal(d_h, full["d_h"]) and torch.equal(d_y, full["d_y"])
        for name, v in grads.items():
            assert torch.equal(v, full[name]), name


@pytest.mark.parametrize("mean", [30.0, -1000.0])
def test_rows_far_from_zero(mean):
    """A layer norm's variance is taken around the mean."""
    c = Case(20, 1536, R.LAYER, R.LAYER, h=F32, y=F32, mean=mean)
    c.check_forward()
    c.check_backward(c.d_h_out, c.d_n)


def test_rows_of_zeros():
    c = Case(4, 520, R.RMS, R.LAYER, alpha=1.0, gate=2)
    c.h.zero_()
    c.y[1:].zero_()
    c.check_forward()
    c.check_backward(c.d_h_out, c.d_n)
    c.c["eps"] = 0.0
    z = M.ResidualNormConfig.make(4, 520, after=M.NORM_NONE, before=M.NORM_RMS, eps=0.0, w_dtype=M.DTYPE_F32)
    n = torch.zeros(4, 520, dtype=BF16, device="cuda")
    M.residual_norm(z, c.h, None, None, n)
    assert torch.isnan(n).all()              # 0 / 0, as defined


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_row(bad):
    c = Case(40, 700, R.RMS, R.RMS, p=0.3)
    want, want_n = c.run()
    c.y[7, 3] = bad
    got, n = c.run()
    rest = [t for t in range(40) if t != 7]
    assert torch.equal(got[rest], want[rest]) and torch.equal(n[rest], want_n[rest])
    # a dropped element is 0 whatever it is
    c = Case(40, 700, R.NONE, R.RMS, p=0.3)
    dropped = (c.m == 0).nonzero()
    want, _ = c.run()
    for t, k in dropped[::97].tolist():
        c.y[t, k] = bad
    assert torch.equal(c.run()[0], want)


def test_outputs_in_the_place_of_inputs():
    for d in (384, 1111, 4096):
        c = Case(33, d, R.RMS, R.RMS, gate=10, p=0.1)
        h_out, n = c.run()
        g = c.gradients(h_out, c.d_h_out, c.d_n)
        h, y = c.h.clone(), c.y.clone()
        M.residual_norm(c.cfg, h, y, h, y, **c.w, rng=c.rng)
        assert torch.equal(h, h_out) and torch.equal(y, n)
        for other in ("d_n", "y"):
            dh, dn, y = c.d_h_out.clone(), c.d_n.clone(), c.y.clone()
            ws = torch.empty(M.residual_norm_workspace_size(c.cfg), dtype=torch.uint8, device="cuda")
            M.residual_norm_backward(c.cfg, h_out, y, dh, dn, dh, dn if other == "d_n" else y, ws,
                                     **{k: v for k, v in c.w.items() if k != "b_before"}, rng=c.rng)
            assert torch.equal(dh, g["d_h"]) and torch.equal(dn if other == "d_n" else y, g["d_y"])


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("T,d,pad", [(1, 1, 0), (4, 1, 0), (3, 2, 1), (5, 256, 0), (5, 255, 2), (4, 513, 0),
                                     (7, 1027, 3), (3, 2304, 1), (2, 8200, 1)])
def test_tensors_that_start_in_the_middle_of_a_word(T, d, pad, dtype):
    """Inputs and outputs one element into their buffers: rows that start on words and between them in turn, nothing
    before the first one, and what lies around the outputs stays."""
    c = Case(T, d, R.RMS, R.LAYER, h=dtype, y=dtype, w=dtype, gate=2, bias=True, p=0.1, pad_h=pad, pad_y=pad)

    def inside(v, pad=0):
        buf = torch.full((T * (d + pad) + 2,), float("nan"), dtype=dtype, device="cuda")
        view = buf[1:-1].view(T, d + pad)[:, :d]
        view.copy_(v)
        return view, buf

    c.h, c.y = inside(c.h, pad)[0], inside(c.y, pad)[0]
    (h_out, h_buf), (n, n_buf) = inside(c.d_n), inside(c.d_n)
    M.residual_norm(c.cfg, c.h, c.y, h_out, n, **c.w, rng=c.rng)
    h64, n64, dh, dn = R.forward(c.c, c.tensors(), c.m)
    R.assert_close("h_out", h_out, h64, dh)
    R.assert_close("n", n, n64, dn)
    c.d_h_out, c.d_n = inside(c.d_h_out)[0], inside(c.d_n)[0]
    c.check_backward(c.d_h_out, c.d_n)
    for buf in (h_buf, n_buf):
        assert buf[0].isnan() and buf[-1].isnan()


@pytest.mark.parametrize("d", [64, 1024, 2304])
def test_32_bit_rows_on_16_bytes_but_not_on_32(d):
    T = 5
    c = Case(T, d, R.RMS, R.LAYER, h=F32, y=F32, gate=1, p=0.1)

    def off():
        buf = torch.full((T * d + 8,), 3.0, device="cuda")
        return buf[4:-4].view(T, d), buf

    want = c.run()
    (h_out, h_buf), (n, n_buf), (d_h, dh_buf), (d_y, dy_buf) = off(), off(), off(), off()
    M.residual_norm(c.cfg, c.h, c.y, h_out, n, **c.w, rng=c.rng)
    assert torch.equal(h_out, want[0]) and torch.equal(n, want[1])
    g = c.gradients(want[0], c.d_h_out, c.d_n)
    (d_gate, dg_buf) = off()
    ws = torch.empty(M.residual_norm_workspace_size(c.cfg), dtype=torch.uint8, device="cuda")
    M.residual_norm_backward(c.cfg, h_out, c.y, c.d_h_out, c.d_n, d_h, d_y, ws,
                             **{k: v for k, v in c.w.items() if k != "b_before"}, rng=c.rng, d_gate=d_gate)
    assert torch.equal(d_h, g["d_h"]) and torch.equal(d_y, g["d_y"]) and torch.equal(d_gate, g["d_gate"])
    x, x_buf = off()
    M.dropout(c.h, 0.1, c.rng, x)
    aligned = torch.empty_like(c.h)
    M.dropout(c.h, 0.1, c.rng, aligned)
    assert torch.equal(x, aligned)
    for buf in (h_buf, n_buf, dh_buf, dy_buf, dg_buf, x_buf):
        assert (buf[:4] == 3).all() and (buf[-4:] == 3).all()


def test_what_lies_between_and_behind_rows_stays():
    T, d, pad = 6, 100, 28
    for base in (torch.full((T + 1, d + pad), 7.0, dtype=BF16, device="cuda"),):
        c = Case(T, d, R.RMS, R.RMS, pad_h=pad, pad_y=pad)
        out = torch.full((T + 2, d), 5.0, dtype=BF16, device="cuda")
        n = torch.full((T + 2, d), 5.0, dtype=BF16, device="cuda")
        before = c.h._base.clone() if c.h._base is not None else None
        M.residual_norm(c.cfg, c.h, c.y, out[:T], n[:T], **c.w)
        assert (out[T:] == 5).all() and (n[T:] == 5).all()
        if before is not None:
            assert torch.equal(c.h._base, before)


def test_gradient_against_differences():
    """Along random directions of every input, the 64-bit definition's central difference is the inner product
    of the gradient with the direction."""
    T, d = 6, 130
    c = Case(T, d, R.LAYER, R.RMS, h=F32, y=F32, gate=4, bias=True, alpha=0.9, beta=1.1, p=0.2)
    t = c.tensors()
    h_out = R.forward(c.c, t, c.m)[0]
    g = c.gradients(h_out.float(), c.d_h_out, c.d_n)

    def loss(u):
        h, n, _, _ = R.forward(c.c, u, c.m)
        return (h * c.d_h_out.double()).sum() + (n * c.d_n.double()).sum()

    gen = torch.Generator().manual_seed(1)
    for name in ("h", "y") + PARAMS:
        v = torch.randn(t[name].shape, generator=gen).double().cuda()
        v /= v.norm()
        step = 1e-4
        diff = (loss({**t, name: t[name] + step * v}) - loss({**t, name: t[name] - step * v})) / (2 * step)
        got = (g["d_" + name].double() * v).sum()
        scale = g["d_" + name].double().norm()
        # the third derivative's share, step^2, and 32 bits
        assert abs(got - diff) <= 1e-5 * scale, name


def test_gradients_repeat_bit_for_bit():
    c = Case(2500, 1000, R.RMS, R.LAYER, gate=333, bias=True, p=0.1)
    h_out = c.stream()
    first = c.gradients(h_out, c.d_h_out, c.d_n)
    for _ in range(5):
        again = c.gradients(h_out, c.d_h_out, c.d_n)
        for name in first:
            assert torch.equal(first[name], again[name]), name


def test_an_empty_batch():
    cfg = M.ResidualNormConfig.make(0, 64, after=M.NORM_RMS, before=M.NORM_RMS, gate_rows=3)
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    M.residual_norm(cfg, e, e, e, e, w_after=w, w_before=w, gate=e)
    g = [torch.full((64,), 3.0, device="cuda") for _ in range(4)]
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    M.residual_norm_backward(cfg, e, e, e, e, e, e, ws, w_after=w, w_before=w, gate=e, d_w_after=g[0],
                             d_b_after=g[1], d_w_before=g[2], d_b_before=g[3],
                             d_gate=torch.empty(0, 64, device="cuda"))
    assert all((v == 0).all() for v in g)
    M.dropout(e, 0.5, torch.zeros(2, dtype=torch.int64, device="cuda"), e)


def test_graphs_streams_and_a_step_that_moves_on():
    """Two captured graphs share a workspace; the mask follows rng as it is when a graph is replayed."""
    c = Case(200, 900, R.RMS, R.RMS, gate=60, p=0.3)
    h_out, n = (torch.empty_like(c.d_h_out) for _ in range(2))
    stream = c.stream()
    side = torch.cuda.Stream()
    ws = torch.empty(M.residual_norm_workspace_size(c.cfg), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g = c.gradients(stream, c.d_h_out, c.d_n, ws)
        x, dx = c.y.clone(), torch.empty_like(c.y)
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    par = {k: v for k, v in c.w.items() if k != "b_before"}
    with torch.cuda.graph(first, stream=side):
        M.residual_norm(c.cfg, c.h, c.y, h_out, n, **c.w, rng=c.rng)
        M.residual_norm_backward(c.cfg, stream, c.y, c.d_h_out, c.d_n, g["d_h"], g["d_y"], ws, **par,
                                 rng=c.rng, d_w_after=g["d_w_after"], d_gate=g["d_gate"],
                                 d_w_before=g["d_w_before"])
        c.rng[1:].add_(1)
    g2 = {k: None if v is None else torch.empty_like(v) for k, v in g.items()}
    with torch.cuda.graph(second, stream=side):
        M.residual_norm_backward(c.cfg, stream, c.y, c.d_n, c.d_h_out, g2["d_h"], g2["d_y"], ws, **par,
                                 rng=c.rng, d_w_after=g2["d_w_after"], d_gate=g2["d_gate"],
                                 d_w_before=g2["d_w_before"])
        M.dropout(x, c.p, c.rng, dx)
    for step in range(3):
        c.rng.copy_(torch.tensor([SEED, STEP + step]))
        first.replay()
        second.replay()
        for i, (got, pair) in enumerate(((g, (c.d_h_out, c.d_n)), (g2, (c.d_n, c.d_h_out)))):
            m = R.factors(SEED, STEP + step + i, c.T, c.d, c.p).cuda()
            if i == 0:
                h64, _, dh, _ = R.forward(c.c, c.tensors(), m)
                R.assert_close("h_out", h_out, h64, dh)
            t = {**c.tensors(), "h_out": stream.double(), "d_h_out": pair[0].double(), "d_n": pair[1].double()}
            want, err = R.backward(c.c, t, m)
            for name, v in got.items():
                if v is not None:
                    R.assert_close(name, v, want[name], err[name])
            if i == 1:
                R.assert_close("dropout", dx, x.double() * m, 2 * R.U * x.double().abs() * m)


# -------------------------------------------------------------------------------------------- dropout
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,d,pad", [(1, 1, 0), (3, 4, 0), (70, 13, 3), (5, 64, 0), (129, 100, 4), (40, 2048, 0),
                                     (33, 2051, 0), (7, 9000, 8)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1 - 2.0 ** -24])
def test_dropout(dtype, T, d, pad, p):
    g = torch.Generator().manual_seed(d)
    x, r = rows(g, T, d, dtype, pad), rows(g, T, d, dtype, 2 * pad)
    rng = torch.tensor([SEED, STEP], device="cuda")
    m = R.factors(SEED, STEP, T, d, p).cuda()
    for residual in (None, r):
        y = torch.full((T, d), float("nan"), dtype=dtype, device="cuda")
        M.dropout(x, p, rng, y, residual=residual)
        if p > 0.9 and dtype is F16:         # kept values leave fp16's range
            continue
        want = x.double() * m + (0 if residual is None else r.double())
        R.assert_close("y", y, want, 2 * R.U * (x.double().abs() * m + want.abs()))
        if residual is None:
            assert torch.equal(y == 0, (m == 0) | (x == 0))
        # in place
        z = x.contiguous().clone()
        M.dropout(z, p, rng, z, residual=residual)
        assert torch.equal(z, y)
        if residual is not None:
            z = r.contiguous().clone()
            M.dropout(x, p, rng, z, residual=z)
            assert torch.equal(z, y)
    if p == 0:
        y = torch.empty(T, d, dtype=dtype, device="cuda")
        M.dropout(x, 0.0, None, y)
        assert torch.equal(y, x)


def test_dropout_depends_on_seed_and_step_in_all_their_bits():
    x = torch.ones(64, 256, device="cuda")
    seen = {}
    for seed in (0, 1, 1 << 32, -1):
        for step in (0, 1, 1 << 32, -1):
            y = torch.empty_like(x)
            M.dropout(x, 0.5, torch.tensor([seed, step], device="cuda"), y)
            assert torch.equal(y.cpu().double(), R.factors(seed, step, 64, 256, 0.5))
            seen[y.cpu().numpy().tobytes()] = 1
    assert len(seen) == 16


def test_dropout_past_2_to_the_31_elements():
    """Offsets are 64 bits wide: 16-bit rows that end past 4 GB."""
    T, d = 300000, 7200
    x = torch.ones(T, d, dtype=BF16, device="cuda")
    rng = torch.tensor([5, 6], device="cuda")
    M.dropout(x, 0.25, rng, x)
    last = x[-3:].double().cpu()
    want = R.factors(5, 6, 3, d, 0.25, row0=T - 3).to(BF16).double()
    assert torch.equal(last, want)
    assert abs((x[::1000] != 0).double().mean().item() - 0.75) < 0.002
