"""Routing from given logits and its gradient against the formulas in 64 bits.

u = 2^-24 below. Tolerances, before any run:
  weights   a sigmoid is within 6 u of its value (exp 4 u, sum u, quotient u); renormalised: two of
            those, 8 u for the sum of eight, 2 u for the quotient and the scale, 22 u in all. A softmax
            term adds the rounding of l - max, at most 16 u for the spans used here: 40 u.
  gradient  every term is at most M = 2 scale max|d_w| + max|d_scores| of its row and within 40 u of it;
            a few are added: 64 u M. A bf16 gradient is the fp32 one of the same values rounded once,
            bit for bit.
  indices   equal wherever 64 bits decide by more than 1e-6 (an fp32 rank is within 2e-7 of its value
            for ranks below 2); exact ties are tested on equal logits, where they are ties in both.
"""
import itertools

import numpy as np
import pytest
import torch

import sparse_moe_layer_route_gb300 as M

U = 2.0 ** -24
NEG = float("-inf")


def scores64(l, sigmoid):
    if sigmoid:
        return 1.0 / (1.0 + np.exp(-l))
    top = l.max(-1, keepdims=True)
    e = np.exp(l - np.where(np.isneginf(top), 0.0, top))
    return e / np.maximum(e.sum(-1, keepdims=True), 1e-300)


def pick64(l, s, bias, k, G, keep, top2, sigmoid):
    """(chosen experts, smallest gap of the decisions) of one token, as the header defines them."""
    E = l.size
    r = s + bias if bias is not None else (s if sigmoid else l)
    r = np.where(np.isneginf(l), NEG, r)
    gap, live = np.inf, np.ones(E, bool)
    if G:
        by = -np.sort(-r.reshape(G, E // G), axis=1)
        rank = by[:, 0].copy()
        if top2 and E // G > 1:
            rank += np.where(np.isneginf(by[:, 1]), 0.0, by[:, 1])
        order = np.argsort(-rank, kind="stable")
        if keep < G and np.isfinite(rank[order[keep]]):
            gap = rank[order[keep - 1]] - rank[order[keep]]
        live = np.zeros((G, E // G), bool)
        live[order[:keep]] = True
        live = live.reshape(E)
    cand = np.flatnonzero(live)
    order = cand[np.argsort(-r[cand], kind="stable")]
    with np.errstate(invalid="ignore"):
        d = r[order[:k]][:min(k, order.size - 1)] - r[order[1:k + 1]]
    d = d[~np.isnan(d)]                                   # -inf - -inf: an exact tie of masked ones
    return order[:k], min([gap] + list(d))


def weights64(l, idx, sigmoid, renorm, scale):
    s = scores64(l, sigmoid)
    if renorm and not sigmoid:
        w = scores64(np.take_along_axis(l, idx, 1), False)
    else:
        w = np.take_along_axis(s, idx, 1)
        if renorm:
            w = w / np.maximum(w.sum(-1, keepdims=True), 1e-300)
    return scale * w, s


def run(l, k, sigmoid, bias=None, G=0, keep=0, top2=False, renorm=True, scale=1.0, full=False,
        ld=0):
    T, E = l.shape
    cfg = M.GateConfig.make(T, E, k, M.SCORE_SIGMOID if sigmoid else M.SCORE_SOFTMAX, G, keep, top2,
                            renorm, scale,
                            M.DTYPE_BF16 if l.dtype == torch.bfloat16 else M.DTYPE_F32, ld)
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    s = torch.full((T, E), float("nan"), device="cuda") if full else None
    M.route_logits(cfg, l, bias, idx, w, s)
    return cfg, idx, w, s


def logits(T, E, dtype, seed, masked=0.0, span=4.0):
    g = torch.Generator().manual_seed(seed)
    l = (torch.randn(T, E, generator=g) * span / 4).clamp(-span, span)
    l[torch.rand(T, E, generator=g) < masked] = NEG
    if T > 3:
        l[2] = NEG                                        # a token with every expert switched off
    return l.to(dtype).cuda()


SHAPES = [(1, 1, 1, 0, 0), (1, 256, 8, 8, 4), (5, 7, 7, 0, 0), (33, 32, 2, 0, 0),
          (9, 33, 8, 3, 2), (64, 60, 4, 30, 11), (17, 128, 2, 64, 3), (7, 96, 5, 2, 1),
          (100, 255, 8, 5, 2), (3, 256, 1, 0, 0), (40, 16, 8, 4, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,G,keep", SHAPES)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_choice_and_weights(T, E, k, G, keep, sigmoid, dtype):
    for n, (with_bias, renorm, top2, masked) in enumerate(itertools.product(
            (False, True), (False, True), (False, True), (0.0, 0.2))):
        if top2 and not G:
            continue
        l = logits(T, E, dtype, 100 * n + T + E, masked)
        g = torch.Generator().manual_seed(n)
        bias = (0.1 * torch.randn(E, generator=g)).cuda() if with_bias else None
        _, idx, w, s = run(l, k, sigmoid, bias, G, keep, top2, renorm, 2.5, full=True)
        l64, i = l.double().cpu().numpy(), idx.cpu().numpy().astype(np.int64)
        assert i.min() >= 0 and i.max() < E
        assert all(len(set(row)) == k for row in i.tolist())
        w64, s64 = weights64(l64, i, sigmoid, renorm, 2.5)
        b64 = bias.double().cpu().numpy() if with_bias else None
        decided = 0
        for t in range(T):
            want, gap = pick64(l64[t], s64[t], b64, k, G, keep, top2, sigmoid)
            if gap > 1e-6 or (np.isneginf(l64[t])).all():
                decided += 1
                assert want.tolist() == i[t].tolist(), (t, gap)
        # fp32 logits are rarely that near; bf16 ones tie often without a bias, and a tie with
        # none is decided by the index in both (below)
        if dtype == torch.float32:
            assert decided >= 0.9 * T
        np.testing.assert_allclose(w.cpu().numpy(), w64, rtol=40 * U, atol=1e-37)
        np.testing.assert_allclose(s.cpu().numpy(), s64, rtol=40 * U, atol=1e-37)


@pytest.mark.gpu
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("G,keep", [(0, 0), (4, 2)])
def test_ties_go_to_the_lowest_index(sigmoid, G, keep):
    # logits on a coarse grid: many equal, and unequal ones differ by 1/4
    g = torch.Generator().manual_seed(3)
    l = torch.randint(-6, 7, (257, 64), generator=g).float() / 4
    l[l == 0.25] = -0.0                                   # -0 and +0 are equal
    _, idx, _, _ = run(l.cuda(), 8, sigmoid, None, G, keep)
    l64 = l.double().numpy()
    s64 = scores64(l64, sigmoid)
    for t in range(l.shape[0]):
        want, _ = pick64(l64[t] + 0.0, s64[t], None, 8, G, keep, False, sigmoid)
        assert want.tolist() == idx[t].tolist()


@pytest.mark.gpu
@pytest.mark.parametrize("sigmoid", [False, True])
def test_nan_and_infinity(sigmoid):
    l = logits(6, 40, torch.float32, 5)
    l[0, 3] = float("nan")
    l[1, 4] = float("inf")
    l[2] = NEG
    l[3] = float("nan")
    l[4] = NEG
    l[4, 17] = 1.5                                        # one live expert
    _, idx, w, _ = run(l, 4, sigmoid)
    i = idx.cpu().numpy()
    assert all(len(set(r)) == 4 and min(r) >= 0 and max(r) < 40 for r in i.tolist())
    assert 3 not in i[0] and torch.isnan(w[0]).all() and torch.isnan(w[3]).all()
    assert i[1, 0] == 4
    assert torch.isfinite(w[1]).all() if sigmoid else torch.isnan(w[1]).all()
    assert i[2].tolist() == [0, 1, 2, 3] and (w[2] == 0).all()
    assert i[4].tolist() == [17, 0, 1, 2] and w[4].tolist() == [1.0, 0.0, 0.0, 0.0]
    # a switched-off expert stays last under a large bias
    bias = torch.zeros(40, device="cuda")
    bias[7] = 100.0
    l = torch.zeros(1, 40, device="cuda")
    l[0, 7] = NEG
    assert 7 not in run(l, 8, sigmoid, bias)[1][0].tolist()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_rows_alignment_and_streams(dtype):
    big = torch.randn(50, 131, device="cuda").to(dtype)
    view = big[:, 3:67]                                   # odd offset, row stride 131
    own = view.contiguous()
    for sigmoid in (False, True):
        _, i0, w0, s0 = run(own, 6, sigmoid, full=True)
        _, i1, w1, s1 = run(view, 6, sigmoid, full=True, ld=131)
        assert torch.equal(i0, i1) and torch.equal(w0, w1) and torch.equal(s0, s1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _, i2, w2, _ = run(own, 6, True)
    side.synchronize()
    _, i0, w0, _ = run(own, 6, True)
    assert torch.equal(i0, i2) and torch.equal(w0, w2)


def grad64(l, idx, dw, ds, sigmoid, renorm, scale):
    """The gradient by automatic differentiation in 64 bits of the forward formulas."""
    x = torch.tensor(l, requires_grad=True)
    i = torch.tensor(idx)
    s = torch.sigmoid(x) if sigmoid else torch.softmax(x, -1)
    if renorm and not sigmoid:
        w = torch.softmax(x.gather(1, i), -1)
    else:
        w = s.gather(1, i)
        if renorm:
            w = w / w.sum(-1, keepdim=True)
    loss = torch.zeros((), dtype=torch.float64)
    if dw is not None:
        loss = loss + (scale * w * torch.tensor(dw)).sum()
    if ds is not None:
        loss = loss + (s * torch.tensor(ds)).sum()
    return torch.nan_to_num(torch.autograd.grad(loss, x)[0], nan=0.0).numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,G,keep", SHAPES)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient(T, E, k, G, keep, sigmoid, dtype):
    for n, (renorm, with_w, with_s, masked) in enumerate(itertools.product(
            (False, True), (False, True), (False, True), (0.0, 0.2))):
        if not (with_w or with_s):
            continue
        l = logits(T, E, dtype, 7 * n + T, masked)
        cfg, idx, _, _ = run(l, k, sigmoid, None, G, keep, False, renorm, 2.5)
        g = torch.Generator().manual_seed(n)
        dw = torch.randn(T, k, generator=g) if with_w else None
        ds = torch.randn(T, E, generator=g) if with_s else None
        out = torch.full((T, E), float("nan"), dtype=dtype, device="cuda")
        M.route_logits_backward(cfg, l, idx, dw.cuda() if with_w else None,
                                ds.cuda() if with_s else None, out)
        want = grad64(l.double().cpu().numpy(), idx.cpu().numpy().astype(np.int64),
                      dw.double().numpy() if with_w else None,
                      ds.double().numpy() if with_s else None, sigmoid, renorm, 2.5)
        top = np.zeros((T, 1))
        if with_w:
            top += 2 * 2.5 * dw.abs().double().numpy().max(1, keepdims=True)
        if with_s:
            top += ds.abs().double().numpy().max(1, keepdims=True)
        if dtype == torch.bfloat16:
            cfg.dtype = M.DTYPE_F32
            full = torch.full((T, E), float("nan"), device="cuda")
            M.route_logits_backward(cfg, l.float(), idx, dw.cuda() if with_w else None,
                                    ds.cuda() if with_s else None, full)
            assert torch.equal(out, full.bfloat16())
            out = full
        got = out.double().cpu().numpy()
        assert (np.abs(got - want) <= 64 * U * top).all(), np.abs(got - want).max()


@pytest.mark.gpu
@pytest.mark.parametrize("sigmoid,renorm", list(itertools.product((False, True), repeat=2)))
def test_gradient_against_differences(sigmoid, renorm):
    """Central differences of the 64-bit forward, step 1e-4: their own error is below 1e-7 (third
    derivatives of order one, sums of a few terms)."""
    T, E, k, scale, h = 3, 20, 4, 1.5, 1e-4
    l = logits(T, E, torch.float32, 11)
    cfg, idx, _, _ = run(l, k, sigmoid, renorm=renorm, scale=scale)
    g = torch.Generator().manual_seed(1)
    dw, ds = torch.randn(T, k, generator=g), torch.randn(T, E, generator=g)
    out = torch.empty(T, E, device="cuda")
    M.route_logits_backward(cfg, l, idx, dw.cuda(), ds.cuda(), out)
    l64, i = l.double().cpu().numpy(), idx.cpu().numpy().astype(np.int64)

    def loss(x):
        w, s = weights64(x, i, sigmoid, renorm, scale)
        return (w * dw.double().numpy()).sum(1) + (s * ds.double().numpy()).sum(1)

    for e in range(E):
        d = np.zeros(E)
        d[e] = h
        diff = (loss(l64 + d) - loss(l64 - d)) / (2 * h)
        np.testing.assert_allclose(out[:, e].cpu().numpy(), diff, rtol=0, atol=64 * U * 12 + 1e-7)


@pytest.mark.gpu
def test_gradient_ignores_indices_out_of_range():
    l = logits(2, 12, torch.float32, 2)
    cfg, idx, _, _ = run(l, 3, True, renorm=False)
    bad = idx.clone()
    bad[0, 1], bad[1, 2] = -1, 12
    dw = torch.ones(2, 3, device="cuda")
    a, b = torch.empty(2, 12, device="cuda"), torch.empty(2, 12, device="cuda")
    M.route_logits_backward(cfg, l, bad, dw, None, a)
    kept = torch.ones(2, 3, device="cuda")
    kept[0, 1] = kept[1, 2] = 0
    M.route_logits_backward(cfg, l, idx, kept, None, b)
    assert torch.equal(a, b)


@pytest.mark.gpu
def test_wrong_tensors_are_refused():
    cfg = M.GateConfig.make(4, 16, 2)
    l = torch.zeros(4, 16, device="cuda")
    idx = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    for bad in ((l.half(), idx, w), (l[:, :8], idx, w), (l.t().contiguous().t(), idx, w),
                (l, idx.long(), w), (l, idx, w.half()), (l, idx[:, :1], w), (l.cpu(), idx, w)):
        with pytest.raises(ValueError):
            M.route_logits(cfg, bad[0], None, bad[1], bad[2])
    with pytest.raises(ValueError):
        M.route_logits_backward(cfg, l, idx, w, None, l.bfloat16())
    with pytest.raises(M.MoeError):
        M.route_logits_backward(cfg, l, idx, None, None, torch.empty_like(l))


@pytest.mark.gpu
def test_repeated_calls_give_the_same_bits():
    l = logits(1000, 256, torch.float32, 9)
    bias = 0.05 * torch.randn(256, device="cuda")
    first = run(l, 8, False, bias, 8, 4, True, full=True)[1:]
    for _ in range(3):
        again = run(l, 8, False, bias, 8, 4, True, full=True)[1:]
        assert all(torch.equal(a, b) for a, b in zip(first, again))
