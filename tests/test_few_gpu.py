"""The MoE layer for a few tokens against 64 bits: sizes, routing modes, capacity, given choices, streams and
graphs."""
import pytest
import torch

import few_reference as R
import sparse_moe_layer_route_gb300 as M

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def weights_of(p, prepared=True):
    return M.make_weights(p["W_g"], p["bias"], p["W_gate"], p["W_up"], p["W_down"], p["Wsh_gate"],
                          p["Wsh_up"], p["Wsh_down"],
                          W_g_t=M.prepare_router(p["W_g"]) if prepared else None)


def routing(T, E, k):
    return {"topk_idx": torch.full((T, k), -7, dtype=I32, device="cuda"),
            "topk_w": torch.empty(T, k, device="cuda"),
            "counts": torch.full((E,), -7, dtype=I32, device="cuda"),
            "offsets": torch.full((E + 1,), -7, dtype=I32, device="cuda"),
            "perm_slot": torch.full((T * k,), -7, dtype=I32, device="cuda"),
            "slot_pos": torch.full((T * k,), -7, dtype=I32, device="cuda")}


@pytest.mark.parametrize("T,d,E,k,f,S,kw", [
    (1, 64, 1, 1, 64, 0, {}), (1, 256, 8, 2, 512, 0, {}), (2, 256, 8, 2, 512, 1, {}),
    (3, 128, 5, 5, 192, 2, dict(mode=R.BIAS)), (8, 512, 16, 2, 384, 0, dict(mode=R.GUMBEL, tau=0.5)),
    (9, 512, 16, 2, 384, 0, dict(mode=R.GUMBEL, tau=2.0)), (16, 256, 8, 8, 256, 4, {}),
    (7, 2048, 64, 6, 1408, 2, dict(mode=R.BIAS)), (16, 1024, 256, 8, 64, 0, dict(groups=8, keep=3)),
    (5, 64, 256, 8, 320, 1, dict(mode=R.BIAS, groups=64, keep=33)),
    (13, 1152, 33, 3, 64, 1, dict(mode=R.BIAS)), (16, 64, 4, 4, 2048, 1, {}),
    (4, 576, 24, 3, 704, 0, dict(cap=1)), (16, 320, 3, 2, 128, 1, dict(cap=5)),
    (11, 2112, 12, 4, 960, 3, dict(mode=R.GUMBEL, cap=2, groups=4, keep=2)),
    (1, 7168, 8, 2, 2048, 1, {}), (16, 7168, 8, 2, 512, 0, {}), (12, 4096, 4, 2, 3584, 0, {}),
    (2, 64, 9, 8, 8192, 0, {}), (10, 8192, 3, 1, 64, 0, {})])
@pytest.mark.parametrize("prepared", [True, False])
def test_layer(T, d, E, k, f, S, kw, prepared):
    mode, cap, groups, keep = (kw.get(n, 0) for n in ("mode", "cap", "groups", "keep"))
    tau = kw.get("tau", 1.0)
    p = R.make(T, d, E, k, f, S, seed=T + d + E)
    cfg = M.MoeConfig.make(T, d, E, k, f, n_shared=S, mode=mode, tau=tau, capacity_override=cap,
                           n_groups=groups, topk_groups=keep)
    ws, ro = M.alloc_few_workspace(cfg), routing(T, E, k)
    out = torch.full((T, d), float("nan"), dtype=BF16, device="cuda")
    for _ in range(2):                       # the second call finds the counters the first one left
        M.layer_forward_few(cfg, weights_of(p, prepared), p["x"], p["u"], out,
                            M.make_route_out(**ro), ws)
    assert M.device_status(ws) == 0
    idx, w, gap = R.choose(p, k, mode, tau, groups, keep)
    assert gap > 1e-6                        # of these inputs: nothing is decided by less
    assert torch.equal(ro["topk_idx"].long(), idx)
    # the logits' error (2^-24 of about 5), twice, and the exponential's: 1e-6 of a gate covers them
    assert (ro["topk_w"].double() - w).abs().max() <= 1e-6 * max(1.0, 1 / tau)
    R.assert_rounded(out, *R.layer(p, idx, ro["topk_w"], cap, S))
    # the dispatch is the stand-alone one's
    want = routing(T, E, k)
    plain = M.alloc_workspace(cfg)
    M.permute(cfg, ro["topk_idx"], want["counts"], want["offsets"], want["perm_slot"],
              want["slot_pos"], plain)
    for name in ("counts", "offsets", "perm_slot", "slot_pos"):
        assert torch.equal(ro[name], want[name]), name


def given(T, d, E, k, f, S, idx, w, cap=0, seed=3, **change):
    p = {**R.make(T, d, E, k, f, S, seed=seed), **change}
    cfg = M.MoeConfig.make(T, d, E, k, f, n_shared=S, capacity_override=cap)
    ws = M.alloc_few_workspace(cfg)
    out = torch.full((T, d), float("nan"), dtype=BF16, device="cuda")
    M.experts_few(cfg, weights_of(p), p["x"], idx, w, out, ws)
    return p, out, M.device_status(ws)


@pytest.mark.parametrize("T,d,E,k,f,S,cap", [
    (1, 128, 4, 1, 64, 0, 0), (5, 2048, 64, 6, 1408, 2, 0), (16, 192, 20, 8, 128, 0, 3),
    (8, 1024, 2, 2, 512, 4, 0), (9, 640, 2, 1, 512, 0, 4), (3, 4096, 16, 2, 1792, 0, 1)])
@pytest.mark.parametrize("gates", [True, False])
def test_experts(T, d, E, k, f, S, cap, gates):
    g = torch.Generator().manual_seed(T)
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int().cuda()
    w = torch.randn(T, k, generator=g).cuda()
    p, out, status = given(T, d, E, k, f, S, idx, w if gates else None, cap)
    assert status == 0
    R.assert_rounded(out, *R.layer(p, idx, w if gates else torch.ones_like(w), cap, S))


@pytest.mark.parametrize("cap", [0, 2, 17])
@pytest.mark.parametrize("T", [3, 16])
def test_an_expert_given_twice(T, cap):
    """Both gates count, both slots take room."""
    E, k = 6, 4
    idx = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(5), dtype=I32)
    idx[0] = 3
    idx[-1] = torch.tensor([1, 2, 1, 1])
    w = torch.randn(T, k, generator=torch.Generator().manual_seed(6))
    p, out, status = given(T, 256, E, k, 192, 1, idx.cuda(), w.cuda(), cap)
    assert status == 0
    R.assert_rounded(out, *R.layer(p, idx, w.cuda(), cap, 1))


@pytest.mark.parametrize("S", [0, 1])
def test_indices_that_are_no_expert(S):
    T, E, k = 4, 5, 2
    idx = torch.tensor([[0, 5], [-1, 4], [2 ** 30, -2 ** 31], [1, 3]], dtype=I32).cuda()
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(6)).cuda()
    p, out, status = given(T, 128, E, k, 64, S, idx, w)
    assert status == M.DEVFAULT_BAD_EXPERT_INDEX
    R.assert_rounded(out, *R.layer(p, idx, w, 0, S))
    none = torch.full((T, k), 9, dtype=I32).cuda()
    p, out, status = given(T, 128, E, k, 64, S, none, w)
    assert status == M.DEVFAULT_BAD_EXPERT_INDEX
    R.assert_rounded(out, *R.layer(p, none, w, 0, S))


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_what_is_not_finite_stays_with_its_token(bad):
    """An expert's weights reach the tokens that chose it, a token's values its own output; experts that
    nobody chose reach nobody."""
    T, d, E, k, f = 10, 256, 6, 2, 128
    p = R.make(T, d, E, k, f, 0, seed=8)
    idx = torch.tensor([[0, 1], [2, 3]] * 5, dtype=I32).cuda()
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(6)).cuda()
    for name in ("W_gate", "W_up", "W_down"):
        change = p[name].clone()
        change[2, 5:9] = bad
        change[4] = bad
        q, out, status = given(T, d, E, k, f, 0, idx, w, seed=8, **{name: change})
        even = torch.arange(0, T, 2, device="cuda")
        want, err = R.layer(p, idx, w)
        R.assert_rounded(out[even], want[even], err[even])
        assert not torch.isfinite(out[even + 1]).all(-1).any()
    x = p["x"].clone()
    x[3, 7] = bad
    q, out, status = given(T, d, E, k, f, 0, idx, w, seed=8, x=x)
    rest = [t for t in range(T) if t != 3]
    R.assert_rounded(out[rest], want[rest], err[rest])
    assert not torch.isfinite(out[3]).any()


@pytest.mark.parametrize("T", [2, 12])
def test_activations_past_fp16(T):
    """H and outputs of about 2^40: nothing is clamped."""
    p = R.make(T, 256, 4, 2, 128, 1, seed=9)
    p["W_up"] = p["W_up"] * 2.0 ** 40
    p["Wsh_up"] = p["Wsh_up"] * 2.0 ** 40
    idx, w, _ = R.choose(p, 2)
    cfg = M.MoeConfig.make(T, 256, 4, 2, 128, n_shared=1)
    ws, out = M.alloc_few_workspace(cfg), torch.empty(T, 256, dtype=BF16, device="cuda")
    ro = routing(T, 4, 2)
    M.layer_forward_few(cfg, weights_of(p), p["x"], None, out, M.make_route_out(**ro), ws)
    assert M.device_status(ws) == 0
    R.assert_rounded(out, *R.layer(p, idx, ro["topk_w"], 0, 1))


def test_nan_logits_choose_different_experts():
    """A token with a NaN has NaN logits: distinct experts, a NaN output, and the others are untouched."""
    T, d, E, k = 6, 128, 16, 4
    p = R.make(T, d, E, k, 64, 0, seed=10)
    p["x"][2, 0] = float("nan")
    cfg = M.MoeConfig.make(T, d, E, k, 64)
    ws, out, ro = M.alloc_few_workspace(cfg), torch.empty(T, d, dtype=BF16, device="cuda"), routing(T, E, k)
    M.layer_forward_few(cfg, weights_of(p), p["x"], None, out, M.make_route_out(**ro), ws)
    assert ro["topk_idx"][2].tolist() == [0, 1, 2, 3]
    rest = [t for t in range(T) if t != 2]
    q = {**p, "x": p["x"][rest]}
    idx, w, _ = R.choose(q, k)
    assert torch.equal(ro["topk_idx"][rest].long(), idx)
    R.assert_rounded(out[rest], *R.layer(q, idx, ro["topk_w"][rest]))


def test_ties_go_to_the_lower_index():
    T, d, E, k = 4, 64, 40, 8
    p = R.make(T, d, E, k, 64, 0, seed=11)
    p["W_g"] = p["W_g"][:, :8].repeat_interleave(5, 1).contiguous()       # experts in fives
    cfg = M.MoeConfig.make(T, d, E, k, 64)
    ws, out, ro = M.alloc_few_workspace(cfg), torch.empty(T, d, dtype=BF16, device="cuda"), routing(T, E, k)
    M.layer_forward_few(cfg, weights_of(p), p["x"], None, out, M.make_route_out(**ro), ws)
    l = (p["x"].double() @ p["W_g"].double()[:, ::5])
    best = l.sort(-1, descending=True).indices[:, :2]
    want = torch.cat([best[:, :1] * 5 + torch.arange(5, device="cuda"),
                      best[:, 1:] * 5 + torch.arange(3, device="cuda")], 1)
    assert torch.equal(ro["topk_idx"].long(), want)


def test_agrees_with_the_layer_of_many_tokens():
    T, d, E, k, f, S = 16, 1024, 32, 4, 768, 1
    p = R.make(T, d, E, k, f, S, seed=12)
    cfg = M.MoeConfig.make(T, d, E, k, f, n_shared=S, mode=M.ROUTE_BIAS_SELECT)
    ws, few = M.alloc_workspace(cfg), M.alloc_few_workspace(cfg)
    a, b = (torch.empty(T, d, dtype=BF16, device="cuda") for _ in range(2))
    ro, ro2 = routing(T, E, k), routing(T, E, k)
    M.layer_forward(cfg, weights_of(p), p["x"], None, a, M.make_route_out(**ro), ws)
    M.layer_forward_few(cfg, weights_of(p), p["x"], None, b, M.make_route_out(**ro2), few)
    for name in ro:
        if name != "topk_w":
            assert torch.equal(ro[name], ro2[name])
    # the bf16 path of layer_forward rounds H to 8 bits: 2^-8 of it and of the output
    assert ((a.float() - b.float()).norm() / b.float().norm()).item() < 2.0 ** -7


def test_calls_repeat_bit_for_bit_and_output_may_replace_the_input():
    T, d, E, k, f, S = 16, 1152, 16, 4, 1408, 1
    p = R.make(T, d, E, k, f, S, seed=13)
    cfg, w = M.MoeConfig.make(T, d, E, k, f, n_shared=S), weights_of(p)
    ws, out = M.alloc_few_workspace(cfg), torch.empty(T, d, dtype=BF16, device="cuda")
    M.layer_forward_few(cfg, w, p["x"], None, out, None, ws)
    for _ in range(20):
        x = p["x"].clone()
        M.layer_forward_few(cfg, w, x, None, x, None, ws)
        assert torch.equal(x.view(torch.int16), out.view(torch.int16))
    assert M.device_status(ws) == 0


def test_configurations_share_a_workspace():
    """Of calls one after the other, with any number of tokens up to the workspace's."""
    d, E, k, f = 768, 12, 3, 512
    big = M.MoeConfig.make(16, d, E, k, f)
    ws = M.alloc_few_workspace(big)
    for T in (16, 1, 9, 8, 3, 16):
        p = R.make(T, d, E, k, f, 0, seed=T)
        cfg = M.MoeConfig.make(T, d, E, k, f)
        assert M.few_workspace_size(cfg) <= ws.numel()
        out, ro = torch.empty(T, d, dtype=BF16, device="cuda"), routing(T, E, k)
        M.layer_forward_few(cfg, weights_of(p), p["x"], None, out, M.make_route_out(**ro), ws)
        R.assert_rounded(out, *R.layer(p, ro["topk_idx"], ro["topk_w"]))
        out2 = torch.empty_like(out)
        M.experts_few(cfg, weights_of(p), p["x"], ro["topk_idx"], ro["topk_w"], out2, ws)
        assert torch.equal(out, out2)
    assert M.device_status(ws) == 0


def test_a_workspace_of_both_layers():
    """The layer of many tokens and of few, in turn on one workspace, as prefill and decoding use it."""
    d, E, k, f, S = 512, 16, 3, 384, 1
    p = R.make(16, d, E, k, f, S, seed=23)
    w = weights_of(p)
    few, many = (M.MoeConfig.make(T, d, E, k, f, n_shared=S) for T in (16, 300))
    ws = M.alloc_workspace(many)
    if ws.numel() < M.few_workspace_size(few):
        ws = M.alloc_int8_workspace(M.few_workspace_size(few))
    x = torch.randn(300, d, generator=torch.Generator().manual_seed(24)).bfloat16().cuda()
    alone, want = torch.empty_like(x), torch.empty_like(p["x"])
    M.layer_forward(many, w, x, None, alone, None, M.alloc_workspace(many))
    M.layer_forward_few(few, w, p["x"], None, want, None, M.alloc_few_workspace(few))
    for _ in range(3):
        for cfg, layer, inp, expected in ((many, M.layer_forward, x, alone),
                                          (few, M.layer_forward_few, p["x"], want)):
            out = torch.full_like(expected, float("nan"))
            layer(cfg, w, inp, None, out, None, ws)
            assert torch.equal(out, expected) and M.device_status(ws) == 0


def test_graphs_and_streams():
    """Two captured graphs share a workspace, replayed in turn; calls on two streams with workspaces of
    their own run side by side."""
    T, d, E, k, f, S = 6, 512, 16, 3, 640, 1
    p = R.make(T, d, E, k, f, S, seed=14)
    cfg, w = M.MoeConfig.make(T, d, E, k, f, n_shared=S), weights_of(p)
    ws = M.alloc_few_workspace(cfg)
    x = p["x"].clone()
    outs = [torch.empty(T, d, dtype=BF16, device="cuda") for _ in range(2)]
    idx, gates, _ = R.choose(p, k)
    idx, gates = idx.int(), gates.float()
    graphs = []
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            if i == 0:
                M.layer_forward_few(cfg, w, x, None, outs[0], None, ws)
            else:
                M.experts_few(cfg, w, x, idx, gates, outs[1], ws)
        graphs.append(graph)
    for step in range(4):
        x.copy_(torch.roll(p["x"], step, 0))
        for graph in graphs:
            graph.replay()
        q = {**p, "x": x}
        i2, g2, _ = R.choose(q, k)
        R.assert_rounded(outs[0], *R.layer(q, i2, g2, 0, S))
        R.assert_rounded(outs[1], *R.layer(q, idx, gates, 0, S))
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [M.alloc_few_workspace(cfg) for _ in streams]
    x.copy_(p["x"])
    torch.cuda.synchronize()
    for _ in range(10):
        for s, ws2, out in zip(streams, spaces, outs):
            M.layer_forward_few(cfg, w, x, None, out, None, ws2, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and all(M.device_status(s) == 0 for s in spaces)
    R.assert_rounded(outs[0], *R.layer(p, idx, gates, 0, S))
    assert M.device_status(ws) == 0


def test_an_empty_batch():
    cfg = M.MoeConfig.make(0, 128, 8, 2, 64)
    assert M.few_workspace_size(cfg) == 512
    ws, ro = M.alloc_few_workspace(cfg), routing(0, 8, 2)
    x = torch.empty(0, 128, dtype=BF16, device="cuda")
    p = R.make(1, 128, 8, 2, 64, 0)
    M.layer_forward_few(cfg, weights_of(p), x, None, x, M.make_route_out(**ro), ws)
    M.experts_few(cfg, weights_of(p), x, ro["topk_idx"], ro["topk_w"], x, ws)
    assert ro["counts"].tolist() == [0] * 8 and ro["offsets"].tolist() == [0] * 9
