"""Workloads of the few-token layer, the norms around a block, and dropout.

Each case is one pass through one operator, either in its plain form (elementary torch operations in
32 bits, `own = False`) or through this package's entry points (`own = True`):

  layer        a whole MoE layer (router, choice, SwiGLU experts, shared experts, combine) for up to
               16 tokens
  experts      its experts and combine, for a choice and weights that the program made itself
  norm         a block's output normed, dropped out, gated and scaled onto the residual stream, and the
               stream normed for the next block
  norm_grad    the gradients of that to the stream, the block's output and every parameter
  dropout      counter-based dropout of rows, alone or onto a residual
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
MASK32 = 0xFFFFFFFF


# ------------------------------------------------------------------------------------------ cases
def _few(op, T, d, E, k, f, S, mode="plain", cap=0, groups=0, keep=0):
    """cap: slots that an expert takes, in token order (0: all)."""
    return {"op": op, "T": T, "d": d, "E": E, "k": k, "f": f, "S": S, "mode": mode, "cap": cap,
            "groups": groups, "keep": keep}


def _norm(op, T, d, after, before, h="bf16", y="bf16", w="bf16", gate=0, bias=False, alpha=1.0,
          beta=1.0, p=0.0, pad=0):
    """gate: consecutive tokens that share a row of gates (0: no gates); pad: elements between rows."""
    return {"op": op, "T": T, "d": d, "after": after, "before": before, "h": h, "y": y, "w": w,
            "gate": gate, "bias": bias, "alpha": alpha, "beta": beta, "p": p, "pad": pad}


def _dropout(T, d, dtype, p, residual, pad=0):
    return {"op": "dropout", "T": T, "d": d, "dtype": dtype, "p": p, "residual": residual,
            "pad": pad}


def listed():
    return [
        # one sequence being decoded on the decode shape: bound by three experts' weights
        dict(_few("layer", 1, 7168, 128, 2, 2048, 1), name="layer_one_token"),
        # sixteen sequences on it, balance bias: most tokens have experts of their own
        dict(_few("layer", 16, 7168, 128, 2, 2048, 1, mode="bias"), name="layer_sixteen"),
        # a small layer: nothing but latency
        dict(_few("layer", 2, 256, 8, 2, 512, 0), name="layer_tiny"),
        # five tokens of a speculative decoder on the fine-grained layer, with a router of its own
        dict(_few("experts", 5, 2048, 64, 6, 1408, 2), name="experts_fine_grained"),
        # three tokens on few wide experts that have room for one token each
        dict(_few("experts", 3, 4096, 16, 2, 14336, 0, cap=1), name="experts_wide_capacity"),
        # one decode step of a block with norms on both sides
        dict(_norm("norm", 16, 7168, "rms", "rms"), name="norm_decode"),
        # the large prefill: gates per channel, a scaled residual
        dict(_norm("norm", 16384, 7168, "rms", "rms", gate=16384, alpha=0.75), name="norm_prefill"),
        # sequences of 333 tokens with a row of gates each, the last one cut off, odd width, layer norms
        # with biases, 32-bit stream, dropout
        dict(_norm("norm", 3001, 1027, "layer", "layer", h="f32", y="bf16", w="f32", gate=333,
                   bias=True, beta=0.5, p=0.1), name="norm_sequences"),
        # a training step's batch: 32-bit stream, gates per channel, dropout
        dict(_norm("norm_grad", 8192, 4096, "rms", "rms", h="f32", gate=8192, p=0.1),
             name="norm_grad_large"),
        # the fine-grained width without a norm after the block, gates per sequence
        dict(_norm("norm_grad", 2051, 2048, "none", "layer", gate=300, bias=True, alpha=0.9),
             name="norm_grad_sequences"),
        # dropout of a large batch onto its residual
        dict(_dropout(16384, 7168, "bf16", 0.1, True), name="dropout_large"),
        # odd rows inside a wider buffer
        dict(_dropout(1000, 1027, "f32", 0.25, False, pad=5), name="dropout_odd"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer", "layer", "experts", "experts", "norm", "norm", "norm_grad",
                     "norm_grad", "dropout"])
    if op in ("layer", "experts"):
        groups = rng.choice([0, 0, 2, 4, 8]) if op == "layer" else 0
        # at most the weights that the largest listed case holds, and that it reads
        held, read = 128 * 7168 * 2048, 32 * 7168 * 2048
        k, S, d = rng.randint(1, 8), rng.choice([0, 1, 2, 4]), _log(rng, 2, 112) * 64
        f = _log(rng, 2, max(2, min(224, read // (d * (k + S) * 64)))) * 64
        E = max(8, min(_log(rng, 8, 256), held // (d * f)))
        E = E // groups * groups if groups else E
        keep = rng.randint((groups + 1) // 2, groups) if groups else 0
        k = min(k, keep * (E // groups)) if groups else k
        T = _log(rng, 1, max(1, min(16, (read // (d * f) - S) // k)))
        return _few(op, T, d, E, k, f, S, mode=rng.choice(["plain", "bias", "gumbel"]),
                    cap=rng.choice([0, 0, 1, 2, 5]), groups=groups, keep=keep)
    if op == "dropout":
        d = _log(rng, 1, 16384)
        T = _log(rng, 1, 16384 * 7168 // max(d, 7168))
        return _dropout(T, d, rng.choice(["bf16", "f16", "f32"]), rng.choice([0.0, 0.1, 0.25, 0.9]),
                        rng.random() < 0.5, pad=rng.choice([0, 0, 5, 64]))
    d = _log(rng, 16, 16384)
    d = d if rng.random() < 0.3 else max(16, d // 64 * 64)
    T = _log(rng, 1, (8192 * 4096 if op == "norm_grad" else 8192 * 7168) // max(d, 2048))
    after, before = rng.choice([("rms", "rms"), ("none", "rms"), ("layer", "layer"), ("rms", "none"),
                                ("none", "layer")])
    return _norm(op, T, d, after, before, h=rng.choice(["bf16", "f32", "f16"]),
                 y=rng.choice(["bf16", "bf16", "f16", "f32"]), w=rng.choice(["bf16", "f32"]),
                 gate=rng.choice([0, 1, T, max(1, T // 3), min(T, 7)]), bias=rng.random() < 0.4,
                 alpha=rng.choice([1.0, 0.9]), beta=rng.choice([1.0, 0.5]),
                 p=rng.choice([0.0, 0.0, 0.1]), pad=rng.choice([0, 0, 3, 64]))


# ----------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows(g, T, d, dtype, pad, scale=1.0):
    """Normal values [T, d], rows `pad` elements apart."""
    return (_randn(g, T, d + pad) * scale).to(DT[dtype])[:, :d]


def _stack(g, n, rows, cols):
    w = torch.empty(n, rows, cols, dtype=torch.bfloat16, device="cuda")
    for e in range(n):
        w[e] = _randn(g, rows, cols) * rows ** -0.5
    return w


def _prepare_few(case, g, st):
    T, d, E, k, f, S = (case[v] for v in ("T", "d", "E", "k", "f", "S"))
    st["x"] = _randn(g, T, d).bfloat16()
    for name, n, rows, cols in (("gate", E, d, f), ("up", E, d, f), ("down", E, f, d),
                                ("sh_gate", S, d, f), ("sh_up", S, d, f), ("sh_down", S, f, d)):
        st[name] = _stack(g, n, rows, cols) if n else None
    st["W_g"] = (_randn(g, d, E) * d ** -0.5).bfloat16()
    st["bias"] = 0.3 * _randn(g, E)
    st["u"] = torch.rand(T, E, generator=g, device="cuda").clamp_(2.0 ** -24, 1 - 2.0 ** -24)
    if case["op"] == "experts":
        like = _randn(g, T, E) + 0.5 * _randn(g, E)      # some experts are more liked than others
        st["idx"] = torch.topk(like, k, dim=-1).indices.to(torch.int32)
        st["topk_w"] = torch.softmax(_randn(g, T, k), -1)
    if own:
        import sparse_moe_layer_route_gb300 as M
        mode = {"plain": M.ROUTE_PLAIN, "bias": M.ROUTE_BIAS_SELECT, "gumbel": M.ROUTE_GUMBEL}
        st["cfg"] = M.MoeConfig.make(T, d, E, k, f, n_shared=S, mode=mode[case["mode"]], tau=0.5,
                                     capacity_override=case["cap"], n_groups=case["groups"],
                                     topk_groups=case["keep"])
        st["W_g_t"] = M.prepare_router(st["W_g"])
        st["weights"] = M.make_weights(st["W_g"], st["bias"], st["gate"], st["up"], st["down"],
                                       st["sh_gate"], st["sh_up"], st["sh_down"],
                                       W_g_t=st["W_g_t"])
        st["ws"] = M.alloc_few_workspace(st["cfg"])
        st["out"] = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
        if case["op"] == "layer":
            st["idx"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
            st["topk_w"] = torch.empty(T, k, device="cuda")
            st["route_out"] = M.make_route_out(st["idx"], st["topk_w"])


def _gates(case):
    """Rows of gates."""
    return -(-case["T"] // case["gate"]) if case["gate"] else 0


def _prepare_norm(case, g, st):
    T, d, w = case["T"], case["d"], DT[case["w"]]

    def params(*shape, mean=1.0):
        return (mean + 0.2 * _randn(g, *shape)).to(w)

    # the stream grows over the blocks, a few channels of it far more than the others
    wide = torch.exp(0.7 * _randn(g, 1, d))
    grad = case["op"] == "norm_grad"
    st["y"] = _rows(g, T, d, case["y"], case["pad"], 0.8)
    st["h"] = (_randn(g, T, d + case["pad"]) * torch.cat(
        [wide, torch.ones(1, case["pad"], device="cuda")], 1)).to(DT[case["h"]])[:, :d]
    normed = case["after"] != "none"
    st["w_after"] = params(d) if normed else None
    st["b_after"] = params(d, mean=0.0) if normed and case["bias"] else None
    st["gate"] = params(_gates(case), d, mean=0.6) if case["gate"] else None
    normed = case["before"] != "none"
    st["w_before"] = params(d) if normed else None
    st["b_before"] = params(d, mean=0.0) if normed and case["bias"] else None
    st["rng"] = torch.randint(-2 ** 62, 2 ** 62, (2,), generator=g, device="cuda")
    if grad:
        st["d_h_out"] = _rows(g, T, d, case["h"], 0)
        st["d_n"] = _rows(g, T, d, case["y"], 0) if normed else None
    if not own:
        return
    import sparse_moe_layer_route_gb300 as M
    kind = {"none": M.NORM_NONE, "rms": M.NORM_RMS, "layer": M.NORM_LAYER}
    code = {"f32": M.DTYPE_F32, "bf16": M.DTYPE_BF16, "f16": M.DTYPE_F16}
    st["cfg"] = M.ResidualNormConfig.make(
        T, d, after=kind[case["after"]], before=kind[case["before"]], h_dtype=code[case["h"]],
        y_dtype=code[case["y"]], w_dtype=code[case["w"]], gate_rows=case["gate"], eps=1e-5,
        alpha=case["alpha"], beta=case["beta"], p_drop=case["p"], ld_h=d + case["pad"],
        ld_y=d + case["pad"])

    def out(dtype, *shape):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if not grad:
        st["h_out"] = out(DT[case["h"]], T, d)
        st["n"] = out(DT[case["y"]], T, d) if normed else None
        return
    st["ws"] = out(torch.uint8, M.residual_norm_workspace_size(st["cfg"]))
    st["d_h"], st["d_y"] = out(DT[case["h"]], T, d), out(DT[case["y"]], T, d)
    f32 = torch.float32
    for name in ("w_after", "b_after", "w_before", "b_before"):
        st["d_" + name] = out(f32, d) if st[name] is not None else None
    st["d_gate"] = out(f32, _gates(case), d) if case["gate"] else None


def prepare(case, seed):
    g, st = _gen(seed), {"case": case}
    if case["op"] in ("layer", "experts"):
        _prepare_few(case, g, st)
    elif case["op"] == "dropout":
        T, d = case["T"], case["d"]
        st["x"] = _rows(g, T, d, case["dtype"], case["pad"])
        st["residual"] = _rows(g, T, d, case["dtype"], 0) if case["residual"] else None
        st["rng"] = torch.randint(-2 ** 62, 2 ** 62, (2,), generator=g, device="cuda")
        st["y"] = torch.empty(T, d, dtype=DT[case["dtype"]], device="cuda")
    else:
        _prepare_norm(case, g, st)
    return st


# ------------------------------------------------------------------------------------ plain forms
def _choice_plain(case, st):
    """Experts [T, k] (best first, ties to the lower index) and gates from the router's logits, which are
    summed in 64 bits so that no order of a sum decides a choice."""
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    l = (st["x"].double()[:, None, :] * st["W_g"].double().t()).sum(-1)
    s = l
    if case["mode"] == "bias":
        s = l + st["bias"]
    elif case["mode"] == "gumbel":
        s = (l - torch.log(-torch.log(st["u"].double()))) / 0.5
    r = s
    if G:
        best = s.view(T, G, E // G).amax(-1)
        best = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :case["keep"]]
        live = torch.zeros(T, G, dtype=torch.bool, device="cuda").scatter_(1, best, True)
        r = torch.where(live[:, :, None].expand(T, G, E // G).reshape(T, E), s, -math.inf)
    idx = torch.sort(r, dim=-1, descending=True, stable=True).indices[:, :k]
    sel = (s if case["mode"] == "gumbel" else l).gather(1, idx)
    w = torch.exp(sel - sel.amax(-1, keepdim=True))
    return idx, (w / w.sum(-1, keepdim=True)).float()


def _expert_plain(x, gate, up, down):
    """x [n, 1, d] through its own expert of each row, in 32 bits."""
    a = torch.bmm(x, gate.float())
    b = torch.bmm(x, up.float())
    return torch.bmm(a / (1.0 + torch.exp(-a)) * b, down.float())[:, 0]


def _few_plain(case, st):
    T, d, k, S = case["T"], case["d"], case["k"], case["S"]
    if case["op"] == "layer":
        idx, w = _choice_plain(case, st)
    else:
        idx, w = st["idx"].long(), st["topk_w"]
    kept = w
    if case["cap"]:
        flat = idx.reshape(-1)
        earlier = (flat[:, None] == flat[None, :]).tril(-1).sum(-1)   # slots of the expert before this one
        kept = torch.where((earlier < case["cap"]).view(T, k), w, 0.0)
    x = st["x"].float()
    out = torch.zeros(T, d, device="cuda")
    for t in range(T):
        e = idx[t]
        y = _expert_plain(x[t].expand(k, 1, d), st["gate"][e], st["up"][e], st["down"][e])
        out[t] = (y * kept[t][:, None]).sum(0)
    if S:
        a = torch.matmul(x, st["sh_gate"].float())
        b = torch.matmul(x, st["sh_up"].float())
        out += torch.matmul(a / (1.0 + torch.exp(-a)) * b, st["sh_down"].float()).sum(0)
    out = out.bfloat16()
    return [out, idx.to(torch.int32), w] if case["op"] == "layer" else out


def _philox(rng, T, d):
    """32 random bits for each element of [T, d]: Philox 4x32 with 10 rounds (Salmon et al., "Parallel
    random numbers: as easy as 1, 2, 3", 2011), key the seed rng[0], counter (column / 4, row, step
    rng[1]), whose four words belong to the four columns."""
    cols = -(-d // 4)
    key = [rng[0] & MASK32, (rng[0] >> 32) & MASK32]
    zero = torch.zeros(T, cols, dtype=torch.int64, device="cuda")
    c = [zero + torch.arange(cols, device="cuda"), zero + torch.arange(T, device="cuda")[:, None],
         zero + (rng[1] & MASK32), zero + ((rng[1] >> 32) & MASK32)]

    def mul(m, v):
        """High and low words of the 64-bit product, by halves of v."""
        lo, hi = m * (v & 0xFFFF), m * (v >> 16)
        mid = hi + (lo >> 16)
        return mid >> 16, ((mid & 0xFFFF) << 16) | (lo & 0xFFFF)

    for _ in range(10):
        h0, l0 = mul(0xD2511F53, c[0])
        h1, l1 = mul(0xCD9E8D57, c[2])
        c = [h1 ^ c[1] ^ key[0], l1, h0 ^ c[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) & MASK32, (key[1] + 0xBB67AE85) & MASK32]
    return torch.stack(c, -1).view(T, cols * 4)[:, :d]


def _kept(rng, T, d, p):
    """Factor of each element: 0, or 1 / (1 - p) where its number is at least p * 2^32, p in 32 bits."""
    p = torch.tensor(p, dtype=torch.float32).double().item()
    return torch.where(_philox(rng, T, d) >= round(p * 2 ** 32), 1.0 / (1.0 - p), 0.0)


def _normed(kind, x, eps=1e-5):
    """x without its mean (layer) and over its deviation, and one over that."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * r, r


def _float(t):
    return None if t is None else t.float()


def _spread(case, gate):
    """The gates of every token [T, d], or 1."""
    if gate is None:
        return 1.0
    return gate[torch.arange(case["T"], device="cuda") // case["gate"]]


def _norm_plain(case, st):
    u = st["y"].float()
    if case["after"] != "none":
        u = _normed(case["after"], u)[0] * st["w_after"].float()
        if st["b_after"] is not None:
            u = u + st["b_after"].float()
    if case["p"]:
        u = u * _kept(st["rng"], case["T"], case["d"], case["p"]).float()
    h = case["alpha"] * st["h"].float() + case["beta"] * _spread(case, _float(st["gate"])) * u
    n = None
    if case["before"] != "none":
        n = _normed(case["before"], h)[0] * st["w_before"].float()
        if st["b_before"] is not None:
            n = n + st["b_before"].float()
        n = n.to(st["y"].dtype)
    return [h.to(st["h"].dtype), n]


def _norm_back(kind, dx, xn, r):
    """Gradient through _normed."""
    dx = dx - xn * (dx * xn).mean(-1, keepdim=True) - (dx.mean(-1, keepdim=True) if kind == "layer"
                                                       else 0.0)
    return dx * r


def _norm_grad_plain(case, st):
    T, d = case["T"], case["d"]
    out = {}
    dh = st["d_h_out"].float()
    if case["before"] != "none":
        xn, r = _normed(case["before"], st["h"].float())
        dn = st["d_n"].float()
        out["d_w_before"] = (dn * xn).sum(0)
        if st["b_before"] is not None:
            out["d_b_before"] = dn.sum(0)
        dh = dh + _norm_back(case["before"], dn * st["w_before"].float(), xn, r)
    out["d_h"] = (case["alpha"] * dh).to(st["h"].dtype)
    u, xn, r = st["y"].float(), None, None
    if case["after"] != "none":
        xn, r = _normed(case["after"], u)
        u = xn * st["w_after"].float()
        if st["b_after"] is not None:
            u = u + st["b_after"].float()
    dv = case["beta"] * dh
    if case["p"]:
        dv = dv * _kept(st["rng"], T, d, case["p"]).float()
    if case["gate"]:
        rows = torch.zeros(_gates(case) * case["gate"], d, device="cuda")
        rows[:T] = dv * u
        out["d_gate"] = rows.view(_gates(case), case["gate"], d).sum(1)
    du = dv * _spread(case, _float(st["gate"]))
    if case["after"] != "none":
        out["d_w_after"] = (du * xn).sum(0)
        if st["b_after"] is not None:
            out["d_b_after"] = du.sum(0)
        du = _norm_back(case["after"], du * st["w_after"].float(), xn, r)
    out["d_y"] = du.to(st["y"].dtype)
    return _gradients(out)


def _gradients(out):
    return [out.get(name) for name in ("d_h", "d_y", "d_w_after", "d_b_after", "d_gate", "d_w_before",
                                       "d_b_before")]


def _dropout_plain(case, st):
    y = st["x"].float() * _kept(st["rng"], case["T"], case["d"], case["p"]).float()
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(st["x"].dtype)


def run(state):
    st, case = state, state["case"]
    op = case["op"]
    if not own:
        if op in ("layer", "experts"):
            return _few_plain(case, st)
        return {"norm": _norm_plain, "norm_grad": _norm_grad_plain,
                "dropout": _dropout_plain}[op](case, st)
    import sparse_moe_layer_route_gb300 as M
    if op == "layer":
        M.layer_forward_few(st["cfg"], st["weights"], st["x"],
                            st["u"] if case["mode"] == "gumbel" else None, st["out"],
                            st["route_out"], st["ws"])
        return [st["out"], st["idx"], st["topk_w"]]
    if op == "experts":
        M.experts_few(st["cfg"], st["weights"], st["x"], st["idx"], st["topk_w"], st["out"], st["ws"])
        return st["out"]
    rng = st["rng"]
    if op == "dropout":
        M.dropout(st["x"], case["p"], rng, st["y"], residual=st["residual"])
        return st["y"]
    rng = rng if case["p"] else None
    if op == "norm":
        M.residual_norm(st["cfg"], st["h"], st["y"], st["h_out"], st["n"], w_after=st["w_after"],
                        b_after=st["b_after"], gate=st["gate"], w_before=st["w_before"],
                        b_before=st["b_before"], rng=rng)
        return [st["h_out"], st["n"]]
    M.residual_norm_backward(
        st["cfg"], st["h"], st["y"], st["d_h_out"], st["d_n"], st["d_h"], st["d_y"], st["ws"],
        w_after=st["w_after"], b_after=st["b_after"], gate=st["gate"], w_before=st["w_before"], rng=rng,
        d_w_after=st["d_w_after"], d_b_after=st["d_b_after"], d_gate=st["d_gate"],
        d_w_before=st["d_w_before"], d_b_before=st["d_b_before"])
    return _gradients(st)


# ---------------------------------------------------------------------------------- work of a pass
def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    op, T, d = case["op"], case["T"], case["d"]
    if op in ("layer", "experts"):
        E, k, f, S = (case[v] for v in ("E", "k", "f", "S"))
        hit = E * (1 - (1 - k / E) ** T)                 # experts that get a token, about
        rows = min(T * k, hit * case["cap"]) if case["cap"] else T * k
        router = d * E if op == "layer" else 0
        return {"bytes": int((hit + S) * 6 * d * f) + 2 * router + 4 * T * d,
                "flops": int(6 * (rows + S * T) * d * f) + 2 * T * router}
    if op == "dropout":
        return {"bytes": T * d * size[case["dtype"]] * (3 if case["residual"] else 2),
                "flops": 3 * T * d}
    h, y = size[case["h"]], size[case["y"]]
    normed, gates = case["before"] != "none", _gates(case) * d
    if op == "norm":
        return {"bytes": T * d * (2 * h + y + (y if normed else 0)) + gates * size[case["w"]],
                "flops": 12 * T * d}
    # read: the stream's gradient, its values and the next input's gradient where a norm follows, the
    # output where a norm or gates came after it; written: two gradients
    out = y if case["after"] != "none" or gates else 0
    return {"bytes": T * d * (2 * h + y + out + (h + y if normed else 0))
            + gates * (size[case["w"]] + 4), "flops": 30 * T * d}


# -------------------------------------------------------------------------- definitions in 64 bits
def _exact_few(case, st):
    T, E, k = case["T"], case["E"], case["k"]
    x = st["x"].double()
    w = idx = None
    if case["op"] == "layer":
        logits = x @ st["W_g"].double()
        # the choice itself is whole numbers; the gates are those of the plain form's choice
        idx = _choice_plain(case, st)[0]
        if case["mode"] == "gumbel":
            logits = (logits - torch.log(-torch.log(st["u"].double()))) * 2.0
        w = torch.softmax(logits.gather(1, idx), -1)
    else:
        idx, w = st["idx"].long(), st["topk_w"].double()
    out = torch.zeros(T, case["d"], dtype=torch.float64, device="cuda")

    def expert(rows, gate, up, down):
        return (torch.nn.functional.silu(rows @ gate.double()) * (rows @ up.double())) @ down.double()

    owners = idx.reshape(-1).tolist()
    for e in sorted(set(owners)):
        slots = [s for s, o in enumerate(owners) if o == e]
        slots = slots[:case["cap"]] if case["cap"] else slots
        tok = torch.tensor([s // k for s in slots], device="cuda")
        g = w.reshape(-1)[torch.tensor(slots, device="cuda")]
        out.index_add_(0, tok, expert(x[tok], st["gate"][e], st["up"][e], st["down"][e]) * g[:, None])
    for s in range(case["S"]):
        out += expert(x, st["sh_gate"][s], st["sh_up"][s], st["sh_down"][s])
    return [out, None, w] if case["op"] == "layer" else out


def _double(t, leaf=True):
    return None if t is None else t.double().requires_grad_(leaf)


def _exact_normed(kind, x, w, b):
    if kind == "none":
        return x
    if kind == "layer":
        return torch.nn.functional.layer_norm(x, x.shape[-1:], w, b, 1e-5)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5) * w
    return x if b is None else x + b


def _exact_join(case, st, y, w, b, gate):
    """What a block with output y adds to the stream."""
    u = _exact_normed(case["after"], y, w, b)
    if case["p"]:
        u = u * _kept(st["rng"], case["T"], case["d"], case["p"])
    if gate is not None:
        u = u * gate.repeat_interleave(case["gate"], 0)[:case["T"]]
    return case["beta"] * u


def _exact_norm(case, st):
    p = {name: _double(st[name], False) for name in ("w_after", "b_after", "gate", "w_before",
                                                     "b_before")}
    h = case["alpha"] * st["h"].double() + _exact_join(case, st, st["y"].double(), p["w_after"],
                                                       p["b_after"], p["gate"])
    n = None if case["before"] == "none" else _exact_normed(case["before"], h, p["w_before"],
                                                            p["b_before"])
    return [h, n]


def _exact_norm_grad(case, st):
    p = {name: _double(st[name]) for name in ("y", "w_after", "b_after", "gate", "w_before",
                                              "b_before")}
    # the stream's values after the block are given: h_out = alpha h + join, as a value of its own
    h0 = torch.zeros(case["T"], case["d"], dtype=torch.float64, device="cuda", requires_grad=True)
    join = _exact_join(case, st, p["y"], p["w_after"], p["b_after"], p["gate"])
    h_out = case["alpha"] * h0 + join
    h_out = h_out + (st["h"].double() - h_out).detach()
    loss = (h_out * st["d_h_out"].double()).sum()
    if case["before"] != "none":
        n = _exact_normed(case["before"], h_out, p["w_before"], p["b_before"])
        loss = loss + (n * st["d_n"].double()).sum()
    names = [name for name in p if p[name] is not None]
    grads = torch.autograd.grad(loss, [h0] + [p[name] for name in names])
    out = dict(zip(["d_h"] + ["d_" + name for name in names], grads))
    return _gradients(out)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("layer", "experts"):
        return _exact_few(case, st)
    if case["op"] == "norm":
        return _exact_norm(case, st)
    if case["op"] == "norm_grad":
        return _exact_norm_grad(case, st)
    y = st["x"].double() * _kept(st["rng"], case["T"], case["d"], case["p"])
    return y if st["residual"] is None else y + st["residual"].double()
