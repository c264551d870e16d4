"""Workloads of the routing and 8-bit expert operators.

Each case is one pass through one operator, either in its plain form (elementary torch operations in
32 bits, `own = False`) or through this package's entry points (`own = True`):

  route      experts and weights of each token from its router logits
  route_grad the gradient of those weights (and of the full scores) to the logits
  quant      8-bit quantization of activations, one scale per token
  matmul     products of 8-bit integers with scales per token and per output channel
  ffn        SwiGLU experts on such products, routed and shared, in slot order
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------------------ cases
def _route(op, T, E, k, score, bias=False, groups=0, keep=0, top2=False, renorm=True, scale=1.0,
           dtype="f32", masked=0.0, full=False):
    """full: the scores of all experts are an output too (route) or carry a gradient (route_grad)."""
    return {"op": op, "T": T, "E": E, "k": k, "score": score, "bias": bias, "groups": groups,
            "keep": keep, "top2": top2, "renorm": renorm, "scale": scale, "dtype": dtype,
            "masked": masked, "full": full}


def _matmul(rows, K, N, n_mat, out="bf16", empty=0):
    return {"op": "matmul", "rows": rows, "K": K, "N": N, "n_mat": n_mat, "out": out,
            "empty": empty}


def _ffn(T, d, E, k, f, S, cap):
    return {"op": "ffn", "T": T, "d": d, "E": E, "k": k, "f": f, "S": S, "cap": cap}


def listed():
    return [
        # one sequence being decoded: latency of a single token's choice
        dict(_route("route", 1, 256, 8, "sigmoid", bias=True, groups=8, keep=4, top2=True,
                    scale=2.5), name="route_one_token"),
        # the fine-grained prefill's 64 experts, bf16 logits, scores kept for a balance loss
        dict(_route("route", 4096, 64, 6, "softmax", renorm=False, dtype="bf16", full=True),
             name="route_fine_grained"),
        # the largest training or prefill batch, group-limited, some experts switched off
        dict(_route("route", 65536, 256, 8, "sigmoid", bias=True, groups=8, keep=4, top2=True,
                    scale=2.5, masked=0.02), name="route_large"),
        # training step of the fine-grained router: weights and balance loss, every expert
        dict(_route("route_grad", 4096, 64, 6, "softmax", renorm=False, dtype="bf16", full=True),
             name="route_grad_fine_grained"),
        # training step of a large batch: only the selected experts' scores carry a gradient
        dict(_route("route_grad", 65536, 256, 8, "sigmoid", scale=2.5), name="route_grad_large"),
        # one decode step's activations, and the skewed prefill's
        {"op": "quant", "T": 64, "d": 7168, "dtype": "bf16", "name": "quant_decode"},
        {"op": "quant", "T": 16384, "d": 7168, "dtype": "bf16", "name": "quant_prefill"},
        # one token through one large matrix: bound by reading it
        dict(_matmul(1, 4096, 14336, 1), name="matmul_one_token"),
        # ragged expert segments, odd sizes, two experts without a token, fp32 out
        dict(_matmul(1337, 1408, 2050, 13, out="f32", empty=2), name="matmul_ragged"),
        # a prefill's dense projection, bound by arithmetic
        dict(_matmul(16384, 7168, 4096, 1), name="matmul_prefill"),
        # the decode shape: 64 tokens, 128 experts and a shared one, bound by the weights
        dict(_ffn(64, 7168, 128, 2, 2048, 1, 8), name="ffn_decode"),
        # the fine-grained prefill with two shared experts and a capacity of 1.25 x the mean
        dict(_ffn(4096, 2048, 64, 6, 1408, 2, 480), name="ffn_prefill"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "quant", "matmul", "matmul", "ffn", "ffn"])
    if op in ("route", "route_grad"):
        groups = rng.choice([0, 0, 2, 4, 8])
        E = groups * rng.randint(2, 256 // groups) if groups else _log(rng, 8, 256)
        keep = rng.randint((groups + 1) // 2, groups) if groups else 0
        most = min(8, keep * (E // groups) if groups else E)
        k = rng.randint(1, most)
        score = rng.choice(["softmax", "sigmoid"])
        return _route(op, _log(rng, 1, 65536), E, k, score, bias=rng.random() < 0.5,
                      groups=groups, keep=keep, top2=bool(groups) and rng.random() < 0.5,
                      renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                      dtype=rng.choice(["f32", "bf16"]), masked=rng.choice([0.0, 0.02]),
                      full=rng.random() < 0.4)
    if op == "quant":
        d = _log(rng, 64, 7168)
        d = d if rng.random() < 0.25 else max(64, d // 64 * 64)
        return {"op": "quant", "T": _log(rng, 1, 16384), "d": d,
                "dtype": rng.choice(["bf16", "f16", "f32"])}
    if op == "matmul":
        n_mat = rng.choice([1, 1, _log(rng, 2, 64)])
        K = max(4, _log(rng, 64, 7168) // 16) * 16
        N = min(_log(rng, 64, 14336), (1 << 29) // (K * n_mat))
        rows = min(_log(rng, 1, 16384), int(16384 * 7168 * 4096 / (K * N)))
        return _matmul(max(1, rows), K, max(1, N), n_mat, out=rng.choice(["bf16", "f16", "f32"]),
                       empty=n_mat // 6)
    d, f = _log(rng, 4, 112) * 64, _log(rng, 4, 32) * 64
    E = min(_log(rng, 8, 128), max(8, int(128 * 7168 * 2048 / (d * f))))
    k, S = rng.randint(1, 6), rng.choice([0, 1, 2])
    most = 4096 * 6 * 2048 * 1408 / (k * d * f)   # the largest listed one's products
    T = _log(rng, 1, max(1, min(4096, int(most))))
    return _ffn(T, d, E, k, f, S, min(T, max(4, math.ceil(1.5 * T * k / E))))


# ----------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _codes(g, n, N, K):
    """Weights of one layer as their 8-bit codes (about normal, largest 127 in a channel) and the
    channels' scales."""
    q = torch.empty(n, N, K, dtype=torch.int8, device="cuda")
    for e in range(n):
        q[e] = (_randn(g, N, K) * 32).round_().clamp_(-127, 127)
    s = (0.8 + 0.4 * torch.rand(n, N, generator=g, device="cuda")) / (32 * math.sqrt(K))
    return q, s


def _choice(g, T, E, k):
    """k different experts per token, some experts more liked than others."""
    return torch.topk(_randn(g, T, E) + 0.3 * _randn(g, E), k, dim=-1).indices.to(torch.int32)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"case": case}
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        logits = _randn(g, T, E)
        if case["masked"]:
            logits[torch.rand(T, E, generator=g, device="cuda") < case["masked"]] = -math.inf
        st["logits"] = logits.to(DT[case["dtype"]])
        spread = 0.05 if case["score"] == "sigmoid" else 0.25 / E
        st["bias"] = spread * _randn(g, E) if case["bias"] else None
        if op == "route":
            st["idx"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
            st["w"] = torch.empty(T, k, device="cuda")
            st["scores"] = torch.empty(T, E, device="cuda") if case["full"] else None
        else:
            st["idx"] = _route_plain(case, st["logits"], st["bias"])[0]
            st["d_w"] = _randn(g, T, k)
            st["d_scores"] = _randn(g, T, E) if case["full"] else None
            st["d_logits"] = torch.empty(T, E, dtype=DT[case["dtype"]], device="cuda")
    elif op == "quant":
        T, d = case["T"], case["d"]
        st["x"] = (_randn(g, T, d) * torch.exp(_randn(g, T, 1))).to(DT[case["dtype"]])
        st["q"] = torch.empty(T, d, dtype=torch.int8, device="cuda")
        st["s"] = torch.empty(T, device="cuda")
    elif op == "matmul":
        rows, K, N, n = (case[v] for v in ("rows", "K", "N", "n_mat"))
        st["qx"] = (_randn(g, rows, K) * 32).round_().clamp_(-127, 127).to(torch.int8)
        st["sx"] = torch.exp(0.5 * _randn(g, rows)) / 32
        st["qw"], st["sw"] = _codes(g, n, N, K)
        st["offsets"], st["cap"] = None, rows
        if n > 1:
            r = random.Random(int(seed))
            at = [r.randrange(case["empty"], n) for _ in range(rows)]
            order = list(range(n))
            r.shuffle(order)
            counts = [0] * n
            for a in at:
                counts[order[a]] += 1
            off = [0]
            for c in counts:
                off.append(off[-1] + c)
            st["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")
            st["cap"] = max(counts)          # rows of the plain form's padded segments
        st["y"] = torch.empty(rows, N, dtype=DT[case["out"]], device="cuda")
    else:
        T, d, E, k, f, S, cap = (case[v] for v in ("T", "d", "E", "k", "f", "S", "cap"))
        st["x"] = _randn(g, T, d).to(torch.bfloat16)
        for name, n, N, K in (("gate", E, f, d), ("up", E, f, d), ("down", E, d, f),
                              ("sh_gate", S, f, d), ("sh_up", S, f, d), ("sh_down", S, d, f)):
            st[name] = _codes(g, n, N, K) if n else None
        # the dispatch that precedes the experts: slots by expert, then in token order, the first
        # `cap` of each expert kept
        idx = _choice(g, T, E, k).reshape(-1).long()
        order = torch.sort(idx, stable=True).indices
        counts = torch.bincount(idx, minlength=E)
        start = torch.cumsum(counts, 0) - counts
        rank = torch.arange(T * k, device="cuda") - start[idx[order]]
        kept = order[rank < cap]
        st["perm_slot"] = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
        st["perm_slot"][:kept.numel()] = kept.to(torch.int32)
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[1:] = torch.cumsum(counts.clamp(max=cap), 0)
        st["offsets"] = off
        st["topk_w"] = torch.softmax(_randn(g, T, k), -1)
        # rows of dropped slots are never written: zero from the start
        st["y"] = torch.zeros(T * k + S * T, d, dtype=torch.float16, device="cuda")
    return st


# ------------------------------------------------------------------------------------ plain forms
def _scores_plain(case, l):
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    top = l.amax(-1, keepdim=True)
    e = torch.exp(l - torch.where(top == -math.inf, 0.0, top))
    # summed in 64 bits and rounded once, so that the order of the sum decides no selection
    total = e.double().sum(-1, keepdim=True).float()
    return e / torch.where(total == 0, 1.0, total)


def _route_plain(case, logits, bias):
    l = logits.float()
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    s = _scores_plain(case, l)
    r = s + bias if bias is not None else (s if case["score"] == "sigmoid" else l)
    r = torch.where(l == -math.inf, -math.inf, r)
    live = torch.zeros_like(r, dtype=torch.bool)
    if G:
        by = torch.sort(r.view(T, G, E // G), dim=-1, descending=True).values
        rank = by[..., 0]
        if case["top2"] and E // G > 1:
            rank = rank + torch.where(by[..., 1] == -math.inf, 0.0, by[..., 1])
        best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[:, :case["keep"]]
        live = live.view(T, G, E // G)
        live.scatter_(1, best[..., None].expand(T, case["keep"], E // G), True)
        live = live.view(T, E)
        # kept experts first (they include masked ones), then by rank, then by index
        order = torch.sort(r, dim=-1, descending=True, stable=True).indices
        first = torch.sort((~live.gather(1, order)).to(torch.uint8), dim=-1, stable=True).indices
        idx = order.gather(1, first[:, :k])
    else:
        idx = torch.sort(r, dim=-1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, idx)
    if case["renorm"]:
        if case["score"] == "softmax":
            sel = l.gather(1, idx)
            top = sel.amax(-1, keepdim=True)
            w = torch.exp(sel - torch.where(top == -math.inf, 0.0, top))
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total == 0, 1.0, total)
    return idx.to(torch.int32), w * case["scale"], s


def _route_grad_plain(case, logits, idx, d_w, d_scores):
    l, idx, c = logits.float(), idx.long(), case["scale"]
    ds = torch.zeros_like(l) if d_scores is None else d_scores
    dl = torch.zeros_like(l)
    if case["score"] == "softmax":
        if case["renorm"]:
            sel = l.gather(1, idx)
            top = sel.amax(-1, keepdim=True)
            u = torch.exp(sel - torch.where(top == -math.inf, 0.0, top))
            total = u.sum(-1, keepdim=True)
            u = u / torch.where(total == 0, 1.0, total)
            dl = dl.scatter(1, idx, c * u * (d_w - (u * d_w).sum(-1, keepdim=True)))
        else:
            ds = ds.scatter_add(1, idx, c * d_w)
        p = _scores_plain(case, l)
        dl = dl + p * (ds - (p * ds).sum(-1, keepdim=True))
    else:
        s = 1.0 / (1.0 + torch.exp(-l))
        g = c * d_w
        if case["renorm"]:
            sel = s.gather(1, idx)
            total = sel.sum(-1, keepdim=True)
            total = torch.where(total == 0, math.inf, total)
            g = (g - (g * sel).sum(-1, keepdim=True) / total) / total
        ds = ds.scatter_add(1, idx, g)
        t = torch.exp(-l.abs())
        dl = ds * (t / ((1.0 + t) * (1.0 + t)))
    return dl.to(logits.dtype)


def _quant_plain(x):
    """Whole numbers (as floats) and scales of the rows of x."""
    x = x.float()
    s = x.abs().amax(-1) / 127.0
    q = torch.round(x / torch.where(s == 0, 1.0, s)[..., None]).clamp(-127, 127)
    return q, s


def _segments(offsets, cap, rows):
    """Rows of the segments padded to `cap`: their numbers, and which are there."""
    at = offsets[:-1, None].long() + torch.arange(cap, device="cuda")
    there = at < offsets[1:, None]
    return torch.where(there, at, 0), there


def _matmul_plain(st):
    case = st["case"]
    rows, N, n = case["rows"], case["N"], case["n_mat"]
    wt = st["qw"].float().transpose(1, 2)
    if n == 1:
        y = torch.mm(st["qx"].float(), wt[0]) * st["sx"][:, None] * st["sw"][0]
        return y.to(st["y"].dtype)
    at, there = _segments(st["offsets"], st["cap"], rows)
    y = torch.bmm(st["qx"].float()[at], wt) * st["sx"][at][..., None] * st["sw"][:, None, :]
    out = torch.empty(rows + 1, N, dtype=st["y"].dtype, device="cuda")
    out[torch.where(there, at, rows)] = y.to(out.dtype)
    return out[:rows]


def _experts_plain(q, s, gate, up, down):
    """q [n, rows, d] whole numbers with scales s [n, rows] through n experts."""
    s = s[..., None]
    a = torch.bmm(q, gate[0].float().transpose(1, 2)) * s * gate[1][:, None, :]
    b = torch.bmm(q, up[0].float().transpose(1, 2)) * s * up[1][:, None, :]
    qh, sh = _quant_plain(a / (1.0 + torch.exp(-a)) * b)
    return torch.bmm(qh, down[0].float().transpose(1, 2)) * sh[..., None] * down[1][:, None, :]


def _ffn_plain(st):
    c = st["case"]
    T, d, k, S = c["T"], c["d"], c["k"], c["S"]
    q, s = _quant_plain(st["x"])
    at, there = _segments(st["offsets"], c["cap"], T * k)
    slot = st["perm_slot"][at].long().clamp(min=0)
    token = slot // k
    y = _experts_plain(q[token], s[token], st["gate"], st["up"], st["down"])
    y = y * st["topk_w"].reshape(-1)[slot][..., None]
    out = torch.zeros((k + S) * T + 1, d, dtype=torch.float16, device="cuda")
    out[torch.where(there, slot, (k + S) * T)] = y.half()
    if S:
        z = _experts_plain(q.expand(S, T, d), s.expand(S, T), st["sh_gate"], st["sh_up"],
                           st["sh_down"])
        out[T * k:(k + S) * T] = z.reshape(S * T, d).half()
    return out[:(k + S) * T]


# ------------------------------------------------------------------------------- the entry points
def _handle(st):
    """What a program makes once and keeps: the call's configuration and its workspace."""
    if "handle" in st:
        return st["handle"]
    import sparse_moe_layer_route_gb300 as M
    c = st["case"]
    if c["op"] in ("route", "route_grad"):
        h = M.GateConfig.make(
            c["T"], c["E"], c["k"],
            score=M.SCORE_SIGMOID if c["score"] == "sigmoid" else M.SCORE_SOFTMAX,
            n_groups=c["groups"], topk_groups=c["keep"], group_top2=c["top2"],
            renormalize=c["renorm"], scale=c["scale"],
            dtype=M.DTYPE_BF16 if c["dtype"] == "bf16" else M.DTYPE_F32)
    elif c["op"] == "matmul":
        h = M.alloc_int8_workspace(M.int8_matmul_workspace_size(c["rows"], c["K"], c["N"],
                                                                c["n_mat"]))
    elif c["op"] == "ffn":
        cfg = M.MoeConfig.make(c["T"], c["d"], c["E"], c["k"], c["f"], n_shared=c["S"],
                               capacity_override=c["cap"])
        ws = M.alloc_int8_workspace(M.grouped_ffn_int8_workspace_size(cfg))
        names = ("gate", "up", "down", "sh_gate", "sh_up", "sh_down")
        h = (cfg, M.make_int8_weights(*[st[n] for n in names]), ws)
    else:
        h = None
    st["handle"] = (M, h)
    return st["handle"]


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        M, h = _handle(st)
        if op == "route":
            M.route_logits(h, st["logits"], st["bias"], st["idx"], st["w"], st["scores"])
            return [st["idx"], st["w"], st["scores"]]
        if op == "route_grad":
            M.route_logits_backward(h, st["logits"], st["idx"], st["d_w"], st["d_scores"],
                                    st["d_logits"])
            return st["d_logits"]
        if op == "quant":
            M.quantize_rows(st["x"], st["q"], st["s"])
            return [st["q"], st["s"]]
        if op == "matmul":
            M.int8_matmul(st["qx"], st["sx"], st["qw"], st["sw"], st["offsets"], st["y"], h)
            return st["y"]
        M.grouped_ffn_int8(h[0], st["x"], st["perm_slot"], st["offsets"], st["topk_w"], h[1],
                           st["y"], h[2])
        return st["y"]
    if op == "route":
        idx, w, s = _route_plain(case, st["logits"], st["bias"])
        return [idx, w, s if case["full"] else None]
    if op == "route_grad":
        return _route_grad_plain(case, st["logits"], st["idx"], st["d_w"], st["d_scores"])
    if op == "quant":
        q, s = _quant_plain(st["x"])
        return [q.to(torch.int8), s]
    if op == "matmul":
        return _matmul_plain(st)
    return _ffn_plain(st)


def work(case):
    op = case["op"]
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        size = 2 if case["dtype"] == "bf16" else 4
        full = 4 * T * E if case["full"] else 0
        if op == "route":
            return {"bytes": T * E * size + 8 * T * k + full + 4 * E, "flops": 8 * T * E}
        # without a gradient of the full scores and with the selected ones' scores alone in the
        # weights, only the selected logits are needed
        dense = case["full"] or (case["score"] == "softmax" and not case["renorm"])
        read = T * E * size if dense else T * k * size
        return {"bytes": read + full + 8 * T * k + T * E * size, "flops": 8 * T * E}
    if op == "quant":
        T, d = case["T"], case["d"]
        return {"bytes": T * d * ((4 if case["dtype"] == "f32" else 2) + 1) + 4 * T,
                "flops": 3 * T * d}
    if op == "matmul":
        rows, K, N = case["rows"], case["K"], case["N"]
        hit = min(rows, case["n_mat"] - case["empty"])
        size = 4 if case["out"] == "f32" else 2
        return {"bytes": hit * N * (K + 4) + rows * (K + 4) + rows * N * size,
                "flops": 2 * rows * N * K}
    T, d, E, k, f, S, cap = (case[v] for v in ("T", "d", "E", "k", "f", "S", "cap"))
    hit = E * (1 - (1 - k / E) ** T)                     # experts that get a token, about
    rows = min(T * k, E * cap) + S * T
    return {"bytes": int((hit + S) * (3 * d * f + 8 * f + 4 * d)) + 2 * T * d + 2 * rows * d,
            "flops": 6 * rows * d * f}


# -------------------------------------------------------------------------- definitions in 64 bits
def _exact_scores(case, l):
    if case["score"] == "sigmoid":
        return torch.sigmoid(l)
    return torch.nan_to_num(torch.softmax(l, -1), nan=0.0)


def _exact_route(case, st):
    l = st["logits"].double()
    s = _exact_scores(case, l)
    # the choice itself is whole numbers; the weights are those of the plain form's choice
    idx = _route_plain(case, st["logits"], st["bias"])[0].long()
    if case["renorm"] and case["score"] == "softmax":
        w = torch.nan_to_num(torch.softmax(l.gather(1, idx), -1), nan=0.0)
    else:
        w = s.gather(1, idx)
        if case["renorm"]:
            w = torch.nan_to_num(w / w.sum(-1, keepdim=True), nan=0.0)
    return [None, case["scale"] * w, s if case["full"] else None]


def _exact_route_grad(case, st):
    l = st["logits"].double().requires_grad_(True)
    idx = st["idx"].long()
    s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, -1)
    if case["renorm"] and case["score"] == "softmax":
        w = torch.softmax(l.gather(1, idx), -1)
    else:
        w = s.gather(1, idx)
        if case["renorm"]:
            w = w / w.sum(-1, keepdim=True)
    loss = (case["scale"] * w * st["d_w"].double()).sum()
    if st["d_scores"] is not None:
        loss = loss + (s * st["d_scores"].double()).sum()
    # a row without a single live expert has no gradient
    return torch.nan_to_num(torch.autograd.grad(loss, l)[0], nan=0.0)


def _exact_quant(x):
    x = x.double()
    s = x.abs().amax(-1, keepdim=True) / 127
    return torch.nan_to_num(x / s).round(), s


def _exact_expert(q, s, gate, up, down, e):
    a = (q @ gate[0][e].double().T) * s * gate[1][e].double()
    b = (q @ up[0][e].double().T) * s * up[1][e].double()
    qh, sh = _exact_quant(torch.nn.functional.silu(a) * b)
    return (qh @ down[0][e].double().T) * sh * down[1][e].double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, st)
    if op == "route_grad":
        return _exact_route_grad(case, st)
    if op == "quant":
        return [None, _exact_quant(st["x"])[1][:, 0]]
    if op == "matmul":
        n = case["n_mat"]
        off = [0, case["rows"]] if n == 1 else st["offsets"].tolist()
        y = torch.empty(case["rows"], case["N"], dtype=torch.float64, device="cuda")
        for e in range(n):
            rows = slice(off[e], off[e + 1])
            y[rows] = (st["qx"][rows].double() @ st["qw"][e].double().T) \
                * st["sx"][rows, None].double() * st["sw"][e].double()
        return y
    T, d, E, k, S = (case[v] for v in ("T", "d", "E", "k", "S"))
    q, s = _exact_quant(st["x"])
    y = torch.zeros((k + S) * T, d, dtype=torch.float64, device="cuda")
    off = st["offsets"].tolist()
    for e in range(E):
        slot = st["perm_slot"][off[e]:off[e + 1]].long()
        if slot.numel():
            z = _exact_expert(q[slot // k], s[slot // k], st["gate"], st["up"], st["down"], e)
            y[slot] = z * st["topk_w"].reshape(-1)[slot, None].double()
    for j in range(S):
        y[(k + j) * T:(k + j + 1) * T] = _exact_expert(q, s, st["sh_gate"], st["sh_up"],
                                                       st["sh_down"], j)
    return y
