"""The MoE layer in 64 bits on torch tensors, written from its definition, with a bound on what a kernel that
sums in 32 bits may differ by; inputs for the tests of the few-token layer."""
import math

import torch

PLAIN, BIAS, GUMBEL = 0, 1, 2


def make(T, d, E, k, f, S, seed=0, device="cuda"):
    g = torch.Generator().manual_seed(seed)

    def w(n, rows, cols):
        return (torch.randn(n, rows, cols, generator=g) / math.sqrt(rows)).bfloat16().to(device)

    return {"x": torch.randn(T, d, generator=g).bfloat16().to(device),
            "W_g": w(1, d, E)[0], "bias": (0.3 * torch.randn(E, generator=g)).to(device),
            "u": torch.rand(T, E, generator=g).clamp_(2.0 ** -24, 1 - 2.0 ** -24).to(device),
            "W_gate": w(E, d, f), "W_up": w(E, d, f), "W_down": w(E, f, d),
            "Wsh_gate": w(S, d, f) if S else None, "Wsh_up": w(S, d, f) if S else None,
            "Wsh_down": w(S, f, d) if S else None}


def choose(p, k, mode=PLAIN, tau=1.0, groups=0, keep=0):
    """Experts [T, k], gates and the smallest gap that decided something."""
    l = p["x"].double() @ p["W_g"].double()
    T, E = l.shape
    s = l
    if mode == BIAS:
        s = l + p["bias"].double()
    elif mode == GUMBEL:
        s = (l - torch.log(-torch.log(p["u"].double()))) / tau
    r, gap = s, math.inf
    if groups:
        best = s.view(T, groups, -1).amax(-1)
        order = torch.sort(best, dim=-1, descending=True, stable=True)
        if keep < groups:
            gap = (order.values[:, keep - 1] - order.values[:, keep]).min().item()
        live = torch.zeros_like(best, dtype=torch.bool).scatter_(1, order.indices[:, :keep], True)
        r = torch.where(live.repeat_interleave(E // groups, 1), s, -math.inf)
    order = torch.sort(r, dim=-1, descending=True, stable=True)
    idx = order.indices[:, :k]
    if E > 1:
        ahead = order.values[:, :min(k, E - 1)] - order.values[:, 1:min(k, E - 1) + 1]
        gap = min(gap, torch.nan_to_num(ahead, nan=math.inf).min().item())
    w = torch.softmax((s if mode == GUMBEL else l).gather(1, idx), -1)
    return idx, w, gap


def _expert(x, gate, up, down):
    """Output and the bound of its error: sums of n products in 32 bits, in chains of n / 8 + 32 at most with
    2^-23 a step (the tensor core's adds truncate), silu' <= 1.1, H rounded to 16 bits (2^-17), exp and
    division within 2^-21."""
    gate, up, down = gate.double(), up.double(), down.double()
    d, f = gate.shape
    a, b = x @ gate, x @ up
    step_d, step_f = (d / 8 + 32) * 2.0 ** -23, (f / 8 + 32) * 2.0 ** -23
    da, db = step_d * (x.abs() @ gate.abs()), step_d * (x.abs() @ up.abs())
    act = torch.nn.functional.silu(a)
    h = act * b
    dh = 1.1 * da * (b.abs() + db) + act.abs() * db + h.abs() * (2.0 ** -17 + 2.0 ** -20)
    return h @ down, dh @ down.abs() + step_f * (h.abs() @ down.abs())


def layer(p, idx, w, cap=0, S=0):
    """Output of the layer with this choice, and how far a kernel may be off before its rounding. Indices that
    are no expert's add nothing; each expert takes its first `cap` slots."""
    x = p["x"].double()
    T, k = idx.shape
    E = p["W_gate"].shape[0]
    out = torch.zeros_like(x)
    err = torch.zeros_like(x)
    flat = idx.reshape(-1).tolist()
    w = w.double().reshape(-1)
    for e in sorted({v for v in flat if 0 <= v < E}):
        slots = [s for s, v in enumerate(flat) if v == e]
        for s in slots[:cap] if cap else slots:
            t = s // k
            y, dy = _expert(x[t:t + 1], p["W_gate"][e], p["W_up"][e], p["W_down"][e])
            out[t] += w[s] * y[0]
            err[t] += w[s].abs() * (dy[0] + 2.0 ** -20 * y[0].abs())
    for s in range(S):
        y, dy = _expert(x, p["Wsh_gate"][s], p["Wsh_up"][s], p["Wsh_down"][s])
        out += y
        err += dy
    return out, err


def assert_rounded(got, want, err):
    """got (bf16) is want within err, then rounded once: half a step of bf16 is 2^-8 of the value."""
    assert torch.isfinite(got).all()
    off = (got.double() - want).abs()
    allowed = err + 2.0 ** -8 * (want.abs() + err)
    worst = (off / allowed.clamp_min(1e-300)).max().item()
    assert (off <= allowed).all(), f"{worst} times what is allowed"
