"""Norms around a block, gates and dropout in 64 bits on torch tensors, from their definitions, with bounds on
what sums in 32 bits may differ by."""
import math

import torch

U = 2.0 ** -24                               # half a step of fp32
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LEAST = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
NONE, RMS, LAYER = 0, 1, 2


def philox(counter, key):
    """Philox 4x32-10 on lists of four and two int64 tensors (or numbers) of 32 bits."""
    c, k = list(counter), list(key)
    mask = 0xFFFFFFFF

    def product(m, v):                       # 64 bits in two halves: int64 would overflow
        low = m * (v & 0xFFFF)
        high = m * (v >> 16) + (low >> 16)
        return high >> 16, ((high & 0xFFFF) << 16) | (low & 0xFFFF)

    for _ in range(10):
        (ha, la), (hb, lb) = product(0xD2511F53, c[0]), product(0xCD9E8D57, c[2])
        c = [hb ^ c[1] ^ k[0], lb, ha ^ c[3] ^ k[1], la]
        k = [(k[0] + 0x9E3779B9) & mask, (k[1] + 0xBB67AE85) & mask]
    return c


def factors(seed, step, T, d, p, row0=0):
    """Dropout's factors of [T, d] on the CPU, float64."""
    cols = torch.arange((d + 3) // 4, dtype=torch.int64)
    rows = torch.arange(row0, row0 + T, dtype=torch.int64)[:, None]
    zero = torch.zeros(T, len(cols), dtype=torch.int64)
    mask = 0xFFFFFFFF
    r = philox([zero + cols, zero + rows, zero + (step & mask), zero + (step >> 32 & mask)],
               [seed & mask, seed >> 32 & mask])
    p = torch.tensor(p, dtype=torch.float32).double().item()
    keep = torch.stack(r, -1).reshape(T, -1)[:, :d] >= round(p * 2 ** 32)
    return keep.double() / (1 - p)


def normed(kind, x, eps):
    """Normed rows, one over their deviation, and the size that sums cancel from: mean |x| of a layer norm."""
    m = x.mean(-1, keepdim=True) if kind == LAYER else 0.0
    r = 1 / torch.sqrt((x - m).square().mean(-1, keepdim=True) + eps)
    return (x - m) * r, r, (x.abs().mean(-1, keepdim=True) if kind == LAYER else 0.0)


def norm_error(kind, x, dx, eps):
    """Error of the normed row whose input is off by dx. A sum of d terms goes over chains of at most 16 + 5 +
    4 + 3 adds, so it is off by 32 U of the terms' sizes; the deviation's relative error is half its square's,
    and division and root add a few U."""
    xn, r, size = normed(kind, x, eps)
    mean = dx.mean(-1, keepdim=True) + 32 * U * size if kind == LAYER else 0.0
    dev = dx + mean + U * (x.abs() + size)
    rel = (xn.abs() * dev * r).mean(-1, keepdim=True) + (dev * r).square().mean(-1, keepdim=True) + 40 * U
    return xn.abs() * rel + r * dev


def forward(c, t, m=None):
    """c: after, before, alpha, beta, eps, gate_rows; t: h, y and parameters (float64 or None); m: dropout's
    factors. Returns h', n and the bounds of their errors before rounding."""
    h, y = t["h"], t["y"]
    T = h.shape[0]
    out, err = c["alpha"] * h, 2 * U * (c["alpha"] * h).abs()
    if y is not None:
        u, du = y, torch.zeros_like(y)
        if c["after"] != NONE:
            du = norm_error(c["after"], y, du, c["eps"])
            u = normed(c["after"], y, c["eps"])[0]
            for w, b in ((t["w_after"], t["b_after"]),):
                if w is not None:
                    u, du = u * w, du * w.abs() + U * (u * w).abs()
                if b is not None:
                    u, du = u + b, du + U * ((u + b).abs() + b.abs())
        if m is not None:
            u, du = torch.where(m > 0, u * m, 0.0), torch.where(m > 0, du * m, 0.0) + 2 * U * (u * m).abs()
        if t["gate"] is not None:
            g = t["gate"].repeat_interleave(c["gate_rows"], 0)[:T]
            u, du = u * g, du * g.abs() + U * (u * g).abs()
        out = out + c["beta"] * u
        err = err + abs(c["beta"]) * (du + 2 * U * u.abs()) + 2 * U * out.abs()
    if c["before"] == NONE:
        return out, None, err, None
    n, dn = normed(c["before"], out, c["eps"])[0], norm_error(c["before"], out, err, c["eps"])
    w, b = t["w_before"], t["b_before"]
    if w is not None:
        n, dn = n * w, dn * w.abs() + U * (n * w).abs()
    if b is not None:
        n, dn = n + b, dn + U * ((n + b).abs() + b.abs())
    return out, n, err, dn


NAMES = ("d_h", "d_y", "d_w_after", "d_b_after", "d_gate", "d_w_before", "d_b_before")


def backward(c, t, m=None):
    """Gradients by the chain rule, term by term, and the bounds of their errors: every value is a sum of
    terms; of those a mean has 32 U of its terms' sizes, a normed value 100 U (of itself and of what its mean
    cancelled), a sum over tokens at most 128 + T / 100 adds. t: h_out, y, d_h_out, d_n and parameters."""
    T, d = (t["d_h_out"] if t["d_h_out"] is not None else t["d_n"]).shape
    out, size = {}, {}
    zero = torch.zeros(T, d, dtype=torch.float64, device=(t["d_h_out"] if t["d_h_out"] is not None
                                                          else t["d_n"]).device)
    g = t["d_h_out"] if t["d_h_out"] is not None else zero
    s = g.abs()

    def back(kind, e, es, xn, xs, r):
        """Gradient through a norm and its size, of the gradient e (size es) to normed values xn (size xs)."""
        v = e - xn * (e * xn).mean(-1, keepdim=True)
        vs = es + xs * (es * xs).mean(-1, keepdim=True)
        if kind == LAYER:
            v, vs = v - e.mean(-1, keepdim=True), vs + es.mean(-1, keepdim=True)
        return r * v, r * vs

    if t["d_n"] is not None:
        xn, r, off = normed(c["before"], t["h_out"], c["eps"])
        xs = xn.abs() + r * off
        n = t["d_n"]
        out["d_w_before"], size["d_w_before"] = (n * xn).sum(0), (n.abs() * xs).sum(0)
        out["d_b_before"], size["d_b_before"] = n.sum(0), n.abs().sum(0)
        e = n if t["w_before"] is None else n * t["w_before"]
        v, vs = back(c["before"], e, e.abs(), xn, xs, r)
        g, s = g + v, s + vs
    out["d_h"], size["d_h"] = c["alpha"] * g, abs(c["alpha"]) * s
    if t["y"] is not None:
        e, es = c["beta"] * g, abs(c["beta"]) * s
        if m is not None:
            e, es = e * m, es * m
        u, xn, xs, r = t["y"], t["y"], t["y"].abs(), None
        us = u.abs()
        w, b = t["w_after"], t["b_after"]
        if c["after"] != NONE:
            xn, r, off = normed(c["after"], t["y"], c["eps"])
            xs = xn.abs() + r * off
            u, us = xn, xs
            if w is not None:
                u, us = u * w, us * w.abs()
            if b is not None:
                u, us = u + b, us + b.abs()
        if t["gate"] is not None:
            rows = c["gate_rows"]
            count = math.ceil(T / rows)

            def sums(v):
                wide = torch.zeros(count * rows, d, dtype=torch.float64, device=v.device)
                wide[:T] = v
                return wide.view(count, rows, d).sum(1)

            out["d_gate"], size["d_gate"] = sums(e * u), sums(es * us)
            gate = t["gate"].repeat_interleave(rows, 0)[:T]
            e, es = e * gate, es * gate.abs()
        if c["after"] != NONE:
            out["d_w_after"], size["d_w_after"] = (e * xn).sum(0), (es * xs).sum(0)
            out["d_b_after"], size["d_b_after"] = e.sum(0), es.sum(0)
            if w is not None:
                e, es = e * w, es * w.abs()
            e, es = back(c["after"], e, es, xn, xs, r)
        out["d_y"], size["d_y"] = e, es
    steps = {name: (500 if name in ("d_h", "d_y") else 700 + T / 100) for name in out}
    return out, {name: steps[name] * U * size[name] for name in out}


def assert_close(name, got, want, err):
    """got is want within err, rounded once to its type."""
    assert torch.isfinite(got).all(), name
    half = HALF[got.dtype]
    allowed = err + half * (want.abs() + err) + LEAST[got.dtype]
    off = (got.double() - want).abs()
    worst = (off / allowed).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst} times what is allowed"
