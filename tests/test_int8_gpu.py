"""8-bit rows, products and experts against plain forms in 64 bits.

Tolerances, before any run (u = 2^-24):
  codes, scales  equal to the rule in fp32 (numpy multiplies, divides and rounds as IEEE does).
  product        integer sums below 2^24 are exact: conversion, scale product and result round once
                 each, 4 u. Larger sums (the all-127 case): at most 2^-23 per 16 products added,
                 K / 16 * 2^-23. bf16 and fp16 outputs are the fp32 output rounded once, bit for bit.
  experts        against 64 bits, x quantized by the rule in fp32 (bf16 values x / scale are often exact
                 ties, which 64 bits would break otherwise). A code of H moves by one where fp32 and 64
                 bits round its value to different sides, one in a few hundred at most:
                 sqrt(1 / 300) / 25 of a row's norm, 2.3e-3. 5e-3 of the norm of the whole, and 5e-2 of
                 the largest output for one value.
"""
import numpy as np
import pytest
import torch

import sparse_moe_layer_route_gb300 as M

U = 2.0 ** -24


def gen(seed):
    return torch.Generator().manual_seed(seed)


# -------------------------------------------------------------------------------- quantization
def rows32(x):
    """The rule in fp32."""
    x = np.asarray(x, dtype=np.float32)
    s = (np.abs(x).max(1) * (np.float32(1) / np.float32(127))).astype(np.float32)
    d = np.where(s == 0, np.float32(1), s)[:, None]
    return np.clip(np.rint((x / d).astype(np.float32)), -127, 127).astype(np.int8), s


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", [(1, 1), (3, 7), (1, 7168), (65, 64), (33, 1000), (5, 2048),
                                 (130, 1409), (2, 20000), (700, 256)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_rows(T, d, dtype):
    x = (torch.randn(T, d, generator=gen(T + d)) * torch.exp(torch.randn(T, 1, generator=gen(d))))
    x = x.to(dtype)
    if T > 2:
        x[1] = 0
        x[2] = -x[2].abs()
    q = torch.full((T, d), 99, dtype=torch.int8, device="cuda")
    s = torch.full((T,), -1.0, device="cuda")
    M.quantize_rows(x.cuda(), q, s)
    q0, s0 = rows32(x.float().numpy())
    assert np.array_equal(q.cpu().numpy(), q0) and np.array_equal(s.cpu().numpy(), s0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_rows_strided_and_unaligned(dtype):
    big = torch.randn(40, 515, device="cuda").to(dtype)
    for lo, hi in ((0, 512), (1, 513), (3, 500), (8, 264)):
        x = big[:, lo:hi]
        q = torch.empty(40, hi - lo, dtype=torch.int8, device="cuda")
        s = torch.empty(40, device="cuda")
        M.quantize_rows(x, q, s)
        q0, s0 = rows32(x.float().cpu().numpy())
        assert np.array_equal(q.cpu().numpy(), q0) and np.array_equal(s.cpu().numpy(), s0)


@pytest.mark.gpu
def test_rows_rounding_ties_and_extremes():
    # x / scale exactly between two codes: scale 1, values n + 1/2, to the even one
    x = torch.zeros(4, 256)
    x[0, 0] = 127.0
    x[0, 1:254] = torch.arange(-126, 127).float() + 0.5
    x[1, :3] = torch.tensor([1e-45, -3e-45, 2e-44])       # subnormal
    x[2, :3] = torch.tensor([3e38, -3.4e38, 1.0])
    x[3, :2] = torch.tensor([127 * 2.0 ** -149, 2.0 ** -149])
    q = torch.empty(4, 256, dtype=torch.int8, device="cuda")
    s = torch.empty(4, device="cuda")
    M.quantize_rows(x.cuda(), q, s)
    q0, s0 = rows32(x.numpy())
    assert np.array_equal(s.cpu().numpy(), s0)
    assert np.array_equal(q.cpu().numpy(), q0)


@pytest.mark.gpu
def test_rows_nan_and_infinity_reach_the_scale():
    x = torch.randn(4, 300)
    x[0, 5] = float("nan")
    x[1, 7] = float("inf")
    x[2, 7], x[2, 200] = float("-inf"), float("nan")
    q = torch.empty(4, 300, dtype=torch.int8, device="cuda")
    s = torch.empty(4, device="cuda")
    M.quantize_rows(x.cuda(), q, s)
    assert torch.isnan(s[0]) and torch.isinf(s[1]) and s[1] > 0 and torch.isnan(s[2])
    assert torch.isfinite(s[3]) and (q[0] == 0).all() and (q[1] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n,K,N", [(1, 16, 1), (3, 128, 96), (2, 70, 33), (1, 640, 1000)])
def test_channels(n, K, N):
    W = torch.randn(n, K, N, generator=gen(K)).to(torch.bfloat16)
    q, s = M.quantize_channels(W.cuda())
    q0, s0 = rows32(W.float().transpose(1, 2).reshape(n * N, K).numpy())
    assert np.array_equal(q.cpu().numpy().reshape(n * N, K), q0)
    assert np.array_equal(s.cpu().numpy().reshape(-1), s0)


# -------------------------------------------------------------------------------------- product
def codes(*shape, seed, full=False):
    lo = -128 if full else -127
    return torch.randint(lo, 128, shape, generator=gen(seed), dtype=torch.int8)


def product64(qx, sx, qw, sw, off):
    y = torch.zeros(qx.shape[0], qw.shape[1], dtype=torch.float64)
    for e in range(qw.shape[0]):
        r = slice(off[e], off[e + 1])
        y[r] = (qx[r].double() @ qw[e].double().T) * sx[r, None].double() * sw[e].double()
    return y


def product(qx, sx, qw, sw, offsets, dtype):
    rows, K = qx.shape
    n, N = qw.shape[:2]
    ws = M.alloc_int8_workspace(M.int8_matmul_workspace_size(rows, K, N, n))
    y = torch.full((rows, N), float("nan"), dtype=dtype, device="cuda")
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    M.int8_matmul(qx.cuda(), sx.cuda(), qw.cuda(), sw.cuda(), off, y, ws)
    return y, M.device_status(ws)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,K,N", [(1, 16, 1), (1, 4096, 130), (2, 48, 64), (3, 128, 257),
                                      (8, 1024, 512), (9, 1008, 128), (16, 512, 384),
                                      (17, 64, 100), (40, 768, 1000), (64, 1024, 256),
                                      (129, 272, 300), (260, 1024, 520), (700, 144, 136),
                                      (530000, 16, 3), (2, 16, 70000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_one_matrix(rows, K, N, dtype):
    qx, qw = codes(rows, K, seed=1, full=True), codes(1, N, K, seed=2, full=True)
    sx, sw = torch.rand(rows, generator=gen(3)) / 64, torch.rand(1, N, generator=gen(4)) / 64
    y, status = product(qx, sx, qw, sw, None, dtype)
    assert status == 0
    y32, _ = product(qx, sx, qw, sw, None, torch.float32)
    want = product64(qx, sx, qw, sw, [0, rows])
    err = (y32.double().cpu() - want).abs()
    assert (err <= 4 * U * want.abs()).all(), err.max()
    assert torch.equal(y, y32.to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("counts,K,N", [
    ([20], 4096, 5200),                                   # K in pieces, rows of one narrow tile
    ([129], 1552, 2100), ([700], 1040, 600),              # K in pieces, several row tiles
    ([10] * 40 + [0] * 4 + [13, 33, 1, 64] * 5, 1232, 520),   # many short segments
    ([100, 128, 129, 1, 0, 60, 97, 128] * 2, 704, 520),   # 128-row tiles of CTA pairs
    ([3000], 272, 523), ([1700, 0, 1, 192, 193, 500], 336, 520)])   # 192-row tiles
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_tensor_core_products(counts, K, N, dtype):
    """Products above the work that integer dot products take."""
    n, rows = len(counts), sum(counts)
    off = [0] + [int(v) for v in np.cumsum(counts)]
    # codes whose sums stay below 2^24: at most 4096 * 60 * 60
    qx, qw = (torch.randint(-60, 61, s, generator=gen(11), dtype=torch.int8)
              for s in ((rows, K), (n, N, K)))
    sx, sw = torch.rand(rows, generator=gen(12)) / 64, torch.rand(n, N, generator=gen(13)) / 64
    y32, status = product(qx, sx, qw, sw, off if n > 1 else None, torch.float32)
    assert status == 0
    if dtype == torch.float32:
        want = torch.zeros(rows, N, dtype=torch.float64, device="cuda")
        for e in range(n):
            r = slice(off[e], off[e + 1])
            want[r] = (qx[r].cuda().double() @ qw[e].cuda().double().T) * sx[r, None].cuda() \
                * sw[e].cuda()
        assert ((y32.double() - want).abs() <= 4 * U * want.abs()).all()
    else:
        y, status = product(qx, sx, qw, sw, off if n > 1 else None, dtype)
        assert status == 0 and torch.equal(y, y32.to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("counts,K,N", [([33], 4096, 3001), ([150, 0, 61], 2064, 1049),
                                        ([90, 3, 0, 61], 2064, 1400), ([40], 7168, 1502)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_pieces_of_k_in_rows_of_any_length(counts, K, N, dtype):
    """K in pieces; y's rows on 16 bytes and not, and y itself one element past 16 bytes."""
    n, rows = len(counts), sum(counts)
    off = [0] + [int(v) for v in np.cumsum(counts)]
    # codes whose sums stay below 2^24: at most 7168 * 48 * 48
    qx, qw = (torch.randint(-48, 49, s, generator=gen(31), dtype=torch.int8)
              for s in ((rows, K), (n, N, K)))
    sx, sw = torch.rand(rows, generator=gen(32)) / 64, torch.rand(n, N, generator=gen(33)) / 64
    y32, status = product(qx, sx, qw, sw, off if n > 1 else None, torch.float32)
    want = product64(qx, sx, qw, sw, off)
    assert status == 0 and ((y32.double().cpu() - want).abs() <= 4 * U * want.abs()).all()
    y = torch.empty(rows * N + 1, dtype=dtype, device="cuda")[1:].view(rows, N)
    ws = M.alloc_int8_workspace(M.int8_matmul_workspace_size(rows, K, N, n))
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda") if n > 1 else None
    M.int8_matmul(qx.cuda(), sx.cuda(), qw.cuda(), sw.cuda(), offsets, y, ws)
    assert M.device_status(ws) == 0 and torch.equal(y, y32.to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[200, 224, 225, 256, 257, 400, 449, 512, 513, 700, 1, 0],
                                    [256] * 9, [400] * 7 + [193, 192] * 3])
@pytest.mark.parametrize("K,N", [(48, 5200), (400, 2050)])
def test_tall_row_tiles(counts, K, N):
    """Segments cut into tiles of up to 256 rows, several units for each pair of CTAs, with K so short that
    a tile's products are over before the one before it is stored."""
    n, rows = len(counts), sum(counts)
    off = [0] + [int(v) for v in np.cumsum(counts)]
    qx, qw = (torch.randint(-60, 61, s, generator=gen(21), dtype=torch.int8)
              for s in ((rows, K), (n, N, K)))
    sx, sw = torch.rand(rows, generator=gen(22)) / 64, torch.rand(n, N, generator=gen(23)) / 64
    y32, status = product(qx, sx, qw, sw, off, torch.float32)
    assert status == 0
    for e in range(n):
        r = slice(off[e], off[e + 1])
        want = (qx[r].cuda().double() @ qw[e].cuda().double().T) * sx[r, None].cuda() * sw[e].cuda()
        assert ((y32[r].double() - want).abs() <= 4 * U * want.abs()).all()
    for dtype in (torch.bfloat16, torch.float16):
        y, status = product(qx, sx, qw, sw, off, dtype)
        assert status == 0 and torch.equal(y, y32.to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,n", [(40, 1), (400, 1), (2000, 1), (1500, 16), (700, 64)])
def test_largest_sums_on_the_tensor_cores(rows, n):
    """Sums far past 2^24, with the bound of test_largest_sums; N such that dot products do not
    take it."""
    K, N = 4096, max(160, 400000000 // (4096 * rows) + 1)
    qx = torch.full((rows, K), 127, dtype=torch.int8)
    qw = torch.full((n, N, K), 127, dtype=torch.int8)
    qw[:, 1::2] = -128
    off = [i * rows // n for i in range(n + 1)]
    y, _ = product(qx, torch.ones(rows), qw, torch.ones(n, N), off if n > 1 else None,
                   torch.float32)
    want = torch.full((rows, N), 127.0 * 127 * K, dtype=torch.float64)
    want[:, 1::2] = -127.0 * 128 * K
    assert ((y.double().cpu() - want).abs() <= (K / 16 * 2.0 ** -23 + 4 * U) * want.abs()).all()


@pytest.mark.gpu
def test_bad_offsets_and_scales_on_the_tensor_cores():
    K, N, n, rows = 512, 520, 8, 1600
    qx, qw = codes(rows, K, seed=1), codes(n, N, K, seed=2)
    sx, sw = torch.ones(rows), torch.ones(n, N)
    sx[7] = float("nan")
    off = [0, 200, 400, 600, 800, 1000, 1200, 1400, 1600]
    y, status = product(qx, sx, qw, sw, off, torch.float32)
    assert status == 0 and torch.isnan(y[7]).all() and torch.isfinite(y[:7]).all()
    assert torch.isfinite(y[8:]).all()
    for bad in (off[:3] + [300] + off[4:], off[:8] + [5000], [-5] + off[1:]):
        y, status = product(qx, torch.ones(rows), qw, sw, bad, torch.float32)
        assert status & M.DEVFAULT_BAD_TILE
        want = product64(qx[400:600], torch.ones(200), qw[2:3], sw[2:3], [0, 200])
        if bad[2:4] == [400, 600]:
            assert (y[400:600].double().cpu() == want).all()


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[5, 0, 130, 1, 64], [0, 0, 3], [1, 1, 1, 1, 1, 1, 1, 1],
                                    [300, 2], [0], [16, 17, 15, 33, 128, 127, 129]])
@pytest.mark.parametrize("K,N", [(96, 130), (1024, 256), (400, 64)])
def test_segments(counts, K, N):
    n, rows = len(counts), sum(counts) + 4                # four rows belong to no segment
    off = [0] + list(np.cumsum(counts))
    qx, qw = codes(rows, K, seed=5), codes(n, N, K, seed=6)
    sx, sw = torch.rand(rows, generator=gen(7)), torch.rand(n, N, generator=gen(8))
    y, status = product(qx, sx, qw, sw, off, torch.float32)
    want = product64(qx, sx, qw, sw, off)
    assert status == 0
    assert ((y[:off[-1]].double().cpu() - want[:off[-1]]).abs()
            <= 4 * U * want[:off[-1]].abs()).all()
    assert torch.isnan(y[off[-1]:]).all()                 # not written


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 5, 40, 200])
def test_largest_sums(rows):
    K, N = 4096, 160
    qx = torch.full((rows, K), 127, dtype=torch.int8)
    qw = torch.full((1, N, K), 127, dtype=torch.int8)
    qw[0, 1::2] = -128
    y, _ = product(qx, torch.ones(rows), qw, torch.ones(1, N), None, torch.float32)
    want = product64(qx, torch.ones(rows), qw, torch.ones(1, N), [0, rows])
    assert ((y.double().cpu() - want).abs() <= (K / 16 * 2.0 ** -23 + 4 * U) * want.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[3, 0, 4], [7], [2, 1, 1, 1, 1, 1], [5, 20, 8], [90, 3]])
def test_segments_of_few_rows_and_long_sums(counts):
    """Up to eight rows in all, and products whose K is done in pieces (K = 2064: 17 stages)."""
    n, rows = len(counts), sum(counts)
    off = [0] + list(np.cumsum(counts))
    for K, N in ((2064, 130), (4096, 258), (16, 5)):
        # codes whose sums stay below 2^24: at most 4096 * 60 * 60
        qx, qw = (torch.randint(-60, 61, s, generator=gen(9), dtype=torch.int8)
                  for s in ((rows, K), (n, N, K)))
        sx, sw = torch.rand(rows, generator=gen(7)), torch.rand(n, N, generator=gen(8))
        y, status = product(qx, sx, qw, sw, off, torch.float32)
        want = product64(qx, sx, qw, sw, off)
        assert status == 0
        assert ((y.double().cpu() - want).abs() <= 4 * U * want.abs()).all()


@pytest.mark.gpu
def test_a_row_is_the_same_among_few_and_many():
    """Integer sums do not depend on the path that a number of rows takes."""
    K, N = 1552, 520
    qx = torch.randint(-90, 91, (900, K), generator=gen(1), dtype=torch.int8)
    qw = torch.randint(-90, 91, (1, N, K), generator=gen(2), dtype=torch.int8)
    sx, sw = torch.rand(900, generator=gen(3)), torch.rand(1, N, generator=gen(4))
    all_rows, _ = product(qx, sx, qw, sw, None, torch.bfloat16)
    for rows in (1, 2, 4, 8, 9, 33, 97, 200, 500):
        y, _ = product(qx[:rows], sx[:rows], qw, sw, None, torch.bfloat16)
        assert torch.equal(y, all_rows[:rows]), rows


@pytest.mark.gpu
def test_bad_offsets_are_reported_and_contained():
    K, N = 64, 64
    qx, qw = codes(20, K, seed=1), codes(3, N, K, seed=2)
    sx, sw = torch.ones(20), torch.ones(3, N)
    for off in ([0, 12, 5, 20], [0, 5, 40, 40], [-3, 5, 9, 20]):
        y, status = product(qx, sx, qw, sw, off, torch.float32)
        assert status & M.DEVFAULT_BAD_TILE
    y, status = product(qx, sx, qw, sw, [0, 12, 5, 20], torch.float32)
    want = product64(qx, sx, qw, sw, [0, 12, 12, 12])
    assert (y[:5].double().cpu() == want[:5]).all()       # rows of the first segment alone


@pytest.mark.gpu
def test_non_finite_scales_reach_the_product():
    qx, qw = codes(3, 64, seed=1), codes(1, 32, 64, seed=2)
    sx = torch.tensor([1.0, float("nan"), 1.0])
    y, _ = product(qx, sx, qw, torch.ones(1, 32), None, torch.float32)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[2]).all()


# -------------------------------------------------------------------------------------- experts
def q64(x):
    s = x.abs().amax(1, keepdim=True) / 127
    return torch.nan_to_num(x / s).round(), s


def expert64(q, s, gate, up, down, e):
    a = (q @ gate[0][e].double().T) * s * gate[1][e].double()
    b = (q @ up[0][e].double().T) * s * up[1][e].double()
    qh, sh = q64(a / (1 + torch.exp(-a)) * b)
    return (qh @ down[0][e].double().T) * sh * down[1][e].double()


def layer(T, d, E, k, f, S, cap, seed, one_expert=False):
    g = gen(seed)
    st = {"x": torch.randn(T, d, generator=g).to(torch.bfloat16).cuda()}
    for name, n, K, N in (("gate", E, d, f), ("up", E, d, f), ("down", E, f, d),
                          ("sh_gate", S, d, f), ("sh_up", S, d, f), ("sh_down", S, f, d)):
        st[name] = M.quantize_channels((torch.randn(n, K, N, generator=g) / K ** 0.5)
                                       .to(torch.bfloat16).cuda()) if n else None
    cfg = M.MoeConfig.make(T, d, E, k, f, n_shared=S, capacity_override=cap)
    score = torch.rand(T, E, generator=g)
    if one_expert:
        score[:, 1] += 2
    st["idx"] = torch.topk(score, k).indices.to(torch.int32).cuda()
    st["topk_w"] = torch.softmax(torch.randn(T, k, generator=g), -1).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    st["counts"], st["offsets"] = torch.empty(E, **i32), torch.empty(E + 1, **i32)
    st["perm_slot"], st["slot_pos"] = torch.empty(T * k, **i32), torch.empty(T * k, **i32)
    M.permute(cfg, st["idx"], st["counts"], st["offsets"], st["perm_slot"], st["slot_pos"],
              M.alloc_workspace(cfg))
    names = ("gate", "up", "down", "sh_gate", "sh_up", "sh_down")
    st["weights"] = M.make_int8_weights(*[st[n] for n in names])
    st["ws"] = M.alloc_int8_workspace(M.grouped_ffn_int8_workspace_size(cfg))
    return cfg, st


def experts64(cfg, st, gates=True):
    T, k, E, S, d = cfg.T, cfg.top_k, cfg.E, cfg.n_shared, cfg.d
    q, s = (torch.from_numpy(v).double().cuda() for v in rows32(st["x"].float().cpu().numpy()))
    s = s[:, None]
    y = torch.full(((k + S) * T, d), float("nan"), dtype=torch.float64, device="cuda")
    off = st["offsets"].tolist()
    for e in range(E):
        slot = st["perm_slot"][off[e]:off[e + 1]].long()
        if slot.numel():
            z = expert64(q[slot // k], s[slot // k], st["gate"], st["up"], st["down"], e)
            y[slot] = z * st["topk_w"].reshape(-1)[slot, None].double() if gates else z
    for j in range(S):
        y[(k + j) * T:(k + j + 1) * T] = expert64(q, s, st["sh_gate"], st["sh_up"],
                                                  st["sh_down"], j)
    return y


def check(y, want):
    y = y.double()
    there = ~torch.isnan(want)
    assert torch.equal(torch.isnan(y), ~there)            # dropped slots' rows are not written
    if there.any():
        off = (y - want)[there]
        assert off.norm() <= 5e-3 * want[there].norm()
        assert off.abs().max() <= 5e-2 * want[there].abs().max()


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,E,k,f,S,cap", [
    (1, 64, 4, 2, 64, 0, 0), (1, 256, 8, 2, 192, 1, 0), (3, 128, 1, 1, 128, 2, 0),
    (7, 192, 16, 4, 320, 1, 0), (16, 512, 8, 8, 256, 0, 0), (64, 256, 32, 2, 128, 1, 2),
    (130, 448, 5, 3, 384, 1, 60), (300, 256, 4, 2, 256, 0, 0), (520, 128, 2, 1, 576, 4, 200),
    (1000, 320, 7, 2, 192, 2, 0), (40, 448, 32, 2, 640, 2, 0), (90, 704, 16, 4, 448, 1, 30),
    (200, 320, 24, 4, 576, 0, 0), (13, 1088, 8, 8, 832, 0, 0)])
def test_experts(T, d, E, k, f, S, cap):
    cfg, st = layer(T, d, E, k, f, S, cap, seed=T + d)
    y = torch.full(((k + S) * T, d), float("nan"), dtype=torch.float16, device="cuda")
    M.grouped_ffn_int8(cfg, st["x"], st["perm_slot"], st["offsets"], st["topk_w"], st["weights"], y,
                       st["ws"])
    assert M.device_status(st["ws"]) == 0
    check(y, experts64(cfg, st))
    # every gate 1, and the same bits from a second call on the same workspace
    outs = []
    for _ in range(2):
        z = torch.full_like(y, float("nan"))
        M.grouped_ffn_int8(cfg, st["x"], st["perm_slot"], st["offsets"], None, st["weights"], z,
                           st["ws"])
        outs.append(z)
    check(outs[0], experts64(cfg, st, gates=False))
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 4, 5, 8, 9])
@pytest.mark.parametrize("E,k,S", [(256, 8, 1), (8, 3, 4), (40, 2, 0)])
def test_experts_of_few_tokens(T, E, k, S):
    cfg, st = layer(T, 192, E, k, 128, S, 0, seed=T + E)
    y = torch.full(((k + S) * T, 192), float("nan"), dtype=torch.float16, device="cuda")
    M.grouped_ffn_int8(cfg, st["x"], st["perm_slot"], st["offsets"], st["topk_w"], st["weights"], y,
                       st["ws"])
    assert M.device_status(st["ws"]) == 0
    check(y, experts64(cfg, st))


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,E,k,f,S,cap", [
    (1200, 1280, 8, 2, 640, 1, 0), (1700, 1088, 12, 2, 896, 0, 250)])
def test_experts_of_tall_row_tiles(T, d, E, k, f, S, cap):
    cfg, st = layer(T, d, E, k, f, S, cap, seed=T)
    y = torch.full(((k + S) * T, d), float("nan"), dtype=torch.float16, device="cuda")
    M.grouped_ffn_int8(cfg, st["x"], st["perm_slot"], st["offsets"], st["topk_w"], st["weights"], y,
                       st["ws"])
    assert M.device_status(st["ws"]) == 0
    check(y, experts64(cfg, st))


@pytest.mark.gpu
def test_every_token_on_one_expert():
    cfg, st = layer(200, 128, 16, 1, 128, 0, 0, seed=1, one_expert=True)
    y = torch.full((200, 128), float("nan"), dtype=torch.float16, device="cuda")
    M.grouped_ffn_int8(cfg, st["x"], st["perm_slot"], st["offsets"], st["topk_w"], st["weights"], y,
                       st["ws"])
    check(y, experts64(cfg, st))


@pytest.mark.gpu
def test_zero_rows_nan_rows_and_range():
    cfg, st = layer(20, 128, 4, 2, 128, 1, 0, seed=3)
    st["x"][4] = 0
    st["x"][5, 3] = float("nan")
    y = torch.zeros(60, 128, dtype=torch.float16, device="cuda")
    M.grouped_ffn_int8(cfg, st["x"], st["perm_slot"], st["offsets"], st["topk_w"], st["weights"], y,
                       st["ws"])
    status = M.device_status(st["ws"])
    assert (y[8:10] == 0).all() and (y[44] == 0).all()
    assert torch.isnan(y[10:12]).all() and torch.isnan(y[45]).all()
    others = [r for r in range(60) if r not in (10, 11, 45)]
    assert torch.isfinite(y[others]).all() and status == M.DEVFAULT_FP16_RANGE
    # activations that take the outputs past fp16's range are clamped and reported
    st["x"] = (torch.randn(20, 128, generator=gen(1)) * 2.0 ** 12).to(torch.bfloat16).cuda()
    M.grouped_ffn_int8(cfg, st["x"], st["perm_slot"], st["offsets"], st["topk_w"], st["weights"], y,
                       st["ws"])
    assert M.device_status(st["ws"]) == M.DEVFAULT_FP16_RANGE and torch.isfinite(y).all()


@pytest.mark.gpu
def test_on_another_stream_and_in_a_graph():
    cfg, st = layer(64, 256, 8, 2, 128, 1, 0, seed=4)

    def call(y):
        M.grouped_ffn_int8(cfg, st["x"], st["perm_slot"], st["offsets"], st["topk_w"],
                           st["weights"], y, st["ws"])

    first = torch.zeros(192, 256, dtype=torch.float16, device="cuda")
    call(first)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = torch.zeros_like(first)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(other)
    side.synchronize()
    assert torch.equal(first, other)
    replay = torch.zeros_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(replay)
    replay.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, replay)


@pytest.mark.gpu
def test_bad_dispatch_is_reported_and_contained():
    cfg, st = layer(32, 128, 4, 2, 128, 0, 0, seed=5)
    perm = st["perm_slot"].clone()
    perm[3], perm[40] = -1, 64
    y = torch.full((64, 128), float("nan"), dtype=torch.float16, device="cuda")
    M.grouped_ffn_int8(cfg, st["x"], perm, st["offsets"], st["topk_w"], st["weights"], y, st["ws"])
    assert M.device_status(st["ws"]) & M.DEVFAULT_BAD_TILE
    want = experts64(cfg, st)
    lost = st["perm_slot"][[3, 40]].long()
    assert torch.isnan(y[lost]).all()
    want[lost] = float("nan")
    check(y, want)


@pytest.mark.gpu
def test_wrong_tensors_are_refused():
    cfg, st = layer(8, 128, 4, 2, 128, 0, 0, seed=6)
    y = torch.zeros(16, 128, dtype=torch.float16, device="cuda")
    a = [st["x"], st["perm_slot"], st["offsets"], st["topk_w"], st["weights"], y]
    for i, bad in ((0, st["x"].float()), (0, st["x"][:, :64]), (1, st["perm_slot"].long()),
                   (2, st["offsets"][:-1]), (5, y.float()), (5, y[:8]), (0, st["x"].cpu())):
        b = list(a)
        b[i] = bad
        with pytest.raises(ValueError):
            M.grouped_ffn_int8(cfg, *b, st["ws"])
    few = (st["gate"][0][:2], st["gate"][1][:2])         # two experts' weights for four
    with pytest.raises(ValueError):
        M.grouped_ffn_int8(cfg, *a[:4], M.make_int8_weights(few, st["up"], st["down"]), y, st["ws"])
    with pytest.raises(M.MoeError):
        M.grouped_ffn_int8(cfg, *a, st["ws"][:1024])
    q, s = torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    with pytest.raises(ValueError):
        M.quantize_rows(torch.zeros(64, 4, device="cuda").t(), q, s)
    with pytest.raises(ValueError):
        M.quantize_rows(torch.zeros(4, 64, dtype=torch.float64, device="cuda"), q, s)
    with pytest.raises(ValueError):
        M.int8_matmul(q, s, q[None].float(), s[None], None, torch.zeros(4, 4, device="cuda"), y)
