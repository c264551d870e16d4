"""Python binding of libmoe_gb300.so (the C ABI in include/moe.h).

Argument marshalling only: every function forwards torch tensors' device pointers and the
current CUDA stream to the entry point of the same name; all computation runs in the library's
CUDA kernels. There is no fallback: if the library is missing the first call raises.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_gb300.so")

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
                3: "MOE_ERR_WORKSPACE", 4: "MOE_ERR_CUDA", 5: "MOE_ERR_DEVICE_FAULT"}
ROUTE_PLAIN, ROUTE_BIAS_SELECT, ROUTE_GUMBEL = 0, 1, 2
DEVFAULT_BAD_EXPERT_INDEX, DEVFAULT_PIPELINE_TIMEOUT, DEVFAULT_BAD_TILE = 0x1, 0x2, 0x4
DEVFAULT_FP16_RANGE = 0x8
Y_F16, Y_F32 = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
DTYPE_F32, DTYPE_BF16, DTYPE_F16 = 0, 1, 2
NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2

EXPORTS = ("moe_workspace_size", "moe_workspace_init", "moe_prepare_router", "moe_route",
           "moe_permute", "moe_permute_noalloc", "moe_overflow_reroute", "moe_grouped_ffn",
           "moe_grouped_ffn_quantized", "moe_quantize_weights", "moe_combine",
           "moe_layer_forward", "moe_layer_forward_profiled", "moe_layer_forward_host",
           "moe_pack_f16", "moe_bias_update", "moe_route_logits", "moe_route_logits_backward",
           "moe_quantize_rows", "moe_quantize_channels", "moe_int8_matmul_workspace_size",
           "moe_int8_matmul", "moe_grouped_ffn_int8_workspace_size", "moe_grouped_ffn_int8",
           "moe_few_workspace_size", "moe_layer_forward_few", "moe_experts_few",
           "moe_residual_norm", "moe_residual_norm_workspace_size", "moe_residual_norm_backward",
           "moe_dropout",
            "moe_check_bounded_waits", "moe_check_few_waits", "moe_device_status",
           "moe_status_string")


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


class MoeConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("n_shared", ctypes.c_int32), ("mode", ctypes.c_int32), ("tau", ctypes.c_float),
                ("capacity_factor", ctypes.c_float), ("capacity_override", ctypes.c_int32),
                ("n_groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("overflow_reroute", ctypes.c_int32), ("weight_bits", ctypes.c_int32)]

    @classmethod
    def make(cls, T, d, E, top_k, d_ff, n_shared=0, mode=ROUTE_PLAIN, tau=1.0,
             capacity_factor=0.0, capacity_override=0, n_groups=0, topk_groups=0,
             overflow_reroute=0, weight_bits=0):
        return cls(T, d, E, top_k, d_ff, n_shared, mode, tau, capacity_factor, capacity_override,
                   n_groups, topk_groups, int(bool(overflow_reroute)), weight_bits)

    @classmethod
    def from_layer(cls, c):
        """From any object with T, d, E, k, f, S, mode, tau, capacity_factor (and optionally
        n_groups, topk_groups, reroute, weight_bits) attributes."""
        return cls.make(c.T, c.d, c.E, c.k, c.f, c.S, c.mode, c.tau, c.capacity_factor,
                        n_groups=getattr(c, "n_groups", 0),
                        topk_groups=getattr(c, "topk_groups", 0),
                        overflow_reroute=getattr(c, "reroute", False),
                        weight_bits=getattr(c, "weight_bits", 0))


class MoeQMatrix(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("zero", ctypes.c_void_p)]


class MoeQWeights(ctypes.Structure):
    _fields_ = [(n, MoeQMatrix) for n in ("gate", "up", "down", "sh_gate", "sh_up", "sh_down")]


class _Holding(ctypes.Structure):
    """Addresses, with the tensors that some of them are of in `_tensors`: a field set anew lets its tensor go."""

    def __setattr__(self, name, value):
        held = self.__dict__.get("_tensors")
        if held is not None and name in held:
            held[name] = None
            self.__dict__.pop("_fit", None)
        super().__setattr__(name, value)


class MoeWeights(_Holding):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("W_g", "expert_bias", "W_gate", "W_up", "W_down", "Wsh_gate", "Wsh_up",
                 "Wsh_down", "W_down_f16", "Wsh_down_f16")] + \
        [("quant", ctypes.POINTER(MoeQWeights)), ("W_g_t", ctypes.c_void_p)]


class MoeRouteOut(_Holding):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("topk_idx", "topk_w", "counts", "offsets", "perm_slot", "slot_pos")]


class GateConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "E", "top_k", "score", "n_groups", "topk_groups", "group_top2",
                 "renormalize")] + \
        [("scale", ctypes.c_float), ("dtype", ctypes.c_int32), ("ld", ctypes.c_int64)]

    @classmethod
    def make(cls, T, E, top_k, score=SCORE_SOFTMAX, n_groups=0, topk_groups=0, group_top2=False,
             renormalize=True, scale=1.0, dtype=DTYPE_F32, ld=0):
        return cls(T, E, top_k, score, n_groups, topk_groups, int(bool(group_top2)),
                   int(bool(renormalize)), scale, dtype, ld)


class ResidualNormConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "d", "after", "before", "h_dtype", "y_dtype", "w_dtype", "gate_rows")] + \
        [(n, ctypes.c_float) for n in ("eps", "alpha", "beta", "p_drop")] + \
        [(n, ctypes.c_int64) for n in ("ld_h", "ld_y")]

    @classmethod
    def make(cls, T, d, after=NORM_NONE, before=NORM_RMS, h_dtype=DTYPE_BF16, y_dtype=DTYPE_BF16,
             w_dtype=DTYPE_BF16, gate_rows=0, eps=1e-6, alpha=1.0, beta=1.0, p_drop=0.0, ld_h=0,
             ld_y=0):
        return cls(T, d, after, before, h_dtype, y_dtype, w_dtype, gate_rows, eps, alpha, beta, p_drop,
                   ld_h, ld_y)


class _NormParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w_after", "b_after", "gate", "w_before", "b_before",
                                               "rng")]


class _NormGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w_after", "b_after", "gate", "w_before", "b_before")]


class MoeInt8Matrix(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


class MoeInt8Weights(ctypes.Structure):
    _names = ("gate", "up", "down", "sh_gate", "sh_up", "sh_down")
    _fields_ = [(n, MoeInt8Matrix) for n in _names]


_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m sparse_moe_layer_route_gb300._build`")
        L = ctypes.CDLL(LIB_PATH)
        P, S, I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        cfgp = ctypes.POINTER(MoeConfig)
        L.moe_workspace_size.argtypes = [cfgp, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_workspace_init.argtypes = [P, S, P]
        L.moe_prepare_router.argtypes = [ctypes.c_int32, ctypes.c_int32, P, P, P]
        L.moe_route.argtypes = [cfgp, P, P, P, P, P, P, P, P, S, P]
        L.moe_permute.argtypes = [cfgp, P, P, P, P, P, P, S, P]
        L.moe_permute_noalloc.argtypes = [cfgp, P, P, P, P, P, P, P]
        L.moe_overflow_reroute.argtypes = [cfgp, P, P, P, P, P, P, P, P, P, S, P]
        i32 = ctypes.c_int32
        L.moe_quantize_weights.argtypes = [i32, i32, i32, i32, P, P, P, P, P]
        L.moe_grouped_ffn_quantized.argtypes = [cfgp, P, P, P, P, ctypes.POINTER(MoeQWeights),
                                                P, P, S, P]
        L.moe_grouped_ffn.argtypes = [cfgp, P, P, P, P, P, P, P, P, P, P, P, P, P, P, S, P]
        L.moe_combine.argtypes = [cfgp, P, ctypes.c_int32, P, P, P, S, P]
        L.moe_layer_forward.argtypes = [cfgp, ctypes.POINTER(MoeWeights), P, P, P,
                                        ctypes.POINTER(MoeRouteOut), P, S, P]
        L.moe_layer_forward_profiled.argtypes = [cfgp, ctypes.POINTER(MoeWeights), P, P, P,
                                                 ctypes.POINTER(MoeRouteOut), P, S, P,
                                                 ctypes.POINTER(ctypes.c_void_p), I]
        L.moe_layer_forward_host.argtypes = [cfgp, ctypes.POINTER(MoeWeights), P, P, P, P, S, P]
        L.moe_pack_f16.argtypes = [P, P, S, P, P]
        L.moe_bias_update.argtypes = [ctypes.c_int32, P, P, ctypes.c_float, ctypes.c_float, P]
        L.moe_device_status.argtypes = [P, P, ctypes.POINTER(ctypes.c_int32)]
        L.moe_check_bounded_waits.argtypes = [ctypes.c_int64, P, P, S, P]
        L.moe_check_few_waits.argtypes = [cfgp, ctypes.POINTER(MoeWeights), P, P, P, P, S, ctypes.c_int32,
                                          ctypes.c_int64, P]
        gcfgp, i64 = ctypes.POINTER(GateConfig), ctypes.c_int64
        L.moe_route_logits.argtypes = [gcfgp, P, P, P, P, P, P]
        L.moe_route_logits_backward.argtypes = [gcfgp, P, P, P, P, P, P]
        L.moe_quantize_rows.argtypes = [i32, i32, i32, P, i64, P, P, P]
        L.moe_quantize_channels.argtypes = [i32, i32, i32, P, P, P, P]
        L.moe_int8_matmul_workspace_size.argtypes = [i32, i32, i32, i32,
                                                     ctypes.POINTER(ctypes.c_size_t)]
        L.moe_int8_matmul.argtypes = [i32, i32, i32, i32, P, P, P, P, P, i32, P, P, S, P]
        L.moe_grouped_ffn_int8_workspace_size.argtypes = [cfgp, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_grouped_ffn_int8.argtypes = [cfgp, P, P, P, P, ctypes.POINTER(MoeInt8Weights), P, P,
                                           S, P]
        L.moe_few_workspace_size.argtypes = [cfgp, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_layer_forward_few.argtypes = [cfgp, ctypes.POINTER(MoeWeights), P, P, P,
                                            ctypes.POINTER(MoeRouteOut), P, S, P]
        L.moe_experts_few.argtypes = [cfgp, ctypes.POINTER(MoeWeights), P, P, P, P, P, S, P]
        normp, paramp = ctypes.POINTER(ResidualNormConfig), ctypes.POINTER(_NormParams)
        L.moe_residual_norm.argtypes = [normp, P, P, paramp, P, P, P]
        L.moe_residual_norm_workspace_size.argtypes = [normp, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_residual_norm_backward.argtypes = [normp, P, P, P, P, paramp, P, P,
                                                 ctypes.POINTER(_NormGrads), P, S, P]
        L.moe_dropout.argtypes = [i32, i32, i32, P, i64, ctypes.c_float, P, P, i64, P, P]
        L.moe_status_string.argtypes = [I]
        L.moe_status_string.restype = ctypes.c_char_p
        for name in EXPORTS:
            if name != "moe_status_string":
                getattr(L, name).restype = I
        _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(status, where):
    if status != MOE_OK:
        raise MoeError(status, where)


def status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def workspace_size(cfg: MoeConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_workspace_size(ctypes.byref(cfg), ctypes.byref(n)), "moe_workspace_size")
    return n.value


def alloc_workspace(cfg: MoeConfig, device="cuda"):
    """A workspace tensor of the right size (torch allocates; 256-byte aligned) with its status
    word cleared."""
    import torch
    ws = torch.empty(workspace_size(cfg), dtype=torch.uint8, device=device)
    workspace_init(ws)
    return ws


def workspace_init(ws, stream=None):
    _check(lib().moe_workspace_init(_ptr(ws), ws.numel(), _stream(stream)), "moe_workspace_init")


def prepare_router(W_g, W_g_t=None, stream=None):
    """W_g [d, E] bf16 transposed into W_g_t [E, d] (a new tensor unless given); one-time."""
    import torch
    d, E = W_g.shape
    if W_g_t is None:
        W_g_t = torch.empty((E, d), dtype=W_g.dtype, device=W_g.device)
    _check(lib().moe_prepare_router(d, E, _ptr(W_g), _ptr(W_g_t), _stream(stream)),
           "moe_prepare_router")
    return W_g_t


def route(cfg, x, W_g, expert_bias, gumbel_u, topk_idx, topk_w, ws, stream=None, W_g_t=None):
    _check(lib().moe_route(ctypes.byref(cfg), _ptr(x), _ptr(W_g), _ptr(W_g_t), _ptr(expert_bias),
                           _ptr(gumbel_u), _ptr(topk_idx), _ptr(topk_w), _ptr(ws), ws.numel(),
                           _stream(stream)), "moe_route")


def permute(cfg, topk_idx, counts, offsets, perm_slot, slot_pos, ws, stream=None):
    _check(lib().moe_permute(ctypes.byref(cfg), _ptr(topk_idx), _ptr(counts), _ptr(offsets),
                             _ptr(perm_slot), _ptr(slot_pos), _ptr(ws), ws.numel(),
                             _stream(stream)), "moe_permute")


NOALLOC_MAX_SLOTS = 262144


def permute_noalloc(cfg, topk_idx, counts, offsets, perm_slot, slot_pos, fault_bits=None,
                    stream=None):
    """moe_permute without a workspace, for callers that cannot allocate device memory: the
    library's own static device array holds the scratch (shared by every call; calls that
    overlap on the GPU race). fault_bits: optional int32 device tensor of one element."""
    _check(lib().moe_permute_noalloc(ctypes.byref(cfg), _ptr(topk_idx), _ptr(counts),
                                     _ptr(offsets), _ptr(perm_slot), _ptr(slot_pos),
                                     _ptr(fault_bits), _stream(stream)), "moe_permute_noalloc")


def overflow_reroute(cfg, x, expert_bias, gumbel_u, topk_idx, topk_w, counts, slot_pos, ws,
                     stream=None, W_g_t=None):
    _check(lib().moe_overflow_reroute(ctypes.byref(cfg), _ptr(x), _ptr(W_g_t), _ptr(expert_bias),
                                      _ptr(gumbel_u), _ptr(topk_idx), _ptr(topk_w), _ptr(counts),
                                      _ptr(slot_pos), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_overflow_reroute")


def grouped_ffn(cfg, x, perm_slot, offsets, topk_w, W_gate, W_up, W_down, Wsh_gate, Wsh_up,
                Wsh_down, y_slot, ws, stream=None, W_down_f16=None, Wsh_down_f16=None):
    """y_slot [T*k + S*T, d]: float16 on the fp16 down path (W_down_f16 given), float32 on the
    bf16 down path."""
    _check(lib().moe_grouped_ffn(ctypes.byref(cfg), _ptr(x), _ptr(perm_slot), _ptr(offsets),
                                 _ptr(topk_w), _ptr(W_gate), _ptr(W_up), _ptr(W_down),
                                 _ptr(Wsh_gate), _ptr(Wsh_up), _ptr(Wsh_down),
                                 _ptr(W_down_f16), _ptr(Wsh_down_f16), _ptr(y_slot),
                                 _ptr(ws), ws.numel(), _stream(stream)), "moe_grouped_ffn")


QUANT_GROUP = 128


def quantize_weights(W, bits, stream=None):
    """Group-wise quantization of bf16 weights W [n, K, N] (or [K, N]) on W's device; returns
    a dict with q (uint8, fragment order), scale (fp16 [n, K/128, N]) and zero (uint8, same)."""
    import torch
    shp = tuple(W.shape)
    n_mat = 1 if len(shp) == 2 else shp[0]
    K, N = shp[-2], shp[-1]
    dev = W.device
    q = torch.empty(n_mat * K * N * bits // 8, dtype=torch.uint8, device=dev)
    sc = torch.empty((n_mat, K // QUANT_GROUP, N), dtype=torch.float16, device=dev)
    z = torch.empty((n_mat, K // QUANT_GROUP, N), dtype=torch.uint8, device=dev)
    _check(lib().moe_quantize_weights(bits, n_mat, K, N, _ptr(W), _ptr(q), _ptr(sc), _ptr(z),
                                      _stream(stream)), "moe_quantize_weights")
    return {"q": q, "scale": sc, "zero": z, "bits": bits, "shape": (n_mat, K, N)}


def make_qweights(gate, up, down, sh_gate=None, sh_up=None, sh_down=None) -> MoeQWeights:
    """From quantize_weights() results (keep those tensors alive while the struct is used)."""
    def m(d):
        return MoeQMatrix(None, None, None) if d is None else \
            MoeQMatrix(_ptr(d["q"]), _ptr(d["scale"]), _ptr(d["zero"]))
    return MoeQWeights(m(gate), m(up), m(down), m(sh_gate), m(sh_up), m(sh_down))


def grouped_ffn_quantized(cfg, x, perm_slot, offsets, topk_w, qweights: MoeQWeights, y_slot,
                          ws, stream=None):
    _check(lib().moe_grouped_ffn_quantized(ctypes.byref(cfg), _ptr(x), _ptr(perm_slot),
                                           _ptr(offsets), _ptr(topk_w), ctypes.byref(qweights),
                                           _ptr(y_slot), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_grouped_ffn_quantized")


def pack_f16(src_bf16, dst_f16, stream=None, fault_bits=None):
    """dst (int16/float16 tensor) = fp16 re-encoding of the bf16 tensor src (same shape).
    fault_bits: optional int32 device tensor into which DEVFAULT_FP16_RANGE is OR-ed when a
    weight had to be clamped."""
    assert src_bf16.numel() == dst_f16.numel()
    _check(lib().moe_pack_f16(_ptr(src_bf16), _ptr(dst_f16), src_bf16.numel(), _ptr(fault_bits),
                              _stream(stream)), "moe_pack_f16")


def packed_f16(src_bf16, stream=None, fault_bits=None):
    """A new float16 tensor holding the fp16 re-encoding of src (torch allocates)."""
    import torch
    dst = torch.empty(src_bf16.shape, dtype=torch.float16, device=src_bf16.device)
    pack_f16(src_bf16, dst, stream, fault_bits)
    return dst


def combine(cfg, y_slot, slot_pos, out, ws, stream=None):
    """y_slot: float16 or float32 slot rows (its dtype selects MOE_Y_F16 / MOE_Y_F32)."""
    import torch
    y_type = Y_F32 if y_slot.dtype == torch.float32 else Y_F16
    _check(lib().moe_combine(ctypes.byref(cfg), _ptr(y_slot), y_type, _ptr(slot_pos), _ptr(out),
                             _ptr(ws), ws.numel(), _stream(stream)), "moe_combine")


def make_weights(W_g, expert_bias, W_gate, W_up, W_down, Wsh_gate=None, Wsh_up=None,
                 Wsh_down=None, W_down_f16=None, Wsh_down_f16=None,
                 quant: MoeQWeights | None = None, W_g_t=None) -> MoeWeights:
    """The weights' addresses. The struct holds the tensors: their memory stays as long as it does, and the few-token
    entry points check them. An address that the program sets in a field itself is its own affair: it is not checked, the
    program keeps its memory, and the tensor that was there is let go."""
    w = MoeWeights(*[_ptr(t) for t in (W_g, expert_bias, W_gate, W_up, W_down, Wsh_gate,
                                        Wsh_up, Wsh_down, W_down_f16, Wsh_down_f16)])
    w.W_g_t = _ptr(W_g_t)
    w._tensors = dict(W_g=W_g, expert_bias=expert_bias, W_gate=W_gate, W_up=W_up, W_down=W_down,
                      Wsh_gate=Wsh_gate, Wsh_up=Wsh_up, Wsh_down=Wsh_down, W_g_t=W_g_t,
                      W_down_f16=W_down_f16, Wsh_down_f16=Wsh_down_f16)
    if quant is not None:
        w.quant = ctypes.pointer(quant)
        w._quant_ref = quant          # keep the struct alive with the weights
    return w


def make_route_out(topk_idx=None, topk_w=None, counts=None, offsets=None, perm_slot=None,
                   slot_pos=None) -> MoeRouteOut:
    """The struct holds its tensors as make_weights' does."""
    tensors = (topk_idx, topk_w, counts, offsets, perm_slot, slot_pos)
    r = MoeRouteOut(*[_ptr(t) for t in tensors])
    r._tensors = {name: t for (name, _), t in zip(MoeRouteOut._fields_, tensors)}
    return r


def layer_forward(cfg, weights: MoeWeights, x, gumbel_u, out, route_out: MoeRouteOut | None,
                  ws, stream=None):
    _check(lib().moe_layer_forward(ctypes.byref(cfg), ctypes.byref(weights), _ptr(x),
                                   _ptr(gumbel_u), _ptr(out),
                                   ctypes.byref(route_out) if route_out is not None else None,
                                   _ptr(ws), ws.numel(), _stream(stream)), "moe_layer_forward")


PROFILE_PHASES = ("router", "dispatch", "tiles_gather", "gate_up_gemm", "down_gemm", "combine")


def layer_forward_profiled(cfg, weights: MoeWeights, x, gumbel_u, out, route_out, ws, events,
                           stream=None):
    """layer_forward recording the 7 torch.cuda.Event objects in `events` at the phase
    boundaries (PROFILE_PHASES lie between consecutive events)."""
    for e in events:
        if not e.cuda_event:      # torch creates the CUDA event on its first record
            e.record()
    arr = (ctypes.c_void_p * 7)(*[e.cuda_event for e in events])
    _check(lib().moe_layer_forward_profiled(
        ctypes.byref(cfg), ctypes.byref(weights), _ptr(x), _ptr(gumbel_u), _ptr(out),
        ctypes.byref(route_out) if route_out is not None else None, _ptr(ws), ws.numel(),
        _stream(stream), arr, 7), "moe_layer_forward_profiled")


def layer_forward_host(cfg, weights: MoeWeights, x_host, gumbel_u_host, out_host, ws,
                       stream=None):
    _check(lib().moe_layer_forward_host(ctypes.byref(cfg), ctypes.byref(weights), _ptr(x_host),
                                        _ptr(gumbel_u_host), _ptr(out_host), _ptr(ws),
                                        ws.numel(), _stream(stream)), "moe_layer_forward_host")


def bias_update(counts, expert_bias, decay=0.99, rate=0.01, stream=None):
    """In place: expert_bias <- decay*expert_bias - rate*counts/(mean(counts)+1e-8)."""
    _check(lib().moe_bias_update(expert_bias.numel(), _ptr(counts), _ptr(expert_bias), decay, rate,
                                 _stream(stream)), "moe_bias_update")


class _Torch:
    """What the tensor checks need of torch, looked up once (the module loads without torch)."""

    def __init__(self):
        import torch
        self.f32, self.bf16, self.f16 = torch.float32, torch.bfloat16, torch.float16
        self.i8, self.i32, self.i64 = torch.int8, torch.int32, torch.int64
        self.code = {self.f32: DTYPE_F32, self.bf16: DTYPE_BF16, self.f16: DTYPE_F16}
        self.dtype = {code: dtype for dtype, code in self.code.items()}
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


_torch_names = None


def _names() -> _Torch:
    global _torch_names
    if _torch_names is None:
        _torch_names = _Torch()
    return _torch_names


def _stream_on(stream, gpu, names):
    """The raw handle of `stream`, or of the current stream of the current GPU, number `gpu`."""
    if stream is None and names.raw_stream is not None:
        return names.raw_stream(gpu)
    return _stream(stream)


def _allocating_for(stream):
    """A context in which torch allocates for `stream`, so that its kernels may write to the memory at
    once: the current stream's allocations may still be written to by what that stream has enqueued."""
    import contextlib

    import torch
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _current_gpu(where, name, t, names):
    """The current GPU's number; launches go there, so tensor t, and with it all others, has to be
    there too."""
    gpu = t.get_device()
    if gpu < 0 or gpu != names.current_device():
        raise ValueError(f"{where}: {name} is on {t.device}, which is not the current GPU")
    return gpu


def _dtype_code(t, where):
    code = _names().code.get(t.dtype)
    if code is None:
        raise ValueError(f"{where}: element type {t.dtype} is not supported")
    return code


def _expect(where, name, t, shape, dtype, gpu):
    """t: a contiguous tensor of this shape and element type on GPU `gpu`. Its address."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != gpu or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be a contiguous tensor {dtype} {shape} on cuda:{gpu}, "
                         f"not {t.dtype} {tuple(t.shape)} (strides {t.stride()}) on {t.device}")
    return t.data_ptr()


def _expect_int32(where, **sizes):
    """Sizes that the library takes as 32-bit numbers: past their range they would arrive as others."""
    for name, n in sizes.items():
        if n >= 2 ** 31:
            raise ValueError(f"{where}: {name} = {n} is not below 2^31")


def _expect_ws(where, ws, gpu):
    """ws: a tensor whose elements fill their memory on GPU `gpu`. Its address and bytes."""
    if ws.get_device() != gpu or not ws.is_contiguous():
        raise ValueError(f"{where}: ws must be a contiguous tensor on cuda:{gpu}, not "
                         f"{tuple(ws.shape)} (strides {ws.stride()}) on {ws.device}")
    return ws.data_ptr(), ws.nbytes


def _expect_logits(where, gcfg, T, E, logits):
    if logits.shape != (T, E) or \
            _names().code.get(logits.dtype) != gcfg.dtype or \
            logits.stride() != (gcfg.ld or E, 1) and not (
                (T <= 1 or logits.stride(0) == (gcfg.ld or E)) and
                (E <= 1 or logits.stride(1) == 1)):
        raise ValueError(f"{where}: logits {logits.dtype} {tuple(logits.shape)} (strides "
                         f"{logits.stride()}) on {logits.device} do not fit the configuration")
    return logits.data_ptr()


def route_logits(gcfg: GateConfig, logits, expert_bias, topk_idx, topk_w, scores=None, stream=None):
    """Experts and weights from given router logits [T, E] (see moe_route_logits); scores: optional
    fp32 [T, E] that receives every expert's score."""
    w, T, E, k, n = "moe_route_logits", gcfg.T, gcfg.E, gcfg.top_k, _names()
    gpu = _current_gpu(w, "logits", logits, n)
    _check(lib().moe_route_logits(
        ctypes.byref(gcfg), _expect_logits(w, gcfg, T, E, logits),
        None if expert_bias is None else _expect(w, "expert_bias", expert_bias, (E,), n.f32, gpu),
        _expect(w, "topk_idx", topk_idx, (T, k), n.i32, gpu),
        _expect(w, "topk_w", topk_w, (T, k), n.f32, gpu),
        None if scores is None else _expect(w, "scores", scores, (T, E), n.f32, gpu),
        _stream_on(stream, gpu, n)), w)


def route_logits_backward(gcfg: GateConfig, logits, topk_idx, d_topk_w, d_scores, d_logits,
                          stream=None):
    """d_logits from the gradients of topk_w and scores (either may be None)."""
    w, T, E, k, n = "moe_route_logits_backward", gcfg.T, gcfg.E, gcfg.top_k, _names()
    gpu = _current_gpu(w, "logits", logits, n)
    _check(lib().moe_route_logits_backward(
        ctypes.byref(gcfg), _expect_logits(w, gcfg, T, E, logits),
        _expect(w, "topk_idx", topk_idx, (T, k), n.i32, gpu),
        None if d_topk_w is None else _expect(w, "d_topk_w", d_topk_w, (T, k), n.f32, gpu),
        None if d_scores is None else _expect(w, "d_scores", d_scores, (T, E), n.f32, gpu),
        _expect(w, "d_logits", d_logits, (T, E), logits.dtype, gpu),
        _stream_on(stream, gpu, n)), w)


def quantize_rows(x, q, scale, stream=None):
    """x [T, d] (fp32, bf16 or fp16; rows may be strided, but not share elements: an expanded row's
    stride of 0 means `contiguous` to the library) to q int8 [T, d] and scale fp32 [T]."""
    w, n = "moe_quantize_rows", _names()
    T, d = x.shape
    _expect_int32(w, T=T, d=d)
    step, unit = x.stride()
    gpu = _current_gpu(w, "x", x, n)
    if (d > 1 and unit != 1) or (T > 1 and step < d):
        raise ValueError(f"{w}: x must have unit stride inside a row and rows at least {d} apart, not "
                         f"strides {x.stride()}")
    _check(lib().moe_quantize_rows(T, d, _dtype_code(x, w), x.data_ptr(), step if T > 1 else d,
                                   _expect(w, "q", q, (T, d), n.i8, gpu),
                                   _expect(w, "scale", scale, (T,), n.f32, gpu),
                                   _stream_on(stream, gpu, n)), w)


def quantize_channels(W, stream=None):
    """One-time preparation of bf16 weights W [n, K, N] (or [K, N]) for the 8-bit products: (q int8
    [n, N, K], scale fp32 [n, N]), new tensors on W's device that belong to `stream`."""
    import torch
    if W.dim() not in (2, 3):
        raise ValueError(f"moe_quantize_channels: W of shape {tuple(W.shape)} is neither [n, K, N] nor "
                         "[K, N]")
    n, (K, N) = (1 if W.dim() == 2 else W.shape[0]), W.shape[-2:]
    _expect_int32("moe_quantize_channels", n=n, K=K, N=N)
    gpu = _current_gpu("moe_quantize_channels", "W", W, _names())
    _expect("moe_quantize_channels", "W", W, tuple(W.shape), torch.bfloat16, gpu)
    with _allocating_for(stream):
        q = torch.empty((n, N, K), dtype=torch.int8, device=W.device)
        scale = torch.empty((n, N), dtype=torch.float32, device=W.device)
    _check(lib().moe_quantize_channels(n, K, N, W.data_ptr(), q.data_ptr(), scale.data_ptr(),
                                       _stream_on(stream, gpu, _names())), "moe_quantize_channels")
    return q, scale


def int8_matmul_workspace_size(rows, K, N, n_mat) -> int:
    """Bytes that products of up to `rows` rows need."""
    n = ctypes.c_size_t(0)
    _expect_int32("moe_int8_matmul_workspace_size", rows=rows, K=K, N=N, n_mat=n_mat)
    _check(lib().moe_int8_matmul_workspace_size(rows, K, N, n_mat, ctypes.byref(n)),
           "moe_int8_matmul_workspace_size")
    return n.value


def grouped_ffn_int8_workspace_size(cfg: MoeConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_grouped_ffn_int8_workspace_size(ctypes.byref(cfg), ctypes.byref(n)),
           "moe_grouped_ffn_int8_workspace_size")
    return n.value


def alloc_int8_workspace(nbytes, device="cuda"):
    """A workspace of nbytes for the 8-bit entry points, its status word cleared."""
    import torch
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.device(ws.device):
        workspace_init(ws)
    return ws


def int8_matmul(q_x, s_x, q_w, s_w, offsets, y, ws, stream=None):
    """y [rows, N] (fp32, bf16 or fp16) = (q_x q_w[e]^T) * s_x * s_w[e] over the row segments of
    offsets (int32 [n + 1] on the device; None: one matrix for every row)."""
    w, t = "moe_int8_matmul", _names()
    rows, K = q_x.shape
    n, N, _ = q_w.shape
    _expect_int32(w, rows=rows, K=K, N=N, n=n)
    gpu = _current_gpu(w, "q_x", q_x, t)
    _check(lib().moe_int8_matmul(
        rows, K, N, n, _expect(w, "q_x", q_x, (rows, K), t.i8, gpu),
        _expect(w, "s_x", s_x, (rows,), t.f32, gpu), _expect(w, "q_w", q_w, (n, N, K), t.i8, gpu),
        _expect(w, "s_w", s_w, (n, N), t.f32, gpu),
        None if offsets is None else _expect(w, "offsets", offsets, (n + 1,), t.i32, gpu),
        _dtype_code(y, w), _expect(w, "y", y, (rows, N), y.dtype, gpu),
        *_expect_ws(w, ws, gpu), _stream_on(stream, gpu, t)), w)


def make_int8_weights(gate, up, down, sh_gate=None, sh_up=None, sh_down=None) -> MoeInt8Weights:
    """From quantize_channels() results (kept alive by the struct), all on one GPU."""
    mats, t, gpu = (gate, up, down, sh_gate, sh_up, sh_down), _names(), gate[0].get_device()
    if not gate[0].is_cuda:
        raise ValueError(f"make_int8_weights: weights on {gate[0].device}")
    for m in mats:
        if m is not None:
            n, N, K = m[0].shape
            _expect("make_int8_weights", "q", m[0], (n, N, K), t.i8, gpu)
            _expect("make_int8_weights", "scale", m[1], (n, N), t.f32, gpu)
    w = MoeInt8Weights(*[MoeInt8Matrix() if m is None else MoeInt8Matrix(_ptr(m[0]), _ptr(m[1]))
                         for m in mats])
    w._tensors, w._gpu = mats, gpu
    w._shapes = tuple(None if m is None else tuple(m[0].shape) for m in mats)
    return w


def grouped_ffn_int8(cfg, x, perm_slot, offsets, topk_w, weights: MoeInt8Weights, y_slot, ws,
                     stream=None):
    """y_slot [T*k + S*T, d] float16: the routed and shared experts on 8-bit weights and
    activations (see moe_grouped_ffn_int8)."""
    w, t = "moe_grouped_ffn_int8", _names()
    T, d, k, E, f, S = cfg.T, cfg.d, cfg.top_k, cfg.E, cfg.d_ff, cfg.n_shared
    into, back = (E, f, d), (E, d, f)
    want = (into, into, back) + (((S, f, d), (S, f, d), (S, d, f)) if S else ())
    gpu = _current_gpu(w, "x", x, t)
    if weights._shapes[:len(want)] != want or weights._gpu != gpu:
        raise ValueError(f"{w}: weights of shapes {weights._shapes} on cuda:{weights._gpu} do not fit "
                         f"the configuration on cuda:{gpu}")
    _check(lib().moe_grouped_ffn_int8(
        ctypes.byref(cfg), _expect(w, "x", x, (T, d), t.bf16, gpu),
        _expect(w, "perm_slot", perm_slot, (T * k,), t.i32, gpu),
        _expect(w, "offsets", offsets, (E + 1,), t.i32, gpu),
        None if topk_w is None else _expect(w, "topk_w", topk_w, (T, k), t.f32, gpu),
        ctypes.byref(weights), _expect(w, "y_slot", y_slot, (T * (k + S), d), t.f16, gpu),
        *_expect_ws(w, ws, gpu), _stream_on(stream, gpu, t)), w)


FEW_MAX_TOKENS = 16


def few_workspace_size(cfg: MoeConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_few_workspace_size(ctypes.byref(cfg), ctypes.byref(n)),
           "moe_few_workspace_size")
    return n.value


def alloc_few_workspace(cfg: MoeConfig, device="cuda"):
    """A workspace for layer_forward_few and experts_few with this configuration, its status word and
    counters cleared."""
    return alloc_int8_workspace(few_workspace_size(cfg), device)


def _expect_experts(where, cfg, weights, gpu, router):
    """The weights' tensors fit the configuration on GPU `gpu` (addresses that the program gave instead of
    tensors are its own affair). Looked at once per configuration."""
    tensors = getattr(weights, "_tensors", None)
    if tensors is None:
        return                        # filled in by hand: addresses alone
    d, E, f, S, t = cfg.d, cfg.E, cfg.d_ff, cfg.n_shared, _names()
    bias = router and cfg.mode == ROUTE_BIAS_SELECT
    fit = weights.__dict__.setdefault("_fit", set())  # configurations that these tensors have been checked against
    key = (d, E, f, S, gpu, router, bias)
    if key in fit:
        return
    want = dict(W_gate=(E, d, f), W_up=(E, d, f), W_down=(E, f, d))
    if S:
        want.update(Wsh_gate=(S, d, f), Wsh_up=(S, d, f), Wsh_down=(S, f, d))
    if router:
        want.update(W_g=(d, E), W_g_t=(E, d))
    for name, shape in want.items():
        m = tensors[name]
        if m is not None and not isinstance(m, int):
            _expect(where, name, m, shape, t.bf16, gpu)
    m = tensors["expert_bias"]
    if bias and m is not None and not isinstance(m, int):
        _expect(where, "expert_bias", m, (E,), t.f32, gpu)
    fit.add(key)


def layer_forward_few(cfg, weights: MoeWeights, x, gumbel_u, out, route_out: MoeRouteOut | None, ws,
                      stream=None):
    """layer_forward for up to FEW_MAX_TOKENS tokens in one kernel (see moe_layer_forward_few), in half its time for
    one token and about the same for sixteen; ws from alloc_few_workspace."""
    w, t = "moe_layer_forward_few", _names()
    T, d, E, k = cfg.T, cfg.d, cfg.E, cfg.top_k
    gpu = _current_gpu(w, "x", x, t)
    _expect_experts(w, cfg, weights, gpu, True)
    if route_out is not None:
        shapes = ((T, k), (T, k), (E,), (E + 1,), (T * k,), (T * k,))
        given = getattr(route_out, "_tensors", {})
        for (name, _), shape in zip(MoeRouteOut._fields_, shapes):
            r = given.get(name)
            if r is not None and not isinstance(r, int):
                _expect(w, name, r, shape, t.f32 if name == "topk_w" else t.i32, gpu)
    _check(lib().moe_layer_forward_few(
        ctypes.byref(cfg), ctypes.byref(weights), _expect(w, "x", x, (T, d), t.bf16, gpu),
        None if gumbel_u is None else _expect(w, "gumbel_u", gumbel_u, (T, E), t.f32, gpu),
        _expect(w, "out", out, (T, d), t.bf16, gpu),
        None if route_out is None else ctypes.byref(route_out), *_expect_ws(w, ws, gpu),
        _stream_on(stream, gpu, t)), w)


def experts_few(cfg, weights: MoeWeights, x, topk_idx, topk_w, out, ws, stream=None):
    """The experts, shared experts and combine of a layer for up to FEW_MAX_TOKENS tokens, with the choice
    topk_idx [T, k] and gates topk_w [T, k] (None: 1) given (see moe_experts_few)."""
    w, t = "moe_experts_few", _names()
    T, d, k = cfg.T, cfg.d, cfg.top_k
    gpu = _current_gpu(w, "x", x, t)
    _expect_experts(w, cfg, weights, gpu, False)
    _check(lib().moe_experts_few(
        ctypes.byref(cfg), ctypes.byref(weights), _expect(w, "x", x, (T, d), t.bf16, gpu),
        _expect(w, "topk_idx", topk_idx, (T, k), t.i32, gpu),
        None if topk_w is None else _expect(w, "topk_w", topk_w, (T, k), t.f32, gpu),
        _expect(w, "out", out, (T, d), t.bf16, gpu), *_expect_ws(w, ws, gpu),
        _stream_on(stream, gpu, t)), w)


def _expect_rows(where, name, t, T, d, ld, dtype, gpu):
    """t [T, d] on GPU `gpu` with unit stride inside a row and rows ld elements apart. Its address."""
    if t.shape != (T, d) or t.dtype is not dtype or t.get_device() != gpu or \
            t.stride() != (ld, 1) and ((d > 1 and t.stride(1) != 1) or (T > 1 and t.stride(0) != ld)):
        raise ValueError(f"{where}: {name} must be a tensor {dtype} {(T, d)} on cuda:{gpu} with strides "
                         f"{(ld, 1)}, not {t.dtype} {tuple(t.shape)} (strides {t.stride()}) on {t.device}")
    return t.data_ptr()


def _norm_params(where, cfg, d, names, gpu, w_after, b_after, gate, w_before, b_before, rng):
    dtype, vector = names.dtype.get(cfg.w_dtype), (d,)
    return _NormParams(
        None if w_after is None else _expect(where, "w_after", w_after, vector, dtype, gpu),
        None if b_after is None else _expect(where, "b_after", b_after, vector, dtype, gpu),
        None if gate is None else _expect(where, "gate", gate, (_gate_count(cfg), d), dtype, gpu),
        None if w_before is None else _expect(where, "w_before", w_before, vector, dtype, gpu),
        None if b_before is None else _expect(where, "b_before", b_before, vector, dtype, gpu),
        None if rng is None else _expect(where, "rng", rng, (2,), names.i64, gpu))


def _gate_count(cfg):
    return -(-cfg.T // cfg.gate_rows) if cfg.gate_rows > 0 else 0


def residual_norm(cfg: ResidualNormConfig, h, y, h_out, n, w_after=None, b_after=None, gate=None,
                  w_before=None, b_before=None, rng=None, stream=None):
    """h_out = alpha h + beta gate drop(norm_after(y)) and n = norm_before(h_out) (see moe_residual_norm); y,
    h_out and n may be None as there. rng: int64 [2] on the GPU, seed and step; every place of dropout needs a
    seed of its own, else it drops what the others drop."""
    w, t = "moe_residual_norm", _names()
    T, d = cfg.T, cfg.d
    gpu = _current_gpu(w, "h", h, t)
    h_type, y_type = t.dtype.get(cfg.h_dtype), t.dtype.get(cfg.y_dtype)
    p = _norm_params(w, cfg, d, t, gpu, w_after, b_after, gate, w_before, b_before, rng)
    _check(lib().moe_residual_norm(
        ctypes.byref(cfg), _expect_rows(w, "h", h, T, d, cfg.ld_h or d, h_type, gpu),
        None if y is None else _expect_rows(w, "y", y, T, d, cfg.ld_y or d, y_type, gpu),
        ctypes.byref(p), None if h_out is None else _expect(w, "h_out", h_out, (T, d), h_type, gpu),
        None if n is None else _expect(w, "n", n, (T, d), y_type, gpu), _stream_on(stream, gpu, t)), w)


def residual_norm_workspace_size(cfg: ResidualNormConfig) -> int:
    """Bytes that the gradient of up to cfg.T tokens needs."""
    n = ctypes.c_size_t(0)
    _check(lib().moe_residual_norm_workspace_size(ctypes.byref(cfg), ctypes.byref(n)),
           "moe_residual_norm_workspace_size")
    return n.value


def residual_norm_backward(cfg: ResidualNormConfig, h_out, y, d_h_out, d_n, d_h, d_y, ws, w_after=None,
                           b_after=None, gate=None, w_before=None, rng=None, d_w_after=None,
                           d_b_after=None, d_gate=None, d_w_before=None, d_b_before=None, stream=None):
    """Gradients of residual_norm (see moe_residual_norm_backward): d_h, d_y and, fp32, those of the
    parameters that are given; h_out (the stream after the block), y, d_h_out, d_n and d_y may be None as
    there."""
    w, t = "moe_residual_norm_backward", _names()
    T, d = cfg.T, cfg.d
    gpu = _current_gpu(w, "d_h", d_h, t)
    h_type, y_type = t.dtype.get(cfg.h_dtype), t.dtype.get(cfg.y_dtype)
    p = _norm_params(w, cfg, d, t, gpu, w_after, b_after, gate, w_before, None, rng)
    vector = (d,)
    g = _NormGrads(
        None if d_w_after is None else _expect(w, "d_w_after", d_w_after, vector, t.f32, gpu),
        None if d_b_after is None else _expect(w, "d_b_after", d_b_after, vector, t.f32, gpu),
        None if d_gate is None else _expect(w, "d_gate", d_gate, (_gate_count(cfg), d), t.f32, gpu),
        None if d_w_before is None else _expect(w, "d_w_before", d_w_before, vector, t.f32, gpu),
        None if d_b_before is None else _expect(w, "d_b_before", d_b_before, vector, t.f32, gpu))
    _check(lib().moe_residual_norm_backward(
        ctypes.byref(cfg),
        None if h_out is None else _expect_rows(w, "h_out", h_out, T, d, cfg.ld_h or d, h_type, gpu),
        None if y is None else _expect_rows(w, "y", y, T, d, cfg.ld_y or d, y_type, gpu),
        None if d_h_out is None else _expect(w, "d_h_out", d_h_out, (T, d), h_type, gpu),
        None if d_n is None else _expect(w, "d_n", d_n, (T, d), y_type, gpu), ctypes.byref(p),
        _expect(w, "d_h", d_h, (T, d), h_type, gpu),
        None if d_y is None else _expect(w, "d_y", d_y, (T, d), y_type, gpu), ctypes.byref(g),
        *_expect_ws(w, ws, gpu), _stream_on(stream, gpu, t)), w)


def dropout(x, p, rng, y, residual=None, stream=None):
    """y [T, d] = residual + x / (1 - p) where the element's number is at least p * 2^32, else residual (0 if
    None); see moe_dropout. rng: int64 [2] on the GPU, seed and step (None where p is 0); every place of
    dropout needs a seed of its own. The gradient to x is the same call on y's."""
    w, t = "moe_dropout", _names()
    if x.dim() != 2:
        raise ValueError(f"{w}: x of shape {tuple(x.shape)} is not [T, d]")
    T, d = x.shape
    _expect_int32(w, T=T, d=d)
    gpu = _current_gpu(w, "x", x, t)
    ld_x, ld_r = (x.stride(0) if T > 1 else d), d
    if ld_x < d:
        raise ValueError(f"{w}: rows of x (strides {x.stride()}) share elements")
    if residual is not None:
        ld_r = residual.stride(0) if T > 1 and residual.dim() == 2 else d
        if ld_r < d:
            raise ValueError(f"{w}: rows of residual (strides {residual.stride()}) share elements")
    _check(lib().moe_dropout(
        T, d, _dtype_code(x, w), _expect_rows(w, "x", x, T, d, ld_x, x.dtype, gpu), ld_x, p,
        None if rng is None else _expect(w, "rng", rng, (2,), t.i64, gpu),
        None if residual is None else _expect_rows(w, "residual", residual, T, d, ld_r, x.dtype, gpu), ld_r,
        _expect(w, "y", y, (T, d), x.dtype, gpu), _stream_on(stream, gpu, t)), w)


def check_bounded_waits(limit_ns, expired, ws, stream=None):
    """Both bounded device waits against conditions that never come true (limit_ns each);
    expired: int32 device tensor of 2. Read the result with device_status()."""
    _check(lib().moe_check_bounded_waits(int(limit_ns), _ptr(expired), _ptr(ws), ws.numel(),
                                         _stream(stream)), "moe_check_bounded_waits")


def check_few_waits(cfg, weights: MoeWeights, x, topk_idx, out, ws, which, limit_ns, stream=None):
    """The waits of experts_few against a condition that never comes true (see moe_check_few_waits): which 0 and 1 the
    grid barriers, 2 a tile of weights. Read the result with device_status()."""
    w, t = "moe_check_few_waits", _names()
    T, d, k = cfg.T, cfg.d, cfg.top_k
    gpu = _current_gpu(w, "x", x, t)
    _expect_experts(w, cfg, weights, gpu, False)
    _check(lib().moe_check_few_waits(
        ctypes.byref(cfg), ctypes.byref(weights), _expect(w, "x", x, (T, d), t.bf16, gpu),
        _expect(w, "topk_idx", topk_idx, (T, k), t.i32, gpu), _expect(w, "out", out, (T, d), t.bf16, gpu),
        *_expect_ws(w, ws, gpu), int(which), int(limit_ns), _stream_on(stream, gpu, t)), w)


def device_status(ws, stream=None) -> int:
    """Synchronises, returns the device fault bits (and clears them)."""
    bits = ctypes.c_int32(0)
    st = lib().moe_device_status(_ptr(ws), _stream(stream), ctypes.byref(bits))
    if st not in (MOE_OK, 5):
        raise MoeError(st, "moe_device_status")
    return bits.value
