"""What the binding of routing from logits and of the 8-bit entry points hands to the library, and what
it refuses before: CPU tensors that say they are on a GPU, and a recorder in the library's place, so
nothing is launched."""
import pytest
import torch

import sparse_moe_layer_route_gb300 as M


class OnGpu:
    """A CPU tensor that says it is on a GPU."""

    is_cuda = True

    def __init__(self, tensor, index=0):
        self._tensor, self._index = tensor, index

    def __getattr__(self, name):
        return getattr(self._tensor, name)

    def get_device(self):
        return self._index

    @property
    def device(self):
        return torch.device("cuda", self._index)


class Recorder:
    """Every entry point succeeds and leaves its arguments in `calls`."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append((name, args))
            return M.MOE_OK
        return entry


@pytest.fixture
def calls(monkeypatch):
    recorder = Recorder()
    monkeypatch.setattr(M, "lib", lambda: recorder)
    monkeypatch.setattr(M._names(), "current_device", lambda: 0, raising=False)
    return recorder.calls


def rows_out(T, d):
    return OnGpu(torch.empty(T, d, dtype=torch.int8)), OnGpu(torch.empty(T))


@pytest.mark.parametrize("x", [torch.zeros(1, 64).expand(1000, 64), torch.zeros(1, 1).expand(9, 1),
                               torch.zeros(200).as_strided((3, 64), (63, 1))])
def test_rows_that_overlap_are_refused(calls, x):
    """A row stride of 0 would reach the library as `contiguous`, and be read far past the row."""
    with pytest.raises(ValueError):
        M.quantize_rows(OnGpu(x), *rows_out(*x.shape), stream=0)
    assert calls == []


@pytest.mark.parametrize("x,ld", [(torch.zeros(5, 64), 64), (torch.zeros(5, 80)[:, :64], 80),
                                  (torch.zeros(5, 3)[:, 1:2], 3), (torch.zeros(1, 64), 64),
                                  (torch.zeros(1, 64).expand(1, 64), 64),
                                  (torch.zeros(0, 64), 64)])
def test_row_strides_of_quantize_rows(calls, x, ld):
    M.quantize_rows(OnGpu(x), *rows_out(*x.shape), stream=0)
    (name, args), = calls
    assert name == "moe_quantize_rows" and args[:2] == tuple(x.shape) and args[4] == ld


def every_call(at, stream=0, odd=None):
    """A call of each entry point with its tensors on GPU `at`, but the one named `odd` on the next."""
    def g(name, *shape, dtype=torch.float32):
        return OnGpu(torch.zeros(*shape, dtype=dtype), at + (name == odd))

    f16, bf16, i8, i32 = torch.float16, torch.bfloat16, torch.int8, torch.int32
    gate = M.GateConfig.make(4, 16, 2)
    cfg = M.MoeConfig.make(8, 128, 4, 2, 64)
    mats = [(g("q", 4, n, k, dtype=i8), g("scale", 4, n)) for n, k in ((64, 128), (64, 128),
                                                                      (128, 64))]
    return {
        "route_logits": lambda: M.route_logits(
            gate, g("logits", 4, 16), g("bias", 16), g("idx", 4, 2, dtype=i32), g("w", 4, 2),
            g("scores", 4, 16), stream=stream),
        "route_logits_backward": lambda: M.route_logits_backward(
            gate, g("logits", 4, 16), g("idx", 4, 2, dtype=i32), g("d_w", 4, 2),
            g("d_scores", 4, 16), g("d_logits", 4, 16), stream=stream),
        "quantize_rows": lambda: M.quantize_rows(
            g("x", 4, 64), g("q", 4, 64, dtype=i8), g("scale", 4), stream=stream),
        "int8_matmul": lambda: M.int8_matmul(
            g("q_x", 4, 64, dtype=i8), g("s_x", 4), g("q_w", 2, 8, 64, dtype=i8), g("s_w", 2, 8),
            g("offsets", 3, dtype=i32), g("y", 4, 8), g("ws", 4096, dtype=torch.uint8),
            stream=stream),
        "grouped_ffn_int8": lambda: M.grouped_ffn_int8(
            cfg, g("x", 8, 128, dtype=bf16), g("perm", 16, dtype=i32), g("offsets", 5, dtype=i32),
            g("w", 8, 2), M.make_int8_weights(*mats), g("y", 16, 128, dtype=f16),
            g("ws", 4096, dtype=torch.uint8), stream=stream),
    }


TENSORS = [(call, odd) for call, names in (
    ("route_logits", "logits bias idx w scores"),
    ("route_logits_backward", "logits idx d_w d_scores d_logits"),
    ("quantize_rows", "x q scale"),
    ("int8_matmul", "q_x s_x q_w s_w offsets y"),
    ("grouped_ffn_int8", "x perm offsets w q scale y")) for odd in names.split()]


@pytest.mark.parametrize("call,odd", TENSORS)
def test_a_tensor_of_another_gpu_is_refused(calls, call, odd):
    """The launch goes to the current GPU, whose kernels would be given another one's addresses."""
    every_call(0)[call]()
    assert [name for name, _ in calls] == ["moe_" + call]
    with pytest.raises(ValueError):
        every_call(0, odd=odd)[call]()
    assert len(calls) == 1


@pytest.mark.parametrize("call", sorted({c for c, _ in TENSORS}))
def test_tensors_of_a_gpu_that_is_not_current_are_refused(calls, monkeypatch, call):
    with pytest.raises(ValueError):
        every_call(1)[call]()
    assert calls == []
    monkeypatch.setattr(M._names(), "current_device", lambda: 1)
    every_call(1)[call]()
    assert len(calls) == 1


@pytest.mark.parametrize("ws", [
    torch.zeros(4096, dtype=torch.uint8), OnGpu(torch.zeros(4096, dtype=torch.uint8), 1),
    OnGpu(torch.zeros(1, dtype=torch.uint8).expand(4096)),
    OnGpu(torch.zeros(8192, dtype=torch.uint8)[::2])])
@pytest.mark.parametrize("call", ["int8_matmul", "grouped_ffn_int8"])
def test_workspaces_that_are_not_bytes_in_a_row_there_are_refused(calls, monkeypatch, call, ws):
    """The library sees an address and a length: host memory, another GPU's, or a view of fewer bytes than
    its elements would be written past."""
    entry = getattr(M, call)
    monkeypatch.setattr(M, call, lambda *a, **kw: entry(*a[:-1], ws, **kw))
    with pytest.raises(ValueError):
        every_call(0)[call]()
    assert calls == []


def test_workspaces_of_any_element_type_count_in_bytes(calls, monkeypatch):
    entry = M.int8_matmul
    ws = OnGpu(torch.zeros(1024))
    monkeypatch.setattr(M, "int8_matmul", lambda *a, **kw: entry(*a[:-1], ws, **kw))
    every_call(0)["int8_matmul"]()
    assert calls[0][1][11:13] == (ws.data_ptr(), 4096)


@pytest.mark.parametrize("shape", [(64,), (2, 3, 64, 32), (1, 2, 2, 16, 8)])
def test_channels_of_one_or_a_row_of_matrices_alone(calls, monkeypatch, shape):
    """Of more dimensions the first would count as the matrices, and the others' be left out."""
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: torch.zeros(*a, **kw))
    monkeypatch.setattr(M._names(), "raw_stream", lambda gpu: 0)
    with pytest.raises(ValueError):
        M.quantize_channels(OnGpu(torch.zeros(*shape, dtype=torch.bfloat16)))
    assert calls == []
    for good in ((64, 32), (3, 64, 32)):
        M.quantize_channels(OnGpu(torch.zeros(*good, dtype=torch.bfloat16)))
    assert [c[1][:3] for c in calls] == [(1, 64, 32), (3, 64, 32)]


def test_a_workspace_is_cleared_on_its_own_gpu(calls, monkeypatch):
    """Not on the current one's stream, which nothing orders before the first call there."""
    entered = []

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            entered.append(self.device)

        def __exit__(self, *exc):
            entered.pop()

    seen = []
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: OnGpu(torch.zeros(n, dtype=dtype), 1))
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(M, "_stream", lambda stream: seen.append(list(entered)) or 7)
    ws = M.alloc_int8_workspace(4096, "cuda:1")
    assert calls == [("moe_workspace_init", (ws.data_ptr(), 4096, 7))]
    assert seen == [[torch.device("cuda", 1)]] and entered == []
