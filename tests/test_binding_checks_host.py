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
