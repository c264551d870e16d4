"""The waits of the few-token layer when what they wait for never comes: each gives up by its own timer, says so in the
status word, takes the copies under way and returns; the context and the workspace stay usable. Nothing faults or hangs:
the kernel itself is told to wait for one CTA more than there are, or not to be told of one tile."""
import time

import pytest
import torch

import few_reference as R
import sparse_moe_layer_route_gb300 as M
from test_few_gpu import weights_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("T,d,E,k,f,S", [(2, 256, 8, 2, 512, 0), (16, 512, 16, 4, 384, 1), (5, 2048, 24, 6, 1408, 2),
                                         (1, 64, 1, 1, 64, 0)])
def test_waits_run_out_report_and_return(T, d, E, k, f, S, which):
    p = R.make(T, d, E, k, f, S, seed=31)
    w = weights_of(p)
    cfg = M.MoeConfig.make(T, d, E, k, f, n_shared=S)
    ws, out = M.alloc_few_workspace(cfg), torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    idx, gates, _ = R.choose(p, k)
    idx, gates = idx.int(), gates.float()
    want = R.layer(p, idx, gates, 0, S)
    for _ in range(2):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        M.check_few_waits(cfg, w, p["x"], idx, out, ws, which, 1_000_000)
        status = M.device_status(ws)
        took = time.perf_counter() - t0
        assert status == M.DEVFAULT_PIPELINE_TIMEOUT
        assert 0.001 <= took < 0.5, took       # the limit at least, not the layer's 2 s
        # the workspace is as good as before
        out.fill_(float("nan"))
        M.experts_few(cfg, w, p["x"], idx, gates, out, ws)
        assert M.device_status(ws) == 0
        R.assert_rounded(out, *want)
        out.fill_(float("nan"))
        M.layer_forward_few(cfg, w, p["x"], None, out, None, ws)
        assert M.device_status(ws) == 0
        R.assert_rounded(out, *want)
