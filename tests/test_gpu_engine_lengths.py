"""Lengths as the engine bounds them on the host: slots that are used again, runs of the native
driver between the other calls, lengths put back, captured steps that are replayed. Outputs are
compared with their definition, as in the serving loop's own test."""
import numpy as np
import pytest
import torch

import sparse_long_context_sfi_gb300 as sfi
from tests.test_gpu_cache_run import D, Loop, built  # noqa: F401  (built: the module's fixture)

pytestmark = pytest.mark.gpu


def test_a_captured_step_is_replayed_at_lengths_that_the_host_has_not_seen():
    """And so is the eager step behind it."""
    lp = Loop(True)
    lp.prefill([60, 20, 1, 33, 40, 50], 64)
    lp.step("window", window=64)
    q, kv = lp.rnd(2, 6, 8, D), lp.rnd(2, 6, 2, D)
    out = torch.zeros((2, 6, 8, D), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lp.st.window_step(q, kv, kv, out, n_window=64)
    host = kv.double().cpu().numpy()
    for _ in range(70):
        graph.replay()
        for b in range(6):
            lp.grow(b, host[:, b:b + 1], host[:, b:b + 1])
    torch.cuda.synchronize()
    assert int(lp.st.err[0]) == 0 and lp.st.seq_len.tolist() == [k.shape[2] for k in lp.k]
    lp.step("window", window=200)
