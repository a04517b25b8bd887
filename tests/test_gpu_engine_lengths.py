"""Lengths as the engine bounds them on the host: slots that are used again, runs of the native
driver between the other calls, lengths put back, captured steps that are replayed. Outputs are
compared with their definition, as in the serving loop's own test."""
import numpy as np
import pytest
import torch

import sparse_long_context_sfi_gb300 as sfi
from tests.test_gpu_cache_run import D, Loop, built  # noqa: F401  (built: the module's fixture)

pytestmark = pytest.mark.gpu


def forget(lp):
    lp.k = [np.zeros((lp.layers, 2, 0, D)) for _ in range(lp.batch)]
    lp.v = [np.zeros((lp.layers, 2, 0, D)) for _ in range(lp.batch)]


def by_run(lp):
    """The loop's slow and fast steps through make_plan and run."""
    st = lp.st
    st.step = lambda q, k, v, slow, out: st.run(st.make_plan(
        np.asarray(slow, np.uint8)[None], q[None], k[None], v[None], out[None]))


@pytest.mark.parametrize("native", [False, True])
def test_slots_are_used_again(native):
    """Released sequences start over: more tokens in all than a slot holds (320)."""
    lp = Loop(True)
    if native:
        by_run(lp)
    for _ in range(4):
        lp.prefill([180, 20, 33, 200, 40, 21], 64)
        lp.step("slow")
        lp.step("window", window=48)
        lp.step("fast")
        lp.st.release()
        forget(lp)
    # and some of them: the others go on
    lp.prefill([30, 20, 30, 20, 30, 20], 64)
    for t in range(8):
        lp.prefill([50, 0, 50, 0, 50, 0], 64)
        lp.step("slow" if t % 2 == 0 else "window", window=32)
        mask = torch.tensor([1, 0, 1, 0, 1, 0], dtype=torch.uint8, device="cuda")
        lp.st.release(active=mask)
        for b in (0, 2, 4):
            lp.k[b], lp.v[b] = (np.zeros((lp.layers, 2, 0, D)) for _ in "kv")


@pytest.mark.parametrize("paged", [False, True])
def test_runs_between_the_other_calls(paged):
    lp = Loop(paged)
    by_run(lp)
    lp.prefill([100, 40, 60, 77, 30, 50], 64)
    lp.step("slow")
    lp.step("window", window=48)
    lp.step("fast")
    lp.step("fast")
    lp.step("window", window=48)
    lp.prefill([10, 0, 1, 0, 33, 2], 64)
    lp.reorder(torch.tensor([1, 1, 2, 0, 3, 3], dtype=torch.int32, device="cuda"))
    for kind in ("slow", "fast", "window", "slow"):
        lp.step(kind, window=48)


@pytest.mark.parametrize("paged", [False, True])
def test_reset_lengths_puts_back_the_first_lengths(paged):
    lp = Loop(paged)
    lp.prefill([100, 0, 0, 77, 0, 0], 64)
    lp.reorder(torch.tensor([0, 0, 0, 3, 3, 3], dtype=torch.int32, device="cuda"))
    lp.st.reset_lengths()
    assert lp.st.seq_len.tolist() == [0] * 6
    if paged:
        lp.st.release()
    forget(lp)
    lp.prefill([10, 20, 30, 40, 50, 60], 64)
    lp.step("slow")


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
    lp.step("slow")
    lp.step("fast")
    by_run(lp)
    lp.step("slow")
    lp.step("fast")


def test_captured_release():
    """A release that is only captured leaves the lengths, and their bounds, as they are."""
    lp = Loop(True)
    lp.prefill([60, 20, 30, 33, 40, 50], 64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lp.st.release()
    lp.step("slow")
    lp.step("fast")
    graph.replay()
    forget(lp)
    lp.prefill([60, 20, 30, 33, 40, 50], 64)
    lp.step("window", window=64)
    lp.step("slow")
