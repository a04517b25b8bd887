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


@pytest.mark.parametrize("out_fp32", [False, True])
def test_a_full_sequence_is_left_out(out_fp32):
    """A contiguous cache: what does not fit its capacity is not attended either; the others are."""
    lp = Loop(False)
    lp.prefill([320, 0, 0, 100, 318, 0], 64)
    st = lp.st
    dt = torch.float32 if out_fp32 else torch.bfloat16
    q, k, v = lp.rnd(2, 10, 8, D), lp.rnd(2, 10, 2, D), lp.rnd(2, 10, 2, D)
    out = torch.full((2, 10, 8, D), -7.0, dtype=dt, device="cuda")
    st.prefill(q, k, v, [1, 0, 0, 5, 3, 0], out, out_fp32=out_fp32, n_window=64)
    torch.cuda.synchronize()
    assert int(st.err[0]) == sfi.SFI_DEVERR_CAPACITY
    assert st.seq_len.tolist() == [320, 0, 0, 105, 318, 0]
    assert (out[:, 0] == -7.0).all() and (out[:, 6:] == -7.0).all()
    assert (out[:, 1:6] != -7.0).any(-1).all()
    q, k, v = lp.rnd(2, 6, 8, D), lp.rnd(2, 6, 2, D), lp.rnd(2, 6, 2, D)
    for mask in (None, [1, 1, 0, 1, 1, 0]):
        out = torch.full((2, 6, 8, D), -7.0, dtype=dt, device="cuda")
        before = st.seq_len.tolist()
        st.err.zero_()
        st.window_step(q, k, v, out, out_fp32=out_fp32, n_window=64,
                       active=None if mask is None else torch.tensor(mask, dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        assert int(st.err[0]) == sfi.SFI_DEVERR_CAPACITY
        on = [b for b in range(6) if b != 0 and (mask is None or mask[b])]
        assert st.seq_len.tolist() == [n + (b in on) for b, n in enumerate(before)]
        for b in range(6):
            assert (out[:, b] != -7.0).any(-1).all() if b in on else (out[:, b] == -7.0).all()


def test_a_sequence_that_fills_up_in_a_replayed_step():
    """The replays beyond its capacity leave the full sequence's output alone and serve the others."""
    lp = Loop(False)
    lp.prefill([318, 20, 1, 33, 40, 50], 64)
    q, kv = lp.rnd(2, 6, 8, D), lp.rnd(2, 6, 2, D)
    out = torch.zeros((2, 6, 8, D), device="cuda")
    lp.st.window_step(q, kv, kv, out, n_window=64)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lp.st.window_step(q, kv, kv, out, n_window=64)
    for t in range(3):
        out.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert int(lp.st.err[0]) == (sfi.SFI_DEVERR_CAPACITY if t else 0)
        assert lp.st.seq_len.tolist() == [320] + [n + 2 + t for n in (20, 1, 33, 40, 50)]
        assert (out[:, 0] == -7.0).all() if t else (out[:, 0] != -7.0).any()
        assert (out[:, 1:] != -7.0).any(-1).all()


def test_lengths_that_a_replayed_reorder_exchanged():
    """A full slot's length has moved to another sequence, which is then the one that is left out."""
    lp = Loop(False)
    lp.prefill([20, 21, 22, 23, 24, 25], 64)
    src = torch.tensor([1, 0, 2, 3, 4, 5], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lp.st.reorder(src)
    lp.prefill([0, 290, 0, 0, 0, 0], 64)
    graph.replay()
    q, k, v = lp.rnd(2, 60, 8, D), lp.rnd(2, 60, 2, D), lp.rnd(2, 60, 2, D)
    out = torch.full((2, 60, 8, D), -7.0, device="cuda")
    lp.st.prefill(q, k, v, [30, 30, 0, 0, 0, 0], out, out_fp32=True, n_window=64)
    torch.cuda.synchronize()
    assert int(lp.st.err[0]) == sfi.SFI_DEVERR_CAPACITY
    assert lp.st.seq_len.tolist() == [311, 50, 22, 23, 24, 25]
    assert (out[:, :30] == -7.0).all() and (out[:, 30:] != -7.0).any(-1).all()


def test_the_pool_is_not_made_in_a_capture():
    lp = Loop(True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError):
            lp.st.reserve()
    lp.prefill([60, 20, 30, 33, 40, 50], 64)
    lp.step("slow")
