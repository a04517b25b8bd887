"""The engine's own workspaces around captured calls: a graph goes on using the one it was captured
with, and a workspace that was made during a capture is not there for eager calls."""
import numpy as np
import pytest
import torch

from sparse_long_context_sfi_gb300.engine import BeamSearch, SfiState
from synth.configs import WORKLOADS
from tests.cache_model import beam_select, window_attention
from tests.test_gpu_cache_run import D, built  # noqa: F401  (built: the module's fixture)

pytestmark = pytest.mark.gpu

WINDOW = 4096


class One:
    """One sequence of a contiguous cache under a window that is split over the GPU."""

    def __init__(self, rows=4500):
        cfg = WORKLOADS["ragged_paged_b32"].scaled(
            batch=1, n_layers=1, n_q_heads=8, n_kv_heads=2, n_sink=4, n_window=16, n_select=24,
            steps=64, page_size=0)
        self.st = SfiState(cfg, np.zeros(1), capacity=8192)
        self.g = torch.Generator(device="cuda").manual_seed(5)
        kv = self.rnd(1, rows, 2, D), self.rnd(1, rows, 2, D)
        self.st.k[0, 0, :, :rows], self.st.v[0, 0, :, :rows] = (t[0].transpose(0, 1) for t in kv)
        self.st.seq_len.fill_(rows)
        self.st.len0[:] = rows
        self.st.reset_lengths()
        self.q, self.kn, self.vn = self.rnd(1, 1, 8, D), self.rnd(1, 1, 2, D), self.rnd(1, 1, 2, D)
        self.out = torch.zeros((1, 1, 8, D), device="cuda")

    def rnd(self, *s):
        return torch.randn(s, generator=self.g, device="cuda").to(torch.bfloat16)

    def step(self):
        self.st.window_step(self.q, self.kn, self.vn, self.out, n_window=WINDOW)

    def check(self):
        torch.cuda.synchronize()
        n = int(self.st.seq_len[0])
        k, v = (t[0, 0, :, :n].double().cpu().numpy() for t in (self.st.k, self.st.v))
        o, mag = window_attention(self.q[0].double().cpu().numpy(), k, v, n, 4, WINDOW)
        assert (np.abs(self.out[0].double().cpu().numpy() - o) <= 1e-4 * mag).all()
        assert int(self.st.err[0]) == 0
        self.out.zero_()


def capture(call):
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    return graph


def test_a_graph_keeps_its_workspace():
    one = One()
    one.step()
    one.check()
    graph = capture(one.step)
    small = one.st._window_ws.now.numel()
    n = 300
    q, k, v = one.rnd(1, n, 8, D), one.rnd(1, n, 2, D), one.rnd(1, n, 2, D)
    one.st.prefill(q, k, v, [n], torch.zeros((1, n, 8, D), device="cuda"), out_fp32=True, n_window=WINDOW)
    assert one.st._window_ws.now.numel() > small
    torch.cuda.synchronize()
    others = [torch.full((small,), 0xa5, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(3):
        graph.replay()
        one.check()
    assert all(bool((t == 0xa5).all()) for t in others)
    one.step()
    one.check()


def test_a_first_call_that_is_captured():
    one = One()
    graph = capture(one.step)
    for _ in range(2):
        one.step()                  # before any replay
        one.check()
    graph.replay()
    one.check()
    one.step()
    one.check()


def test_a_first_selection_that_is_captured():
    g = torch.Generator(device="cuda").manual_seed(1)
    many = torch.randn((4, 6, 20000), generator=g, device="cuda") * 2
    beam, logits = BeamSearch(2, 3, 20000, eos=7), many[0].clone()
    beam.cum.copy_(-torch.rand(6, generator=g, device="cuda"))
    graph = capture(lambda: beam.select(logits))
    for t in range(4):
        logits.copy_(many[t])
        cum, done = beam.cum.cpu().numpy(), beam.done.cpu().numpy()
        graph.replay() if t % 2 else beam.select(logits)
        want = beam_select(many[t].cpu().numpy(), cum, done, None, 7, 3)
        np.testing.assert_array_equal(beam.parent.cpu().numpy(), want[0])
        np.testing.assert_array_equal(beam.token.cpu().numpy(), want[1])
