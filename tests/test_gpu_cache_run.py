"""The cache-side operators together with the decode path, as a serving loop uses them: prompts
enter a paged cache in chunks, are forked into beams, and every step selects, reorders and
reserves; slow and fast steps, windowed steps, eviction, release and compaction in between.
Every attention output is compared with its definition on the host's own copy of each
sequence's keys and values. Tolerances as in the windowed attention's tests (fp32 outputs:
1e-4 of sum_j w_j |v_j|, twice for the decode kernels, whose weights go through a merge)."""
import numpy as np
import pytest
import torch

import sparse_long_context_sfi_gb300 as sfi
from sparse_long_context_sfi_gb300.engine import BeamSearch, SfiState
from synth.configs import WORKLOADS
from tests.cache_model import beam_select, window_attention

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def attend(q, k, v, at):
    """q [Hq][D] over the rows `at` of k, v [Hkv][L][D]: output and sum of weights * |v|."""
    group = q.shape[0] // k.shape[0]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(q.shape[0]):
        z = k[h // group][at] @ q[h] / np.sqrt(D)
        w = np.exp(z - z.max())
        w /= w.sum()
        out[h], mag[h] = w @ v[h // group][at], w @ np.abs(v[h // group][at])
    return out, mag


class Loop:
    def __init__(self, paged, groups=2, beams=3, layers=2):
        self.groups, self.beams, self.layers = groups, beams, layers
        self.batch = groups * beams
        cfg = WORKLOADS["ragged_paged_b32"].scaled(
            batch=self.batch, n_layers=layers, n_q_heads=8, n_kv_heads=2, n_sink=4, n_window=16,
            n_select=24, steps=64, page_size=16 if paged else 0)
        cols = 20
        table = np.full((self.batch, cols), -1, np.int32) if paged else None
        self.st = SfiState(cfg, np.zeros(self.batch), page_table=table, n_pages=90 if paged else 0,
                           capacity=None if paged else cols * 16)
        self.cfg, self.paged = cfg, paged
        self.g = torch.Generator(device="cuda").manual_seed(3)
        self.k = [np.zeros((layers, 2, 0, D)) for _ in range(self.batch)]
        self.v = [np.zeros((layers, 2, 0, D)) for _ in range(self.batch)]

    def rnd(self, *s):
        return torch.randn(s, generator=self.g, device="cuda").to(torch.bfloat16)

    def check(self, got, want, mag, factor=1e-4):
        got = got.double().cpu().numpy()
        assert (np.abs(got - want) <= factor * mag).all(), float(np.abs(got - want).max())

    def grow(self, b, k, v):
        self.k[b] = np.concatenate([self.k[b], k.transpose(0, 2, 1, 3)], 2)
        self.v[b] = np.concatenate([self.v[b], v.transpose(0, 2, 1, 3)], 2)

    def prefill(self, rows, window):
        n = int(sum(rows)) + 1
        q, k, v = self.rnd(self.layers, n, 8, D), self.rnd(self.layers, n, 2, D), self.rnd(self.layers, n, 2, D)
        out = torch.zeros((self.layers, n, 8, D), device="cuda")
        self.st.prefill(q, k, v, rows, out, out_fp32=True, n_window=window)
        qh, kh, vh = (t.double().cpu().numpy() for t in (q, k, v))
        r0 = 0
        for b, m in enumerate(rows):
            if m:
                self.grow(b, kh[:, r0:r0 + m], vh[:, r0:r0 + m])
                for ly in range(self.layers):
                    want, mag = window_attention(qh[ly, r0:r0 + m], self.k[b][ly], self.v[b][ly],
                                                 self.k[b].shape[2], 4, window)
                    self.check(out[ly, r0:r0 + m], want, mag)
            r0 += m

    def reorder(self, src):
        self.st.reorder(src)
        s = src.cpu().numpy()
        self.k, self.v = [self.k[i] for i in s], [self.v[i] for i in s]

    def step(self, kind, window=None):
        """One decode step of every sequence: 'slow', 'fast' or 'window'."""
        shape = (self.layers, self.batch)
        q, k, v = self.rnd(*shape, 8, D), self.rnd(*shape, 2, D), self.rnd(*shape, 2, D)
        out = torch.zeros((*shape, 8, D), device="cuda")
        st = self.st
        if kind == "window":
            st.window_step(q, k, v, out, n_window=window)
        else:
            if self.paged:
                st.reserve()
            st.step(q, k, v, np.full(self.batch, kind == "slow"), out)
        qh, kh, vh = (t.double().cpu().numpy() for t in (q, k, v))
        sel = st.sel_idx.cpu().numpy().reshape(self.layers, self.batch, 2, -1)
        cnt = st.sel_cnt.cpu().numpy().reshape(self.layers, self.batch, 2)
        for b in range(self.batch):
            self.grow(b, kh[:, b:b + 1], vh[:, b:b + 1])
            n = self.k[b].shape[2]
            for ly in range(self.layers):
                kb, vb = self.k[b][ly], self.v[b][ly]
                if kind == "slow":
                    want, mag = attend(qh[ly, b], kb, vb, np.arange(n))
                elif kind == "window":
                    want, mag = window_attention(qh[ly, b:b + 1], kb, vb, n, 4, window)
                    want, mag = want[0], mag[0]
                else:
                    want, mag = np.zeros((8, D)), np.zeros((8, D))
                    for h in range(2):
                        at = np.concatenate([np.arange(4), sel[ly, b, h, :cnt[ly, b, h]],
                                             np.arange(n - 16, n)])
                        w, m = attend(qh[ly, b, 4 * h:4 * h + 4], kb[h:h + 1], vb[h:h + 1], at)
                        want[4 * h:4 * h + 4], mag[4 * h:4 * h + 4] = w, m
                self.check(out[ly, b], want, mag, 2e-4)
        torch.cuda.synchronize()
        assert int(st.err[0]) == 0


@pytest.mark.parametrize("paged", [True, False])
def test_serving_loop(paged):
    lp = Loop(paged)
    st = lp.st
    lp.prefill([100, 0, 0, 77, 0, 0], 64)
    lp.prefill([33, 0, 0, 60, 0, 0], 64)
    lp.prefill([1, 0, 0, 1, 0, 0], 1000)
    lp.reorder(torch.tensor([0, 0, 0, 3, 3, 3], dtype=torch.int32, device="cuda"))
    beam = BeamSearch(2, 3, 500, eos=7)
    lp.step("slow")
    for t in range(6):
        logits = torch.randn((6, 500), generator=lp.g, device="cuda") * 2
        cum, done = beam.cum.cpu().numpy(), beam.done.cpu().numpy()
        want = beam_select(logits.cpu().numpy(), cum, done, None, 7, 3)
        parent, token = beam.select(logits)
        np.testing.assert_array_equal(parent.cpu().numpy(), want[0])
        np.testing.assert_array_equal(token.cpu().numpy(), want[1])
        lp.reorder(parent)
        lp.step("slow" if t == 3 else "fast")
    if paged:
        refs = st.page_refs.cpu().numpy()
        table = st.page_table.cpu().numpy()
        np.testing.assert_array_equal(np.bincount(table[table >= 0], minlength=90), refs)
        st.evict(n_window=48)
        assert int(st.page_refs.sum()) < int(refs.sum())
        used = st.compact_pages()
        torch.cuda.synchronize()
        n = int(used[0])
        assert (st.page_refs[:n] > 0).all() and not st.page_refs[n:].any()
    for _ in range(3):
        lp.step("window", window=48)
    if paged:
        st.release()
        torch.cuda.synchronize()
        assert not st.page_refs.any() and (st.page_table == -1).all() and not st.seq_len.any()


def test_two_states_at_once():
    """Two caches with their own workspaces, stepped on two streams at once: neither disturbs the
    other."""
    a, b = Loop(True), Loop(True)
    for lp in (a, b):
        lp.prefill([120, 0, 0, 90, 0, 0], 40)
        lp.reorder(torch.tensor([0, 0, 0, 3, 3, 3], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for lp, s in ((a, s1), (b, s2)):
        with torch.cuda.stream(s):
            q, k, v = lp.rnd(2, 6, 8, D), lp.rnd(2, 6, 2, D), lp.rnd(2, 6, 2, D)
            out = torch.zeros((2, 6, 8, D), device="cuda")
            for _ in range(4):
                lp.st.window_step(q, k, v, out, n_window=40)
            outs.append(out)
    torch.cuda.synchronize()
    assert torch.equal(a.st.seq_len, b.st.seq_len) and torch.equal(a.st.page_table, b.st.page_table)
    assert torch.equal(outs[0], outs[1])     # the same seeds: the same bits


def test_exhausted_pool_leaves_the_others_alone():
    """Three beams on one page and no page to copy to: the step leaves them as they are and serves
    the sequence that needs none."""
    lp = Loop(True)
    st = lp.st
    lp.prefill([60, 0, 0, 1200 // 8, 0, 0], 64)
    lp.reorder(torch.tensor([0, 0, 0, 3, 4, 5], dtype=torch.int32, device="cuda"))
    st.page_refs[st.page_refs == 0] = 7                 # (nothing is free)
    before = st.k.clone()
    q, k, v = lp.rnd(2, 6, 8, D), lp.rnd(2, 6, 2, D), lp.rnd(2, 6, 2, D)
    out = torch.full((2, 6, 8, D), -7.0, device="cuda")
    st.window_step(q, k, v, out, n_window=64)
    torch.cuda.synchronize()
    assert int(st.err[0]) == sfi.SFI_DEVERR_POOL
    assert st.seq_len.tolist() == [60, 60, 60, 151, 0, 0]
    page = int(st.page_table[3, 150 // 16])
    assert torch.equal(st.k[:, page, :, 150 % 16], k[:, 3])
    before[:, page, :, 150 % 16] = k[:, 3]
    assert torch.equal(st.k, before)
    assert (out[:, [0, 1, 2, 4, 5]] == -7.0).all() and (out[:, 3] != -7.0).all()


def test_captured_beam_step():
    """A captured step (select, reorder, reserve) replayed: the same beams as eager steps."""
    def setup():
        lp, beam = Loop(True), BeamSearch(2, 3, 500, eos=7)
        lp.prefill([60, 0, 0, 33, 0, 0], 64)
        lp.reorder(torch.tensor([0, 0, 0, 3, 3, 3], dtype=torch.int32, device="cuda"))
        return lp, beam

    def step(lp, beam, logits, out, q, kv):
        parent, token = beam.select(logits)
        lp.st.reorder(parent)
        lp.st.window_step(q, kv, kv, out, n_window=64)

    g = torch.Generator(device="cuda").manual_seed(1)
    many = torch.randn((5, 6, 500), generator=g, device="cuda") * 2
    q = torch.randn((2, 6, 8, D), generator=g, device="cuda").to(torch.bfloat16)
    kv = torch.randn((2, 6, 2, D), generator=g, device="cuda").to(torch.bfloat16)
    outs = []
    for captured in (False, True):
        lp, beam = setup()
        out, logits = torch.zeros((2, 6, 8, D), device="cuda"), many[0].clone()
        step(lp, beam, logits, out, q, kv)              # (workspaces are made here)
        if captured:
            torch.cuda.synchronize()
            lp.st.len0 = lp.st.len0 + 8                 # a bound for the steps to come
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step(lp, beam, logits, out, q, kv)
        for t in range(1, 5):
            logits.copy_(many[t])
            graph.replay() if captured else step(lp, beam, logits, out, q, kv)
        torch.cuda.synchronize()
        assert int(lp.st.err[0]) == 0
        outs.append((out, beam.parent, beam.token, beam.cum, beam.done, lp.st.seq_len, lp.st.page_table))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_engine_refuses():
    lp = Loop(False)
    with pytest.raises(ValueError):
        lp.st.pool()
    q = lp.rnd(2, 4, 8, D)
    kv = lp.rnd(2, 4, 2, D)
    with pytest.raises(ValueError):
        lp.st.prefill(q, kv, kv, [5, 0, 0, 0, 0, 0], torch.zeros_like(q))
    beam = BeamSearch(1, 2, 50)
    for bad in (torch.zeros((2, 49), device="cuda"), torch.zeros((2, 50), device="cuda", dtype=torch.float16),
                torch.zeros((50, 2), device="cuda").t()):
        with pytest.raises(ValueError):
            beam.select(bad)
