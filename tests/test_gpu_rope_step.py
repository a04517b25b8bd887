"""Steps with rotary positions on the rows of one projection, as a model's split leaves them, against steps
on packed copies of them: outputs, keys and values bit for bit, and the values in the cache those given."""
import numpy as np
import pytest
import torch

from sparse_long_context_sfi_gb300.engine import Rope, SfiState
from synth.configs import WORKLOADS

pytestmark = pytest.mark.gpu

D, BF, PAGE = 128, torch.bfloat16, 16
HQ, HKV, BATCH, LAYERS, COLS, LEN0 = 8, 2, 3, 2, 6, 20


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def make_state(paged):
    cfg = WORKLOADS["ragged_paged_b32" if paged else "gqa4_ctx4k_hh"].scaled(
        n_layers=LAYERS, batch=BATCH, n_q_heads=HQ, n_kv_heads=HKV, n_sink=4, n_window=16, n_select=16, steps=4)
    if not paged:
        return SfiState(cfg, np.full(BATCH, 0), capacity=COLS * PAGE)
    return SfiState(cfg, np.full(BATCH, 0), page_table=np.full((BATCH, COLS), -1), n_pages=BATCH * COLS)


def values_at(st, pos):
    """[layers][sequences][heads][D] values held at position pos of every sequence."""
    if st.page_table is None:
        return st.v[:, :, :, pos]
    return st.v[:, st.page_table[:, pos // PAGE].long()][:, :, :, pos % PAGE]


@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("paged", [True, False])
def test_rows_of_one_projection(paged, fused, given, side):
    rope = Rope(rot_dim=96, base=500000.0)
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)
    a, b = make_state(paged), make_state(paged)
    q, k, v = rnd(LAYERS, BATCH * LEN0, HQ + 2 * HKV, D).split([HQ, HKV, HKV], 2)
    for st in (a, b):
        st.prefill(q, k, v, [LEN0] * BATCH, torch.zeros((LAYERS, BATCH * LEN0, HQ, D), dtype=BF, device="cuda"), rope=rope)
    stream = torch.cuda.Stream() if side else None
    for t, slow in enumerate(([1, 1, 1], [0, 0, 0], [1, 0, 1], [0, 0, 0])):
        q, k, v = rnd(LAYERS, BATCH, HQ + 2 * HKV, D).split([HQ, HKV, HKV], 2)
        assert not v.is_contiguous()
        pos = torch.tensor([7, 100000, 3], dtype=torch.int32, device="cuda") + t if given else None
        outs = [torch.zeros((LAYERS, BATCH, HQ, D), device="cuda") for _ in "ab"]
        torch.cuda.synchronize()
        for st, o, rows in ((a, outs[0], (q, k, v)), (b, outs[1], [x.contiguous() for x in (q, k, v)])):
            torch.cuda.synchronize()
            active = st.reserve(stream=stream) if paged else None
            st.step(*rows, np.array(slow, bool), o, rope=rope, pos=pos, fused=fused, active=active, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.isfinite(outs[0]).all() and outs[0].abs().sum() > 0
        assert torch.equal(values_at(a, LEN0 + t), v)
        assert a.seq_len.tolist() == [LEN0 + t + 1] * BATCH
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    assert int(a.err[0]) == 0 and int(b.err[0]) == 0


def test_in_a_graph():
    """The packing of the values is part of a captured step."""
    rope = Rope()
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)
    st = make_state(False)
    q, k, v = rnd(LAYERS, BATCH, HQ + 2 * HKV, D).split([HQ, HKV, HKV], 2)
    st.prefill(q, k, v, [1] * BATCH, torch.zeros((LAYERS, BATCH, HQ, D), dtype=BF, device="cuda"), rope=rope)
    x = rnd(LAYERS, BATCH, HQ + 2 * HKV, D)
    q, k, v = x.split([HQ, HKV, HKV], 2)
    out = torch.zeros((LAYERS, BATCH, HQ, D), device="cuda")
    st.step(q, k, v, np.ones(BATCH, bool), out, rope=rope)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.step(q, k, v, np.zeros(BATCH, bool), out, rope=rope)
    for t in range(2, 5):
        x.copy_(rnd(*x.shape))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(values_at(st, t), v) and st.seq_len.tolist() == [t + 1] * BATCH
    assert int(st.err[0]) == 0
