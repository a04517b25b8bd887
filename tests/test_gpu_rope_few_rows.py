"""Chunks without rows, and of one row whose own stride says nothing, with rotary positions."""
import pytest
import torch

from sparse_long_context_sfi_gb300.engine import Rope
from tests.test_gpu_rope_step import BF, D, HKV, HQ, LAYERS, make_state, values_at

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("paged", [True, False])
def test_no_rows(paged):
    st, rope = make_state(paged), Rope()
    x = torch.zeros((LAYERS, 4, HQ + 2 * HKV, D), dtype=BF, device="cuda")
    out = torch.full((LAYERS, 0, HQ, D), 7.0, dtype=BF, device="cuda")
    st.prefill(*x[:, :0].split([HQ, HKV, HKV], 2), [0, 0, 0], out, rope=rope)
    # rows that no sequence has: left as they are
    out = torch.full((LAYERS, 4, HQ, D), 7.0, dtype=BF, device="cuda")
    st.prefill(*x.split([HQ, HKV, HKV], 2), [0, 0, 0], out, rope=rope)
    torch.cuda.synchronize()
    assert st.seq_len.tolist() == [0, 0, 0] and int(st.err[0]) == 0 and (out == 7.0).all()


def test_one_row():
    """Rows of one sequence whose single-row dimension has any stride, against packed ones."""
    rope = Rope(rot_dim=64)
    g = torch.Generator(device="cuda").manual_seed(1)
    wide = (HQ + 2 * HKV) * D
    outs, states = [], []
    for own in (wide, 1, HQ * D):
        g.manual_seed(1)
        st = make_state(False)
        for t in range(3):
            x = torch.randn((LAYERS, wide), generator=g, device="cuda").to(BF)
            q, k, v = (x[:, a * D:b * D].as_strided((LAYERS, 1, b - a, D), (wide, own, D, 1), a * D)
                       for a, b in ((0, HQ), (HQ, HQ + HKV), (HQ + HKV, HQ + 2 * HKV)))
            out = torch.zeros((LAYERS, 1, HQ, D), dtype=BF, device="cuda")
            st.prefill(q, k, v, [1, 0, 0], out, rope=rope)
        torch.cuda.synchronize()
        assert torch.equal(values_at(st, 2)[:, 0], v[:, 0]) and int(st.err[0]) == 0
        outs.append(out)
        states.append(st)
    for o, st in zip(outs[1:], states[1:]):
        assert torch.equal(o, outs[0]) and torch.equal(st.k, states[0].k) and torch.equal(st.v, states[0].v)
    assert outs[0].abs().sum() > 0 and states[0].seq_len.tolist() == [3, 0, 0]
