"""Which rows of heads a call with rotary positions takes: none at all, one, rows of a projection. On the
CPU, with the library's calls replaced."""
import types

import numpy as np
import pytest
import torch

import sparse_long_context_sfi_gb300.engine as engine
from tests.test_engine_checks import B, BF, D, HKV, HQ, LAYERS, arrays, state
from tests.test_rope_step_rows import rope, whole_state

CPU = torch.device("cpu")


@pytest.mark.parametrize("slices", [False, True])
def test_no_rows(monkeypatch, slices):
    """A chunk without rows is taken with positions as it is without."""
    monkeypatch.setattr(engine, "_torch_stream", lambda stream: None)
    calls = []
    monkeypatch.setattr(engine, "sfi_append_chunk", lambda *a, **kw: calls.append("append"))
    monkeypatch.setattr(engine, "sfi_rope_append", lambda kv, r, io, *a, **kw: calls.append(io))
    monkeypatch.setattr(engine.SfiState, "_fitting", lambda self, *a: None)
    monkeypatch.setattr(engine.SfiState, "_window", lambda self, *a: calls.append("window"))
    a = {k: t[:, :0] if slices else torch.zeros((LAYERS, 0) + t.shape[2:], dtype=t.dtype) for k, t in arrays(B).items()}
    for r in (None, rope()):
        st = state(paged=False)
        st.kv = types.SimpleNamespace()
        st.prefill(rows=[0] * B, out_fp32=False, rope=r, **a)
    assert [calls[i] for i in (0, 1, 3)] == ["append", "window", "window"]
    # (the library takes a pair of addresses or none)
    assert not calls[2].q and not calls[2].q_out and not calls[2].k and not calls[2].v


def one(layers, stride):
    """One row a layer, rows `stride` apart; the stride of the single row itself says nothing."""
    x = torch.zeros(layers * stride + 2 * HQ * D, dtype=BF)
    return [x.as_strided((layers, 1, HQ, D), (stride, own, D, 1)) for own in (stride, HQ * D, 1, 13)]


@pytest.mark.parametrize("layers", [1, 3])
def test_one_row(layers):
    stride = (HQ + 2 * HKV) * D
    for t in one(layers, stride):
        step = engine._want_rows("q", t, (layers, 1, HQ, D), CPU)
        # what a kernel reads for layer l: (l * rows + 0) * step elements on
        assert layers == 1 or step == stride
        assert step >= HQ * D and step % 8 == 0
    for stride in (HQ * D - 8, HQ * D + 4):
        for t in one(3, stride):
            with pytest.raises(ValueError):
                engine._want_rows("q", t, (3, 1, HQ, D), CPU)


@pytest.mark.parametrize("which", ["q", "k_new", "v_new"])
def test_what_is_no_tensor(which):
    a = {**arrays(B), "rope": rope(), which: None if which != "q" else np.zeros((LAYERS, B, HQ, D))}
    with pytest.raises(ValueError):
        state().window_step(out_fp32=False, **a)
    with pytest.raises(ValueError):
        whole_state().step(slow_b=np.ones(B, bool), out_fp32=False, **a)
