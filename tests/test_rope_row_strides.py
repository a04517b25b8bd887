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
