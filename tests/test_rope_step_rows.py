"""Which arrays a step with rotary positions hands on to the cache's calls, which read them as packed. On
the CPU, with the library's calls replaced."""
import types

import numpy as np
import pytest
import torch

import sparse_long_context_sfi_gb300.engine as engine
from tests.test_engine_checks import B, BF, D, HKV, HQ, LAYERS, arrays, state


@pytest.fixture
def handed(monkeypatch):
    """The arrays of a step's inner calls."""
    monkeypatch.setattr(engine, "_torch_stream", lambda stream: None)
    monkeypatch.setattr(engine, "sfi_rope_apply", lambda *a, **kw: None)
    got = []
    monkeypatch.setattr(engine.SfiState, "_step", lambda self, *a: got.append(a))
    return got


def rope():
    return types.SimpleNamespace(device=torch.device("cpu"), desc=None)


def whole_state():
    st = state()
    st.kv = types.SimpleNamespace()
    return st


@pytest.mark.parametrize("out_fp32", [False, True])
def test_values_of_a_fused_projection_are_packed(handed, out_fp32):
    x = torch.randn((LAYERS, B, HQ + 2 * HKV, D)).to(BF)
    q, k, v = x.split([HQ, HKV, HKV], 2)
    out = torch.zeros((LAYERS, B, HQ, D), dtype=torch.float32 if out_fp32 else BF)
    whole_state().step(q, k, v, np.ones(B, bool), out, out_fp32=out_fp32, rope=rope())
    (tq, tk, tv, *_, ), = handed
    for t, like in ((tq, q), (tk, k), (tv, v)):
        assert t.is_contiguous() and t.shape == like.shape and t.dtype == BF
    assert torch.equal(tv, v)


def test_packed_values_are_not_copied(handed):
    a = arrays(B)
    whole_state().step(a["q"], a["k_new"], a["v_new"], np.ones(B, bool), a["out"], out_fp32=False, rope=rope())
    assert handed[0][2] is a["v_new"]


WRONG = [
    dict(v_new=torch.zeros((LAYERS, B - 1, HKV, D), dtype=BF)), dict(v_new=torch.zeros((LAYERS, B, HKV, D))),
    dict(v_new=torch.zeros((LAYERS, B, 2 * HKV, D), dtype=BF)[:, :, ::2]),              # heads apart
    dict(v_new=torch.zeros((LAYERS, B, HKV, D), dtype=BF, device="meta")),
    dict(out=torch.zeros((LAYERS, B, HQ, D), dtype=torch.float64)), dict(out=torch.zeros((LAYERS, B, HQ, D))),
    dict(out=torch.zeros((LAYERS, B, HKV, D), dtype=BF)),
    dict(out=torch.zeros((LAYERS, B, HQ + HKV, D), dtype=BF)[:, :, :HQ]),               # not packed
]


@pytest.mark.parametrize("wrong", range(len(WRONG)))
def test_values_and_outputs_are_checked(handed, wrong):
    a = {**arrays(B), **WRONG[wrong]}
    with pytest.raises(ValueError):
        whole_state().step(slow_b=np.ones(B, bool), out_fp32=False, rope=rope(), **a)
    assert not handed
