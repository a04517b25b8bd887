"""What the engine refuses before any call of the library: arrays that a kernel, which gets their
addresses alone, would read or write wrongly. On the CPU, with states that have no cache."""
import types

import numpy as np
import pytest
import torch

from sparse_long_context_sfi_gb300.engine import BeamSearch, SfiState

B, LAYERS, HQ, HKV, D = 3, 2, 8, 2, 128
BF = torch.bfloat16


def state(paged=True):
    st = SfiState.__new__(SfiState)
    st.cfg = types.SimpleNamespace(batch=B, n_layers=LAYERS, n_q_heads=HQ, n_kv_heads=HKV, head_dim=D,
                                   n_window=16, n_sink=4)
    st.device = torch.device("cpu")
    st.page_table = torch.zeros((B, 4), dtype=torch.int32) if paged else None
    st.capacity, st._upto, st._replayed = 64, np.zeros(B, np.int64), False
    return st


def arrays(n, fp32=False):
    return dict(q=torch.zeros((LAYERS, n, HQ, D), dtype=BF), k_new=torch.zeros((LAYERS, n, HKV, D), dtype=BF),
                v_new=torch.zeros((LAYERS, n, HKV, D), dtype=BF),
                out=torch.zeros((LAYERS, n, HQ, D), dtype=torch.float32 if fp32 else BF))


WRONG = [
    dict(out=torch.zeros((LAYERS, B, HQ, D), dtype=torch.float64)),
    dict(q=torch.zeros((LAYERS, B, HQ, D))),
    dict(q=torch.zeros((LAYERS, HQ, B, D), dtype=BF).transpose(1, 2)),      # not contiguous
    dict(k_new=torch.zeros((LAYERS, B - 1, HKV, D), dtype=BF)),             # too few rows
    dict(v_new=torch.zeros((LAYERS, B, HKV, D), dtype=torch.float16)),
    dict(v_new=torch.zeros((LAYERS, B, HQ, D), dtype=BF)),
    dict(k_new=np.zeros((LAYERS, B, HKV, D), np.uint16)),
    dict(out=torch.zeros((LAYERS, B, HQ, D), dtype=BF, device="meta")),
]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("wrong", range(len(WRONG)))
def test_chunk_arrays(wrong, fp32, paged):
    a = {**arrays(B, fp32), **WRONG[wrong]}
    with pytest.raises(ValueError):
        state(paged).prefill(rows=[1, 1, 1], out_fp32=fp32, **a)
    with pytest.raises(ValueError):
        state(paged).window_step(out_fp32=fp32, **a)


def test_output_type_and_flag_disagree():
    for fp32 in (False, True):
        with pytest.raises(ValueError):
            state().window_step(out_fp32=not fp32, **arrays(B, fp32))
        with pytest.raises(ValueError):
            state().prefill(rows=[1, 1, 1], out_fp32=not fp32, **arrays(B, fp32))


@pytest.mark.parametrize("rows", [[1, 1], [1, 1, 1, 0], [2, -1, 2], [[1, 1, 1]], [1, 1, 2]])
def test_rows(rows):
    with pytest.raises(ValueError):
        state().prefill(rows=rows, **arrays(B))


@pytest.mark.parametrize("bad", [torch.ones(B), torch.ones(B - 1, dtype=torch.uint8),
                                 torch.ones(B, dtype=torch.int32), np.ones(B, np.uint8),
                                 torch.ones(2 * B, dtype=torch.uint8)[::2]])
def test_masks(bad):
    st = state()
    for call in (lambda: st.reserve(active=bad), lambda: st.evict(active=bad), lambda: st.release(active=bad),
                 lambda: st.window_step(active=bad, out_fp32=False, **arrays(B))):
        with pytest.raises(ValueError):
            call()


def test_counts_maps_and_flags():
    st = state()
    with pytest.raises(ValueError):
        st.reserve(n_new=torch.ones(B, dtype=torch.int64))
    with pytest.raises(ValueError):
        st.reserve(ok=torch.ones(B, dtype=torch.int32))
    for src in (torch.arange(B), torch.arange(B - 1, dtype=torch.int32), [0, 1, 2]):
        with pytest.raises(ValueError):
            st.reorder(src)


def test_beam_arrays():
    beam = BeamSearch(2, 2, 50, device="cpu")
    x = torch.zeros((4, 50))
    for logits, scale in ((x.to("meta"), None), (x.half(), None), (x[:3], None), (x, torch.ones(4).double()),
                          (x, torch.ones(3)), (x, torch.ones((4, 2))[:, 0])):
        with pytest.raises(ValueError):
            beam.select(logits, rank_scale=scale)


def test_another_device_than_the_current_one(monkeypatch):
    """Kernels run on the current device: a state on another one refuses (the devices are made up)."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    st = state()
    st.device, st._pool = torch.device("cuda", 1), None
    with pytest.raises(ValueError, match="not the current device"):
        st.reserve()
    with pytest.raises(ValueError, match="not the current device"):
        st.step(None, None, None, [True] * B, None)
    with pytest.raises(ValueError, match="not the current device"):
        st.run(None)
    with pytest.raises(ValueError):
        st.reorder(torch.zeros(B, dtype=torch.int32))
