"""What the engine refuses of rotary rows, encoder states and scores before any call of the library. On
the CPU, with objects that have no device memory behind them."""
import types

import numpy as np
import pytest
import torch

from sparse_long_context_sfi_gb300.engine import EncoderStates, Rope, TokenScores
from tests.test_engine_checks import B, BF, D, HKV, HQ, LAYERS, arrays, state

CPU = torch.device("cpu")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def rope(device=CPU):
    return types.SimpleNamespace(device=device, desc=None)


WRONG = [
    dict(q=torch.zeros((LAYERS, B, HQ, D))),                                    # fp32
    dict(q=torch.zeros((LAYERS, B, HQ, 2 * D), dtype=BF)[..., ::2]),            # dimensions apart
    dict(q=torch.zeros((LAYERS, B, 2 * HQ, D), dtype=BF)[:, :, ::2]),           # heads apart
    dict(q=torch.zeros((LAYERS, B, HQ * D + 4), dtype=BF)[..., :HQ * D].view(LAYERS, B, HQ, D)),   # rows off 8
    dict(q=torch.zeros((LAYERS, 2 * B, HQ, D), dtype=BF)[:, :B]),               # layers apart
    dict(q=torch.zeros((LAYERS, 1, HQ, D), dtype=BF).expand(LAYERS, B, HQ, D)),     # one row thrice
    dict(q=torch.zeros(LAYERS * B * HQ * D + 4, dtype=BF)[4:].view(LAYERS, B, HQ, D)),      # 8 bytes off
    dict(k_new=torch.zeros((LAYERS, B, HQ, D), dtype=BF)), dict(v_new=torch.zeros((LAYERS, B - 1, HKV, D), dtype=BF)),
    dict(k_new=torch.zeros((LAYERS, B, HKV, D), dtype=BF, device="meta")),
    dict(pos=torch.zeros(B, dtype=torch.int64)), dict(pos=torch.zeros(B + 1, dtype=torch.int32)),
    dict(rope=rope(torch.device("meta"))), dict(out=torch.zeros((LAYERS, B, HQ, D), dtype=torch.float64)),
]


@pytest.mark.parametrize("wrong", range(len(WRONG)))
def test_rope_rows(wrong):
    a = {**arrays(B), "rope": rope(), **WRONG[wrong]}
    with pytest.raises(ValueError):
        state().prefill(rows=[1, 1, 1], out_fp32=False, **a)
    with pytest.raises(ValueError):
        state().window_step(out_fp32=False, **a)
    if "v_new" in WRONG[wrong] or "out" in WRONG[wrong]:
        return
    with pytest.raises(ValueError):
        state().step(slow_b=np.ones(B, bool), out_fp32=False, **a)


def test_positions_without_rope():
    with pytest.raises(ValueError):
        state().window_step(out_fp32=False, pos=torch.zeros(B, dtype=torch.int32), **arrays(B))


def test_step_positions_without_rope():
    a = {k: v for k, v in arrays(B).items()}
    with pytest.raises(ValueError):
        state().step(a["q"], a["k_new"], a["v_new"], np.ones(B, bool), a["out"],
                     pos=torch.zeros(B, dtype=torch.int32))


def test_rope_arguments():
    w = torch.ones(D, dtype=BF)
    for kw in (dict(q_norm=w.float()), dict(k_norm=torch.ones(64, dtype=BF)), dict(q_norm=w, norm_eps=0.0),
               dict(k_norm=w, norm_eps=float("inf")), dict(scaling="none at all"),
               dict(q_norm=torch.ones(D + 4, dtype=BF)[4:])):
        with pytest.raises(ValueError):
            Rope(device="cpu", **kw)
    with pytest.raises(RuntimeError):
        Rope(rot_dim=7, device="cpu")
    r = Rope(rot_dim=64, scaling="linear", factor=2.0, q_norm=w, device="cpu")
    assert r.turns.shape == (32,) and r.desc.q_norm == w.data_ptr() and r.desc.k_norm is None


def encoder():
    return EncoderStates(LAYERS, B, HQ, HKV, 64, device="cpu")


def test_encoder_arguments():
    e = encoder()
    kv = lambda n: torch.zeros((LAYERS, n, HKV, D), dtype=BF)
    for rows, k, v in (([1, 1], kv(2), kv(2)), ([1, -1, 1], kv(1), kv(1)), ([60, 65, 1], kv(126), kv(126)),
                       ([1, 1, 1], kv(4), kv(3)), ([1, 1, 1], kv(3), kv(3).float())):
        with pytest.raises(ValueError):
            e.write(k, v, rows)
    with pytest.raises(ValueError):
        e.clear([B])
    q = lambda n, **kw: torch.zeros((LAYERS, n, HQ, D), **{"dtype": BF, **kw})
    for a, kw in (((q(3), q(3)), dict(rows=[1, 1])), ((q(3), q(3)), dict(rows=[1, 1, -1])),
                  ((q(3), q(3)), dict(rows=2)), ((q(3), q(4)), {}), ((q(3, dtype=torch.float32), q(3)), {}),
                  ((q(3), q(3)), dict(out_fp32=True)), ((q(3), q(3, dtype=torch.float32)), {}),
                  ((q(3).transpose(0, 1).contiguous().transpose(0, 1), q(3)), {}), ((None, q(3)), {}),
                  ((q(3), q(3)), dict(active=torch.ones(B + 1, dtype=torch.uint8))),
                  ((q(3), q(3)), dict(active=torch.ones(B)))):
        with pytest.raises(ValueError):
            e.attend(*a, **kw)


def test_score_arguments():
    s = TokenScores(device="cpu")
    x, t = torch.zeros((4, 100)), torch.zeros(4, dtype=torch.int32)
    for a, kw in (((x[0], t), {}), ((x.half(), t), {}), ((x.t(), t), {}), ((x, t.long()), {}), ((x, t[:3]), {}),
                  ((x,), {}), ((x,), dict(rank=True, entropy=True)), ((x, t), dict(n_top=33)),
                  ((x, t), dict(n_top=-1)), ((x[:, :5], t), dict(n_top=6)), ((x[:1].expand(4, 100), t), {}),
                  ((x.to("meta"), t), {}), ((x[:, :0], t), {})):
        with pytest.raises(ValueError):
            s.score(*a, **kw)
