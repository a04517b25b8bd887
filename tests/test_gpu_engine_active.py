"""Slow and fast steps and runs of some of the sequences: what a reserve refused stays as it is."""
import numpy as np
import pytest
import torch

import sparse_long_context_sfi_gb300 as sfi
from tests.test_gpu_cache_run import D, Loop, attend, built  # noqa: F401  (built: the module's fixture)

pytestmark = pytest.mark.gpu


def check_row(lp, b, q, out, kind):
    """Sequence b's row against its definition; its new key and value are in lp.k and lp.v."""
    st, n = lp.st, lp.k[b].shape[2]
    sel = st.sel_idx.cpu().numpy().reshape(lp.layers, lp.batch, 2, -1)
    cnt = st.sel_cnt.cpu().numpy().reshape(lp.layers, lp.batch, 2)
    qh = q.double().cpu().numpy()
    for ly in range(lp.layers):
        for h in range(2):
            at = np.arange(n) if kind == "slow" else np.concatenate(
                [np.arange(4), sel[ly, b, h, :cnt[ly, b, h]], np.arange(n - 16, n)])
            want, mag = attend(qh[ly, b, 4 * h:4 * h + 4], lp.k[b][ly][h:h + 1], lp.v[b][ly][h:h + 1], at)
            lp.check(out[ly, b, 4 * h:4 * h + 4], want, mag, 2e-4)


@pytest.mark.parametrize("how", ["step", "unfused", "run"])
def test_refused_sequences_stay_as_they_are(how):
    """Beams 0 to 2 are on one page and there is no page to copy to; the others need none."""
    lp = Loop(True)
    lp.prefill([60, 0, 0, 150, 70, 71], 64)
    lp.reorder(torch.tensor([0, 0, 0, 3, 4, 5], dtype=torch.int32, device="cuda"))
    st = lp.st
    st.page_refs[st.page_refs == 0] = 7                 # (nothing is free)
    lens = [60, 60, 60, 150, 70, 71]
    for kind, slow in (("slow", [1, 1, 1, 1, 1, 1]), ("fast", [0, 0, 0, 0, 0, 0]), ("mixed", [1, 0, 1, 0, 1, 0])):
        ok = st.reserve()
        assert int(st.err[0]) == sfi.SFI_DEVERR_POOL
        assert ok.tolist() == [0, 0, 0, 1, 1, 1]
        st.err.zero_()
        shared = int(st.page_table[0, 3])
        before = st.k[:, shared].clone()
        q, k, v = lp.rnd(2, 6, 8, D), lp.rnd(2, 6, 2, D), lp.rnd(2, 6, 2, D)
        out = torch.full((2, 6, 8, D), -7.0, device="cuda")
        slow = np.array(slow, bool)
        if how == "run":
            plan = st.make_plan(slow.astype(np.uint8)[None], q[None], k[None], v[None], out[None])
            st.run(plan, active=ok)
        else:
            st.step(q, k, v, slow, out, active=ok, fused=how == "step")
        torch.cuda.synchronize()
        assert int(st.err[0]) == 0
        lens = [n + (b > 2) for b, n in enumerate(lens)]
        assert st.seq_len.tolist() == lens
        assert torch.equal(st.k[:, shared], before) and (out[:, :3] == -7.0).all()
        kh, vh = k.double().cpu().numpy(), v.double().cpu().numpy()
        for b in (3, 4, 5):
            lp.grow(b, kh[:, b:b + 1], vh[:, b:b + 1])
            check_row(lp, b, q, out, "slow" if slow[b] else "fast")


@pytest.mark.parametrize("dense_only", [False, True])
def test_a_run_of_some_equals_the_run_of_all(dense_only):
    """Several steps, mixed and not: the active sequences have what a run of all gives them, the
    others keep lengths and outputs. Steps of their own launches: equal up to the order of sums."""
    steps, slow = 4, np.array([[1] * 6, [0, 1, 0, 1, 0, 1], [0] * 6, [0, 0, 0, 1, 1, 1]], np.uint8)
    outs = []
    for some in (False, True):
        lp = Loop(True)
        lp.prefill([60, 90, 33, 150, 70, 71], 64)
        st = lp.st
        q, k, v = lp.rnd(steps, 2, 6, 8, D), lp.rnd(steps, 2, 6, 2, D), lp.rnd(steps, 2, 6, 2, D)
        out = torch.full((steps, 2, 6, 8, D), -7.0, device="cuda")
        st.reserve(torch.full((6,), steps, dtype=torch.int32, device="cuda"))
        plan = st.make_plan(slow, q, k, v, out, dense_only=dense_only)
        on = torch.tensor([1, 0, 1, 1, 0, 1], dtype=torch.uint8, device="cuda")
        st.run(plan, active=on if some else None)
        torch.cuda.synchronize()
        assert int(st.err[0]) == 0
        outs.append(out)
        want = [60, 90, 33, 150, 70, 71]
        assert st.seq_len.tolist() == [n + steps * (not some or b not in (1, 4)) for b, n in enumerate(want)]
    a, b = outs[0][:, :, [0, 2, 3, 5]], outs[1][:, :, [0, 2, 3, 5]]
    assert ((a - b).abs() <= 1e-4).all() and (outs[1][:, :, [1, 4]] == -7.0).all()


def test_events_are_refused_with_active():
    lp = Loop(True)
    lp.prefill([60, 90, 33, 150, 70, 71], 64)
    q, k, v = lp.rnd(1, 2, 6, 8, D), lp.rnd(1, 2, 6, 2, D), lp.rnd(1, 2, 6, 2, D)
    out = torch.zeros((1, 2, 6, 8, D), device="cuda")
    plan = lp.st.make_plan(np.ones((1, 6), np.uint8), q, k, v, out,
                           events=[torch.cuda.Event(enable_timing=True) for _ in range(2)])
    with pytest.raises(ValueError):
        lp.st.run(plan, active=torch.ones(6, dtype=torch.uint8, device="cuda"))
    assert lp.st.seq_len.tolist() == [60, 90, 33, 150, 70, 71]
