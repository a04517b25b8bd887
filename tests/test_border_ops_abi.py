"""Rotary frequencies, and the argument checks of rotary positions, attention to an encoder and log
probabilities: refused before any launch, without a GPU. The pointers are never dereferenced."""
import ctypes as C
import math

import numpy as np
import pytest

import sparse_long_context_sfi_gb300 as sfi
from tests.border_model import frequencies

DUMMY = 1 << 20
INVALID, UNSUPPORTED, WORKSPACE = sfi.SFI_ERR_INVALID_ARG, sfi.SFI_ERR_UNSUPPORTED, sfi.SFI_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return sfi.lib()


def cache(**kw):
    a = dict(n_layers=1, batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, capacity=64, page_size=16,
             n_pages=16, max_pages_per_seq=4, max_len=10, k=DUMMY, v=DUMMY, page_table=DUMMY,
             seq_len=DUMMY, err=DUMMY)
    return sfi.SfiKvCache(**{**a, **kw})


def test_struct_layouts():
    assert C.sizeof(sfi.SfiRope) == 40 and sfi.SfiRope.turns.offset == 16
    assert C.sizeof(sfi.SfiRopeScaling) == 48
    assert C.sizeof(sfi.SfiRopeRows) == 72 and sfi.SfiRopeRows.pos.offset == 64
    assert C.sizeof(sfi.SfiScoring) == 80 and sfi.SfiScoring.logits.offset == 24


SCALINGS = [dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0),
            dict(scaling="base", factor=8.0), dict(scaling="ramp", factor=32.0, original_len=4096.0),
            dict(scaling="ramp", factor=4.0, original_len=8192.0, low=2.0, high=3.0),
            dict(scaling="ramp", factor=1.0, original_len=40.0),
            dict(scaling="smooth", base=500000.0, factor=8.0, original_len=8192.0, low=1.0, high=4.0)]


@pytest.mark.parametrize("rot", [2, 4, 34, 64, 126, 128])
@pytest.mark.parametrize("kw", SCALINGS, ids=[str(i) for i in range(len(SCALINGS))])
def test_frequencies(lib, rot, kw):
    """Both sides compute in doubles, with a handful of roundings each, for which 2^-46 relative is far
    more than enough; and the turns are rounded to 2^-64 of a turn: by up to pi 2^-64 radians."""
    if kw.get("scaling") == "base" and rot == 2:
        pytest.skip("refused")
    turns, amplitude = sfi.sfi_rope_turns(rot, **kw)
    want, c = frequencies(rot, **kw)
    got = np.array([int(t) / 2 ** 64 * 2 * math.pi for t in turns])
    assert turns.dtype == np.uint64 and np.all(np.abs(got - want) <= 2.0 ** -46 * want + math.pi * 2.0 ** -64)
    assert abs(amplitude - c) <= 2.0 ** -23 * c


@pytest.mark.parametrize("rot,kw", [
    (0, {}), (3, {}), (130, {}), (-2, {}), (64, dict(base=1.0)), (64, dict(base=math.inf)),
    (64, dict(base=math.nan)), (64, dict(scaling="linear", factor=0.5)), (64, dict(scaling="linear", factor=math.nan)),
    (2, dict(scaling="base", factor=2.0)), (64, dict(scaling="ramp", factor=2.0)),
    (64, dict(scaling="ramp", factor=2.0, original_len=100.0, low=0.0)),
    (64, dict(scaling="smooth", factor=2.0, original_len=100.0, low=4.0, high=4.0)),
    (64, dict(scaling="smooth", factor=2.0, original_len=100.0, low=1.0, high=math.inf))])
def test_frequencies_refused(lib, rot, kw):
    with pytest.raises(sfi.SfiError):
        sfi.sfi_rope_turns(rot, **kw)


def test_scaling_names(lib):
    with pytest.raises(ValueError):
        sfi.sfi_rope_turns(64, scaling="dynamic")
    sc = sfi.SfiRopeScaling(kind=5, base=10000.0, factor=1.0)
    buf = (C.c_uint64 * 32)()
    amp = C.c_float()
    assert lib.sfi_rope_turns(64, C.byref(sc), buf, C.byref(amp)) == INVALID
    sc.kind, sc.reserved = 0, 1
    assert lib.sfi_rope_turns(64, C.byref(sc), buf, C.byref(amp)) == INVALID
    sc.reserved = 0
    assert lib.sfi_rope_turns(64, None, buf, C.byref(amp)) == INVALID
    assert lib.sfi_rope_turns(64, C.byref(sc), None, C.byref(amp)) == INVALID
    assert lib.sfi_rope_turns(64, C.byref(sc), buf, None) == INVALID


def rope(**kw):
    return sfi.SfiRope(**{**dict(rot_dim=128, amplitude=1.0, turns=DUMMY), **kw})


def rows(append, **kw):
    a = dict(q=DUMMY, q_out=2 * DUMMY, k=3 * DUMMY, q_stride=1024, k_stride=256)
    a.update(dict(v=5 * DUMMY, v_stride=256) if append else dict(k_out=4 * DUMMY))
    return sfi.SfiRopeRows(**{**a, **kw})


def call(lib, append, kv=None, r=None, io=None, start=DUMMY, n=5, most=5):
    f = lib.sfi_rope_append if append else lib.sfi_rope_apply
    kv, r, io = kv or cache(), r or rope(), io or rows(append)
    return f(C.byref(kv), C.byref(r), C.byref(io), start, n, most, None, None)


@pytest.mark.parametrize("append", [False, True])
def test_rope_refusals(lib, append):
    for r in (rope(rot_dim=0), rope(rot_dim=7), rope(rot_dim=130), rope(turns=None), rope(turns=DUMMY + 4),
              rope(amplitude=math.inf), rope(amplitude=math.nan), rope(q_norm=DUMMY),        # eps 0
              rope(k_norm=DUMMY, norm_eps=math.nan), rope(q_norm=DUMMY + 8, norm_eps=1e-6)):
        assert call(lib, append, r=r) == INVALID
    for io in (rows(append, q=None), rows(append, q_out=None), rows(append, q_stride=1016),
               rows(append, q_stride=1028), rows(append, q=DUMMY + 8), rows(append, q_out=DUMMY + 8),
               rows(append, k_stride=128), rows(append, k=DUMMY + 2),
               rows(append, q=DUMMY, q_out=DUMMY, q_stride=1536)):      # in place, not packed
        assert call(lib, append, io=io) == INVALID
    assert call(lib, append, n=-1) == INVALID
    assert call(lib, append, start=None, n=5) == INVALID            # one each: n_rows is the batch
    assert call(lib, append, kv=cache(head_dim=64)) == UNSUPPORTED
    assert call(lib, append, kv=cache(max_len=65)) == sfi.SFI_ERR_CAPACITY
    f = lib.sfi_rope_append if append else lib.sfi_rope_apply
    kv, r, io = cache(), rope(), rows(append)
    assert f(None, C.byref(r), C.byref(io), DUMMY, 5, 5, None, None) == INVALID
    assert f(C.byref(kv), None, C.byref(io), DUMMY, 5, 5, None, None) == INVALID
    assert f(C.byref(kv), C.byref(r), None, DUMMY, 5, 5, None, None) == INVALID
    assert call(lib, append, n=0, most=0) == sfi.SFI_OK


def test_rope_refusals_of_one_form(lib):
    assert call(lib, True, io=rows(True, k_out=DUMMY)) == INVALID
    assert call(lib, True, io=rows(True, k=None)) == INVALID
    assert call(lib, True, io=rows(True, v=None)) == INVALID
    assert call(lib, True, io=rows(True, v_stride=250)) == INVALID
    assert call(lib, False, io=rows(False, k=None)) == INVALID
    assert call(lib, False, io=sfi.SfiRopeRows()) == INVALID        # nothing to turn


def test_cross_refusals(lib):
    kv = cache()
    need = sfi.sfi_cross_workspace_bytes(kv, 5, 5)

    def go(kv=kv, q=DUMMY, out=DUMMY, start=DUMMY, n=5, most=5, ws=DUMMY, nb=need):
        return lib.sfi_cross_attn(C.byref(kv), q, out, 1, start, n, most, None, ws, nb, None)

    assert go(q=None) == INVALID and go(out=None) == INVALID and go(q=DUMMY + 8) == INVALID
    assert go(out=DUMMY + 8) == INVALID and go(n=-1) == INVALID and go(most=-1) == INVALID
    assert go(start=None) == INVALID and go(kv=cache(k=None)) == INVALID
    assert go(ws=None) == WORKSPACE and go(ws=DUMMY + 16) == WORKSPACE and go(nb=need - 1) == WORKSPACE
    assert go(kv=cache(n_q_heads=6)) == UNSUPPORTED
    assert go(n=0, most=0) == sfi.SFI_OK
    with pytest.raises(sfi.SfiError):
        sfi.sfi_cross_workspace_bytes(kv, -1, 1)
    with pytest.raises(sfi.SfiError):
        sfi.sfi_cross_workspace_bytes(cache(head_dim=64), 1, 1)


def scoring(**kw):
    return sfi.SfiScoring(**{**dict(n_rows=3, vocab=100, row_stride=100, n_top=4, logits=DUMMY, token=DUMMY,
                                    logprob=DUMMY, rank=DUMMY, entropy=DUMMY, top_token=DUMMY,
                                    top_logprob=DUMMY), **kw})


def test_scoring_refusals(lib):
    def go(sc, ws=DUMMY, nb=1 << 30):
        return lib.sfi_score_tokens(C.byref(sc), ws, nb, None)

    for kw in (dict(n_rows=-1), dict(vocab=0), dict(row_stride=99), dict(n_top=-1), dict(logits=None),
               dict(logits=DUMMY + 1), dict(logits=DUMMY + 2, logits_fp32=1), dict(token=None),
               dict(token=None, logprob=None), dict(token=None, rank=None), dict(top_token=None),
               dict(top_logprob=None), dict(n_top=101, vocab=100),
               dict(n_top=0, logprob=None, rank=None, entropy=None)):
        assert go(scoring(**kw)) == INVALID, kw
    assert go(scoring(n_top=33)) == UNSUPPORTED
    assert go(scoring(vocab=(1 << 30) + 1, row_stride=1 << 31)) == UNSUPPORTED
    need = sfi.sfi_scoring_workspace_bytes(scoring())
    for ws, nb in ((None, need), (DUMMY, need - 1), (DUMMY + 16, need)):
        assert go(scoring(), ws, nb) == WORKSPACE
    assert go(scoring(n_rows=0, logits=None)) == sfi.SFI_OK
    assert lib.sfi_score_tokens(None, DUMMY, need, None) == INVALID
    with pytest.raises(sfi.SfiError):
        sfi.sfi_scoring_workspace_bytes(scoring(n_top=33))
