"""Argument checks of the cache-side entry points: refused before any launch, without a GPU.
The pointers are never dereferenced."""
import ctypes as C

import pytest

import sparse_long_context_sfi_gb300 as sfi

DUMMY = 1 << 20


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return sfi.lib()


def cache(**kw):
    a = dict(n_layers=1, batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, capacity=64, page_size=16,
             n_pages=16, max_pages_per_seq=4, max_len=10, k=DUMMY, v=DUMMY, page_table=DUMMY,
             seq_len=DUMMY, err=DUMMY)
    a.update(kw)
    return sfi.SfiKvCache(**a)


def pool(**kw):
    return sfi.SfiPagePool(**{**dict(page_table=DUMMY, refs=DUMMY), **kw})


def test_struct_layouts():
    assert C.sizeof(sfi.SfiPagePool) == 16
    assert C.sizeof(sfi.SfiBeam) == 4 * 4 + 8 + 8 + 8 * 8
    assert sfi.SfiBeam.logits.offset == 32 and sfi.SfiBeam.done_out.offset == 88


@pytest.mark.parametrize("kv,pl", [
    (cache(page_size=0), pool()),                 # a contiguous cache has no pages
    (cache(), pool(refs=None)),
    (cache(), pool(page_table=None)),
    (cache(), pool(page_table=2 * DUMMY)),        # not the table that the cache reads
    (cache(k=None), pool()),
])
def test_page_calls_refuse(lib, kv, pl):
    for st in (lib.sfi_pages_reserve(C.byref(kv), C.byref(pl), None, None, None, DUMMY, 1 << 30, None),
               lib.sfi_pages_release(C.byref(kv), C.byref(pl), None, None),
               lib.sfi_pages_evict(C.byref(kv), C.byref(pl), 4, 64, None, None),
               lib.sfi_pages_compact(C.byref(kv), C.byref(pl), DUMMY, DUMMY, 1 << 30, None)):
        assert st == sfi.SFI_ERR_INVALID_ARG
    assert lib.sfi_pages_evict(C.byref(kv), None, 4, 64, None, None) == sfi.SFI_ERR_INVALID_ARG


def test_page_workspace_and_arguments(lib):
    kv, pl = cache(), pool()
    need = sfi.sfi_pages_workspace_bytes(kv)
    assert need >= 3 * 4 * kv.n_pages
    for ws, n in ((None, need), (DUMMY, need - 1), (DUMMY + 16, need)):
        assert lib.sfi_pages_reserve(C.byref(kv), C.byref(pl), None, None, None, ws, n, None) == \
            sfi.SFI_ERR_WORKSPACE
        assert lib.sfi_pages_compact(C.byref(kv), C.byref(pl), DUMMY, ws, n, None) == \
            sfi.SFI_ERR_WORKSPACE
    assert lib.sfi_pages_compact(C.byref(kv), C.byref(pl), None, DUMMY, need, None) == \
        sfi.SFI_ERR_INVALID_ARG
    for sink, window in ((-1, 64), (4, 0), (4, -5)):
        assert lib.sfi_pages_evict(C.byref(kv), C.byref(pl), sink, window, None, None) == \
            sfi.SFI_ERR_INVALID_ARG
    with pytest.raises(sfi.SfiError):
        sfi.sfi_pages_workspace_bytes(cache(page_size=0))


def test_chunk_calls_refuse(lib):
    kv = cache()
    big = 1 << 30
    ap = lambda *a: lib.sfi_append_chunk(C.byref(kv), *a, None, None)
    assert ap(DUMMY, DUMMY, DUMMY, -1, 4) == sfi.SFI_ERR_INVALID_ARG
    assert ap(DUMMY, DUMMY, None, 3, 1) == sfi.SFI_ERR_INVALID_ARG     # one row each: n_rows == batch
    assert ap(DUMMY, DUMMY, None, 2, 0) == sfi.SFI_ERR_INVALID_ARG
    assert ap(None, DUMMY, DUMMY, 4, 4) == sfi.SFI_ERR_INVALID_ARG
    assert ap(DUMMY + 8, DUMMY, DUMMY, 4, 4) == sfi.SFI_ERR_INVALID_ARG
    assert ap(DUMMY, DUMMY, DUMMY, big, 4) == sfi.SFI_ERR_UNSUPPORTED
    assert ap(None, None, DUMMY, 0, 4) == sfi.SFI_OK                   # nothing to append
    at = lambda q, out, start, n, m, sink, window, ws, nb: lib.sfi_window_attn(
        C.byref(kv), q, out, 0, start, n, m, sink, window, None, ws, nb, None)
    assert at(DUMMY, DUMMY, DUMMY, 4, 4, -1, 8, DUMMY, big) == sfi.SFI_ERR_INVALID_ARG
    assert at(DUMMY, DUMMY, DUMMY, 4, 4, 4, 0, DUMMY, big) == sfi.SFI_ERR_INVALID_ARG
    assert at(DUMMY, DUMMY, None, 4, 1, 4, 8, DUMMY, big) == sfi.SFI_ERR_INVALID_ARG
    assert at(DUMMY, DUMMY, DUMMY, 4, 4, 4, 8, None, big) == sfi.SFI_ERR_WORKSPACE
    assert at(DUMMY, DUMMY, DUMMY, 4, 4, 4, 8, DUMMY + 32, big) == sfi.SFI_ERR_WORKSPACE
    assert at(DUMMY, DUMMY, DUMMY, 4, 4, 4, 8, DUMMY, 0) == sfi.SFI_ERR_WORKSPACE
    assert at(None, DUMMY, DUMMY, 4, 4, 4, 8, DUMMY, big) == sfi.SFI_ERR_INVALID_ARG
    assert at(DUMMY, DUMMY + 8, DUMMY, 4, 4, 4, 8, DUMMY, big) == sfi.SFI_ERR_INVALID_ARG
    assert at(None, None, DUMMY, 0, 4, 4, 8, DUMMY, big) == sfi.SFI_OK
    for sink, window in ((-1, 8), (0, 0)):
        with pytest.raises(sfi.SfiError):
            sfi.sfi_window_workspace_bytes(kv, 4, 4, sink, window)


def test_reorder_refuses(lib):
    paged, flat = cache(), cache(page_size=0)
    bud = sfi.SfiBudget(n_sink=4, n_window=64, n_select=16, prior_tau=64, lambda_=0.1)
    mem = sfi.SfiSparseMem(kc=DUMMY, vc=DUMMY, sel_idx=DUMMY, sel_cnt=DUMMY, rows=DUMMY)
    bad = sfi.SFI_ERR_INVALID_ARG
    call = lambda kv, pl, b, m, src: lib.sfi_reorder(
        C.byref(kv), None if pl is None else C.byref(pl), None if b is None else C.byref(b),
        None if m is None else C.byref(m), src, None)
    assert call(paged, None, None, None, DUMMY) == bad        # the table needs its counts
    assert call(flat, pool(), None, None, DUMMY) == bad
    assert call(paged, pool(), None, None, None) == bad
    assert call(paged, pool(), None, mem, DUMMY) == bad       # packed memory without its sizes
    mem.kc = DUMMY + 8
    assert call(paged, pool(), bud, mem, DUMMY) == bad
    mem.kc, mem.sel_idx = DUMMY, None
    assert call(paged, pool(), bud, mem, DUMMY) == bad


@pytest.mark.parametrize("change,status", [
    (dict(n_groups=0), sfi.SFI_ERR_INVALID_ARG),
    (dict(n_beams=0), sfi.SFI_ERR_INVALID_ARG),
    (dict(n_beams=17), sfi.SFI_ERR_UNSUPPORTED),
    (dict(n_groups=16384), sfi.SFI_ERR_UNSUPPORTED),
    (dict(vocab=0), sfi.SFI_ERR_INVALID_ARG),
    (dict(row_stride=99), sfi.SFI_ERR_INVALID_ARG),
    (dict(eos=100), sfi.SFI_ERR_INVALID_ARG),
    (dict(vocab=1 << 30, row_stride=1 << 30), sfi.SFI_ERR_UNSUPPORTED),
])
def test_beam_sizes_refused(lib, change, status):
    beam = sfi.SfiBeam(**{**dict(n_groups=2, n_beams=4, vocab=100, row_stride=100, eos=2), **change})
    assert lib.sfi_beam_select(C.byref(beam), DUMMY, 1 << 30, None) == status
    with pytest.raises(sfi.SfiError):
        sfi.sfi_beam_workspace_bytes(beam)


def test_beam_pointers_refused(lib):
    names = ("logits", "cum", "parent", "token", "cum_out")
    for name in names:
        beam = sfi.SfiBeam(n_groups=2, n_beams=4, vocab=100, row_stride=100, eos=2,
                           **{n: DUMMY for n in names if n != name})
        assert lib.sfi_beam_select(C.byref(beam), DUMMY, 1 << 30, None) == sfi.SFI_ERR_INVALID_ARG
    beam = sfi.SfiBeam(n_groups=2, n_beams=4, vocab=100, row_stride=100, eos=-1, done=DUMMY,
                       **{n: DUMMY for n in names})
    assert lib.sfi_beam_select(C.byref(beam), DUMMY, 1 << 30, None) == sfi.SFI_ERR_INVALID_ARG
    beam.done = None
    beam.logits = DUMMY + 1
    assert lib.sfi_beam_select(C.byref(beam), DUMMY, 1 << 30, None) == sfi.SFI_ERR_INVALID_ARG
    beam.logits = DUMMY
    for ws, n in ((None, 1 << 30), (DUMMY + 64, 1 << 30), (DUMMY, 0)):
        assert lib.sfi_beam_select(C.byref(beam), ws, n, None) == sfi.SFI_ERR_WORKSPACE
