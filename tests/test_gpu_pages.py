"""Pages, chunk appends and reordering against a plain model: integers and moved bytes equal."""
import numpy as np
import pytest
import torch

import sparse_long_context_sfi_gb300 as sfi
from tests.cache_model import PAGE, PoolModel

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def bits(t):
    return t.view(torch.int16).cpu().numpy()


class Pool:
    """A paged cache that starts empty, its pool filled with noise, and the model beside it."""

    def __init__(self, batch, cols, pages, hkv=2, layers=1, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.batch, self.cols, self.pages, self.hkv, self.layers = g, batch, cols, pages, hkv, layers
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((batch, cols), -1, **i32)
        # one word past a 16-byte boundary: nothing may count on alignment
        self.refs = torch.zeros(pages + 1, **i32)[1:]
        self.seq_len = torch.zeros(batch, **i32)
        self.err = torch.zeros(4, **i32)
        shape = (layers, pages, hkv, PAGE, D)
        self.k, self.v = (torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv")
        self.kv = sfi.SfiKvCache(
            n_layers=layers, batch=batch, n_q_heads=hkv, n_kv_heads=hkv, head_dim=D,
            capacity=cols * PAGE, page_size=PAGE, n_pages=pages, max_pages_per_seq=cols,
            max_len=cols * PAGE, k=self.k.data_ptr(), v=self.v.data_ptr(),
            page_table=self.table.data_ptr(), seq_len=self.seq_len.data_ptr(), err=self.err.data_ptr())
        self.pool = sfi.SfiPagePool(page_table=self.table.data_ptr(), refs=self.refs.data_ptr())
        self.nb = sfi.sfi_pages_workspace_bytes(self.kv)
        self.ws = torch.full((self.nb,), 0x5a, dtype=torch.uint8, device="cuda")
        self.model = PoolModel(self.table.cpu().numpy(), self.refs.cpu().numpy(),
                               self.seq_len.cpu().numpy(), bits(self.k), bits(self.v), cols * PAGE)

    def check(self, bytes_too=True):
        torch.cuda.synchronize()
        m = self.model
        np.testing.assert_array_equal(self.table.cpu().numpy(), m.table)
        np.testing.assert_array_equal(self.refs.cpu().numpy(), m.refs)
        np.testing.assert_array_equal(self.seq_len.cpu().numpy(), m.seq_len)
        assert int(self.err[0]) == m.err
        if bytes_too:
            assert np.array_equal(bits(self.k), m.k) and np.array_equal(bits(self.v), m.v)
        held = np.bincount(m.table[m.table >= 0], minlength=self.pages)
        np.testing.assert_array_equal(held, m.refs)

    def mask(self, mask):
        return None if mask is None else torch.tensor(mask, dtype=torch.uint8, device="cuda")

    def reserve(self, n_new=None, mask=None):
        ok = torch.full((self.batch,), 9, dtype=torch.uint8, device="cuda")
        n = None if n_new is None else torch.tensor(n_new, dtype=torch.int32, device="cuda")
        sfi.sfi_pages_reserve(self.kv, self.pool, n, self.ws, self.nb, active=self.mask(mask), ok=ok)
        want = self.model.reserve(n_new, mask)
        np.testing.assert_array_equal(ok.cpu().numpy(), want)
        return want

    def append(self, rows, mask=None):
        start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        n = int(start[-1]) + 2
        k, v = (torch.randn((self.layers, n, self.hkv, D), generator=self.g, device="cuda").to(
            torch.bfloat16) for _ in "kv")
        sfi.sfi_append_chunk(self.kv, k, v, torch.from_numpy(start).cuda(), n, max(rows),
                             active=self.mask(mask))
        self.model.append(bits(k), bits(v), start, mask)

    def reorder(self, src):
        sfi.sfi_reorder(self.kv, torch.tensor(src, dtype=torch.int32, device="cuda"), pool=self.pool)
        self.model.reorder(np.array(src))

    def release(self, mask):
        sfi.sfi_pages_release(self.kv, self.pool, active=self.mask(mask))
        self.model.release(mask)

    def compact(self):
        n = torch.full((1,), -1, dtype=torch.int32, device="cuda")
        sfi.sfi_pages_compact(self.kv, self.pool, n, self.ws, self.nb)
        assert int(n[0]) == self.model.compact()


def test_prompt_pages_lowest_first():
    p = Pool(3, 40, 100, layers=2)
    p.reserve([100, 0, 333])
    p.check()
    p.append([100, 0, 333])
    p.check()
    p.reserve([0, 16, 1])
    p.append([0, 16, 1])
    p.check()
    assert p.table[0, :7].tolist() == list(range(7))


def test_forks_copy_on_write():
    p = Pool(6, 10, 60, layers=2, hkv=3)
    p.reserve([37, 0, 0, 32, 0, 0])
    p.append([37, 0, 0, 32, 0, 0])
    p.reorder([0, 0, 0, 3, 3, 3])
    p.check()
    p.reserve()                      # tails of 0..2 shared: two copies; 3..5 start a new page
    p.check()
    p.append([1] * 6)
    p.check()
    p.reserve()                      # nothing shared any more, nothing missing
    p.check()
    p.reorder([0, 0, 2, 5, 4, 3])    # pages reserved ahead are shared too
    p.reserve(mask=[0, 1, 1, 1, 0, 1])
    p.check()


def test_one_of_the_holders_writes():
    """A holder that does not reserve keeps the shared page: every other one copies."""
    p = Pool(4, 4, 20)
    p.reserve([20, 0, 0, 0])
    p.append([20, 0, 0, 0])
    p.reorder([0, 0, 0, 0])
    p.reserve([0, 1, 1, 0])
    p.check()
    p.reserve([1, 0, 0, 1])
    p.check()


def test_pool_exhausted_and_capacity():
    p = Pool(4, 8, 10)
    p.reserve([64, 64, 64, 16])      # 4 + 4 fit, the third does not, nor anything after it
    assert p.model.err == sfi.SFI_DEVERR_POOL
    p.check()
    p.append([64, 64, 0, 0])
    p.reserve([65, 0, 0, 0])         # past the capacity of 128
    assert p.model.err == sfi.SFI_DEVERR_POOL | sfi.SFI_DEVERR_CAPACITY
    p.check()
    p.reserve([0, 1, 1, 0])
    p.check()


def test_last_holder_of_a_page_when_the_others_are_refused():
    """With no page left to copy to, the first holders stay on the shared page, so the last one
    may not write there either; a sequence that needs nothing is served all the same."""
    p = Pool(4, 4, 4)
    p.reserve([20, 0, 0, 17])
    p.append([20, 0, 0, 17])
    p.reorder([0, 0, 0, 3])
    ok = p.reserve()
    assert p.model.err == sfi.SFI_DEVERR_POOL and ok.tolist() == [0, 0, 0, 1]
    p.check()
    p.release([0, 0, 0, 1])
    ok = p.reserve(mask=[1, 1, 1, 0])   # two pages: both copies, and the last keeps the page
    assert ok.tolist() == [1, 1, 1, 0]
    p.check()
    p.append([1, 1, 1, 0])
    p.check()


def test_release_and_evict():
    p = Pool(5, 30, 200)
    p.reserve([400, 100, 480, 33, 0])
    p.append([400, 100, 480, 33, 0])
    for sink, window in ((4, 64), (0, 100), (40, 17), (4, 16)):
        sfi.sfi_pages_evict(p.kv, p.pool, sink, window, active=p.mask([1, 1, 0, 1, 1]))
        p.model.evict(sink, window, [1, 1, 0, 1, 1])
        p.check()
    p.reserve([1, 1, 0, 1, 1])
    p.check()
    sfi.sfi_pages_release(p.kv, p.pool, active=p.mask([1, 0, 1, 0, 1]))
    p.model.release([1, 0, 1, 0, 1])
    p.check()
    sfi.sfi_pages_release(p.kv, p.pool)
    p.model.release()
    p.check()
    assert int(p.refs.sum()) == 0


def test_counts_that_disagree_are_reported():
    p = Pool(2, 4, 8)
    p.table[0, 0] = 3                # an entry that no count knows
    p.table[1, 0] = 99               # an entry past the pool
    sfi.sfi_pages_release(p.kv, p.pool)
    torch.cuda.synchronize()
    assert int(p.err[0]) == sfi.SFI_DEVERR_REFS | sfi.SFI_DEVERR_PAGE_RANGE
    assert (p.refs == 0).all() and (p.table == -1).all()


def test_compact_reports_entries_of_free_pages():
    """An entry whose page counts as free is reported and stays; the others follow their pages."""
    p = Pool(2, 6, 40)
    p.table[0, :3] = torch.tensor([30, 39, 12], dtype=torch.int32)
    p.refs[30] = p.refs[12] = 1                      # 39 is held by the table alone
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    sfi.sfi_pages_compact(p.kv, p.pool, n, p.ws, p.nb)
    torch.cuda.synchronize()
    assert int(n[0]) == 2 and int(p.err[0]) == sfi.SFI_DEVERR_REFS
    assert p.table[0, :3].tolist() == [1, 39, 0] and p.refs.sum() == 2


@pytest.mark.parametrize("layers,hkv", [(1, 2), (3, 1)])
def test_compact(layers, hkv):
    p = Pool(6, 20, 120, hkv=hkv, layers=layers)
    p.compact()                      # empty
    p.check()
    p.reserve([300, 10, 100, 5, 160, 0])
    p.append([300, 10, 100, 5, 160, 0])
    p.compact()                      # already at the front
    p.check()
    p.reorder([0, 1, 2, 3, 4, 4])
    sfi.sfi_pages_release(p.kv, p.pool, active=p.mask([1, 0, 1, 0, 0, 0]))
    p.model.release([1, 0, 1, 0, 0, 0])
    p.compact()
    p.check()
    assert int((p.refs > 0).nonzero().max()) == int((p.refs > 0).sum()) - 1


def test_random_life():
    """Two hundred calls in random order on a pool of more than one scan chunk."""
    rng = np.random.default_rng(7)
    p = Pool(40, 40, 17000, hkv=1, seed=1)
    p.refs[:16300] = 1                # another user's pages; the model knows them too
    p.model.refs[:16300] = 1
    base = p.model.refs.copy()
    for step in range(60):
        what = rng.integers(6)
        mask = None if rng.random() < 0.3 else (rng.random(40) < 0.6).astype(np.uint8).tolist()
        if what <= 1:
            n = rng.integers(0, 50, 40).tolist()
            ok = p.reserve(n, mask)
            p.append([a if o else 0 for a, o in zip(n, ok)])
        elif what == 2:
            p.reorder(rng.integers(0, 40, 40).tolist())
        elif what == 3:
            sfi.sfi_pages_evict(p.kv, p.pool, 4, 100, active=p.mask(mask))
            p.model.evict(4, 100, mask)
        elif what == 4:
            some = (rng.random(40) < 0.2).astype(np.uint8).tolist()
            sfi.sfi_pages_release(p.kv, p.pool, active=p.mask(some))
            p.model.release(some)
        else:
            p.reserve(rng.integers(0, 50, 40).tolist(), mask)   # ahead
        torch.cuda.synchronize()
        np.testing.assert_array_equal(p.table.cpu().numpy(), p.model.table)
        np.testing.assert_array_equal(p.refs.cpu().numpy(), p.model.refs)
        np.testing.assert_array_equal(p.seq_len.cpu().numpy(), p.model.seq_len)
        assert int(p.err[0]) == p.model.err
    assert np.array_equal(bits(p.k), p.model.k) and np.array_equal(bits(p.v), p.model.v)
    assert (p.model.refs[:16300] == base[:16300]).all()


def test_append_reports_and_skips():
    p = Pool(3, 4, 16)
    p.reserve([40, 8, 0])
    start = torch.tensor([0, 30, 20, 25], dtype=torch.int32, device="cuda")   # runs backwards
    rows = torch.zeros((1, 25, 2, D), dtype=torch.bfloat16, device="cuda")
    sfi.sfi_append_chunk(p.kv, rows, rows, start, 25, 30)
    torch.cuda.synchronize()
    assert int(p.err[0]) & sfi.SFI_DEVERR_ROWS
    assert p.seq_len[:2].tolist() == [0, 0]
    p.err.zero_()
    start = torch.tensor([0, 9, 18, 18], dtype=torch.int32, device="cuda")
    sfi.sfi_append_chunk(p.kv, rows, rows, start, 25, 30, active=p.mask([0, 1, 1]))
    torch.cuda.synchronize()
    assert int(p.err[0]) == 0 and p.seq_len.tolist() == [0, 9, 0]   # 8 reserved: one page holds 16
    start = torch.tensor([0, 0, 8, 8], dtype=torch.int32, device="cuda")
    sfi.sfi_append_chunk(p.kv, rows, rows, start, 25, 30)
    torch.cuda.synchronize()
    assert int(p.err[0]) == sfi.SFI_DEVERR_PAGE_RANGE and p.seq_len.tolist() == [0, 9, 0]


def test_append_contiguous():
    g = torch.Generator(device="cuda").manual_seed(2)
    layers, batch, hkv, cap = 2, 3, 2, 50
    k, v = (torch.zeros((layers, batch, hkv, cap, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    length = torch.tensor([0, 20, 45], dtype=torch.int32, device="cuda")
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    kv = sfi.SfiKvCache(n_layers=layers, batch=batch, n_q_heads=4, n_kv_heads=hkv, head_dim=D,
                        capacity=cap, max_len=45, k=k.data_ptr(), v=v.data_ptr(),
                        seq_len=length.data_ptr(), err=err.data_ptr())
    new = torch.randn((layers, 60, hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    start = torch.tensor([0, 50, 51, 57], dtype=torch.int32, device="cuda")
    sfi.sfi_append_chunk(kv, new, -new, start, 60, 50)
    torch.cuda.synchronize()
    assert int(err[0]) == sfi.SFI_DEVERR_CAPACITY       # 45 + 6 > 50
    assert length.tolist() == [50, 21, 45]
    assert torch.equal(k[:, 0], new[:, :50].transpose(1, 2))
    assert torch.equal(v[:, 1, :, 20], -new[:, 50]) and not k[:, 2].any()
    one = new[:, :3].contiguous()
    kv.max_len = 50
    err.zero_()
    sfi.sfi_append_chunk(kv, one, one, None, 3, 1, active=torch.tensor([0, 1, 1], dtype=torch.uint8,
                                                                      device="cuda"))
    torch.cuda.synchronize()
    assert int(err[0]) == 0 and length.tolist() == [50, 22, 46]
    assert torch.equal(k[:, 2, :, 45], one[:, 2])


@pytest.mark.parametrize("batch,paged", [(1, True), (7, True), (7, False), (200, True), (33, False)])
def test_reorder_whole_state(batch, paged):
    """Packed memory, selections, lengths, and contiguous rows, under a map with cycles and
    repeats; rows past a source's counts and lengths stay what they were."""
    g = torch.Generator(device="cuda").manual_seed(batch)
    rng = np.random.default_rng(batch)
    layers, hkv, sink, select = 2, 2, 3, 21
    i32 = dict(dtype=torch.int32, device="cuda")
    comp = sink + select
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    kc, vc = rnd(layers, batch, hkv, comp, D), rnd(layers, batch, hkv, comp, D)
    sel = torch.randint(0, 1000, (layers, batch, hkv, select), generator=g, **i32)
    rows = torch.randint(0, comp + 1, (layers, batch, hkv), generator=g, **i32)
    cnt = (rows - sink).clamp(min=0)
    length = torch.randint(0, 41, (batch,), generator=g, **i32)
    err = torch.zeros(4, **i32)
    if paged:
        cols, pages = 3, 3 * batch + 4
        table = torch.full((batch, cols), -1, **i32)
        for b in range(batch):
            for c in range((int(length[b]) + 15) // 16):
                table[b, c] = 3 * b + c
        refs = torch.bincount(table[table >= 0], minlength=pages).to(torch.int32)
        k, v = rnd(layers, pages, hkv, PAGE, D), rnd(layers, pages, hkv, PAGE, D)
        cap = 48
    else:
        cap, pages, cols, table = 41, 0, 0, None
        k, v = rnd(layers, batch, hkv, cap, D), rnd(layers, batch, hkv, cap, D)
    kv = sfi.SfiKvCache(n_layers=layers, batch=batch, n_q_heads=hkv, n_kv_heads=hkv, head_dim=D,
                        capacity=cap, page_size=PAGE if paged else 0, n_pages=pages,
                        max_pages_per_seq=cols, max_len=41, k=k.data_ptr(), v=v.data_ptr(),
                        page_table=table.data_ptr() if paged else None,
                        seq_len=length.data_ptr(), err=err.data_ptr())
    pool = sfi.SfiPagePool(page_table=table.data_ptr(), refs=refs.data_ptr()) if paged else None
    bud = sfi.SfiBudget(n_sink=sink, n_window=8, n_select=select, prior_tau=8, lambda_=0.1)
    mem = sfi.SfiSparseMem(kc=kc.data_ptr(), vc=vc.data_ptr(), sel_idx=sel.data_ptr(),
                           sel_cnt=cnt.data_ptr(), rows=rows.data_ptr())
    src = rng.integers(0, batch, batch)
    if batch > 3:
        src[:3] = [1, 2, 0]
    m = torch.from_numpy(src).cuda()
    at = torch.arange(comp, device="cuda")[None, None, None, :, None]
    live = (at < rows[:, m][..., None, None]) & (m != torch.arange(batch, device="cuda"))[None, :, None, None, None]
    want = [torch.where(live, t[:, m], t) for t in (kc, vc)] + [sel[:, m], cnt[:, m], rows[:, m], length[m]]
    if paged:
        want += [table[m], torch.bincount(table[m][table[m] >= 0], minlength=pages).to(torch.int32), k.clone(), v.clone()]
    else:
        pos = torch.arange(cap, device="cuda")[None, None, None, :, None]
        liv = pos < length[m][None, :, None, None, None]
        want += [torch.where(liv, t[:, m], t) for t in (k, v)]
    sfi.sfi_reorder(kv, m.to(torch.int32), pool=pool, budget=bud, mem=mem)
    torch.cuda.synchronize()
    have = [kc, vc, sel, cnt, rows, length] + ([table, refs, k, v] if paged else [k, v])
    assert int(err[0]) == 0
    for i, (a, b) in enumerate(zip(have, want)):
        assert torch.equal(a, b), i


def test_reorder_bad_source_left_alone():
    p = Pool(4, 4, 16)
    p.reserve([20, 5, 40, 0])
    p.append([20, 5, 40, 0])
    sfi.sfi_reorder(p.kv, torch.tensor([2, -1, 7, 0], dtype=torch.int32, device="cuda"), pool=p.pool)
    p.model.reorder(np.array([2, 1, 2, 0]))
    p.model.err = sfi.SFI_DEVERR_SEQ
    p.check()


def test_captured_step():
    """Reserve, append and reorder recorded once and replayed: the replays do what the calls do."""
    p = Pool(4, 12, 64)
    p.reserve([30, 0, 0, 17])
    p.append([30, 0, 0, 17])
    p.reorder([0, 0, 0, 3])
    p.check()
    start = np.arange(5, dtype=np.int32)
    new = torch.randn((1, 4, 2, D), device="cuda").to(torch.bfloat16)
    src, ok = torch.tensor([1, 0, 0, 3], dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sfi.sfi_pages_reserve(p.kv, p.pool, None, p.ws, p.nb, ok=ok)
        sfi.sfi_append_chunk(p.kv, new, new, None, 4, 1, active=ok)
        sfi.sfi_reorder(p.kv, src, pool=p.pool)
    for _ in range(5):
        graph.replay()
        p.model.reserve()
        p.model.append(bits(new), bits(new), start)
        p.model.reorder(src.cpu().numpy())
        p.check()
