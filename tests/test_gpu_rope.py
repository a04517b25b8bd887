"""Rotary positions against their definition in 64 bits.

Tolerance, from the arithmetic in fp32: the angle is a float of at most one half turn (2^-25 of it
off, and 2^-31 from the product's cut-off lower half: 2^-25 pi < 2^-23 radians in all), sincospif is within
2^-22, the amplitude and the products add three roundings of 2^-24: under 2^-21 of the magnitudes
that meet. The norm adds the sum of 128 squares (12 roundings in a row and halved by the root), the mean,
rsqrtf (2^-22) and two products: under 2^-20 more. bf16 outputs add half a step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import sparse_long_context_sfi_gb300 as sfi
from tests.border_model import angles, turned

pytestmark = pytest.mark.gpu

D, PAGE, EPS = 128, 16, 1e-5


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def host(t):
    return t.double().cpu().numpy()


class Case:
    """A cache of random rows (kept beside), a packed chunk of q, k and v and what turns them."""

    def __init__(self, lens, rows, hq=8, hkv=2, layers=1, rot=128, inter=False, paged=False, packed=True,
                 norm="", amplitude=1.0, tail=3, seed=0, room=20, turns=None, pages=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
        self.lens, self.rows, self.hq, self.hkv, self.layers, self.rot = lens, rows, hq, hkv, layers, rot
        self.inter, self.amplitude = inter, amplitude
        batch = len(lens)
        cols = (max(a + r for a, r in zip(lens, rows)) + room + PAGE - 1) // PAGE
        self.capacity = cols * PAGE
        self.table = None
        if paged:
            n = pages or batch * cols + 3
            self.table = torch.randperm(n, generator=g, device="cuda")[:batch * cols].to(torch.int32).view(batch, cols)
            shape = (layers, n, hkv, PAGE, D)
        else:
            shape = (layers, batch, hkv, self.capacity, D)
        self.k, self.v = rnd(*shape), rnd(*shape)
        self.k0, self.v0 = self.k.clone(), self.v.clone()
        self.starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.row_start = torch.from_numpy(self.starts).cuda()
        self.total = int(self.starts[-1]) + tail
        if packed:
            self.q, self.kn, self.vn = (rnd(layers, self.total, h, D) for h in (hq, hkv, hkv))
        else:       # rows of one projection with something behind each
            x = rnd(layers, self.total, hq + 2 * hkv + 1, D)
            self.q, self.kn, self.vn, _ = x.split([hq, hkv, hkv, 1], 2)
        self.q_out = torch.full((layers, self.total, hq, D), -7.0, device="cuda", dtype=torch.bfloat16)
        self.k_out = torch.full((layers, self.total, hkv, D), -7.0, device="cuda", dtype=torch.bfloat16)
        self.seq_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.turns = sfi.sfi_rope_turns(rot)[0] if turns is None else turns
        self.dev_turns = torch.from_numpy(self.turns.view(np.int64)).cuda()
        self.q_w, self.k_w = rnd(D) + 1, rnd(D) - 1
        self.rope = sfi.SfiRope(rot_dim=rot, interleaved=1 if inter else 0, amplitude=amplitude, norm_eps=EPS,
                                turns=self.dev_turns.data_ptr(),
                                q_norm=self.q_w.data_ptr() if "q" in norm else None,
                                k_norm=self.k_w.data_ptr() if "k" in norm else None)
        self.norm = norm
        self.kv = sfi.SfiKvCache(
            n_layers=layers, batch=batch, n_q_heads=hq, n_kv_heads=hkv, head_dim=D, capacity=self.capacity,
            page_size=PAGE if paged else 0, n_pages=shape[1] if paged else 0, max_pages_per_seq=cols if paged else 0,
            max_len=max(lens), k=self.k.data_ptr(), v=self.v.data_ptr(),
            page_table=self.table.data_ptr() if paged else None, seq_len=self.seq_len.data_ptr(),
            err=self.err.data_ptr())

    def io(self, append, pos=None, **kw):
        a = dict(q=self.q.data_ptr(), q_out=self.q_out.data_ptr(), k=self.kn.data_ptr(),
                 q_stride=self.q.stride(1), k_stride=self.kn.stride(1), v_stride=self.vn.stride(1),
                 pos=None if pos is None else pos.data_ptr())
        a.update(dict(v=self.vn.data_ptr()) if append else dict(k_out=self.k_out.data_ptr()))
        return sfi.SfiRopeRows(**{**a, **kw})

    def run(self, append, pos=None, active=None, single=False, most=None, stream=None, **kw):
        call = sfi.sfi_rope_append if append else sfi.sfi_rope_apply
        call(self.kv, self.rope, self.io(append, pos, **kw), None if single else self.row_start, self.total,
             max(max(self.rows), 1) if most is None else most, active=active, stream=stream)

    def want(self, x, weight, pos):
        return turned(host(x), angles(pos, self.turns), self.rot, self.inter, self.amplitude,
                      None if weight is None else host(weight), EPS)

    def places(self, pos=None):
        p = np.zeros(self.total, np.int64)
        for b, r in enumerate(self.rows):
            p[self.starts[b]:self.starts[b + 1]] = self.lens[b] + np.arange(r)
        return p if pos is None else host(pos).astype(np.int64)

    def close(self, got, x, which, pos, at):
        w = {"q": self.q_w, "k": self.k_w}[which] if which in self.norm else None
        y, mag = self.want(x, w, pos)
        tol = 2.0 ** (-21 if w is None else -19) * mag + 2.0 ** -8 * np.abs(y)
        bad = ~(np.abs(host(got) - y) <= tol)[:, at]
        assert not bad.any(), (which, np.argwhere(bad)[0], bad.mean())

    def slots(self, b):
        """The rows of sequence b in the cache: [layers][hkv][positions][D] views of k, v and as they were."""
        def of(t):
            if self.table is None:
                return t[:, b]
            return t[:, self.table[b].long()].permute(0, 2, 1, 3, 4).reshape(self.layers, self.hkv, -1, D)
        return tuple(of(t) for t in (self.k, self.v, self.k0, self.v0))

    def check(self, append, pos=None, skip=(), err=0):
        torch.cuda.synchronize()
        assert int(self.err[0]) == err
        at = self.places(pos)
        rows = [r for b in range(len(self.rows)) if b not in skip
                for r in range(self.starts[b], self.starts[b + 1])]
        self.close(self.q_out, self.q, "q", at, rows)
        rest = np.setdiff1d(np.arange(self.total), rows)
        assert (self.q_out[:, rest] == -7.0).all()
        if not append:
            self.close(self.k_out, self.kn, "k", at, rows)
            assert (self.k_out[:, rest] == -7.0).all()
            assert torch.equal(self.k, self.k0) and torch.equal(self.v, self.v0)
            assert self.seq_len.tolist() == self.lens
            return
        assert (self.k_out == -7.0).all()
        turned_k = torch.zeros(self.kn.shape, dtype=torch.bfloat16, device="cuda")
        for b, (n, r) in enumerate(zip(self.lens, self.rows)):
            r = 0 if b in skip else r
            assert int(self.seq_len[b]) == n + r
            k, v, k0, v0 = self.slots(b)
            s0 = self.starts[b]
            turned_k[:, s0:s0 + r] = k[:, :, n:n + r].transpose(1, 2)
            assert torch.equal(v[:, :, n:n + r].transpose(1, 2), self.vn[:, s0:s0 + r])
            keep = torch.ones(k.shape[2], dtype=torch.bool)
            keep[n:n + r] = False
            assert torch.equal(k[:, :, keep], k0[:, :, keep]) and torch.equal(v[:, :, keep], v0[:, :, keep])
        self.close(turned_k, self.kn, "k", at, rows)


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [2, 6, 16, 40, 64, 66, 96, 126, 128])
def test_layouts(rot, inter, append):
    """Part of the head and all of it; half-head distances that are no multiple of 8 among them."""
    c = Case([5, 33], [7, 20], rot=rot, inter=inter, paged=True, seed=rot)
    c.run(append)
    c.check(append)


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("norm", ["q", "k", "qk"])
@pytest.mark.parametrize("rot,inter", [(128, False), (64, True), (20, False)])
def test_norms(rot, inter, norm, append):
    c = Case([0, 100], [3, 30], rot=rot, inter=inter, norm=norm, amplitude=1.25, packed=False, seed=1)
    c.run(append)
    c.check(append)


SHAPES = [
    ([0], [1], 1, 1, 1), ([0], [1], 8, 8, 3), ([15], [2], 2, 1, 1), ([4096], [1], 8, 2, 1), ([16], [16], 16, 2, 1),
    ([7, 0, 99, 31], [0, 5, 0, 1], 8, 2, 2), ([1] * 40, [1] * 40, 32, 8, 1), ([3] * 256, [1] * 256, 2, 2, 1),
    ([100, 20], [1501, 333], 32, 4, 2), ([0, 50, 10], [2000, 1, 3000], 4, 4, 1),
    # one cluster, up to its bounds, and just beyond them
    ([9], [1], 8, 1, 8), ([9], [1], 8, 1, 9), ([5] * 16, [1] * 16, 16, 2, 1), ([5] * 17, [1] * 17, 16, 2, 1),
    ([5, 6, 7, 8], [3, 9, 1, 7], 64, 8, 1), ([30] * 8, [8] * 8, 32, 8, 1), ([30, 2], [2, 6], 32, 8, 8),
    ([15] + [0] * 15, [2] + [0] * 15, 8, 2, 1),
]


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_shapes(shape, packed, paged, append):
    lens, rows, hq, hkv, layers = SHAPES[shape]
    c = Case(lens, rows, hq, hkv, layers, paged=paged, packed=packed, seed=shape)
    c.run(append)
    c.check(append)


@pytest.mark.parametrize("append", [False, True])
def test_one_row_each(append):
    """row_start NULL, as the single tokens of a decode step."""
    c = Case([5, 0, 77], [1, 1, 1], tail=0, paged=True)
    c.run(append, single=True, most=1)
    c.check(append)


@pytest.mark.parametrize("inter", [False, True])
def test_far_and_negative_positions(inter):
    """Given positions up to the ends of 32 bits: the angle loses nothing. The cache rows of an
    append do not follow them."""
    c = Case([3, 9], [4, 6], inter=inter, tail=2)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 131071, 1, -1, 10 ** 9, -131072, 65536, 2 ** 30, 5, 5],
                       dtype=torch.int32, device="cuda")
    for append in (False, True):
        c.q_out.fill_(-7.0)
        c.run(append, pos=pos)
        if append:
            c.k_out.fill_(-7.0)
        c.check(append, pos=pos)


def test_far_positions_of_the_cache():
    """A sequence near 2^20 positions whose old pages are gone."""
    n = (1 << 20) - 5
    c = Case([n, 20], [30, 3], paged=True, pages=3 * ((1 << 20) // PAGE + 10), hkv=1, hq=1)
    c.table[0, :n // PAGE] = -1
    c.run(True)
    torch.cuda.synchronize()
    assert int(c.err[0]) == 0 and c.seq_len.tolist() == [n + 30, 23]
    c.close(c.q_out, c.q, "q", c.places(), list(range(33)))
    page = c.table[0].long()
    got = torch.stack([c.k[:, page[p // PAGE], :, p % PAGE] for p in range(n, n + 30)], 1)
    full = torch.zeros_like(c.kn)
    full[:, :30] = got
    c.close(full, c.kn, "k", c.places(), list(range(30)))


def test_turned_back():
    """The same call with the positions negated is the inverse, and so the gradient: <R x, y> = <x, R' y>."""
    c = Case([100, 7], [9, 5], tail=0, seed=5)
    pos = torch.from_numpy(c.places().astype(np.int32)).cuda()
    c.run(False, pos=pos)
    once = c.q_out.clone()
    y = torch.randn(c.q.shape, device="cuda").to(torch.bfloat16)
    back = torch.empty_like(y)
    neg = -pos
    c.run(False, pos=neg, q=y.data_ptr(), q_out=back.data_ptr(), k=None, k_out=None)
    torch.cuda.synchronize()
    # (each output is rounded by at most 2^-8 of itself)
    a, b = (once.double() * y.double()), (c.q.double() * back.double())
    assert abs(float(a.sum() - b.sum())) <= 2.0 ** -8 * float(a.abs().sum() + b.abs().sum())


@pytest.mark.parametrize("rot,inter", [(128, False), (64, False), (20, False), (64, True)])
@pytest.mark.parametrize("norm", ["", "qk"])
def test_in_place(rot, inter, norm):
    c = Case([40, 9], [12, 25], rot=rot, inter=inter, norm=norm)
    c.run(False)
    q, k = c.q_out.clone(), c.k_out.clone()
    old = c.q[:, -3:].clone()
    c.run(False, q_out=c.q.data_ptr(), k_out=c.kn.data_ptr())
    torch.cuda.synchronize()
    assert torch.equal(c.q[:, :-3], q[:, :-3]) and torch.equal(c.kn[:, :-3], k[:, :-3])
    assert torch.equal(c.q[:, -3:], old)


def test_either_pair_alone():
    c = Case([4, 5], [6, 7])
    c.run(False, k=None, k_out=None)
    torch.cuda.synchronize()
    assert (c.k_out == -7.0).all() and not (c.q_out[:, :13] == -7.0).any()
    first = c.q_out.clone()
    c.q_out.fill_(-7.0)
    c.run(False, q=None, q_out=None)
    torch.cuda.synchronize()
    assert (c.q_out == -7.0).all() and not (c.k_out[:, :13] == -7.0).any()
    c.run(True, q=None, q_out=None)
    torch.cuda.synchronize()
    assert (c.q_out == -7.0).all() and c.seq_len.tolist() == [10, 12]
    c.seq_len.copy_(torch.tensor(c.lens))
    c.run(True)
    c.k_out.fill_(-7.0)
    c.check(True)
    assert torch.equal(first, c.q_out)


def test_infinities_stay_where_they_are():
    """A dimension that is not turned keeps its infinity, and no other dimension meets it."""
    c = Case([3], [4], rot=64, tail=0)
    c.q[:, 1, :, 100] = float("inf")
    c.run(False)
    torch.cuda.synchronize()
    assert torch.isinf(c.q_out[:, 1, :, 100]).all() and torch.isinf(c.q_out).sum() == c.hq
    assert not torch.isnan(c.q_out).any()


def test_inactive_and_empty():
    c = Case([5, 6, 7], [3, 4, 2], paged=True)
    off = torch.tensor([1, 0, 1], dtype=torch.uint8, device="cuda")
    for append in (False, True):
        c.q_out.fill_(-7.0)
        c.k_out.fill_(-7.0)
        c.run(append, active=off)
        c.check(append, skip=(1,))
    c = Case([5, 6], [0, 0])
    for append in (False, True):
        c.run(append)
        c.check(append)


def test_bad_rows_and_lengths():
    """What sfi_append_chunk skips: a full sequence, too many rows, a length beyond max_len, starts
    that run backwards."""
    for append in (False, True):
        c = Case([20, 30, 40], [5, 6, 7], paged=True)
        c.run(append, most=6)
        c.check(append, skip=(2,), err=sfi.SFI_DEVERR_ROWS)
        c = Case([20, 30, 40], [5, 6, 7], paged=True)
        c.kv.max_len = 39
        c.run(append)
        c.check(append, skip=(2,), err=sfi.SFI_DEVERR_LENGTH)
        c = Case([20, 30, 40], [5, 6, 7], paged=True)
        c.row_start = torch.tensor([0, 5, 2, 9], dtype=torch.int32, device="cuda")
        c.rows, c.starts = [5, 0, 0], np.array([0, 5, 5, 5], np.int32)     # sequence 1 backwards, 2 within 0's rows
        c.run(append, most=7)
        c.check(append, skip=(1, 2), err=sfi.SFI_DEVERR_ROWS)
    c = Case([20, 30], [5, 6], paged=True, room=0)
    c.kv.capacity -= 16                       # (a table of one column less)
    c.kv.max_pages_per_seq -= 1
    c.table = c.table.view(-1)[:2 * (c.kv.max_pages_per_seq)].view(2, -1).contiguous()
    c.kv.page_table = c.table.data_ptr()
    c.kv.max_len = 30
    c.run(True)
    c.check(True, skip=(1,), err=sfi.SFI_DEVERR_CAPACITY)


def test_missing_page():
    """q is turned, the rows that have a page are written, the length stays."""
    c = Case([20, 30], [20, 6], paged=True)
    c.table[0, 2] = -1
    c.run(True)
    torch.cuda.synchronize()
    assert int(c.err[0]) == sfi.SFI_DEVERR_PAGE_RANGE and c.seq_len.tolist() == [20, 36]
    c.close(c.q_out, c.q, "q", c.places(), list(range(26)))
    page = int(c.table[0, 1])
    full = torch.zeros_like(c.kn)
    full[:, :12] = c.k[:, page, :, 4:16].transpose(1, 2)
    c.close(full, c.kn, "k", c.places(), list(range(12)))


def test_same_as_apply_then_append():
    c, d = (Case([100, 31, 0], [17, 40, 3], 16, 4, layers=2, paged=True, norm="qk", rot=96, seed=8) for _ in "ab")
    c.run(True)
    d.run(False)
    sfi.sfi_append_chunk(d.kv, d.k_out, d.vn, d.row_start, d.total, max(d.rows))
    torch.cuda.synchronize()
    assert torch.equal(c.q_out, d.q_out) and torch.equal(c.k, d.k) and torch.equal(c.v, d.v)
    assert torch.equal(c.seq_len, d.seq_len)


def test_captured_and_on_another_stream():
    c = Case([100, 31], [1, 1], tail=0, paged=True, room=40)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.run(True, single=True, most=1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    c.check(True)
    first = c.q_out.clone()
    c.kv.max_len = c.capacity
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(True, single=True, most=1)
    c.seq_len.copy_(torch.tensor(c.lens))
    c.q_out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, c.q_out) and c.seq_len.tolist() == [101, 32]
    graph.replay()                      # at the next positions
    torch.cuda.synchronize()
    assert c.seq_len.tolist() == [102, 33] and int(c.err[0]) == 0
    c.close(c.q_out, c.q, "q", np.array([101, 32]), [0, 1])
