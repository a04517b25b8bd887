"""Attention of a chunk under sinks and a sliding window, against its definition in 64 bits.

Tolerances, from the arithmetic: a weight's relative error is at most its logit's absolute
error (fp32 sums of 128 bf16 products and one fp32 scaling, logits below 64 here: under
2^-16) plus the exponential's 2^-22, twice for the normalisation: under 1e-4 / 2 in all with
the output's fp32 sum. A bf16 weight adds half a step, 2^-8; one in three bf16 parts (fp32 outputs)
adds 2^-24. So an output is off by at most (1e-4 + [bf16: 2^-8]) * sum_j w_j |v_j|, and a bf16
output by 2^-8 |o| more."""
import numpy as np
import pytest
import torch

import sparse_long_context_sfi_gb300 as sfi
from tests.cache_model import PAGE, window_attention

pytestmark = pytest.mark.gpu

D = 128
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


class Case:
    """A cache whose rows beyond the lengths (and unused pages) are NaN, and a packed chunk."""

    def __init__(self, lens, rows, hq=8, hkv=2, paged=False, layers=1, seed=0, tail=3, spare=5):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.rows, self.hq, self.hkv, self.layers = lens, rows, hq, hkv, layers
        batch, cols = len(lens), (max(max(lens), 1) + PAGE - 1) // PAGE + 1
        cap = cols * PAGE
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
        self.flat_k, self.flat_v = (rnd(layers, batch, hkv, cap, D) for _ in "kv")
        for b, n in enumerate(lens):
            self.flat_k[:, b, :, n:] = NAN
            self.flat_v[:, b, :, n:] = NAN
        self.table, pages = None, 0
        if paged:
            pages = batch * cols + spare
            perm = torch.randperm(pages, generator=g, device="cuda")[:batch * cols]
            self.table = perm.to(torch.int32).view(batch, cols)
            self.k, self.v = (torch.full((layers, pages, hkv, PAGE, D), NAN, device="cuda",
                                         dtype=torch.bfloat16) for _ in "kv")
            for t, f in ((self.k, self.flat_k), (self.v, self.flat_v)):
                t[:, perm] = f.view(layers, batch, hkv, cols, PAGE, D).permute(
                    0, 1, 3, 2, 4, 5).reshape(layers, batch * cols, hkv, PAGE, D)
        else:
            self.k, self.v = self.flat_k, self.flat_v
        self.n_rows = sum(rows)
        starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.starts = starts
        self.row_start = torch.from_numpy(starts).cuda()
        self.total = self.n_rows + tail       # rows behind the last sequence
        self.q = rnd(layers, self.total, hq, D)
        self.seq_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.kv = sfi.SfiKvCache(
            n_layers=layers, batch=batch, n_q_heads=hq, n_kv_heads=hkv, head_dim=D, capacity=cap,
            page_size=PAGE if paged else 0, n_pages=pages, max_pages_per_seq=cols if paged else 0,
            max_len=max(lens), k=self.k.data_ptr(), v=self.v.data_ptr(),
            page_table=self.table.data_ptr() if paged else None,
            seq_len=self.seq_len.data_ptr(), err=self.err.data_ptr())

    def run(self, sink, window, fp32=True, active=None, single=False, ws=None, max_rows=None):
        n = self.total
        m = max(max(self.rows), 1) if max_rows is None else max_rows
        dt = torch.float32 if fp32 else torch.bfloat16
        self.out = torch.full((self.layers, n, self.hq, D), -7.0, dtype=dt, device="cuda")
        if ws is None:
            nb = sfi.sfi_window_workspace_bytes(self.kv, n, m, sink, window)
            ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
            sfi.sfi_workspace_init(ws, nb)
        sfi.sfi_window_attn(self.kv, self.q, self.out, fp32, None if single else self.row_start, n,
                            m, sink, window, ws, ws.numel(), active=active)
        self.ws = ws
        return self.out

    def check(self, sink, window, fp32=True, skip=(), err=0):
        torch.cuda.synchronize()
        assert int(self.err[0]) == err
        got = self.out.double().cpu().numpy()
        q, k, v = (t.double().cpu().numpy() for t in (self.q, self.flat_k, self.flat_v))
        for b, (n, m) in enumerate(zip(self.lens, self.rows)):
            r0, r1 = self.starts[b], self.starts[b + 1]
            for layer in range(self.layers):
                if b in skip:
                    assert (got[layer, r0:r1] == -7.0).all()
                    continue
                if m == 0:
                    continue
                o, mag = window_attention(q[layer, r0:r1], k[layer, b, :, :n], v[layer, b, :, :n],
                                          n, sink, window)
                tol = 1e-4 * mag if fp32 else (1e-4 + 2.0 ** -8) * mag + 2.0 ** -8 * np.abs(o)
                bad = ~(np.abs(got[layer, r0:r1] - o) <= tol)
                assert not bad.any(), (b, layer, np.argwhere(bad)[0], bad.mean())
        assert (got[:, self.starts[-1]:] == -7.0).all()


# lengths, rows, query and kv heads, sinks, window
SHAPES = [
    ([1], [1], 2, 2, 4, 64),
    ([17], [17], 8, 2, 4, 5),                          # whole short prompt, window inside a page
    ([300], [300], 8, 2, 4, 64),
    ([300], [300], 4, 4, 0, 1),                        # only itself
    ([700], [140], 8, 2, 0, 100),                      # no sinks
    ([1000], [33], 16, 2, 17, 200),                    # group 8, sinks over a page's edge
    ([513], [513], 2, 2, 600, 64),                     # sinks longer than the sequence
    ([900], [260], 8, 2, 130, 16),                     # sinks over more than one tile
    ([640, 1, 0, 77, 129], [640, 1, 0, 0, 129], 8, 2, 4, 128),   # empty sequences and chunks
    ([1500, 257, 1024], [1, 2, 3], 4, 2, 4, 256),
    ([2000], [700], 4, 1, 4, 2000),                    # full causal
]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
def test_against_definition(shape, fp32, paged):
    lens, rows, hq, hkv, sink, window = shape
    c = Case(lens, rows, hq, hkv, paged=paged, seed=len(rows))
    c.run(sink, window, fp32)
    c.check(sink, window, fp32)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("window", [16, 1000, 4096])
def test_single_token(group, window, paged):
    lens = [4001, 1, 16, 2500, 127, 128, 129]
    c = Case(lens, [1] * len(lens), 2 * group, 2, paged=paged, layers=2, seed=group, tail=0)
    for fp32 in (True, False):
        c.run(4, window, fp32, single=True)
        c.check(4, window, fp32)


def test_one_row_among_long_history():
    """Few rows over a long window: the window is split over the GPU and joined."""
    c = Case([20000, 12345], [1, 3], 8, 2, seed=9)
    for window in (20000, 9000):
        c.run(64, window)
        c.check(64, window)


def test_fp32_sums_over_a_long_window():
    """The tensor core's own sums do not round to nearest; over 8000 keys the fp32 outputs stay
    within 2e-6 of the definition in the 2-norm (a single chain of such sums had 1e-5 there)."""
    c = Case([9000, 8200], [3, 130], 8, 2, seed=2)
    c.run(4, 8000)
    c.check(4, 8000)
    q, k, v = (t.double().cpu().numpy() for t in (c.q, c.flat_k, c.flat_v))
    for b, (n, m) in enumerate(zip(c.lens, c.rows)):
        r0, r1 = c.starts[b], c.starts[b + 1]
        o, _ = window_attention(q[0, r0:r1], k[0, b, :, :n], v[0, b, :, :n], n, 4, 8000)
        d = c.out[0, r0:r1].double().cpu().numpy() - o
        assert np.linalg.norm(d) <= 2e-6 * np.linalg.norm(o)


def test_layers_and_inactive_sequences():
    c = Case([500, 320, 640], [90, 320, 1], 8, 2, paged=True, layers=3)
    active = torch.tensor([1, 0, 1], dtype=torch.uint8, device="cuda")
    c.run(4, 100, False, active=active)
    c.check(4, 100, False, skip=(1,))
    c.run(4, 100, True, active=torch.zeros_like(active))
    c.check(4, 100, True, skip=(0, 1, 2))


def test_evicted_pages_are_not_read():
    """Pages outside sinks and window may be gone (the last row's window reaches back to
    length - window) and positions that nobody sees may hold anything."""
    c = Case([1600, 900], [40, 1], 8, 2, paged=True)
    sink, window = 20, 300
    for b, (n, m) in enumerate(zip(c.lens, c.rows)):
        low = n - m - window + 1
        for p in range(n):
            if sink <= p < low:
                page, r = int(c.table[b, p // PAGE]), p % PAGE
                c.k[:, page, :, r] = NAN
                c.v[:, page, :, r] = NAN
        c.table[b, (sink + PAGE - 1) // PAGE:low // PAGE] = -1
    c.run(sink, window)
    c.check(sink, window)


def test_infinite_key_and_extreme_logits():
    """A visible key of huge norm takes all the weight; logits of -1e4 underflow to zero."""
    c = Case([400], [64], 2, 2)
    c.flat_k[:, 0, :, 390] = 100 * c.q[:, 60:61, :2].mean(1)
    c.run(4, 128)
    torch.cuda.synchronize()
    assert torch.isfinite(c.out[:, :64]).all()


def test_bad_inputs_are_reported_and_skipped():
    c = Case([300, 200, 100], [50, 60, 70], 8, 2, paged=True)
    keep = c.seq_len.clone()
    c.seq_len[1] = 40                       # more rows than positions
    c.run(4, 64)
    c.check(4, 64, skip=(1,), err=sfi.SFI_DEVERR_LENGTH)
    c.seq_len.copy_(keep)
    c.err.zero_()
    c.run(4, 64, max_rows=60)               # sequence 2 has 70 rows
    c.check(4, 64, skip=(2,), err=sfi.SFI_DEVERR_ROWS)
    c.err.zero_()
    c.table[0, 17] = 10 ** 6                # visible to sequence 0
    c.run(4, 64)
    torch.cuda.synchronize()
    assert int(c.err[0]) == sfi.SFI_DEVERR_PAGE_RANGE
    assert torch.isfinite(c.out[:, 50:180].float()).all()


@pytest.mark.parametrize("fp32", [True, False])
def test_output_aligned_to_16_bytes_only(fp32):
    c = Case([300, 140], [150, 1], 8, 2, paged=True)
    c.run(4, 64, fp32)
    want = c.out.clone()
    flat = torch.full((c.out.numel() + 8,), -7.0, dtype=c.out.dtype, device="cuda")
    at = 4 if fp32 else 8
    out = flat[at:at + c.out.numel()].view(c.out.shape)
    assert out.data_ptr() % 32 == 16
    sfi.sfi_window_attn(c.kv, c.q, out, fp32, c.row_start, c.total, max(c.rows), 4, 64, c.ws, c.ws.numel())
    torch.cuda.synchronize()
    assert torch.equal(out, want) and (flat[:at] == -7.0).all() and (flat[at + out.numel():] == -7.0).all()


def test_overlapping_rows_stay_in_bounds():
    """A row_start that runs backwards: what is skipped is reported, rows of sound sequences in
    front of it are right, and no other memory is touched."""
    c = Case([3000, 2000, 2500], [2, 2, 2], 8, 2)
    c.row_start = torch.tensor([0, 2, 0, 2], dtype=torch.int32, device="cuda")
    c.n_rows, c.total = 2, 2
    c.run(4, 2048, max_rows=2)
    torch.cuda.synchronize()
    assert int(c.err[0]) == sfi.SFI_DEVERR_ROWS
    q, k, v = (t.double().cpu().numpy() for t in (c.q, c.flat_k, c.flat_v))
    o, mag = window_attention(q[0, :2], k[0, 0, :, :3000], v[0, 0, :, :3000], 3000, 4, 2048)
    assert (np.abs(c.out[0, :2].double().cpu().numpy() - o) <= 1e-4 * mag).all()


def test_cache_beyond_32_bit_offsets():
    """Rows whose byte offset passes 2^32 and whose element offset passes 2^31."""
    cap, hkv, n = 1 << 21, 4, 1000
    k = torch.zeros((1, 3, hkv, cap, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    assert k.numel() > 1 << 31
    length = torch.tensor([0, 0, cap - n - 3], dtype=torch.int32, device="cuda")
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    kv = sfi.SfiKvCache(n_layers=1, batch=3, n_q_heads=8, n_kv_heads=hkv, head_dim=D, capacity=cap,
                        max_len=cap, k=k.data_ptr(), v=v.data_ptr(), seq_len=length.data_ptr(),
                        err=err.data_ptr())
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    q, kn, vn = rnd(1, n, 8, D), rnd(1, n, hkv, D), rnd(1, n, hkv, D)
    start = torch.tensor([0, 0, 0, n], dtype=torch.int32, device="cuda")
    sfi.sfi_append_chunk(kv, kn, vn, start, n, n)
    assert torch.equal(k[0, 2, :, cap - n - 3:cap - 3], kn[0].transpose(0, 1))
    out = torch.zeros((1, n, 8, D), device="cuda")
    nb = sfi.sfi_window_workspace_bytes(kv, n, n, 0, 200)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    sfi.sfi_workspace_init(ws, nb)
    sfi.sfi_window_attn(kv, q, out, True, start, n, n, 0, 200, ws, nb)
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    # rows from 200 on see new rows alone
    o, mag = window_attention(q[0].double().cpu().numpy(), kn[0].transpose(0, 1).double().cpu().numpy(),
                              vn[0].transpose(0, 1).double().cpu().numpy(), n, 0, 200)
    assert (np.abs(out[0, 200:].double().cpu().numpy() - o[200:]) <= 1e-4 * mag[200:]).all()
    del k, v
    torch.cuda.empty_cache()


def test_calls_of_other_shapes_share_a_workspace():
    """Split items of a small call, then of a larger one whose tickets reach further, and back."""
    small = Case([4000], [1], tail=0)
    large = Case([4000] * 16, [1] * 16, hkv=8, hq=16, tail=0, seed=1)
    chunk = Case([3000, 2000], [9, 40], seed=2)
    nb = max(sfi.sfi_window_workspace_bytes(c.kv, c.total, max(c.rows), 4, 4096) for c in (small, large, chunk))
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    sfi.sfi_workspace_init(ws, nb)
    for c in (small, chunk, large, small, large, chunk):
        c.run(4, 4096, ws=ws)
        c.check(4, 4096)


def test_repeatable_and_captured():
    """The same call gives the same bits: again, on another stream, and replayed from a graph
    whose inputs changed in place; and the workspace is ready for the next call."""
    c = Case([3000, 1700], [2, 1], 8, 2, paged=True, seed=4)
    first = c.run(4, 2048).clone()
    ws = c.ws
    assert torch.equal(first, c.run(4, 2048, ws=ws))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = c.run(4, 2048, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = c.run(4, 2048, ws=ws)
    old = c.q.clone()
    c.q.copy_(old.flip(1))
    graph.replay()
    c.out = out
    c.check(4, 2048)
    c.q.copy_(old)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out)
