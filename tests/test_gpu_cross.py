"""Attention to an encoder's states, against its definition in 64 bits. Tolerances as in
test_gpu_window.py: (1e-4 + [one bf16 part: 2^-8]) * sum_j w_j |v_j|, and 2^-8 |o| of a bf16 output."""
import numpy as np
import pytest
import torch

import sparse_long_context_sfi_gb300 as sfi
from tests.border_model import cross_attention

pytestmark = pytest.mark.gpu

D, PAGE, NAN = 128, 16, float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


class Case:
    """Encoder states whose rows beyond the lengths (and unused pages) are NaN, and packed rows."""

    def __init__(self, lens, rows, hq=8, hkv=2, paged=False, layers=1, seed=0, tail=3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.rows, self.hq, self.hkv, self.layers = lens, rows, hq, hkv, layers
        batch, cols = len(lens), max(lens) // PAGE + 2
        cap = cols * PAGE
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
        self.flat_k, self.flat_v = (rnd(layers, batch, hkv, cap, D) for _ in "kv")
        for b, n in enumerate(lens):
            self.flat_k[:, b, :, n:] = NAN
            self.flat_v[:, b, :, n:] = NAN
        self.table, pages = None, 0
        self.k, self.v = self.flat_k, self.flat_v
        if paged:
            pages = batch * cols + 5
            perm = torch.randperm(pages, generator=g, device="cuda")[:batch * cols]
            self.table = perm.to(torch.int32).view(batch, cols)
            self.k, self.v = (torch.full((layers, pages, hkv, PAGE, D), NAN, device="cuda",
                                         dtype=torch.bfloat16) for _ in "kv")
            for t, f in ((self.k, self.flat_k), (self.v, self.flat_v)):
                t[:, perm] = f.view(layers, batch, hkv, cols, PAGE, D).permute(
                    0, 1, 3, 2, 4, 5).reshape(layers, batch * cols, hkv, PAGE, D)
            for b, n in enumerate(lens):        # pages behind the end are missing
                self.table[b, (n + PAGE - 1) // PAGE:] = -1
        self.starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.row_start = torch.from_numpy(self.starts).cuda()
        self.total = int(self.starts[-1]) + tail
        self.q = rnd(layers, self.total, hq, D)
        self.seq_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.kv = sfi.SfiKvCache(
            n_layers=layers, batch=batch, n_q_heads=hq, n_kv_heads=hkv, head_dim=D, capacity=cap,
            page_size=PAGE if paged else 0, n_pages=pages, max_pages_per_seq=cols if paged else 0,
            max_len=max(lens), k=self.k.data_ptr(), v=self.v.data_ptr(),
            page_table=self.table.data_ptr() if paged else None,
            seq_len=self.seq_len.data_ptr(), err=self.err.data_ptr())
        self.ws = None

    def run(self, fp32=True, active=None, single=False, ws=None, max_rows=None, stream=None):
        n = self.total
        m = max(max(self.rows), 1) if max_rows is None else max_rows
        self.out = torch.full((self.layers, n, self.hq, D), -7.0, device="cuda",
                              dtype=torch.float32 if fp32 else torch.bfloat16)
        if ws is None:
            nb = sfi.sfi_cross_workspace_bytes(self.kv, n, m)
            ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
            sfi.sfi_workspace_init(ws, nb)
        sfi.sfi_cross_attn(self.kv, self.q, self.out, fp32, None if single else self.row_start, n, m, ws,
                           ws.numel(), active=active, stream=stream)
        self.ws = ws
        return self.out

    def check(self, fp32=True, skip=(), err=0):
        torch.cuda.synchronize()
        assert int(self.err[0]) == err
        got = self.out.double().cpu().numpy()
        q, k, v = (t.double().cpu().numpy() for t in (self.q, self.flat_k, self.flat_v))
        parts = fp32 or max(self.rows) * (self.hq // self.hkv) <= 16
        for b, n in enumerate(self.lens):
            r0, r1 = self.starts[b], self.starts[b + 1]
            for layer in range(self.layers):
                if b in skip:
                    assert (got[layer, r0:r1] == -7.0).all()
                    continue
                o, mag = cross_attention(q[layer, r0:r1], k[layer, b, :, :n], v[layer, b, :, :n])
                tol = (1e-4 + (0 if parts else 2.0 ** -8)) * mag + (0 if fp32 else 2.0 ** -8) * np.abs(o)
                bad = ~(np.abs(got[layer, r0:r1] - o) <= tol)
                assert not bad.any(), (b, layer, np.argwhere(bad)[0], bad.mean())
                if n == 0:
                    assert (got[layer, r0:r1] == 0).all()
        assert (got[:, self.starts[-1]:] == -7.0).all()


# encoder lengths, rows, query and kv heads
SHAPES = [
    ([1], [1], 2, 2), ([0], [1], 8, 2), ([0, 0], [40, 3], 8, 2), ([15, 16, 17], [1, 1, 1], 8, 8),
    ([63, 64, 65], [4, 2, 3], 8, 2), ([127, 128, 129], [33, 32, 31], 8, 2),
    ([601], [1], 8, 2), ([1000, 0, 3, 511], [200, 9, 65, 0], 16, 2),
    ([513, 512], [257, 256], 2, 2), ([2000, 700], [300, 129], 4, 1), ([40], [1000], 4, 4),
    ([3000, 0, 2500], [2, 3, 1], 16, 2), ([1300] * 5, [64, 0, 1, 700, 128], 8, 1),
]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_against_definition(shape, fp32, paged):
    lens, rows, hq, hkv = SHAPES[shape]
    c = Case(lens, rows, hq, hkv, paged=paged, seed=shape)
    c.run(fp32)
    c.check(fp32)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_one_row_each(group, paged):
    lens = [4001, 1, 16, 0, 127, 128, 129]
    c = Case(lens, [1] * len(lens), 2 * group, 2, paged=paged, layers=2, seed=group, tail=0)
    for fp32 in (True, False):
        c.run(fp32, single=True)
        c.check(fp32)


def test_few_rows_of_long_states():
    """Split over the GPU and joined; one of the sequences is empty."""
    c = Case([20000, 0, 12345], [1, 2, 3], 8, 2, seed=9)
    for fp32 in (True, False):
        c.run(fp32)
        c.check(fp32)


def test_fp32_sums_over_long_states():
    c = Case([9000, 8200], [3, 130], 8, 2, seed=2)
    c.run()
    c.check()
    q, k, v = (t.double().cpu().numpy() for t in (c.q, c.flat_k, c.flat_v))
    for b, n in enumerate(c.lens):
        r0, r1 = c.starts[b], c.starts[b + 1]
        o, _ = cross_attention(q[0, r0:r1], k[0, b, :, :n], v[0, b, :, :n])
        d = c.out[0, r0:r1].double().cpu().numpy() - o
        assert np.linalg.norm(d) <= 2e-6 * np.linalg.norm(o)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("paged", [False, True])
def test_many_short_items(paged, fp32):
    """More items than twice the CTAs, of very different lengths, empty ones in rows: a queue."""
    g = np.random.default_rng(5)
    lens = [0] * 9 + g.integers(0, 300, 20).tolist() + [0] * 10 + [1, 2, 16, 17, 400] + [0] * 6
    rows = g.integers(0, 90, len(lens)).tolist()
    c = Case(lens, rows, 16, 16, paged=paged, seed=1)
    c.run(fp32)
    c.check(fp32)


@pytest.mark.parametrize("paged", [False, True])
def test_many_long_items(paged):
    """The same with items of two q tiles."""
    lens = [700, 0, 0, 900, 513, 1, 0, 640, 64, 0]
    c = Case(lens, [257, 300, 256, 200, 129, 700, 128, 40, 300, 255], 32, 16, paged=paged, seed=2)
    c.run(False)
    c.check(False)
    again = c.out.clone()
    c.run(False, ws=c.ws)
    torch.cuda.synchronize()
    assert torch.equal(again, c.out)


@pytest.mark.parametrize("rows", [1, 3])
def test_widest_batch(rows):
    lens = [(37 * i) % 97 for i in range(256)]
    c = Case(lens, [rows if i % 5 else 0 for i in range(256)], 8, 2, paged=True, seed=3)
    for fp32 in (True, False):
        c.run(fp32)
        c.check(fp32)


def test_queue_and_shares_use_a_workspace_in_turn():
    many = Case([100] * 50, [60] * 50, 16, 16, seed=1)
    few = Case([3000, 10], [4, 2], 8, 2, seed=2)
    nb = max(sfi.sfi_cross_workspace_bytes(c.kv, c.total, max(c.rows)) for c in (many, few))
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    sfi.sfi_workspace_init(ws, nb)
    for c in (many, few, many, many, few):
        c.run(ws=ws)
        c.check()


def test_layers_and_inactive_sequences():
    c = Case([500, 320, 0], [90, 320, 4], 8, 2, paged=True, layers=3)
    active = torch.tensor([1, 0, 1], dtype=torch.uint8, device="cuda")
    c.run(False, active=active)
    c.check(False, skip=(1,))
    c.run(True, active=torch.zeros_like(active))
    c.check(True, skip=(0, 1, 2))


def test_jumps_of_the_maximum():
    """Ever larger logits, and one key that takes all the weight."""
    c = Case([1500], [64], 2, 2)
    c.flat_k[0, 0] *= torch.linspace(0.1, 6, c.flat_k.shape[3], device="cuda").to(torch.bfloat16)[None, :, None]
    c.flat_k[0, 0, :, 1400] = 100 * c.q[0, 60:61, :2].mean(1)
    c.run()
    torch.cuda.synchronize()
    assert torch.isfinite(c.out[:, :64]).all()


def jump_case(rows, hq, hkv, n, places, sizes, seed=3):
    """Keys that a row's query finds at `places` with ever larger logits, of `sizes` in powers of e."""
    c = Case([n], [rows], hq, hkv, seed=seed)
    for i, (at, size) in enumerate(zip(places, sizes)):
        for h in range(hkv):
            # (the first query head of the group, one row after the other)
            q = c.q[0, i % rows, h * (hq // hkv)].double()
            c.flat_k[0, 0, h, at] = (q * (size * D ** 0.5 / float(q @ q))).to(torch.bfloat16)
    return c


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("rows,hq,hkv", [(100, 8, 2), (40, 2, 2), (3, 4, 2)])
@pytest.mark.parametrize("column", [0, 5, 33, 40, 64, 70, 97, 127])
def test_maxima_far_above_the_first_tile(column, rows, hq, hkv, fp32):
    """Jumps by 2^64 and more in every 32-column piece of later tiles, of either size of tiles."""
    n = 1400
    places = [256 + column, 256 + (column + 31) % 128, 512 + column, 640 + column, 1024 + (column + 64) % 128]
    c = jump_case(rows, hq, hkv, n, places, [60.0, 120.0, 180.0, 300.0, 500.0], seed=column)
    c.run(fp32)
    torch.cuda.synchronize()
    got = c.out.double().cpu().numpy()[0, :rows]
    q, k, v = (t.double().cpu().numpy() for t in (c.q, c.flat_k, c.flat_v))
    o, mag = cross_attention(q[0, :rows], k[0, 0, :, :n], v[0, 0, :, :n])
    # Logits of up to 500 and more: a weight's relative error is its logit's absolute one, 128 products and a
    # scaling in fp32 at 2^-24 each of sum |q_d k_d| / sqrt(128) <= |q| |k| / sqrt(128), twice
    norm = np.linalg.norm(q[0, :rows], axis=-1).max() * np.linalg.norm(k[0, 0, :, :n], axis=-1).max() / 128 ** 0.5
    err = 2 * 130 * 2.0 ** -24 * norm
    parts = fp32 or rows * (hq // hkv) <= 16
    tol = (1e-4 + err + (0 if parts else 2.0 ** -8)) * mag + (0 if fp32 else 2.0 ** -8) * np.abs(o)
    assert (np.abs(got - o) <= tol).all(), np.abs(got - o).max()


def test_keys_of_minus_infinity_first():
    """A first tile whose logits are all -inf, and a sequence that has no others: its sum is nothing."""
    c = Case([400, 100], [40, 2], 2, 2)
    c.q[..., 0] = 1.0
    c.flat_k[0, 0, :, :300] = 0
    c.flat_k[0, 0, :, :300, 0] = float("-inf")
    c.run(False)
    torch.cuda.synchronize()
    q, k, v = (t.double().cpu().numpy() for t in (c.q, c.flat_k, c.flat_v))
    o, mag = cross_attention(q[0, :40], k[0, 0, :, 300:400], v[0, 0, :, 300:400])
    got = c.out.double().cpu().numpy()
    assert (np.abs(got[0, :40] - o) <= (1e-4 + 2.0 ** -8) * mag + 2.0 ** -8 * np.abs(o)).all()
    assert np.isfinite(got[0, 40:42]).all()


def test_bad_inputs_are_reported_and_skipped():
    c = Case([300, 200, 100], [50, 60, 70], 8, 2, paged=True)
    c.run(max_rows=60)
    c.check(skip=(2,), err=sfi.SFI_DEVERR_ROWS)
    c.err.zero_()
    c.kv.max_len = 250
    c.run()
    c.check(skip=(0,), err=sfi.SFI_DEVERR_LENGTH)
    c.err.zero_()
    c.kv.max_len = 300
    c.seq_len[1] = -1
    c.run()
    c.check(skip=(1,), err=sfi.SFI_DEVERR_LENGTH)
    c.err.zero_()
    c.seq_len[1] = 200
    c.table[0, 17] = 10 ** 6
    c.run()
    torch.cuda.synchronize()
    assert int(c.err[0]) == sfi.SFI_DEVERR_PAGE_RANGE
    assert torch.isfinite(c.out[:, 50:180]).all()


def test_more_rows_than_states():
    """Rows and lengths have nothing to do with each other (a chunk of the cache itself would be refused)."""
    c = Case([3, 1], [500, 2], 8, 2)
    c.run(False)
    c.check(False)


@pytest.mark.parametrize("fp32", [True, False])
def test_output_aligned_to_16_bytes_only(fp32):
    c = Case([300, 0], [150, 1], 8, 2, paged=True)
    want = c.run(fp32).clone()
    flat = torch.full((c.out.numel() + 8,), -7.0, dtype=c.out.dtype, device="cuda")
    at = 4 if fp32 else 8
    out = flat[at:at + c.out.numel()].view(c.out.shape)
    sfi.sfi_cross_attn(c.kv, c.q, out, fp32, c.row_start, c.total, max(c.rows), c.ws, c.ws.numel())
    torch.cuda.synchronize()
    assert torch.equal(out, want) and (flat[:at] == -7.0).all() and (flat[at + out.numel():] == -7.0).all()


def test_calls_of_other_shapes_share_a_workspace():
    small = Case([4000], [1], tail=0)
    large = Case([4000] * 16, [1] * 16, hkv=8, hq=16, tail=0, seed=1)
    chunk = Case([3000, 2000], [9, 40], seed=2)
    nb = max(sfi.sfi_cross_workspace_bytes(c.kv, c.total, max(c.rows)) for c in (small, large, chunk))
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    sfi.sfi_workspace_init(ws, nb)
    for c in (small, chunk, large, small, large, chunk):
        c.run(ws=ws)
        c.check()


def test_repeatable_captured_and_on_another_stream():
    c = Case([3000, 1700], [2, 1], 8, 2, paged=True, seed=4)
    first = c.run().clone()
    ws = c.ws
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = c.run(ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = c.run(ws=ws)
    old = c.q.clone()
    c.q.copy_(old.flip(1))
    graph.replay()
    c.out = out
    c.check()
    c.q.copy_(old)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out)
