"""Packed chunks whose row_start is not ascending: sfi_append_chunk and sfi_window_attn leave out
the same sequences, and of those nothing is written."""
import numpy as np
import pytest
import torch

import sparse_long_context_sfi_gb300 as sfi
from tests.cache_model import PAGE, window_attention
from tests.test_gpu_pages import D, Pool, bits, built  # noqa: F401  (built: the module's fixture)

pytestmark = pytest.mark.gpu


def served(start, n_rows, max_rows):
    """Sequences that are taken: rows within bounds, and none before the end of an earlier start."""
    out = []
    for b in range(len(start) - 1):
        s0, s1 = start[b], start[b + 1]
        ok = 0 <= s0 <= s1 <= n_rows and s1 - s0 <= max_rows
        out.append(ok and (s0 == s1 or max(start[:b + 1]) == s0))
    return out


@pytest.mark.parametrize("start,n_rows,max_rows", [
    ([0, 5, 3, 8], 8, 8),           # the middle runs backwards; the last begins inside the first
    ([0, 5, 3, 4, 9], 12, 8),
    ([0, 2, 0, 2], 2, 2),
    ([4, 9, 2, 3, 9, 12], 12, 12),
    ([0, 6, 6, 20, 9, 11], 16, 16),     # one runs past n_rows
    ([-2, 3, 7, 7], 8, 8),
    ([0, 40, 40, 37, 60] + list(range(60, 100)), 100, 64),     # more starts than a warp has lanes
])
def test_starts_that_run_backwards(start, n_rows, max_rows):
    batch = len(start) - 1
    p = Pool(batch, 8, batch * 8 + 3, layers=2)
    first = [17 + b % 5 for b in range(batch)]
    p.reserve(first)
    p.append(first)
    p.reserve([80] * batch)
    p.check()
    k, v, q = (torch.randn((2, n_rows, 2, D), generator=p.g, device="cuda").to(torch.bfloat16)
               for _ in "kvq")
    dev = torch.tensor(start, dtype=torch.int32, device="cuda")
    sfi.sfi_append_chunk(p.kv, k, v, dev, n_rows, max_rows)
    ok = served(start, n_rows, max_rows)
    assert not all(ok)
    kn, vn = bits(k), bits(v)
    for b in range(batch):
        for i in range(start[b], start[b + 1]) if ok[b] else ():
            at = int(p.model.seq_len[b])
            page = p.model.table[b, at // PAGE]
            p.model.k[:, page, :, at % PAGE], p.model.v[:, page, :, at % PAGE] = kn[:, i], vn[:, i]
            p.model.seq_len[b] += 1
    p.model.err = sfi.SFI_DEVERR_ROWS
    p.check()
    # and the attention of the same rows
    p.err.zero_()
    out = torch.full(q.shape, -7.0, device="cuda")
    nb = sfi.sfi_window_workspace_bytes(p.kv, n_rows, max_rows, 4, 30)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    sfi.sfi_workspace_init(ws, nb)
    sfi.sfi_window_attn(p.kv, q, out, True, dev, n_rows, max_rows, 4, 30, ws, nb)
    torch.cuda.synchronize()
    assert int(p.err[0]) == sfi.SFI_DEVERR_ROWS
    got = out.double().cpu().numpy()
    cache = [t.double().cpu().numpy() for t in (p.k, p.v)]
    want_rows = set()
    for b in range(batch):
        m = start[b + 1] - start[b]
        if not ok[b] or m == 0:
            continue
        n = int(p.model.seq_len[b])
        pages = p.model.table[b, :(n + PAGE - 1) // PAGE]
        for layer in range(2):
            kb, vb = (t[layer, pages].transpose(1, 0, 2, 3).reshape(2, -1, D)[:, :n] for t in cache)
            o, mag = window_attention(q[layer, start[b]:start[b + 1]].double().cpu().numpy(), kb, vb, n, 4, 30)
            assert (np.abs(got[layer, start[b]:start[b + 1]] - o) <= 1e-4 * mag).all(), b
        want_rows |= set(range(start[b], start[b + 1]))
    rest = [r for r in range(n_rows) if r not in want_rows]
    assert (got[:, rest] == -7.0).all()
