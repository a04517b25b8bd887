"""Page upkeep one step beyond the sizes that its kernels hold on chip: pools of several chunks of
16384 pages, reserves of more than 1024 column tasks and more than 2048 pages, against the model."""
import numpy as np
import pytest
import torch

import sparse_long_context_sfi_gb300 as sfi
from tests.test_gpu_pages import Pool, built  # noqa: F401  (built: the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [16384, 16385, 40001])
def test_compaction_of_several_chunks(pages):
    """Pages all over the pool are held, some twice: tables, counts and bytes follow."""
    rng = np.random.default_rng(pages)
    p = Pool(40, 300, pages, hkv=1)
    ids = rng.permutation(pages)[:40 * 250].reshape(40, 250)
    ids[0, :4] = [pages - 1, 16383, 0, pages // 2]
    flat = np.full((40, 300), -1, np.int32)
    for b in range(40):
        n = int(rng.integers(1, 251))
        flat[b, :n] = ids[b, :n]
    flat[39] = flat[38]                                     # a fork
    seen, first = np.unique(flat[flat >= 0], return_counts=True)
    refs = np.zeros(pages, np.int32)
    refs[seen] = first
    p.table.copy_(torch.from_numpy(flat))
    p.refs.copy_(torch.from_numpy(refs))
    p.model.table, p.model.refs = flat.copy(), refs.copy()
    p.compact()
    p.check()
    used = int((refs > 0).sum())
    assert used < pages and (p.model.refs[:used] > 0).all() and not p.model.refs[used:].any()
    p.reserve([300] * 40, None)                             # and the freed ids are handed out again
    p.check(bytes_too=False)


@pytest.mark.parametrize("rows", [
    [2048 * 16], [2049 * 16], [1024 * 16 + 1] * 2,          # around the list on chip, one and two takers
    [31, 33, 511, 513, 1025, 16 * 1500, 0, 16 * 700],
])
def test_reserve_of_more_pages_than_are_listed_on_chip(rows):
    p = Pool(len(rows), 2100, 17000, hkv=1)
    p.refs[::3] = 1                                         # held by somebody else
    p.model.refs[::3] = 1
    p.reserve(rows)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(p.table.cpu().numpy(), p.model.table)
    np.testing.assert_array_equal(p.refs.cpu().numpy(), p.model.refs)
    assert int(p.err[0]) == p.model.err == 0


def test_reserve_of_more_tasks_than_fit_on_chip():
    """256 sequences of five tasks of 32 columns each, forks and refused ones among them."""
    rng = np.random.default_rng(3)
    p = Pool(256, 160, 36000, hkv=1)
    p.reserve([37] * 256)
    p.append([37] * 256)
    p.reorder([b - b % 4 for b in range(256)])
    n = (16 * 130 + rng.integers(0, 16, 256)).tolist()
    n[5] = 16 * 160                                         # past its capacity
    n[9] = 0
    for b in range(0, 256, 7):
        n[b] = 1
    ok = p.reserve(n)
    p.check(bytes_too=False)
    assert not ok[5] and ok.sum() >= 250
    p.reserve([16 * 150] * 256)                             # more than there is
    assert p.model.err & sfi.SFI_DEVERR_POOL
    p.check(bytes_too=True)
