"""Windowed attention where values go to the edge: keys that are not numbers."""
import pytest
import torch

from tests.test_gpu_window import NAN, Case, built  # noqa: F401  (built: the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("at,window", [(10000, 20000), (20, 9000), (11001, 9000)])
def test_nan_key_shows_in_the_rows_that_see_it(at, window, paged, fp32):
    """One key that is not a number, in a window that is split over the GPU: the rows that see it
    are not numbers either, the others are what they are without it. 11001 is the first key of
    the first of three rows alone, 20 a sink."""
    c = Case([20000, 20003], [1, 3], 8, 2, paged=paged, seed=9)
    c.run(64, window, fp32)
    clean = c.out.clone()
    head = 1
    for b in (0, 1):
        c.flat_k[0, b, head, at, 5] = NAN
        if paged:
            c.k[0, int(c.table[b, at // 16]), head, at % 16, 5] = NAN
    c.run(64, window, fp32)
    torch.cuda.synchronize()
    assert int(c.err[0]) == 0
    seen = [at < 64 or at > p - window for p in (19999, 20000, 20001, 20002)]
    for row, s in enumerate(seen):
        out = c.out[0, row].float()
        assert torch.isnan(out[4:]).all() if s else torch.equal(c.out[0, row, 4:], clean[0, row, 4:]), row
        assert torch.equal(c.out[0, row, :4], clean[0, row, :4]), row
    assert any(seen)
