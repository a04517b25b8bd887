"""Windowed attention where values go to the edge: keys that are not numbers or infinite, maxima that
jump, weights that nearly cancel."""
import numpy as np
import pytest
import torch

from tests.cache_model import window_attention
from tests.test_gpu_window import D, NAN, Case, built  # noqa: F401  (built: the module's fixture)

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


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("group,rows", [(1, 1), (1, 16), (2, 5), (4, 1), (4, 4), (8, 2)])
@pytest.mark.parametrize("window", [16, 300, 4096])
def test_bf16_outputs_of_few_rows_round_once(group, rows, window, paged):
    """Items of up to 16 operand rows hold their weights in two bf16 parts: half a step of the first,
    2^-8, and of the second, 2^-8 of that, leave 2^-16, which the 1e-4 of fp32 outputs covers;
    beside it an output is off by its own rounding, half a step of 2^-8, and no more."""
    lens = [4001, rows, 16, 2500, 127, 129]
    c = Case(lens, [rows] * len(lens), 2 * group, 2, paged=paged, seed=rows)
    c.run(4, window, False)
    torch.cuda.synchronize()
    got = c.out.double().cpu().numpy()
    q, k, v = (t.double().cpu().numpy() for t in (c.q, c.flat_k, c.flat_v))
    for b, n in enumerate(lens):
        r0, r1 = c.starts[b], c.starts[b + 1]
        o, mag = window_attention(q[0, r0:r1], k[0, b, :, :n], v[0, b, :, :n], n, 4, window)
        assert (np.abs(got[0, r0:r1] - o) <= 1e-4 * mag + 2.0 ** -8 * np.abs(o)).all(), b


# items of 16, 128 and (bf16 outputs) 256 operand rows; the first also split over the GPU
FORMS = [([1000, 700], [1, 2], 1000), ([20000], [1], 20000), ([1000, 700], [200, 33], 300),
         ([1100, 700], [200, 33], 1000)]


def offsets(n, how):
    """What is added to the logits of each position, in steps of 64 keys."""
    step = np.arange(n) // 64
    if how == "ascending":
        return 15.0 * (step % 12)
    if how == "descending":
        return 15.0 * (11 - step % 12)
    out = np.zeros(n)
    at = {"first": 2, "middle": n - 150, "last": n - 1, "window": n - 301}[how]
    out[max(at, 0)] = 120.0
    return out


@pytest.mark.parametrize("how", ["ascending", "descending", "first", "middle", "last", "window"])
@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_jumps_of_the_maximum(form, fp32, how):
    """Logits whose running maximum climbs by 15 every 64 keys, falls, or meets one key 120 above the
    others. A logit is off by 128 fp32 additions and a scaling, which 2^-16 of sum |q k| / sqrt(D)
    covers; a weight by twice that (its own and its row's maximum), normalised twice that."""
    lens, rows, window = FORMS[form]
    c = Case(lens, rows, 4, 1, seed=form)
    unit = torch.ones(D, device="cuda") * D ** -0.5
    c.q += (8 * unit).to(c.q.dtype)
    for b, n in enumerate(lens):
        # (8 unit . x unit / sqrt(D) = the offset, but for what q has along it already)
        x = torch.tensor(offsets(n, how) * D ** 0.5 / 8, device="cuda", dtype=torch.float32)
        c.flat_k[0, b, 0, :n] = (c.flat_k[0, b, 0, :n].float() + x[:, None] * unit).to(c.q.dtype)
    c.run(4, window, fp32)
    torch.cuda.synchronize()
    assert int(c.err[0]) == 0
    got = c.out.double().cpu().numpy()
    q, k, v = (t.double().cpu().numpy() for t in (c.q, c.flat_k, c.flat_v))
    for b, n in enumerate(lens):
        r0, r1 = c.starts[b], c.starts[b + 1]
        o, mag = window_attention(q[0, r0:r1], k[0, b, :, :n], v[0, b, :, :n], n, 4, window)
        size = np.abs(q[0, r0:r1]) @ np.abs(k[0, b, 0, :n]).T / np.sqrt(D)          # [rows][Hq][n]
        err = 4 * 2.0 ** -16 * size.max(-1)[..., None]
        tol = (1e-4 + err) * mag + (0 if fp32 else 2.0 ** -8 * (mag + np.abs(o)))
        assert (np.abs(got[0, r0:r1] - o) <= tol).all(), (b, np.abs(got[0, r0:r1] - o).max())


@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_infinite_keys(form, fp32):
    """A key with an infinite element: rows that do not see it are as without it, rows whose logit is
    -inf give it no weight, rows whose logit is +inf are not numbers."""
    lens, rows, window = FORMS[form]
    c = Case(lens, rows, 4, 1, seed=form)
    for b, n in enumerate(lens):
        for at in (n - 1, n - 80, n - window, 3):
            if at >= 0:
                c.flat_k[0, b, 0, at, 7] = float("inf")
    c.run(4, window, fp32)
    torch.cuda.synchronize()
    assert int(c.err[0]) == 0
    got = c.out.double().cpu().numpy()
    q, k, v = (t.double().cpu().numpy() for t in (c.q, c.flat_k, c.flat_v))
    kinds = set()
    for b, n in enumerate(lens):
        r0, r1 = c.starts[b], c.starts[b + 1]
        with np.errstate(invalid="ignore"):
            o, mag = window_attention(q[0, r0:r1], k[0, b, :, :n], v[0, b, :, :n], n, 4, window)
        np.testing.assert_array_equal(np.isnan(got[0, r0:r1]), np.isnan(o))
        tol = 1e-4 * mag + (0 if fp32 else 2.0 ** -8 * (mag + np.abs(o)))
        fine = ~np.isnan(o)
        assert (np.abs(got[0, r0:r1] - o)[fine] <= tol[fine]).all()
        kinds |= set(np.isnan(o).reshape(-1).tolist())
    assert kinds == {True, False} or rows == [1]
