"""Attention to an encoder's states whose logits rise all along the states, so that the running maximum
moves, and what is summed is rescaled, again and again: against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from tests.border_model import cross_attention
from tests.test_gpu_cross import D, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def rising(c, most, first=0.0):
    """Keys along the mean query of their head, so that logits rise from `first` to about `most` for all rows."""
    n = c.lens[0]
    group = c.hq // c.hkv
    for h in range(c.hkv):
        # queries of a head: a common direction and something of their own
        common = torch.randn(D, generator=torch.Generator().manual_seed(h)).cuda()
        common /= common.norm()
        heads = c.q[0, :, h * group:(h + 1) * group].float()
        c.q[0, :, h * group:(h + 1) * group] = (0.3 * heads + 6.0 * common).to(torch.bfloat16)
        size = torch.linspace(first, most, n, device="cuda") * D ** 0.5 / 6.0
        own = c.flat_k[0, 0, h, :n].float()
        c.flat_k[0, 0, h, :n] = (0.3 * own + size[:, None] * common).to(torch.bfloat16)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("most", [40.0, 400.0, -400.0])
@pytest.mark.parametrize("rows,hq,hkv,n", [(64, 2, 2, 1500), (300, 8, 2, 2100), (3, 8, 2, 5000), (1, 4, 4, 3100)])
def test_rising_logits(rows, hq, hkv, n, most, fp32):
    """Of either size of items, shared out and whole; falling for a negative `most`."""
    c = Case([n], [rows], hq, hkv, seed=rows)
    rising(c, abs(most), 0.0)
    if most < 0:
        c.flat_k[0, 0, :, :n] = c.flat_k[0, 0, :, :n].flip(1)
    c.run(fp32)
    torch.cuda.synchronize()
    assert int(c.err[0]) == 0
    got = c.out.double().cpu().numpy()[0, :rows]
    q, k, v = (t.double().cpu().numpy() for t in (c.q, c.flat_k, c.flat_v))
    o, mag = cross_attention(q[0, :rows], k[0, 0, :, :n], v[0, 0, :, :n])
    # A weight's relative error is its logit's absolute one: 128 products and a scaling in fp32, 2^-24 each of
    # sum |q_d k_d| / sqrt(128) <= |q| |k| / sqrt(128), in the weight and in the sum it is divided by
    norm = np.linalg.norm(q[0, :rows], axis=-1).max() * np.linalg.norm(k[0, 0, :, :n], axis=-1).max() / D ** 0.5
    err = 2 * 130 * 2.0 ** -24 * norm
    parts = fp32 or rows * (hq // hkv) <= 16
    tol = (1e-4 + err + (0 if parts else 2.0 ** -8)) * mag + (0 if fp32 else 2.0 ** -8) * np.abs(o)
    bad = ~(np.abs(got - o) <= tol)
    assert not bad.any(), (np.argwhere(bad)[0], bad.mean(), np.abs(got - o).max())
    # (what is compared is a mean of many states' values, or, at the steepest, of a few)
    assert 1e-3 < np.abs(o).max() < 5
