"""Dimensions behind rot_dim come out of a rotation without norms as they went in, bit for bit: signed
zeros, the smallest and the largest numbers, infinities."""
import pytest
import torch

from tests.test_gpu_rope import D, Case

pytestmark = pytest.mark.gpu

VALUES = [0.0, -0.0, 2.0 ** -133, -2.0 ** -133, 2.0 ** -126, 3.3895e38, -3.3895e38, float("inf"), -float("inf"), 1.0, -1.5]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [2, 20, 40, 64, 66, 96, 126])
def test_bits(rot, inter, append):
    c = Case([3, 40], [11, 30], rot=rot, inter=inter, paged=True, amplitude=1.25, seed=rot)
    rest = D - rot
    for t in (c.q, c.kn):
        n = t.shape[0] * t.shape[1] * t.shape[2] * rest
        t[..., rot:] = torch.tensor(VALUES, device="cuda").repeat(n // len(VALUES) + 1)[:n].view(
            *t.shape[:3], rest).to(torch.bfloat16)
    c.run(append)
    torch.cuda.synchronize()
    assert int(c.err[0]) == 0
    bits = lambda t: t[..., rot:].contiguous().view(torch.int16)
    n = int(c.starts[-1])
    assert (bits(c.q_out[:, :n]) == bits(c.q[:, :n])).all()
    if not append:
        assert (bits(c.k_out[:, :n]) == bits(c.kn[:, :n])).all()
        return
    for b, (a, r) in enumerate(zip(c.lens, c.rows)):
        k = c.slots(b)[0][:, :, a:a + r].transpose(1, 2)
        assert (bits(k) == bits(c.kn[:, c.starts[b]:c.starts[b + 1]])).all()
