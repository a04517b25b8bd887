"""The rotation's inverse, which is its gradient: the same call with the positions negated, element by
element. Against its definition, against the forward call undone, and against the forward call's differences.

Tolerances: an output is within 2^-21 of the magnitudes that meet in it (the derivation stands with the other
tests of rotary positions) and half a step of bf16, 2^-8 of its value."""
import numpy as np
import pytest
import torch

from tests.border_model import angles, turned
from tests.test_gpu_rope import D, Case, host

pytestmark = pytest.mark.gpu

LAYOUTS = [(128, False), (128, True), (64, False), (20, False), (20, True), (66, True)]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def device_positions(p):
    return torch.from_numpy(np.asarray(p).astype(np.int32)).cuda()


@pytest.mark.parametrize("rot,inter", LAYOUTS)
def test_against_definition_and_undone(rot, inter):
    c = Case([100, 7], [9, 5], rot=rot, inter=inter, tail=0, seed=5)
    at = c.places()
    pos, neg = device_positions(at), device_positions(-at)
    c.run(False, pos=pos)
    once = c.q_out.clone()
    g = torch.Generator(device="cuda").manual_seed(6)
    y = torch.randn(c.q.shape, generator=g, device="cuda").to(torch.bfloat16)
    back, undone = torch.empty_like(y), torch.empty_like(y)
    for x, out in ((y, back), (once, undone)):
        c.run(False, pos=neg, q=x.data_ptr(), q_out=out.data_ptr(), k=None, k_out=None)
    torch.cuda.synchronize()
    assert int(c.err[0]) == 0
    want, mag = turned(host(y), angles(-at, c.turns), rot, inter)
    assert (np.abs(host(back) - want) <= 2.0 ** -21 * mag + 2.0 ** -8 * np.abs(want)).all()
    # forwards each of the two values that meet was rounded: 2^-8 of itself, 2^-21 of what met in it (at most
    # sqrt 2 of mag, as a rotation keeps the norm; 2^-19.5 for both); then as above, of what came out of that
    _, mag = turned(host(once), angles(-at, c.turns), rot, inter)
    x = host(c.q)
    first = (2.0 ** -8 * (1 + 2.0 ** -7) + 2.0 ** -19) * mag
    assert (np.abs(host(undone) - x) <= first + 2.0 ** -21 * mag + 2.0 ** -8 * (np.abs(x) + first)).all()
    assert not torch.equal(undone, once) and not torch.equal(back, y)


@pytest.mark.parametrize("position", [1, 77, 100003, -5])
@pytest.mark.parametrize("rot,inter", LAYOUTS)
def test_against_differences(rot, inter, position):
    """Of f(x) = <R x, y> the derivative by x_d is f(e_d), f being linear: the forward call on unit vectors."""
    c = Case([0], [D], rot=rot, inter=inter, tail=0, hq=2, hkv=1, seed=8)
    c.q[0] = torch.eye(D, device="cuda", dtype=torch.bfloat16)[:, None]
    pos, neg = device_positions(np.full(D, position)), device_positions(np.full(D, -position))
    c.run(False, pos=pos, k=None, k_out=None)
    g = torch.Generator(device="cuda").manual_seed(9)
    y = torch.randn((1, 1, 2, D), generator=g, device="cuda").to(torch.bfloat16).expand(1, D, 2, D).contiguous()
    grad = torch.empty_like(y)
    c.run(False, pos=neg, q=y.data_ptr(), q_out=grad.data_ptr(), k=None, k_out=None)
    torch.cuda.synchronize()
    each = host(c.q_out)[0] * host(y)[0]                    # [e_d][head][dimension]
    want, mag = each.sum(-1).T, np.abs(each).sum(-1).T      # [head][d]
    # (the forward call's factors: half a step of bf16, 2^-21 of 1 where they are small, and the same of the gradient)
    top = np.abs(host(y)[0, 0]).max(-1)[:, None]
    tol = 2.0 ** -8 * (1 + 2.0 ** -7) * mag + 2.0 ** -19 * top + 2.0 ** -8 * np.abs(want)
    assert (np.abs(host(grad)[0, 0] - want) <= tol * (1 + 2.0 ** -7)).all()
