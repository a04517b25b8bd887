"""Beam selection over the whole range of finite logits: where two different logits differ by so much
that one has all the weight, equal ones still share it."""
import pytest
import torch

from tests.test_gpu_beam import built, check, run  # noqa: F401  (built: the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [600, 20001])
def test_logits_up_to_the_types_largest(dtype, vocab):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    top = torch.finfo(dtype).max
    x = torch.randn((12, vocab), generator=g, device="cuda").to(dtype)
    x[0, 300] = top                                   # one forced token
    x[1, 5] = x[1, 599] = top                         # two equal ones share the weight
    x[2, 77], x[2, 78], x[2, 79] = top, top / 2, 2.0 ** 126
    x[3, :] = top                                     # a uniform row
    x[4, 9] = 2.0 ** 126
    x[5, 9] = 2.0 ** 125
    x[6, 17], x[6, 18] = 2.4e38, -top
    x[7, 1] = 1e38
    x[8, 3] = x[8, vocab - 1] = 9e37
    x[9, :] = -top
    x[9, 4] = top
    x[10, 8] = 2.0 ** 124
    x[11, :] = 2.0 ** 126
    cum = -torch.rand(12, generator=g, device="cuda")
    # a beam a group: each row's score is seen (the logarithm of 20001 is the largest, under 64)
    for rows in range(12):
        one, c = x[rows:rows + 1].contiguous(), cum[rows:rows + 1].contiguous()
        o = run(one, c, 1)
        check(o, one, c, 1)
    for beams in (3, 4, 12):
        o = run(x, cum, beams)
        check(o, x, cum, beams)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_logits_of_every_size(dtype, sign):
    """Rows whose largest logits lie at 2^10 to 2^126 in size, next to each other and equal."""
    g = torch.Generator(device="cuda").manual_seed(4)
    cum = -torch.rand(3, generator=g, device="cuda")
    step = torch.finfo(dtype).eps
    for e in list(range(10, 40)) + [60, 100, 124, 125, 126]:
        for m in (1.0, 1.3, 1.9):
            big = sign * m * 2.0 ** e
            x = (torch.randn((3, 9001), generator=g, device="cuda") * 3).to(dtype)
            if sign < 0:
                x = (x.float() * 2.0 ** (e - 4) + 4 * big).to(dtype)      # all of them below
            near = torch.tensor(big, dtype=dtype).item()
            x[0, 8000] = near
            x[1, 5] = x[1, 6000] = x[1, 6001] = near
            x[2, 100] = near
            x[2, 99] = torch.tensor(near - abs(near) * step, dtype=dtype).item()
            x = x.clamp(torch.finfo(dtype).min, torch.finfo(dtype).max)
            o = run(x, cum, 3)
            check(o, x, cum, 3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masks_beside_each_other(dtype):
    """A row of the type's lowest value and -inf: the first share the weight, the others stay -inf."""
    lo = torch.finfo(dtype).min
    x = torch.full((4, 5000), -float("inf"), device="cuda", dtype=dtype)
    x[0, 70] = x[0, 4000] = lo
    x[1, 3] = lo
    x[2, 9], x[2, 4999] = lo, lo / 2
    x[3, 11] = -2.0 ** 126
    cum = -torch.arange(4, device="cuda", dtype=torch.float32)
    for beams in (1, 2, 4):
        o = run(x, cum, beams)
        check(o, x, cum, beams)
