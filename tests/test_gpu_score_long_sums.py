"""Log probabilities of rows that one or two warps go through in 60 to 130 chunks, and of which a lane sums
thousands of terms, with references that move in every chunk among them.

Tolerance, in units of 2^-24 of a sum, for n chunks of a warp: a chunk's terms are added up 16 times at most
(bf16: 32 tokens of a lane in pairs; fp32: 16, 8 times), the pair's halves once. Every chunk after a term's own
adds once and may move the reference: a product and an ex2 of 2^-22, 5 units. Lanes, warps and CTAs join by 5 moved
sums and 5 additions each, and a CTA's lanes by two more of each: 17 + 6 n + 40 in all. A term's distance to the
reference rounds to 2^-24 of itself, below 24 powers of two for terms that count: 1.0e-6; the moves' distances, which
add up to as much, the same; logf is within an ulp of at most 16: 1.0e-6. Entropy takes the sum's error once and the
mean distance's, at most ln vocab, twice."""
import math

import numpy as np
import pytest
import torch

from tests.border_model import score
from tests.test_gpu_score import Run, logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def check(run, rows, chunks):
    """The numbers of some rows."""
    torch.cuda.synchronize()
    at = torch.tensor(rows, device="cuda")
    vocab = run.x.shape[1]
    tol = (57 + 6 * chunks) * 2.0 ** -24 + 3.2e-6
    lp, rank, ent, top, top_lp = score(run.x[at].double().cpu().numpy(), run.token[at].cpu().numpy(), run.n_top)
    host = lambda t: t[at].double().cpu().numpy()

    def close(got, want, more=1.0):
        bad = ~(np.abs(got - want) <= tol * more + 2.0 ** -23 * np.abs(want))
        assert not bad.any(), (np.argwhere(bad)[0], np.abs(got - want).max())

    close(host(run.lp), lp)
    close(host(run.ent), ent, 1 + 2 * math.log(vocab))
    assert (host(run.rank) == rank).all()
    if run.n_top:
        assert (host(run.top)[:, :run.n_top] == top).all()
        close(host(run.top_lp)[:, :run.n_top], top_lp)


# rows, vocabulary, type, alternatives, chunks of a warp (of 1024 tokens of bf16, 512 of fp32)
SHAPES = [
    (2048, 128001, torch.bfloat16, 0, 63), (2048, 128001, torch.bfloat16, 8, 63),       # two warps a row
    (4256, 65000, torch.bfloat16, 3, 64), (4200, 128001, torch.bfloat16, 3, 126),       # one
    (2100, 64001, torch.float32, 3, 63),                                                # two
    (4256, 33000, torch.float32, 0, 65), (4256, 64001, torch.float32, 3, 126),          # one
]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("kind", ["random", "rising", "falling", "far"])
def test_sums(shape, kind):
    rows, vocab, dtype, n_top, chunks = SHAPES[shape]
    x, token = logits(rows, vocab, dtype, seed=shape)
    if kind in ("rising", "falling"):
        # (steep enough that every chunk's highest logit is above the last one's, flat enough that many count)
        x += torch.linspace(0, 60, vocab, device="cuda").to(dtype)
        if kind == "falling":
            x.copy_(x.flip(1))
    elif kind == "far":
        x -= 1000.0
    run = Run(x, token, n_top)
    some = [0, 1, 2, rows // 3, rows // 2, rows - 2, rows - 1]
    check(run, some, chunks)
    del x, run
    torch.cuda.empty_cache()


def test_like_terms():
    """Rows of the same logit throughout: every addition rounds the same way, and the answer is known."""
    for rows, vocab, dtype, _, chunks in SHAPES[:1] + SHAPES[3:5] + SHAPES[6:]:
        x = torch.full((rows, vocab), -3.25, dtype=dtype, device="cuda")
        token = torch.arange(rows, dtype=torch.int32, device="cuda") * 7 % vocab
        run = Run(x, token, 2)
        torch.cuda.synchronize()
        tol = (57 + 6 * chunks) * 2.0 ** -24 + 3.2e-6 + 2.0 ** -23 * math.log(vocab)
        assert float((run.lp[:rows].double() + math.log(vocab)).abs().max()) <= tol
        assert float((run.ent[:rows].double() - math.log(vocab)).abs().max()) <= tol * (1 + 2 * math.log(vocab))
        assert (run.rank[:rows] == token).all()
        assert (run.top[:rows, 0] == 0).all() and (run.top[:rows, 1] == 1).all()
        del x, run
        torch.cuda.empty_cache()
