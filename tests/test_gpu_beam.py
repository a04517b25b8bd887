"""Beam selection against its definition in 64 bits. Candidates are drawn so that the kept and
the dropped differ by far more than the fp32 scores' error (|s| < 64: under 64 * 2^-22), except
where they tie exactly; scores are compared at 1e-5 + 2^-20 |s|."""
import numpy as np
import pytest
import torch

import sparse_long_context_sfi_gb300 as sfi
from tests.cache_model import beam_select

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def run(x, cum, n_beams, done=None, scale=None, eos=2, stride=None, done_out=True, ws=None):
    rows, vocab = x.shape
    if stride:
        wide = torch.full((rows, stride), INF, dtype=x.dtype, device="cuda")
        wide[:, :vocab] = x
        x = wide
    o = dict(parent=torch.full((rows,), -1, dtype=torch.int32, device="cuda"),
             token=torch.full((rows,), -1, dtype=torch.int32, device="cuda"),
             cum=torch.zeros(rows, device="cuda"),
             done=torch.full((rows,), 9, dtype=torch.uint8, device="cuda"))
    ptr = lambda t: None if t is None else t.data_ptr()
    beam = sfi.SfiBeam(
        n_groups=rows // n_beams, n_beams=n_beams, vocab=vocab,
        logits_fp32=1 if x.dtype == torch.float32 else 0, row_stride=x.shape[1], eos=eos,
        logits=ptr(x), cum=ptr(cum), done=ptr(done), rank_scale=ptr(scale), parent=ptr(o["parent"]),
        token=ptr(o["token"]), cum_out=ptr(o["cum"]), done_out=ptr(o["done"]) if done_out else None)
    n = sfi.sfi_beam_workspace_bytes(beam)
    if ws is None:
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        sfi.sfi_workspace_init(ws, n)
    sfi.sfi_beam_select(beam, ws, ws.numel())
    o["keep"] = (x, ws, beam)
    return o


def check(o, x, cum, n_beams, done=None, scale=None, eos=2, done_out=True):
    torch.cuda.synchronize()
    c = lambda t: None if t is None else t.cpu().numpy()
    p, t, s, f = beam_select(x.float().cpu().numpy(), c(cum), c(done), c(scale), eos, n_beams)
    np.testing.assert_array_equal(c(o["parent"]), p)
    np.testing.assert_array_equal(c(o["token"]), t)
    got, fin = c(o["cum"]).astype(np.float64), np.isfinite(s)
    np.testing.assert_array_equal(got[~fin], s[~fin])
    assert (np.abs(got[fin] - s[fin]) <= 1e-5 + 2.0 ** -20 * np.abs(s[fin])).all()
    np.testing.assert_array_equal(c(o["done"]), f if done_out else 9)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("groups,beams,vocab", [
    (1, 1, 1), (1, 1, 50257), (1, 4, 4), (3, 5, 7), (2, 16, 1000), (1, 16, 3), (5, 2, 32000),
    (1, 4, 128001), (32, 8, 2049), (7, 3, 8191), (1, 3, 262147),
])
def test_against_definition(groups, beams, vocab, dtype):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    rows = groups * beams
    x = (torch.randn((rows, vocab), generator=g, device="cuda") * 3).to(dtype)
    cum = -30 * torch.rand(rows, generator=g, device="cuda")
    eos = min(2, vocab - 1)
    o = run(x, cum, beams, eos=eos)
    check(o, x, cum, beams, eos=eos)
    done = (torch.rand(rows, generator=g, device="cuda") < 0.4).to(torch.uint8)
    scale = 0.5 + torch.rand(rows, generator=g, device="cuda")
    o = run(x, cum, beams, done, scale, eos, stride=vocab + 5, done_out=False)
    check(o, x, cum, beams, done, scale, eos, done_out=False)


def test_first_step_expands_one_beam():
    x = torch.randn((4, 5000), device="cuda")
    cum = torch.tensor([0.0, -INF, -INF, -INF], device="cuda")
    o = run(x, cum, 4)
    check(o, x, cum, 4)
    assert o["parent"].tolist() == [0, 0, 0, 0]


def test_ties_go_to_the_lowest_place():
    x = torch.zeros((6, 4097), device="cuda", dtype=torch.bfloat16)
    x[:, 4000:4005] = 3
    x[2, 77] = 3
    cum = torch.tensor([-1.0, -1.0, -1.0, -2.0, -2.0, -2.0], device="cuda")
    o = run(x, cum, 3)
    torch.cuda.synchronize()
    # rows 0 and 1 have equal sums; row 2 has one more high logit, so a lower score
    assert o["parent"].tolist() == [0, 0, 0, 3, 3, 3]
    assert o["token"].tolist() == [4000, 4001, 4002] * 2


def test_masked_tokens_and_dead_rows():
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((8, 3001), generator=g, device="cuda") * 2
    x[0, 5:] = -INF                 # five tokens left
    x[1] = -INF                     # none left
    x[2, 17] = float("nan")
    x[3, 99] = INF
    x[4, :] = -INF
    x[4, 2999] = 0.0                # one token left, and the rest of its group has none
    x[5:] = -INF
    cum = -torch.rand(8, generator=g, device="cuda")
    o = run(x, cum, 4)
    check(o, x, cum, 4)
    assert o["token"][4].item() == 2999 and o["cum"][4].item() == pytest.approx(cum[4].item())
    x[:] = -INF
    done = torch.ones(8, dtype=torch.uint8, device="cuda")
    o = run(x, cum, 4, done=done, eos=7)
    check(o, x, cum, 4, done=done, eos=7)
    assert sorted(o["parent"].tolist()) == list(range(8))


def test_lowest_finite_logits():
    """Masks of the type's lowest value and huge logits."""
    lo = torch.finfo(torch.float32).min
    x = torch.full((2, 600), lo, device="cuda")
    x[0, 300], x[0, 10], x[1, 5] = 1e4, 1e4 - 1, -1e4
    cum = torch.tensor([-3.0, -2.5], device="cuda")
    o = run(x, cum, 2)
    check(o, x, cum, 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_masked_with_the_lowest_value(dtype):
    """A row of nothing but the type's lowest value is uniform; beside a real logit such a
    token keeps its own (hopeless, finite) score."""
    x = torch.full((6, 9001), torch.finfo(dtype).min, device="cuda", dtype=dtype)
    x[3, 4000], x[4, 17], x[4, 18], x[5, 9000] = 2.0, 1.0, 0.5, -3.0
    cum = torch.tensor([-1.0, -2.0, -3.0, -1.0, -1.5, -40.0], device="cuda")
    o = run(x, cum, 3)
    check(o, x, cum, 3)
    x[3:, :] = torch.finfo(dtype).min
    x[3, 4000] = 2.0
    cum[4:] = -float("inf")
    o = run(x, cum, 3)
    check(o, x, cum, 3)


def test_large_logits_keep_their_differences():
    g = torch.Generator(device="cuda").manual_seed(8)
    x = 20000 + torch.randn((8, 5000), generator=g, device="cuda")
    x[4:] -= 40000
    cum = -torch.rand(8, generator=g, device="cuda")
    o = run(x, cum, 4)
    check(o, x, cum, 4)


def test_sorted_logits():
    """Ascending and descending logits: every chunk beats the ones before it, or none does."""
    x = torch.arange(40000, device="cuda", dtype=torch.float32).repeat(4, 1) * 1e-3
    x[2:] = x[2:].flip(1)
    cum = -torch.arange(4, device="cuda", dtype=torch.float32)
    for beams in (1, 4):
        o = run(x, cum, beams)
        check(o, x, cum, beams)


def test_selections_of_other_shapes_share_a_workspace():
    ws = torch.empty(4 << 20, dtype=torch.uint8, device="cuda")
    sfi.sfi_workspace_init(ws, ws.numel())
    g = torch.Generator(device="cuda").manual_seed(6)
    for groups, beams, vocab in ((1, 4, 40000), (64, 4, 9001), (3, 16, 128001), (200, 2, 700), (1, 4, 40000)):
        x = torch.randn((groups * beams, vocab), generator=g, device="cuda")
        cum = -torch.rand(groups * beams, generator=g, device="cuda")
        check(run(x, cum, beams, ws=ws), x, cum, beams)


def test_scores_in_place():
    """cum_out = cum and done_out = done."""
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn((12, 60001), generator=g, device="cuda") * 2
    cum = -torch.rand(12, generator=g, device="cuda")
    done = torch.zeros(12, dtype=torch.uint8, device="cuda")
    done[[1, 6, 7]] = 1
    want = run(x, cum, 4, done)
    parent, token = (torch.zeros(12, dtype=torch.int32, device="cuda") for _ in "pt")
    beam = sfi.SfiBeam(n_groups=3, n_beams=4, vocab=60001, logits_fp32=1, row_stride=60001, eos=2,
                       logits=x.data_ptr(), cum=cum.data_ptr(), done=done.data_ptr(),
                       rank_scale=None, parent=parent.data_ptr(), token=token.data_ptr(),
                       cum_out=cum.data_ptr(), done_out=done.data_ptr())
    ws = want["keep"][1]
    sfi.sfi_beam_select(beam, ws, ws.numel())
    torch.cuda.synchronize()
    assert torch.equal(parent, want["parent"]) and torch.equal(token, want["token"])
    assert torch.equal(cum, want["cum"]) and torch.equal(done, want["done"])


def test_repeatable_and_captured():
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((16, 40000), generator=g, device="cuda")
    cum = -torch.rand(16, generator=g, device="cuda")
    o = run(x, cum, 4)
    ws = o["keep"][1]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = run(x, cum, 4, ws=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for name in ("parent", "token", "cum", "done"):
        assert torch.equal(o[name], c[name])
    x.neg_()
    graph.replay()
    check(c, x, cum, 4)
