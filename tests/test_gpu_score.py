"""Log probabilities, ranks, entropies and best tokens against their definition in 64 bits. Whole
numbers are equal. Tolerances: a lane sums up to 500 terms of a row of 128001 (16 per chunk: 9 roundings
and 3 of the running sum in each of at most 32 chunks, then 9 joins): under 400 of 2^-24 = 2.4e-5; a term
itself is off by 2^-22 and by 2^-24 of its distance to the reference, which for terms that count is
below 24 in powers of two: 1.2e-6. So log sums are off by at most 2.6e-5, log probabilities by a rounding
more; entropy takes the sum's error once and the mean distance's, at most ln vocab, twice."""
import math

import numpy as np
import pytest
import torch

import sparse_long_context_sfi_gb300 as sfi
from tests.border_model import score

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


class Run:
    def __init__(self, x, token, n_top, rank=True, entropy=True, ws=None, stream=None, room=2):
        rows, vocab = x.shape
        self.x, self.token, self.n_top = x, token, n_top
        f = lambda *s: torch.full(s, 55.0, device="cuda")
        i = lambda *s: torch.full(s, 55, dtype=torch.int32, device="cuda")
        # (rows behind the last are nobody's)
        self.lp, self.rank, self.ent = f(rows + room), i(rows + room), f(rows + room)
        self.top, self.top_lp = i(rows + room, max(1, n_top)), f(rows + room, max(1, n_top))
        self.sc = sfi.SfiScoring(
            n_rows=rows, vocab=vocab, logits_fp32=1 if x.dtype == torch.float32 else 0, n_top=n_top,
            row_stride=x.stride(0), logits=x.data_ptr(), token=None if token is None else token.data_ptr(),
            logprob=None if token is None else self.lp.data_ptr(),
            rank=self.rank.data_ptr() if rank and token is not None else None,
            entropy=self.ent.data_ptr() if entropy else None,
            top_token=self.top.data_ptr() if n_top else None, top_logprob=self.top_lp.data_ptr() if n_top else None)
        if ws is None:
            nb = sfi.sfi_scoring_workspace_bytes(self.sc)
            ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
            sfi.sfi_workspace_init(ws, nb)
        self.ws = ws
        sfi.sfi_score_tokens(self.sc, ws, ws.numel(), stream=stream)

    def outs(self):
        return [t.clone() for t in (self.lp, self.rank, self.ent, self.top, self.top_lp)]

    def check(self, tol=2.6e-5):
        torch.cuda.synchronize()
        rows, vocab = self.x.shape
        token = np.full(rows, -1) if self.token is None else self.token.cpu().numpy()
        lp, rank, ent, top, top_lp = score(self.x.double().cpu().numpy(), token, self.n_top)

        def close(got, want, more=1.0):
            got = got.double().cpu().numpy()
            same = (np.isnan(got) & np.isnan(want)) | (got == want)
            with np.errstate(invalid="ignore"):
                ok = np.abs(got - want) <= tol * more + 2.0 ** -23 * np.abs(want)
            assert (same | ok).all(), np.argwhere(~(same | ok))[0]

        if self.sc.logprob:
            close(self.lp[:rows], lp)
        if self.sc.rank:
            assert (self.rank[:rows].cpu().numpy() == rank).all()
        if self.sc.entropy:
            close(self.ent[:rows], ent, 1 + 2 * math.log(vocab + 1))
        if self.n_top:
            assert (self.top[:rows].cpu().numpy() == top).all()
            close(self.top_lp[:rows], top_lp)
        for t in (self.lp, self.rank, self.ent, self.top, self.top_lp):
            assert (t[rows:] == 55).all()
        return self


def logits(rows, vocab, kind=torch.float32, seed=0, gap=0, shift=0, scale=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = torch.full((rows * (vocab + gap) + shift,), NAN, dtype=kind, device="cuda")
    x = flat[shift:].view(rows, vocab + gap)[:, :vocab]
    x.copy_(torch.randn((rows, vocab), generator=g, device="cuda") * scale)
    token = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    return x, token


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab,n_top", [
    (1, 1, 1), (1, 2, 2), (3, 5, 5), (2, 31, 31), (7, 32, 32), (2, 500, 0), (1, 4097, 9), (5, 32000, 5),
    (1, 128001, 20), (40, 8191, 8), (300, 8192, 32), (700, 1000, 3), (33, 33000, 1), (700, 513, 0)])
def test_against_definition(rows, vocab, n_top, kind):
    x, token = logits(rows, vocab, kind, seed=vocab)
    Run(x, token, n_top).check()


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n_top", [0, 4, 20])
@pytest.mark.parametrize("rank", [False, True])
@pytest.mark.parametrize("entropy", [False, True])
def test_what_is_asked_for(entropy, rank, n_top, kind):
    for rows in (2, 650):
        x, token = logits(rows, 6001, kind, gap=3)
        Run(x, token, n_top, rank, entropy).check()
        if n_top or entropy:
            Run(x, None, n_top, rank, entropy).check()


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 1, 3, 7])
@pytest.mark.parametrize("gap", [0, 1, 6])
def test_strides_and_alignment(gap, shift, kind):
    """Rows that start anywhere in a 16-byte piece, NaN around them."""
    x, token = logits(9, 1234, kind, gap=gap, shift=shift)
    Run(x, token, 6).check()


@pytest.mark.parametrize("n_top", [3, 8, 9, 32])
def test_ties(n_top):
    """Few distinct logits: ties go to the lowest token, in lists and in ranks."""
    for rows in (2, 640):
        x, token = logits(rows, 9000, seed=n_top)
        x.copy_(torch.round(x / 2.5))
        Run(x, token, n_top).check()
    x.fill_(1.5)
    Run(x, token, n_top).check()


@pytest.mark.parametrize("n_top", [0, 5, 32])
@pytest.mark.parametrize("unit", [1.0, 2.0 ** -130])
def test_ties_around_zero(unit, n_top):
    """Zeros of both signs and their neighbours (the smallest numbers of the type), in bf16 and fp32."""
    for kind in (torch.bfloat16, torch.float32):
        x, token = logits(6, 3000, kind, seed=n_top)
        g = torch.Generator(device="cuda").manual_seed(1)
        pick = torch.randint(0, 5, x.shape, generator=g, device="cuda")
        values = torch.tensor([0.0, -0.0, unit, -unit, 2 * unit], device="cuda").to(kind)
        x.copy_(values[pick])
        for r in range(5):              # a given token of each value
            token[r] = int((pick[r] == r).nonzero()[200])
        Run(x, token, n_top).check()


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [255, 256, 257, 300, 511, 600, 1500, 33000])
def test_equal_logits(vocab, kind):
    """All tokens are among the best, more than wait anywhere; some of them higher, some masked."""
    for rows in (1, 700 if vocab < 1000 else 30):
        x, token = logits(rows, vocab, kind, gap=5)
        x.fill_(0.25)
        for n_top in (3, 32):
            Run(x, token, n_top).check()
        x[:, vocab // 2:vocab // 2 + 40] = 7.0
        x[:, :3] = -INF
        Run(x, token, 32).check()
        x[:, 5:] = -INF                 # fewer tokens than places
        Run(x, token, 32).check()


@pytest.mark.parametrize("n_top", [4, 20, 32])
@pytest.mark.parametrize("vocab", [4000, 40000])
def test_best_tokens_of_few_lanes(vocab, n_top):
    """The best tokens side by side, and at the distances at which one lane meets them."""
    for rows in (2, 300):
        x, token = logits(rows, vocab, torch.bfloat16)
        x[:, 1000:1040] += 30.0
        Run(x, token, n_top).check()
        x, token = logits(rows, vocab, seed=1)
        x[:, 7::512] += 30.0
        x[:, 8::1024] += 60.0
        Run(x, token, n_top).check()


@pytest.mark.parametrize("n_top", [1, 16, 32])
@pytest.mark.parametrize("down", [False, True])
def test_sorted_rows(down, n_top):
    x = torch.arange(20000, device="cuda").float().repeat(3, 1) / 1000
    x = (x.flip(1) if down else x).contiguous()
    Run(x, torch.tensor([0, 19999, 777], dtype=torch.int32, device="cuda"), n_top).check()


@pytest.mark.parametrize("rows", [4, 620])
def test_masked_tokens(rows):
    """Most tokens at -inf, a row with one token left, the given token masked."""
    x, token = logits(rows, 5000)
    g = torch.Generator(device="cuda").manual_seed(3)
    x.masked_fill_(torch.rand(x.shape, generator=g, device="cuda") < 0.9, -INF)
    x[1] = -INF
    x[1, 4321] = -3.0
    token[2] = int((x[2] == -INF).nonzero()[5])
    r = Run(x, token, 32).check()
    # (certainty up to the tolerance above, and never less than none or more than certain)
    assert 0 <= float(r.ent[1]) <= 2.6e-5 and -2.6e-5 <= float(r.top_lp[1, 0]) <= 0 and int(r.top[1, 0]) == 4321
    assert float(r.lp[2]) == -INF


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(2, 40), (3, 5000), (1, 60000), (700, 2000), (40, 40000)])
@pytest.mark.parametrize("left", [1, 2, 7, 19, 20, 21, 40])
def test_few_tokens_left(left, rows, vocab, kind):
    """A grammar's mask: fewer tokens than places (or as many, or a few more), near each other and apart;
    the places behind them are the lowest masked tokens."""
    x, token = logits(rows, vocab, kind, gap=1)
    keep = torch.zeros((rows, vocab), dtype=torch.bool, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(left)
    for r in range(rows):
        if r % 3 == 0:
            keep[r, torch.randperm(vocab, generator=g, device="cuda")[:left]] = True
        elif r % 3 == 1:
            keep[r, :left] = True
        else:
            keep[r, vocab - left:] = True
    x[~keep] = -INF
    Run(x, token, 20).check()
    Run(x, token, 32).check()


@pytest.mark.parametrize("lowest", [-3.0e38, torch.finfo(torch.float32).min])
def test_masks_of_the_lowest_value(lowest):
    x, token = logits(3, 5000)
    x[:, 10:4000] = lowest
    Run(x, token, 12).check()
    x.fill_(lowest)                     # all masked alike: a uniform distribution
    r = Run(x, token, 12).check()
    assert abs(float(r.ent[0]) - math.log(5000)) < 1e-4


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [6, 630])
def test_rows_without_a_distribution(rows, kind):
    x, token = logits(rows, 7000, kind)
    x[0, 5000] = NAN
    x[1, 3] = INF
    x[2] = -INF
    x[3, :] = NAN
    x[4, 17] = NAN
    token[4] = 17
    r = Run(x, token, 5).check()
    assert (r.top[:5] == -1).all() and (r.rank[:5] == -1).all() and torch.isnan(r.lp[:5]).all()
    assert torch.isfinite(r.lp[5:rows]).all()


@pytest.mark.parametrize("size", [1e4, 2e9, 1e30, 3e38])
@pytest.mark.parametrize("sign", [1, -1])
def test_huge_logits(size, sign):
    """Logits of any size (a float's neighbours are far apart there): the highest take all."""
    x, token = logits(4, 3000)
    x.copy_(torch.rand(x.shape, device="cuda") * 0.5 + 0.5)
    x *= sign * size
    x[1, 100:110] = x[1].max()
    x[2, ::7] = float(torch.randn(1))
    token[1] = 104
    # (fp32 logits differ by 2^-24 of their size: log probabilities are rounded like them)
    Run(x, token, 15).check()


def test_tokens_outside():
    x, token = logits(5, 640)
    token[:4] = torch.tensor([-1, -2 ** 31, 640, 2 ** 31 - 1])
    r = Run(x, token, 2).check()
    assert r.lp[:2].tolist() == [0.0, 0.0] and torch.isnan(r.lp[2:4]).all() and (r.rank[:4] == -1).all()


def test_sampled_tokens_sum_to_one():
    """exp of all tokens' log probabilities of one row, each asked for as its own row."""
    x, _ = logits(1, 900)
    r = Run(x.expand(900, 900).contiguous(), torch.arange(900, dtype=torch.int32, device="cuda"), 0)
    torch.cuda.synchronize()
    assert abs(float(r.lp[:900].double().exp().sum()) - 1) < 3e-5
    assert sorted(r.rank[:900].tolist()) == list(range(900))


def test_offsets_beyond_32_bits():
    rows, vocab = 3, 1000
    flat = torch.empty((1 << 31) + 5000, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(flat, (rows, vocab), ((1 << 30) + 3, 1))
    x.copy_(torch.randn((rows, vocab), device="cuda"))
    Run(x, torch.tensor([5, 6, 999], dtype=torch.int32, device="cuda"), 4).check()
    del flat, x
    torch.cuda.empty_cache()


def test_calls_of_other_shapes_share_a_workspace():
    sizes = [(1, 32000, 20), (300, 9000, 32), (8, 128001, 3), (700, 500, 1), (2, 20000, 0)]
    made = [logits(r, v, seed=v) + (k,) for r, v, k in sizes]
    nb = max(Run(*m).ws.numel() for m in made)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    sfi.sfi_workspace_init(ws, nb)
    for i in (0, 2, 1, 3, 4, 2, 0, 1):
        Run(*made[i], ws=ws).check()


def test_repeatable_captured_and_on_another_stream():
    x, token = logits(3, 50000, torch.bfloat16)
    first = Run(x, token, 7)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = Run(x, token, 7, ws=first.ws, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(first.outs(), again.outs()):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sfi.sfi_score_tokens(first.sc, first.ws, first.ws.numel())
    old = x.clone()
    x.copy_(old.flip(1))
    graph.replay()
    first.check()
    x.copy_(old)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first.outs(), again.outs()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n_top", [3, 20])
@pytest.mark.parametrize("masked", [False, True])
def test_chunks_of_one_lane(masked, n_top, kind):
    """One warp a row (so many rows), and one to four chunks of a lane hold the best, others masked."""
    rows, piece = 8500, 16 // (4 if kind == torch.float32 else 2)
    chunk = 128 * piece
    x, token = logits(rows, 4 * chunk + 5, kind, seed=4)
    g = torch.Generator(device="cuda").manual_seed(5)
    pick = lambda n: torch.randint(0, n, (rows,), generator=g, device="cuda")
    r = torch.arange(rows, device="cuda")
    for c in range(4):
        some = pick(4) >= c if not masked else pick(2) > 0
        at = (r * 5 + c) % 4 * chunk + pick(4) * 32 * piece + r % 32 * piece + pick(piece)
        x[r[some], at[some]] += 12.0
        if masked:
            x[~some, c * chunk:(c + 1) * chunk] = -INF
    Run(x, token, n_top).check()


@pytest.mark.parametrize("rows", [2, 8500])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_logits_that_differ_in_the_last_bits(sign, rows):
    """The best differ by less than the keys of chunks tell apart, of either sign and around zero."""
    x, token = logits(rows, 2053, torch.float32)
    g = torch.Generator(device="cuda").manual_seed(6)
    step = torch.randint(0, 5000, x.shape, generator=g, device="cuda").float()
    near = sign * (1.0 + step * 2.0 ** -23)
    best = torch.rand(x.shape, generator=g, device="cuda") < 0.02
    x.copy_(torch.where(best, near, x.clamp(max=0.0) - 1.5))
    for n_top in (1, 6, 32):
        Run(x, token, n_top).check()
    x.copy_(torch.where(best, sign * (step - 2500).clamp(min=0.0) * 2.0 ** -149, x))
    Run(x, token, 20).check()


def test_longest_row():
    """2^30 logits: more chunks to a warp than a key counts, the best among those behind."""
    n = 1 << 30
    x = torch.full((1, n), -20.0, device="cuda")
    last = [n - 1, n - 3, n - 1 - 4 * 128, n - 5 - 64 * 8 * 512, n - 70000, n - 70001, 5, 77777, 512 * 512 * 8 + 9, n // 2]
    for i, v in enumerate(last):
        x[0, v] = 10.0 - i
    token = torch.tensor([77777], dtype=torch.int32, device="cuda")
    run = Run(x, token, 12)
    torch.cuda.synchronize()
    want = last + sorted(set(range(20)) - set(last))[:2]
    assert run.top[0].tolist() == want and int(run.rank[0]) == 7
    # 2^30 e^-20 = 2.2 beside e^10 and less: every lane's sum has 2^14 like terms, an error of at most
    # 2^-10 of what is 1e-4 of the whole
    lse = math.log((n - len(last)) * math.exp(-20.0) + sum(math.exp(10.0 - i) for i in range(len(last))))
    got = run.top_lp[0].double().cpu().numpy()
    assert np.abs(got - ([10.0 - i - lse for i in range(len(last))] + [-20 - lse] * 2)).max() <= 1e-5
    del x, run
    torch.cuda.empty_cache()
