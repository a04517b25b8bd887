"""A decoder around the cache, as a server runs it: rotary positions into a paged cache, windowed
attention, attention to an encoder, logits, scores and beam selection, forks of the pages. Every step's
numbers are compared with a plain model in 64 bits that follows the beams chosen."""
import math

import numpy as np
import pytest
import torch

import sparse_long_context_sfi_gb300 as sfi
from sparse_long_context_sfi_gb300.engine import BeamSearch, EncoderStates, Rope, SfiState, TokenScores
from synth.configs import WORKLOADS
from tests.border_model import cross_attention, score, turned
from tests.cache_model import window_attention

pytestmark = pytest.mark.gpu

D, BF = 128, torch.bfloat16
GROUPS, BEAMS, HQ, HKV, VOCAB, WINDOW, SINK = 2, 3, 8, 2, 997, 32, 4
BATCH = GROUPS * BEAMS


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def host(t):
    return t.double().cpu().numpy()


def make_state(batch=BATCH, cols=8, paged=True, **kw):
    cfg = WORKLOADS["ragged_paged_b32" if paged else "gqa4_ctx4k_hh"].scaled(
        n_layers=1, batch=batch, n_q_heads=HQ, n_kv_heads=HKV, n_sink=SINK, n_window=WINDOW, n_select=16, steps=4, **kw)
    if not paged:
        return SfiState(cfg, np.full(batch, 0), capacity=cols * 16)
    return SfiState(cfg, np.full(batch, 0), page_table=np.full((batch, cols), -1), n_pages=batch * cols)


class Model:
    """Projections of token embeddings and their definition in 64 bits, from the bf16 values on."""

    def __init__(self, rope, kw):
        g = torch.Generator(device="cuda").manual_seed(3)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.table = rnd(VOCAB, (HQ + 2 * HKV) * D).to(BF)       # a token's fused projection
        self.cross_q = rnd(VOCAB, HQ * D).to(BF)
        self.out = rnd(2 * HQ * D, VOCAB) / math.sqrt(2 * HQ * D) * 8
        self.rope, self.kw = rope, kw

    def rows(self, tokens):
        """[1][n] rows of q, k and v of the tokens: views of one projection."""
        x = self.table[tokens.long()].view(1, -1, HQ + 2 * HKV, D)
        return x.split([HQ, HKV, HKV], 2)

    def angle(self, pos):
        i = np.arange(self.kw["rot_dim"] // 2)
        f = self.kw["base"] ** (-2 * i / self.kw["rot_dim"]) / self.kw["factor"]
        return np.asarray(pos)[:, None] * f[None]

    def turn(self, x, pos):
        return turned(host(x)[None] if x.dim() == 3 else host(x), self.angle(pos), self.kw["rot_dim"], False)[0]

    def history(self, tokens):
        """k (rounded as the cache holds it) and v of a token sequence: [hkv][n][D], and its queries."""
        q, k, v = self.rows(torch.tensor(tokens, device="cuda"))
        pos = np.arange(len(tokens))
        bf = lambda y: host(torch.from_numpy(y).to(BF))
        return bf(self.turn(q, pos))[0], bf(self.turn(k, pos))[0].transpose(1, 0, 2), host(v)[0].transpose(1, 0, 2)


@pytest.mark.parametrize("paged", [True, False])
def test_beams_with_encoder(paged):
    kw = dict(rot_dim=96, base=10000.0, factor=2.0)
    rope = Rope(scaling="linear", **kw)
    m = Model(rope, kw)
    st = make_state(paged=paged)
    enc = EncoderStates(1, GROUPS, HQ, HKV, 200)
    g = torch.Generator(device="cuda").manual_seed(8)
    lens = [131, 64]
    ek, ev = (torch.randn((1, sum(lens), HKV, D), generator=g, device="cuda").to(BF) for _ in "kv")
    enc.write(ek[:, :100].contiguous(), ev[:, :100].contiguous(), [100, 0])
    enc.write(ek[:, 100:].contiguous(), ev[:, 100:].contiguous(), [31, 64])
    beams, scores = BeamSearch(GROUPS, BEAMS, VOCAB, eos=-1), TokenScores()
    prompt = torch.randint(0, VOCAB, (2, 41), generator=g, device="cuda")
    # each prompt into the first slot of its group, the others empty
    rows = np.array([41 if b % BEAMS == 0 else 0 for b in range(BATCH)])
    q, k, v = m.rows(prompt.flatten())
    out = torch.zeros((1, 82, HQ, D), dtype=BF, device="cuda")
    st.prefill(q, k, v, rows, out, rope=rope)
    held = [prompt[b // BEAMS].tolist() for b in range(BATCH)]
    for i in range(2):
        mq, mk, mv = m.history(held[i * BEAMS])
        o, mag = window_attention(mq, mk, mv, 41, SINK, WINDOW)
        # (q and k are rounded a second time: 2^-8 of a logit's magnitudes, logits of |q||k|/sqrt(D) below 20)
        err = np.abs(host(out)[0, 41 * i:41 * (i + 1)] - o)
        assert (err <= 0.05 * mag + 2.0 ** -7 * np.abs(o)).all()
        assert np.linalg.norm(err) <= 0.01 * np.linalg.norm(o)
    st.reorder(torch.tensor([b // BEAMS * BEAMS for b in range(BATCH)], dtype=torch.int32, device="cuda"))
    token = torch.tensor([h[-1] for h in held], dtype=torch.int32, device="cuda")
    for step in range(4):
        # the last token goes into the cache (again, for the prompts' own last one: as a new position)
        held = [h + [int(t)] for h, t in zip(held, token.tolist())]
        q, k, v = m.rows(token)
        self_out = torch.zeros((1, BATCH, HQ, D), device="cuda")
        st.window_step(q, k, v, self_out, rope=rope)
        cq = m.cross_q[token.long()].view(1, BATCH, HQ, D)
        cross_out = torch.zeros((1, BATCH, HQ, D), device="cuda")
        enc.attend(cq, cross_out, rows=BEAMS, out_fp32=True)
        for b in range(BATCH):
            mq, mk, mv = m.history(held[b])
            o, _ = window_attention(mq[-1:], mk, mv, len(held[b]), SINK, WINDOW)
            err = host(self_out)[0, b] - o[0]
            assert np.linalg.norm(err) <= 0.01 * np.linalg.norm(o), (step, b)
            e0 = sum(lens[:b // BEAMS])
            part = slice(0, 100) if b // BEAMS == 0 else slice(100 + 31, None)
            kk = torch.cat([ek[0, :100], ek[0, 100:131]]) if b // BEAMS == 0 else ek[0, 131:]
            vv = torch.cat([ev[0, :100], ev[0, 100:131]]) if b // BEAMS == 0 else ev[0, 131:]
            o, mag = cross_attention(host(cq)[0, b:b + 1], host(kk).transpose(1, 0, 2), host(vv).transpose(1, 0, 2))
            assert (np.abs(host(cross_out)[0, b] - o[0]) <= 1e-4 * mag[0]).all(), (step, b)
        logits = torch.cat([self_out.view(BATCH, -1), cross_out.view(BATCH, -1)], 1) @ m.out
        before = beams.cum.clone()
        parent, token = beams.select(logits)
        # the chosen tokens' log probabilities, and the beams' scores made of them
        chosen = scores.score(logits[parent.long()], token, n_top=5, rank=True, entropy=True)
        want = score(host(logits[parent.long()]), token.cpu().numpy(), 5)
        for name, w, tol in (("logprob", want[0], 2e-5), ("entropy", want[2], 3e-4), ("top_logprob", want[4], 2e-5)):
            assert np.abs(host(chosen[name]) - w).max() <= tol, (step, name)
        assert (chosen["rank"].cpu().numpy() == want[1]).all() and (chosen["top_token"].cpu().numpy() == want[3]).all()
        cum = before[parent.long()].double() + chosen["logprob"].double()
        assert (cum - beams.cum.double()).abs().max() <= 1e-4
        st.reorder(parent)
        held = [held[p] for p in parent.tolist()]
    torch.cuda.synchronize()
    assert int(st.err[0]) == 0 and int(enc.err[0]) == 0


@pytest.mark.parametrize("fused", [True, False])
def test_slow_and_fast_steps_with_rope(fused):
    """step(rope=) is the step on queries and keys that were turned before, bit for bit."""
    kw = dict(rot_dim=128, base=500000.0)
    rope = Rope(**kw)
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)
    states = [make_state(batch=4), make_state(batch=4)]
    x = rnd(1, 4 * 50, HQ + 2 * HKV, D)
    q, k, v = x.split([HQ, HKV, HKV], 2)
    outs = [torch.zeros((1, 200, HQ, D), dtype=BF, device="cuda") for _ in states]
    for st, o in zip(states, outs):
        st.prefill(q, k, v, [50] * 4, o, rope=rope)
    for slow in ([1, 1, 1, 1], [0, 0, 0, 0], [1, 0, 0, 1], [0, 0, 0, 0]):
        x = rnd(1, 4, HQ + 2 * HKV, D)
        q, k, v = x.split([HQ, HKV, HKV], 2)
        a, b = (torch.zeros((1, 4, HQ, D), device="cuda") for _ in "ab")
        v = v.contiguous()
        ok = [st.reserve() for st in states]
        states[0].step(q, k, v, np.array(slow, bool), a, rope=rope, fused=fused, active=ok[0])
        io = sfi.SfiRopeRows(q=q.data_ptr(), q_stride=q.stride(1), k=k.data_ptr(), k_stride=k.stride(1))
        tq, tk = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty_like(
            k, memory_format=torch.contiguous_format)
        io.q_out, io.k_out = tq.data_ptr(), tk.data_ptr()
        sfi.sfi_rope_apply(states[1]._whole(), rope.desc, io, None, 4, 1)
        states[1].step(tq, tk, v, np.array(slow, bool), b, fused=fused, active=ok[1])
        torch.cuda.synchronize()
        assert torch.equal(a, b) and torch.isfinite(a).all() and a.abs().sum() > 0
    assert torch.equal(states[0].k, states[1].k) and torch.equal(states[0].seq_len, states[1].seq_len)
    assert int(states[0].err[0]) == 0


def test_captured_step():
    """One whole step in a graph, replayed: positions and lengths move on, encoder states may change."""
    rope = Rope(interleaved=True)
    st = make_state(batch=4, cols=6)
    enc = EncoderStates(1, 2, HQ, HKV, 64)
    scores = TokenScores()
    g = torch.Generator(device="cuda").manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)
    enc.write(rnd(1, 30, HKV, D), rnd(1, 30, HKV, D), [20, 10])
    q, k, v = rnd(1, 4, HQ, D), rnd(1, 4, HKV, D), rnd(1, 4, HKV, D)
    out, cross = torch.zeros((1, 4, HQ, D), device="cuda"), torch.zeros((1, 4, HQ, D), device="cuda")
    w = torch.randn((HQ * D, 500), generator=g, device="cuda")
    token = torch.tensor([3, 4, 5, 6], dtype=torch.int32, device="cuda")

    def whole():
        st.window_step(q, k, v, out, rope=rope)
        enc.attend(q, cross, rows=2, out_fp32=True)
        return scores.score(out.view(4, -1) @ w, token, n_top=3, entropy=True)

    whole()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = whole()
    for n in range(3):
        if n == 1:
            enc.clear([1])
            enc.write(rnd(1, 7, HKV, D), rnd(1, 7, HKV, D), [0, 7])
        q.copy_(rnd(1, 4, HQ, D))
        graph.replay()
        o, _ = cross_attention(host(q)[0, 2:], host(enc.k)[0, 1, :, :enc.lens[1]], host(enc.v)[0, 1, :, :enc.lens[1]])
        assert np.abs(host(cross)[0, 2:] - o).max() <= 1e-3
        want = score(host(out.view(4, -1) @ w), token.cpu().numpy(), 3)
        assert np.abs(host(got["logprob"]) - want[0]).max() <= 1e-3
        assert st.seq_len.tolist() == [n + 2] * 4
    assert int(st.err[0]) == 0 and int(enc.err[0]) == 0


def test_encoder_inputs_come_and_go():
    enc = EncoderStates(2, 3, HQ, HKV, 40)
    g = torch.Generator(device="cuda").manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)
    enc.write(rnd(2, 50, HKV, D), rnd(2, 50, HKV, D), [20, 0, 30])
    q = rnd(2, 6, HQ, D)
    for fp32, active in ((True, None), (False, torch.tensor([0, 1, 1], dtype=torch.uint8, device="cuda"))):
        out = torch.full((2, 6, HQ, D), -7.0, device="cuda", dtype=torch.float32 if fp32 else BF)
        enc.attend(q, out, rows=[1, 2, 2], out_fp32=fp32, active=active)
        for layer in range(2):
            for e, (a, b) in enumerate(((0, 1), (1, 3), (3, 5))):
                if active is not None and not active[e]:
                    assert (out[layer, a:b] == -7.0).all()
                    continue
                n = enc.lens[e]
                o, mag = cross_attention(host(q)[layer, a:b], host(enc.k)[layer, e, :, :n], host(enc.v)[layer, e, :, :n])
                tol = 1e-4 * mag + (0 if fp32 else 2.0 ** -8) * np.abs(o)
                assert (np.abs(host(out)[layer, a:b] - o) <= tol).all()
        assert (out[:, 5] == -7.0).all()
    enc.clear()
    out = torch.ones((2, 3, HQ, D), dtype=BF, device="cuda")
    enc.attend(q[:, :3].contiguous(), out)
    torch.cuda.synchronize()
    assert (out == 0).all() and int(enc.err[0]) == 0 and enc.lens.tolist() == [0, 0, 0]


def test_nothing_to_score():
    s = TokenScores()
    out = s.score(torch.zeros((0, 50), device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"), n_top=3)
    assert out["logprob"].shape == (0,) and out["top_token"].shape == (0, 3)


def test_rope_rows_of_one_projection():
    """prefill on rows of a fused projection, and with given positions, as on packed rows turned before."""
    rope = Rope(rot_dim=64, scaling="ramp", factor=4.0, original_len=64.0)
    g = torch.Generator(device="cuda").manual_seed(6)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)
    x = rnd(1, 30, HQ + 2 * HKV, D)
    q, k, v = x.split([HQ, HKV, HKV], 2)
    pos = torch.randint(0, 100000, (30,), generator=g, device="cuda", dtype=torch.int32)
    for given in (None, pos):
        a, b = make_state(batch=2), make_state(batch=2, paged=False)
        outs = [torch.zeros((1, 30, HQ, D), dtype=BF, device="cuda") for _ in "ab"]
        a.prefill(q, k, v, [10, 20], outs[0], rope=rope, pos=given)
        io = sfi.SfiRopeRows(q=q.data_ptr(), q_stride=q.stride(1), k=k.data_ptr(), k_stride=k.stride(1),
                             pos=None if given is None else given.data_ptr())
        tq, tk = torch.empty((1, 30, HQ, D), dtype=BF, device="cuda"), torch.empty((1, 30, HKV, D), dtype=BF, device="cuda")
        io.q_out, io.k_out = tq.data_ptr(), tk.data_ptr()
        start = torch.tensor([0, 10, 30], dtype=torch.int32, device="cuda")
        sfi.sfi_rope_apply(b._whole(), rope.desc, io, start, 30, 20)
        b.prefill(tq, tk, v.contiguous(), [10, 20], outs[1])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and outs[0].abs().sum() > 0
        assert int(a.err[0]) == 0 and int(b.err[0]) == 0
