"""What the operators at the borders of the decode path are measured on.

Three families, each as a user's program calls it: rotary positions of queries and keys on their
way to the cache (with the per-head norm in front of them); attention of decoder rows to an
encoder's states; and the log probabilities of given tokens with rank, entropy and alternatives.
"""
from __future__ import annotations

import math

import torch

own = False

D = 128        # head dimension
PAGE = 16      # tokens of a page
BF = torch.bfloat16
DEV = "cuda"
EPS = 1e-6     # of the per-head norm


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # the smallest decode: one token of one sequence, two kv heads, into the 4K cache
        dict(name="rope_token_4k", kind="rope", append=True, batch=1, lo=4096, hi=4096, rows_lo=1,
             rows_hi=1, hq=8, hkv=2, layers=1, rot=128, inter=False, scaling="none", factor=1.0,
             norm=False, paged=False, packed=False),
        # one token each of the ragged batch at far positions, out of one fused projection; the
        # rows then go to the fused fast step, which appends them itself
        dict(name="rope_tokens_far_b32", kind="rope", append=False, batch=32, lo=60000, hi=131000,
             rows_lo=1, rows_hi=1, hq=32, hkv=8, layers=1, rot=128, inter=False, scaling="smooth",
             factor=8.0, norm=False, paged=True, packed=True),
        # four prompts' first 8192 tokens enter the cache
        dict(name="rope_prompt_4x8k", kind="rope", append=True, batch=4, lo=0, hi=0, rows_lo=8192,
             rows_hi=8192, hq=32, hkv=8, layers=1, rot=128, inter=False, scaling="none",
             factor=1.0, norm=False, paged=False, packed=True),
        # ragged chunks of odd lengths in pages, half of each head turned in neighbouring pairs,
        # positions stretched, queries and keys normed per head, two layers
        dict(name="rope_ragged_norm", kind="rope", append=True, batch=8, lo=1000, hi=9001,
             rows_lo=700, rows_hi=1501, hq=32, hkv=4, layers=2, rot=64, inter=True,
             scaling="linear", factor=4.0, norm=True, paged=True, packed=False),
        # one decoder row against a short encoder; fp32 outputs
        dict(name="cross_token_601", kind="cross", batch=1, lo=601, hi=601, rows_lo=1, rows_hi=1,
             hq=8, hkv=2, paged=False, fp32=True),
        # four beams each of 32 prompts, encoder states of uneven lengths in pages
        dict(name="cross_beams_32x4", kind="cross", batch=32, lo=1000, hi=4001, rows_lo=4,
             rows_hi=4, hq=32, hkv=8, paged=True, fp32=False),
        # the decoder's prompts against long encoder states
        dict(name="cross_chunk_4x2k_8k", kind="cross", batch=4, lo=8192, hi=8192, rows_lo=2048,
             rows_hi=2048, hq=32, hkv=8, paged=False, fp32=False),
        # ragged chunks of a mixed batch, eight query heads a kv head; one has no encoder states
        dict(name="cross_ragged_empty", kind="cross", batch=8, lo=0, hi=1601, rows_lo=100,
             rows_hi=701, hq=64, hkv=8, paged=True, fp32=False),
        # the sampled token of one sequence with five alternatives
        dict(name="score_1_v32000", kind="score", rows=1, vocab=32000, fp32=False, pad=0.0, top=5,
             rank=True, entropy=True, banned=0.0, gap=0),
        # scoring a prompt: every position's own token, of a large odd vocabulary, some padding
        dict(name="score_2048_v128001", kind="score", rows=2048, vocab=128001, fp32=False, pad=0.05,
             top=0, rank=False, entropy=False, banned=0.0, gap=0),
        # the widest batch in fp32 rows of a padded buffer, a third of the vocabulary masked
        dict(name="score_256_top20", kind="score", rows=256, vocab=128001, fp32=True, pad=0.0,
             top=20, rank=True, entropy=True, banned=0.33, gap=63),
        # 8192 prompt tokens with everything asked for
        dict(name="score_8k_all", kind="score", rows=8192, vocab=32000, fp32=False, pad=0.0, top=3,
             rank=True, entropy=True, banned=0.0, gap=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "rope", "cross", "cross", "score", "score"])
    hkv = rng.choice([2, 4, 8])
    if kind == "rope":
        batch = _log(rng, 1, 32)
        rows = _log(rng, 1, max(1, 16384 // batch))
        paged = rng.random() < 0.5
        # (far positions where pages out of the window are given up; a contiguous cache is whole)
        hi = _log(rng, 1, 131072 if paged else max(1, 65536 // batch))
        scaling = rng.choice(["none", "linear", "base", "ramp", "smooth"])
        return dict(kind="rope", append=rng.random() < 0.7, batch=batch, lo=hi // 3, hi=hi,
                    rows_lo=rows // 2 + 1 if rows > 1 else 1, rows_hi=rows,
                    hq=hkv * rng.choice([1, 2, 4, 8]), hkv=hkv, layers=rng.choice([1, 1, 2]),
                    rot=rng.choice([128, 128, 64, 32, 96, 40, 2 * rng.randint(2, 63)]),
                    inter=rng.random() < 0.5, scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]),
                    norm=rng.random() < 0.4, paged=paged, packed=rng.random() < 0.5)
    if kind == "cross":
        batch, group = _log(rng, 1, 32), rng.choice([1, 2, 4, 8])
        hi = _log(rng, 1, 8192)
        few = rng.random() < 0.5
        rows = rng.randint(1, 8) if few else _log(rng, 9, 2048)
        hq = hkv * group
        # at most the (row, head, key) products of the longest listed one
        while batch * rows * hq * hi > 4 * 2048 * 32 * 8192:
            rows = max(1, rows // 2)
        return dict(kind="cross", batch=batch, lo=rng.choice([0, hi // 2, hi]), hi=hi,
                    rows_lo=max(1, rows // 2), rows_hi=rows, hq=hq, hkv=hkv,
                    paged=rng.random() < 0.5, fp32=rng.random() < 0.25)
    vocab = _log(rng, 500, 128001)
    rows = _log(rng, 1, 2048 * 128001 // vocab if vocab > 32000 else 8192)
    return dict(kind="score", rows=rows, vocab=vocab, fp32=rng.random() < 0.4 and rows <= 1024,
                pad=rng.choice([0.0, 0.0, 0.1]), top=rng.choice([0, 1, 3, 5, 20, 32]),
                rank=rng.random() < 0.5, entropy=rng.random() < 0.5,
                banned=rng.choice([0.0, 0.0, 0.5]), gap=rng.choice([0, 0, 3, 64]))


def _spread(lo, hi, n):
    """n sizes in [lo, hi], fixed by the case: hi first, the others strewn over the range."""
    return [hi - (i * 40503) % (hi - lo + 1) for i in range(n)]


def _shapes(case):
    """Lengths and row counts of the case's sequences."""
    n = case["batch"]
    lens = _spread(case["lo"], case["hi"], n)
    if case["kind"] == "cross" and case["lo"] == 0 and n > 1:
        lens[n // 2] = 0
    return lens, _spread(case["rows_lo"], case["rows_hi"], n)


def _columns(length):
    return (length + PAGE - 1) // PAGE


# ------------------------------------------------------------------------- bytes and flops

def work(case):
    if case["kind"] == "score":
        n = case["rows"]
        out = n * 8 + (4 * n if case["rank"] else 0) + (4 * n if case["entropy"] else 0)
        return {"bytes": n * case["vocab"] * (4 if case["fp32"] else 2) + out + 8 * n * case["top"],
                "flops": n * case["vocab"] * (6 if case["entropy"] else 4)}
    lens, rows = _shapes(case)
    total = sum(rows)
    if case["kind"] == "rope":
        heads = case["hq"] + case["hkv"]
        moved = heads + (case["hkv"] if case["append"] else 0)
        each = total * case["layers"]
        return {"bytes": 2 * each * moved * D * 2,
                "flops": each * heads * (3 * case["rot"] + (3 * D if case["norm"] else 0))}
    q = total * case["hq"] * D
    return {"bytes": q * 2 + q * (4 if case["fp32"] else 2) + sum(lens) * case["hkv"] * D * 4,
            "flops": 4 * D * case["hq"] * sum(a * r for a, r in zip(lens, rows))}


# ------------------------------------------------------------------------------ the inputs

def _rng(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(0xA5F1 + seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=BF)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _starts(rows):
    return _ints([sum(rows[:i]) for i in range(len(rows) + 1)])


def _rope_scaling(case):
    """Arguments of the frequencies: base, and what a stretched context adds."""
    return dict(base=500000.0 if case["scaling"] == "smooth" else 10000.0, scaling=case["scaling"],
                factor=case["factor"], original_len=8192.0,
                low=1.0, high=32.0 if case["scaling"] == "ramp" else 4.0)


def _rope_inputs(case, seed):
    g = _rng(seed)
    lens, rows = _shapes(case)
    n, hq, hkv, layers = case["batch"], case["hq"], case["hkv"], case["layers"]
    total = sum(rows)
    s = dict(lens=lens, rows=rows, start=_starts(rows), n_rows=total, seq_len=_ints(lens))
    s["saved"] = s["seq_len"].clone()
    # values of a projection: a few strong dimensions, as queries and keys have them
    strong = 1 + 4 * (torch.rand((D,), generator=g, device=DEV) < 0.05).to(BF)
    if case["packed"]:  # one fused projection's rows: q heads, k heads, v heads
        x = _randn(g, layers, total, hq + 2 * hkv, D) * strong
        s["x"] = x
        s["q"], s["k_new"], s["v_new"] = x.split([hq, hkv, hkv], 2)
    else:
        s["q"], s["k_new"], s["v_new"] = (_randn(g, layers, total, h, D) * strong
                                          for h in (hq, hkv, hkv))
    s["q_out"] = torch.zeros((layers, total, hq, D), dtype=BF, device=DEV)
    if case["norm"]:
        s["q_norm"], s["k_norm"] = ((1 + 0.3 * torch.randn((D,), generator=g, device=DEV)).to(BF)
                                    for _ in "qk")
    else:
        s["q_norm"] = s["k_norm"] = None
    if not case["append"]:
        s["k_out"] = torch.zeros((layers, total, hkv, D), dtype=BF, device=DEV)
    # the cache behind the rows; of the far sequences only the last page and the new ones are held
    cols = _columns(max(a + r for a, r in zip(lens, rows)))
    s["cols"] = cols
    if case["paged"]:
        held = [_columns(a + r) - a // PAGE for a, r in zip(lens, rows)]
        pages = sum(held) + 7
        ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = torch.full((n, cols), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b in range(n):
            c = lens[b] // PAGE
            table[b, c:c + held[b]] = ids[at:at + held[b]]
            at += held[b]
        s["table"] = table
        shape = (layers, pages, hkv, PAGE, D)
    else:
        s["table"] = None
        shape = (layers, n, hkv, cols * PAGE, D)
    if case["append"]:
        s["k"], s["v"] = (_randn(g, *shape) for _ in "kv")
    else:       # (nothing of the cache is touched: a small one stands in)
        s["k"] = s["v"] = None
    return s


def _cross_inputs(case, seed):
    """Queries lean towards a direction that some encoder positions share: attention finds a few
    positions and spreads the rest."""
    g = _rng(seed)
    lens, rows = _shapes(case)
    n, hq, hkv, total = case["batch"], case["hq"], case["hkv"], sum(rows)
    s = dict(lens=lens, rows=rows, start=_starts(rows), n_rows=total, seq_len=_ints(lens))
    cols = max(1, _columns(max(lens)))
    lean = torch.randn((hkv, D), generator=g, device=DEV)
    lean = lean / lean.norm(dim=1, keepdim=True) * math.sqrt(D) / 2
    q = _randn(g, total, hkv, hq // hkv, D)
    s["q"] = (q + (lean * 0.5).to(BF)[None, :, None]).reshape(1, total, hq, D)
    if case["paged"]:
        pages = n * cols + 5
        s["table"] = torch.randperm(pages, generator=g, device=DEV)[:n * cols].to(torch.int32).view(n, cols)
        shape = (1, pages, hkv, PAGE, D)
    else:
        s["table"] = None
        shape = (1, n, hkv, cols * PAGE, D)
    s["k"], s["v"] = (_randn(g, *shape) for _ in "kv")
    heavy = torch.rand(shape[:-1], generator=g, device=DEV) < 0.01
    s["k"] += heavy[..., None] * lean.to(BF)[None, None, :, None]
    s["cols"] = cols
    return s


def _score_inputs(case, seed):
    g = _rng(seed + 77)
    n, vocab = case["rows"], case["vocab"]
    kind = torch.float32 if case["fp32"] else BF
    buf = torch.empty((n, vocab + case["gap"]), dtype=kind, device=DEV)
    token = torch.empty((n,), dtype=torch.int32, device=DEV)
    for lo in range(0, n, 256):
        x = torch.randn((min(256, n - lo), vocab), generator=g, device=DEV) * 2.5
        if case["banned"]:
            x.masked_fill_(torch.rand(x.shape, generator=g, device=DEV) < case["banned"], -math.inf)
        buf[lo:lo + 256, :vocab] = x.to(kind)
        # a token drawn from the row's own distribution
        noise = -torch.log(-torch.log(torch.rand(x.shape, generator=g, device=DEV).clamp(1e-12, 1 - 1e-7)))
        token[lo:lo + 256] = (x + noise).argmax(1).to(torch.int32)
    if case["gap"]:
        buf[:, vocab:] = math.nan       # what lies between the rows is nobody's
    if case["pad"]:
        token[torch.rand((n,), generator=g, device=DEV) < case["pad"]] = -1
    return dict(logits=buf[:, :vocab], token=token)


def prepare(case, seed):
    make = dict(rope=_rope_inputs, cross=_cross_inputs, score=_score_inputs)[case["kind"]]
    s = make(case, seed)
    s["case"] = case
    if case["kind"] == "cross":
        s["out"] = torch.zeros(s["q"].shape, dtype=torch.float32 if case["fp32"] else BF, device=DEV)
    elif case["kind"] == "score":
        n, f, i = case["rows"], dict(device=DEV), dict(device=DEV, dtype=torch.int32)
        s["logprob"] = torch.zeros(n, **f)
        if case["rank"]:
            s["rank"] = torch.zeros(n, **i)
        if case["entropy"]:
            s["entropy"] = torch.zeros(n, **f)
        if case["top"]:
            s["top_token"] = torch.zeros((n, case["top"]), **i)
            s["top_logprob"] = torch.zeros((n, case["top"]), **f)
    if own:
        _handles(s)
    return s


# ----------------------------------------------------------------- the framework's own calls

def _cache(s, n_q_heads, k, v, capacity):
    import sparse_long_context_sfi_gb300 as sfi
    case, paged = s["case"], s["table"] is not None
    s["err"] = torch.zeros(4, dtype=torch.int32, device=DEV)
    return sfi.SfiKvCache(
        n_layers=case.get("layers", 1), batch=case["batch"], n_q_heads=n_q_heads,
        n_kv_heads=case["hkv"], head_dim=D, capacity=capacity, page_size=PAGE if paged else 0,
        n_pages=k.shape[1] if paged else 0, max_pages_per_seq=s["cols"] if paged else 0,
        max_len=max(s["lens"]), k=k.data_ptr(), v=v.data_ptr(),
        page_table=s["table"].data_ptr() if paged else None, seq_len=s["seq_len"].data_ptr(),
        err=s["err"].data_ptr())


def _handles(s):
    """The descriptors, frequencies and workspaces that a user's program keeps."""
    import sparse_long_context_sfi_gb300 as sfi
    case = s["case"]
    if case["kind"] == "score":
        s["scoring"] = sfi.SfiScoring(
            n_rows=case["rows"], vocab=case["vocab"], logits_fp32=1 if case["fp32"] else 0,
            n_top=case["top"], row_stride=s["logits"].stride(0), logits=s["logits"].data_ptr(),
            token=s["token"].data_ptr(), logprob=s["logprob"].data_ptr(),
            **{k: s[k].data_ptr() for k in ("rank", "entropy", "top_token", "top_logprob") if k in s})
        s["ws_bytes"] = sfi.sfi_scoring_workspace_bytes(s["scoring"])
    elif case["kind"] == "cross":
        s["kv"] = _cache(s, case["hq"], s["k"], s["v"], s["cols"] * PAGE)
        s["ws_bytes"] = sfi.sfi_cross_workspace_bytes(s["kv"], s["n_rows"], max(s["rows"]))
    else:
        hq, hkv = case["hq"], case["hkv"]
        if case["append"]:
            k, v = s["k"], s["v"]
        else:
            k = v = torch.zeros((case["layers"], s["table"].max().item() + 1 if s["table"] is not None
                                 else case["batch"], hkv, PAGE if s["table"] is not None else
                                 s["cols"] * PAGE, D), dtype=BF, device=DEV)
            s["stand_in"] = k
        s["kv"] = _cache(s, hq, k, v, s["cols"] * PAGE)
        turns, amplitude = sfi.sfi_rope_turns(case["rot"], **_rope_scaling(case))
        s["turns"] = torch.from_numpy(turns.view("int64")).to(DEV)
        s["rope"] = sfi.SfiRope(
            rot_dim=case["rot"], interleaved=1 if case["inter"] else 0, amplitude=amplitude,
            norm_eps=EPS, turns=s["turns"].data_ptr(),
            q_norm=s["q_norm"].data_ptr() if case["norm"] else None,
            k_norm=s["k_norm"].data_ptr() if case["norm"] else None)
        s["io"] = sfi.SfiRopeRows(
            q=s["q"].data_ptr(), q_out=s["q_out"].data_ptr(), k=s["k_new"].data_ptr(),
            k_out=None if case["append"] else s["k_out"].data_ptr(),
            v=s["v_new"].data_ptr() if case["append"] else None, q_stride=s["q"].stride(1),
            k_stride=s["k_new"].stride(1), v_stride=s["v_new"].stride(1))
        return
    s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=DEV)
    sfi.sfi_workspace_init(s["ws"], s["ws_bytes"])


def _own_run(s):
    import sparse_long_context_sfi_gb300 as sfi
    case, kind = s["case"], s["case"]["kind"]
    if kind == "score":
        sfi.sfi_score_tokens(s["scoring"], s["ws"], s["ws_bytes"])
        return _score_out(s)
    one = case["rows_hi"] == 1
    start, most = None if one else s["start"], max(s["rows"])
    if kind == "cross":
        sfi.sfi_cross_attn(s["kv"], s["q"], s["out"], case["fp32"], start, s["n_rows"], most, s["ws"],
                           s["ws_bytes"])
        return s["out"]
    if not case["append"]:
        sfi.sfi_rope_apply(s["kv"], s["rope"], s["io"], start, s["n_rows"], most)
        return dict(q=s["q_out"], k=s["k_out"])
    s["seq_len"].copy_(s["saved"])
    sfi.sfi_rope_append(s["kv"], s["rope"], s["io"], start, s["n_rows"], most)
    return dict(q=s["q_out"], k=s["k"], v=s["v"], seq_len=s["seq_len"])


def _score_out(s):
    return {k: s[k] for k in ("logprob", "rank", "entropy", "top_token", "top_logprob") if k in s}


# ------------------------------------------------------------------------- the plain forms

def _frequencies(case):
    """Radians per position of each pair, and the factor on the turned dimensions."""
    a = _rope_scaling(case)
    rot, factor, length = case["rot"], a["factor"], a["original_len"]
    base, amplitude = a["base"], 1.0
    if a["scaling"] == "base" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    theta = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if a["scaling"] == "linear":
        theta = [t / factor for t in theta]
    elif a["scaling"] == "ramp":
        def dim(turns):
            return rot * math.log(length / (2 * math.pi * turns)) / (2 * math.log(base))
        first = max(0, math.floor(dim(a["high"])))
        last = min(rot - 1, math.ceil(dim(a["low"])))
        for i, t in enumerate(theta):
            share = min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
            theta[i] = t * (1 - share) + t / factor * share
        amplitude = 0.1 * math.log(factor) + 1.0
    elif a["scaling"] == "smooth":
        for i, t in enumerate(theta):
            turns = length * t / (2 * math.pi)      # over the original length
            keep = min(1.0, max(0.0, (turns - a["low"]) / (a["high"] - a["low"])))
            theta[i] = t * keep + t / factor * (1 - keep)
    return theta, amplitude


def _places(s):
    """Sequence and position of every packed row."""
    row = torch.arange(s["n_rows"], device=DEV)
    b = torch.searchsorted(s["start"], row.to(torch.int32), right=True) - 1
    return b, s["saved"].long()[b] + row - s["start"].long()[b]


def _turned(s, x, weight, at):
    """x [layers][rows][heads][D] normed and turned to the positions `at`, in fp32."""
    case = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    theta, amplitude = _frequencies(case)
    half = case["rot"] // 2
    angle = at.double()[:, None] * torch.tensor(theta, dtype=torch.float64, device=DEV)
    cos, sin = ((f(angle) * amplitude).float()[None, :, None] for f in (torch.cos, torch.sin))
    y = x.clone()
    if case["inter"]:
        a, b = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
    else:
        a, b = slice(0, half), slice(half, 2 * half)
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _plain_rope(s):
    case = s["case"]
    b, at = _places(s)
    s["q_out"].copy_(_turned(s, s["q"], s["q_norm"], at))
    k = _turned(s, s["k_new"], s["k_norm"], at)
    if not case["append"]:
        s["k_out"].copy_(k)
        return dict(q=s["q_out"], k=s["k_out"])
    if s["table"] is None:
        s["k"][:, b, :, at] = k.to(BF).transpose(0, 1)
        s["v"][:, b, :, at] = s["v_new"].transpose(0, 1)
    else:
        page, slot = s["table"][b, at // PAGE].long(), at % PAGE
        s["k"][:, page, :, slot] = k.to(BF).transpose(0, 1)
        s["v"][:, page, :, slot] = s["v_new"].transpose(0, 1)
    s["seq_len"].copy_(s["saved"]).add_(s["start"][1:] - s["start"][:-1])
    return dict(q=s["q_out"], k=s["k"], v=s["v"], seq_len=s["seq_len"])


def _states(s, b):
    """K and V of encoder b: [hkv][length][D]."""
    if s["table"] is None:
        return s["k"][0, b, :, :s["lens"][b]], s["v"][0, b, :, :s["lens"][b]]
    pages = s["table"][b, :_columns(s["lens"][b])].long()
    return (t[0, pages].transpose(0, 1).reshape(s["case"]["hkv"], -1, D)[:, :s["lens"][b]]
            for t in (s["k"], s["v"]))


def _plain_cross(s):
    case = s["case"]
    hkv, group, done = case["hkv"], case["hq"] // case["hkv"], 0
    for b, (length, rows) in enumerate(zip(s["lens"], s["rows"])):
        out = s["out"][0, done:done + rows]
        if length == 0:
            out.zero_()
        else:
            k, v = (t.float() for t in _states(s, b))
            for lo in range(0, rows, 1024):
                n = min(1024, rows - lo)
                q = s["q"][0, done + lo:done + lo + n].float().view(n, hkv, group, D)
                q = q.permute(1, 2, 0, 3).reshape(hkv, group * n, D)
                z = torch.matmul(q, k.transpose(1, 2)) / math.sqrt(D)
                w = torch.exp(z - z.amax(-1, keepdim=True))
                o = torch.matmul(w, v) / w.sum(-1, keepdim=True)
                out[lo:lo + n] = o.view(hkv, group, n, D).permute(2, 0, 1, 3).reshape(n, -1, D).to(out.dtype)
        done += rows
    return s["out"]


def _plain_score(s):
    case = s["case"]
    for lo in range(0, case["rows"], 256):
        at = slice(lo, min(case["rows"], lo + 256))
        x, token = s["logits"][at].float(), s["token"][at].long()
        top = x.amax(-1, keepdim=True)
        w = torch.exp(x - top)
        total = w.double().sum(-1)
        lse = top.double().squeeze(1) + torch.log(total)
        mine = x.gather(1, token.clamp(min=0)[:, None])
        s["logprob"][at] = torch.where(token >= 0, mine.squeeze(1).double() - lse, 0.0).float()
        if case["rank"]:
            before = torch.arange(case["vocab"], device=DEV) < token[:, None]
            rank = ((x > mine) | ((x == mine) & before)).sum(-1)
            s["rank"][at] = torch.where(token >= 0, rank, -1).int()
        if case["entropy"]:
            share = torch.where(w > 0, w * (x - top), 0.0).double().sum(-1) / total
            s["entropy"][at] = (torch.log(total) - share).float()
        if case["top"]:
            best, index = torch.sort(x, dim=1, descending=True, stable=True)
            s["top_token"][at] = index[:, :case["top"]].int()
            s["top_logprob"][at] = (best[:, :case["top"]].double() - lse[:, None]).float()
    return _score_out(s)


def run(state):
    if own:
        return _own_run(state)
    return dict(rope=_plain_rope, cross=_plain_cross, score=_plain_score)[state["case"]["kind"]](state)


# ------------------------------------------------------- the definitions, in 64 bits

def _exact_rope(case, seed):
    """Pairs as complex numbers, turned by multiplication with exp(i angle)."""
    s = _rope_inputs(case, seed)
    s["case"] = case
    theta, amplitude = _frequencies(case)
    b, at = _places(s)
    turn = torch.polar(torch.full((s["n_rows"], len(theta)), amplitude, dtype=torch.float64, device=DEV),
                       torch.outer(at.double(), torch.tensor(theta, dtype=torch.float64, device=DEV)))
    rot = case["rot"]

    def turned(x, weight):
        y = x.double()
        if weight is not None:
            y = y / (y.square().sum(-1, keepdim=True) / D + EPS).sqrt() * weight.double()
        head, rest = y[..., :rot], y[..., rot:]
        order = (..., rot // 2, 2) if case["inter"] else (..., 2, rot // 2)
        pairs = head.reshape(*head.shape[:-1], *order[1:])
        pairs = pairs if case["inter"] else pairs.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[None, :, None])
        z = z if case["inter"] else z.transpose(-1, -2)
        return torch.cat([z.reshape(head.shape), rest], -1)

    q, k = turned(s["q"], s["q_norm"]), turned(s["k_new"], s["k_norm"])
    if not case["append"]:
        return dict(q=q, k=k)
    cache = s["k"].double()
    if s["table"] is None:
        cache[:, b, :, at] = k.transpose(0, 1)
    else:
        cache[:, s["table"][b, at // PAGE].long(), :, at % PAGE] = k.transpose(0, 1)
    return dict(q=q, k=cache, v=None, seq_len=None)     # (values and lengths are moved)


def _exact_cross(case, seed):
    s = _cross_inputs(case, seed)
    s["case"] = case
    group, done = case["hq"] // case["hkv"], 0
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, (length, rows) in enumerate(zip(s["lens"], s["rows"])):
        if length:
            k, v = (t.double() for t in _states(s, b))
            for h in range(case["hq"]):
                q = s["q"][0, done:done + rows, h].double()
                w = torch.softmax(torch.einsum("nd,md->nm", q, k[h // group]) * D ** -0.5, -1)
                out[0, done:done + rows, h] = torch.einsum("nm,md->nd", w, v[h // group])
        done += rows
    return out


def _exact_score(case, seed):
    s = _score_inputs(case, seed)
    parts = []
    for lo in range(0, case["rows"], 128):
        x, token = s["logits"][lo:lo + 128].double(), s["token"][lo:lo + 128].long()
        lp = torch.log_softmax(x, -1)
        none = token < 0
        mine = lp.gather(1, token.clamp(min=0)[:, None])[:, 0]
        part = dict(logprob=torch.where(none, 0.0, mine))
        if case["rank"]:
            xt = x.gather(1, token.clamp(min=0)[:, None])
            tie = (x == xt) & (torch.arange(case["vocab"], device=DEV)[None] < token[:, None])
            rank = (x > xt).sum(1) + tie.sum(1)
            part["rank"] = torch.where(none, -1, rank).int()
        if case["entropy"]:
            part["entropy"] = -torch.where(lp > -math.inf, lp.exp() * lp, 0.0).sum(-1)
        if case["top"]:
            # (stable: the lowest token of equal logits first)
            order = torch.argsort(-x, dim=1, stable=True)[:, :case["top"]]
            part["top_token"] = order.int()
            part["top_logprob"] = lp.gather(1, order)
        parts.append(part)
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


def exact(case, seed):
    return dict(rope=_exact_rope, cross=_exact_cross, score=_exact_score)[case["kind"]](case, seed)
