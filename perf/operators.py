"""What the cache-side operators around the decode path are measured on.

Three families, each as a user's program calls it: attention of prompt chunks and single
tokens with sinks and a sliding window over the KV cache; the upkeep of a paged cache
(reserving with copy on write, appending, evicting, forking, compacting); and one step of
beam search (selection over beams and vocabulary, reordering, reserving).
"""
from __future__ import annotations

import math

import torch

own = False

D = 128        # head dimension
PAGE = 16      # tokens of a page
BF = torch.bfloat16
DEV = "cuda"


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # the prompts of the 32K batch-4 configuration, whole, with its sinks and window
        dict(name="prompt_32k_w64", kind="attn", batch=4, lo=32768, hi=32768, rows_lo=32768,
             rows_hi=32768, hq=32, hkv=8, sink=4, window=64, paged=False, fp32=False),
        # chunked prefill: the last 8192 tokens of a 32K prompt under a long window
        dict(name="chunk_8k_w4096", kind="attn", batch=1, lo=32768, hi=32768, rows_lo=8192,
             rows_hi=8192, hq=32, hkv=8, sink=4, window=4096, paged=False, fp32=False),
        # a ragged batch of prompts of odd lengths in pages, eight query heads a kv head
        dict(name="ragged_paged_w1000", kind="attn", batch=8, lo=1537, hi=8191, rows_lo=700,
             rows_hi=1500, hq=64, hkv=8, sink=5, window=1000, paged=True, fp32=False),
        # one new token each for the ragged paged batch of 32, long window
        dict(name="token_paged_b32_w4096", kind="attn", batch=32, lo=8192, hi=32768, rows_lo=1,
             rows_hi=1, hq=32, hkv=8, sink=4, window=4096, paged=True, fp32=False),
        # the smallest decode: one sequence, two kv heads, the 4K configuration; fp32 outputs
        dict(name="token_4k_w64", kind="attn", batch=1, lo=4096, hi=4096, rows_lo=1, rows_hi=1,
             hq=8, hkv=2, sink=4, window=64, paged=False, fp32=True),
        # four prompt chunks of 8K enter a paged cache: reserve their pages, write their rows
        dict(name="pages_prompt_4x8k", kind="grow", batch=4, lo=8192, hi=24576, rows_lo=8192,
             rows_hi=8192, hkv=8, layers=1, shared=1, evict=0),
        # a serving step of a ragged batch: dead pages out of the window freed, tails that four
        # forks share copied before they are written, a few rows each appended, four layers
        dict(name="pages_step_b32", kind="grow", batch=32, lo=500, hi=5000, rows_lo=1, rows_hi=40,
             hkv=8, layers=4, shared=4, evict=1024),
        # a pool after many requests came and went: the pages in use moved to the front
        dict(name="pages_compact_16k", kind="compact", batch=32, pages=16384, used=0.5, hkv=8,
             layers=1),
        # eight prompts become four beams each: tables, lengths and packed sparse memory
        dict(name="fork_8x4", kind="fork", batch=32, beams=4, lo=8192, hi=32768, hkv=8, sink=4,
             select=956, layers=1),
        # beam search of one prompt
        dict(name="beam_1x4_v32000", kind="beam", groups=1, beams=4, vocab=32000, fp32=False,
             done=0.0),
        # the widest batch the cache takes, odd vocabulary, some beams finished
        dict(name="beam_32x8_v128001", kind="beam", groups=32, beams=8, vocab=128001, fp32=True,
             done=0.1),
        # one whole step for eight prompts: select, reorder the tables, reserve the next token
        dict(name="beam_step_8x4", kind="step", groups=8, beams=4, vocab=32000, fp32=False,
             done=0.0, lo=1000, hi=8000, hkv=8, layers=1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attn", "attn", "token", "grow", "compact", "fork", "beam", "beam", "step"])
    hkv = rng.choice([2, 4, 8])
    if kind == "attn":
        batch, window = rng.randint(1, 8), _log(rng, 16, 4096)
        # at most the tokens x window of the largest chunk, and the tokens of the largest batch
        rows = _log(rng, 2, max(2, min(16384, 8192 * 4096 // (batch * (window + 256)))))
        hi = rows + _log(rng, 1, 16384)
        return dict(kind="attn", batch=batch, lo=max(rows, hi * 2 // 3), hi=hi,
                    rows_lo=max(1, rows // 2), rows_hi=rows, hq=hkv * rng.choice([1, 2, 4]),
                    hkv=hkv, sink=rng.choice([0, 1, 4, 17, 64]), window=window,
                    paged=rng.random() < 0.5, fp32=rng.random() < 0.25)
    if kind == "token":
        hi = _log(rng, 40, 32768)
        return dict(kind="attn", batch=_log(rng, 1, 32), lo=hi // 2 + 1, hi=hi, rows_lo=1,
                    rows_hi=1, hq=hkv * rng.choice([1, 2, 4, 8]), hkv=hkv,
                    sink=rng.choice([0, 1, 4, 17, 64]), window=_log(rng, 16, 8192),
                    paged=rng.random() < 0.5, fp32=rng.random() < 0.5)
    if kind == "grow":
        shared = rng.choice([1, 2, 4])
        batch, rows = shared * rng.randint(1, 8), _log(rng, 1, 1024)
        hi = _log(rng, 20, 16384)
        return dict(kind="grow", batch=batch, lo=hi // 3 + 1, hi=hi, rows_lo=rows // 2,
                    rows_hi=rows, hkv=hkv, layers=rng.choice([1, 2, 3]), shared=shared,
                    evict=rng.choice([0, 0, 100, 1024]))
    if kind == "compact":
        return dict(kind="compact", batch=rng.randint(1, 64), pages=_log(rng, 64, 16384),
                    used=rng.uniform(0.05, 0.95), hkv=hkv, layers=1)
    if kind == "fork":
        beams = rng.choice([2, 3, 4, 8])
        hi = _log(rng, 100, 32768)
        return dict(kind="fork", batch=beams * rng.randint(1, 32 // beams), beams=beams,
                    lo=hi // 2 + 1, hi=hi, hkv=hkv, sink=rng.choice([0, 4, 16]),
                    select=_log(rng, 16, 956), layers=1)
    groups, beams = _log(rng, 1, 32), rng.randint(1, 8)
    case = dict(kind=kind, groups=groups, beams=beams, vocab=_log(rng, 500, 128001),
                fp32=rng.random() < 0.5, done=rng.choice([0.0, 0.1, 0.3]))
    if kind == "step":
        hi = _log(rng, 40, 8000)
        case.update(lo=hi // 2 + 1, hi=hi, hkv=hkv, layers=1, vocab=min(case["vocab"], 32000))
    return case


def _spread(lo, hi, n):
    """n sizes in [lo, hi], fixed by the case: hi first, the others strewn over the range."""
    return [hi - (i * 40503) % (hi - lo + 1) for i in range(n)]


def _shapes(case):
    """Lengths and row counts of the case's sequences."""
    n = case["batch"]
    rows = _spread(case["rows_lo"], case["rows_hi"], n) if "rows_lo" in case else [1] * n
    lens = [max(a, r) for a, r in zip(_spread(case["lo"], case["hi"], n), rows)]
    return lens, rows


# ------------------------------------------------------------------------- bytes and flops

def _visible(length, rows, sink, window):
    """(query, key) pairs that are visible, and distinct keys seen, over the last `rows` rows."""
    pairs, first = 0, length - rows
    low = max(0, first - window + 1)
    keys = length - low + min(sink, low)
    # rows whose window still reaches position 0 see everything; the others window + sinks
    full = max(0, min(length, window) - first)
    pairs += sum(range(first + 1, first + full + 1)) if full else 0
    for i in (range(first + full, min(length, window + sink))):  # sinks partly in the window
        pairs += window + min(sink, i - window + 1)
    rest = length - max(first + full, window + sink)
    return pairs + max(0, rest) * (window + sink), keys


def work(case):
    kind = case["kind"]
    if kind == "attn":
        lens, rows = _shapes(case)
        seen = [_visible(a, r, case["sink"], case["window"]) for a, r in zip(lens, rows)]
        q = sum(rows) * case["hq"] * D
        return {"bytes": q * 2 + q * (4 if case["fp32"] else 2)
                + sum(s[1] for s in seen) * case["hkv"] * D * 4,
                "flops": 4 * D * case["hq"] * sum(s[0] for s in seen)}
    if kind == "grow":
        lens, rows = _shapes(case)
        moved = sum(rows)
        if case["shared"] > 1:  # all but one of each set of forks copy their tail's rows
            moved += sum(a % PAGE for i, a in enumerate(_fork_lens(case)) if i % case["shared"])
        pages = _pool_pages(case)
        return {"bytes": 2 * moved * case["hkv"] * D * 4 * case["layers"] + 4 * pages, "flops": 0}
    if kind == "compact":
        n = case["pages"]
        move = n * case["used"] * (1 - case["used"])
        return {"bytes": int(2 * move * case["layers"] * case["hkv"] * PAGE * D * 4 + 8 * n
                             + 8 * n * case["used"]), "flops": 0}
    if kind == "fork":
        n, cols = case["batch"], _columns(max(_spread(case["lo"], case["hi"], case["batch"])))
        src, dst = n // case["beams"], n - n // case["beams"]
        row = case["sink"] + case["select"]
        return {"bytes": case["layers"] * case["hkv"] * row * D * 4 * (src + dst)
                + 4 * cols * (n + dst) + 8 * n * cols, "flops": 0}
    rows = case["groups"] * case["beams"]
    total = {"bytes": rows * (case["vocab"] * (4 if case["fp32"] else 2) + 24),
             "flops": rows * case["vocab"] * 4}
    if kind == "step":
        cols = _columns(case["hi"] + 1)
        total["bytes"] += 8 * rows * cols + 4 * (rows * cols)
        total["bytes"] += rows * (PAGE // 2) * case["hkv"] * D * 8 * case["layers"]
    return total


def _columns(length):
    return (length + PAGE - 1) // PAGE


def _fork_lens(case):
    """Lengths before a `grow` case's rows are appended: forks of one prompt have one length."""
    lens = _spread(case["lo"], case["hi"], case["batch"])
    return [lens[i - i % case["shared"]] for i in range(case["batch"])]


def _pool_pages(case):
    lens, (_, rows) = _fork_lens(case), _shapes(case)
    return sum(_columns(a + r) + 1 for a, r in zip(lens, rows)) + case["batch"]


# ------------------------------------------------------------------------------ the inputs

def _rng(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(0x5F1 + seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(BF)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _starts(rows):
    return _ints([sum(rows[:i]) for i in range(len(rows) + 1)])


def _attn_inputs(case, seed):
    """q, the cache, its table and the lengths. Queries lean towards a direction that the
    sinks' keys and a few heavy positions share, as in attention with sinks."""
    g = _rng(seed)
    lens, rows = _shapes(case)
    n, hq, hkv = case["batch"], case["hq"], case["hkv"]
    s = dict(lens=lens, rows=rows, seq_len=_ints(lens), start=_starts(rows), n_rows=sum(rows))
    cols = _columns(max(lens) + 16)
    lean = torch.randn((hkv, D), generator=g, device=DEV)
    lean = lean / lean.norm(dim=1, keepdim=True) * math.sqrt(D) / 2
    q = torch.randn((s["n_rows"], hkv, hq // hkv, D), generator=g, device=DEV, dtype=BF)
    s["q"] = (q + (lean * 0.5).to(BF)[None, :, None]).reshape(1, s["n_rows"], hq, D)
    if case["paged"]:
        pages = n * cols + 7
        s["table"] = torch.randperm(pages, generator=g, device=DEV)[:n * cols].to(torch.int32)
        s["table"] = s["table"].view(n, cols)
        shape = (1, pages, hkv, PAGE, D)
    else:
        s["table"] = None
        shape = (1, n, hkv, cols * PAGE, D)
    s["k"], s["v"] = (torch.randn(shape, generator=g, device=DEV, dtype=BF) for _ in "kv")
    heavy = torch.rand(shape[:-1], generator=g, device=DEV) < 0.01
    if case["paged"]:
        heavy[:, s["table"][:, 0].long(), :, :4] = True
    else:
        heavy[:, :, :, :4] = True
    s["k"] += heavy[..., None] * lean.to(BF)[None, None, :, None]
    return s


def _pool_inputs(case, seed, lens, ahead, forks):
    """A pool in use: shuffled pages, tables of `lens`, `forks` neighbours sharing one table;
    the integers in one buffer so that a pass can put them back with one copy."""
    g = _rng(seed)
    n, cols = case["batch"], _columns(max(a + r for a, r in zip(lens, ahead)))
    pages = sum(_columns(a + r) + 1 for a, r in zip(lens, ahead)) + n
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    ints = torch.zeros(n * cols + pages + n, dtype=torch.int32, device=DEV)
    s = dict(ints=ints, n=n, cols=cols, pages=pages)
    _views(s)
    held = _ints([_columns(a) for a in lens])
    owner = torch.arange(n, device=DEV) // forks * forks
    first = torch.cumsum(held, 0) - held
    at = first[owner][:, None] + torch.arange(cols, device=DEV)
    have = torch.arange(cols, device=DEV) < held[:, None]
    s["table"].copy_(torch.where(have, ids[at.clamp(max=pages - 1)], -1))
    s["refs"].copy_(torch.bincount(s["table"][have], minlength=pages))
    s["seq_len"].copy_(_ints(lens))
    s["saved"] = ints.clone()
    shape = (case["layers"], pages, case["hkv"], PAGE, D)
    s["k"], s["v"] = (torch.randn(shape, generator=g, device=DEV, dtype=BF) for _ in "kv")
    return s, g


def _views(s):
    a, b = s["n"] * s["cols"], s["n"] * s["cols"] + s["pages"]
    s["table"], s["refs"] = s["ints"][:a].view(s["n"], s["cols"]), s["ints"][a:b]
    s["seq_len"] = s["ints"][b:]


def _grow_inputs(case, seed):
    lens, (_, rows) = _fork_lens(case), _shapes(case)
    s, g = _pool_inputs(case, seed, lens, rows, case["shared"])
    total = sum(rows)
    s.update(rows=_ints(rows), start=_starts(rows), n_rows=total)
    s["k_new"], s["v_new"] = (_randn(g, case["layers"], total, case["hkv"], D) for _ in "kv")
    return s


def _compact_inputs(case, seed):
    g = _rng(seed)
    n, pages = case["batch"], case["pages"]
    used = max(1, int(pages * case["used"]))
    cols = (used + n - 1) // n
    s = dict(n=n, cols=cols, pages=pages,
             ints=torch.full((n * cols + pages + n,), -1, dtype=torch.int32, device=DEV))
    _views(s)
    ids = torch.randperm(pages, generator=g, device=DEV)[:used].to(torch.int32)
    s["table"].view(-1)[:used] = ids
    s["refs"].copy_(torch.bincount(ids, minlength=pages))
    s["seq_len"].copy_((s["table"] >= 0).sum(1) * PAGE)
    s["saved"] = s["ints"].clone()
    s["n_used"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    shape = (case["layers"], pages, case["hkv"], PAGE, D)
    s["k"], s["v"] = (torch.randn(shape, generator=g, device=DEV, dtype=BF) for _ in "kv")
    return s


def _fork_inputs(case, seed):
    lens = _spread(case["lo"], case["hi"], case["batch"])
    s, g = _pool_inputs({**case, "layers": 1}, seed, lens, [1] * len(lens), 1)
    n, beams, keep = case["batch"], case["beams"], case["sink"] + case["select"]
    # every slot but the first of each set is empty before the fork
    empty = torch.arange(n, device=DEV) % beams != 0
    s["table"][empty] = -1
    s["seq_len"][empty] = 0
    s["refs"].copy_(torch.bincount(s["table"][s["table"] >= 0], minlength=s["pages"]))
    s["saved"] = s["ints"].clone()
    s["src"] = (torch.arange(n, device=DEV) // beams * beams).to(torch.int32)
    shape = (case["layers"], n, case["hkv"])
    s["kc"], s["vc"] = (_randn(g, *shape, keep, D) for _ in "kv")
    s["sel"] = torch.randint(0, case["lo"], (*shape, case["select"]), generator=g, device=DEV,
                             dtype=torch.int32).sort(-1).values
    s["cnt"] = torch.full(shape, case["select"], dtype=torch.int32, device=DEV)
    s["have"] = torch.full(shape, keep, dtype=torch.int32, device=DEV)
    return s


def _beam_inputs(case, seed):
    g = _rng(seed + 77)
    rows, vocab = case["groups"] * case["beams"], case["vocab"]
    x = torch.randn((rows, vocab), generator=g, device=DEV) * 2.5
    return dict(logits=x if case["fp32"] else x.to(BF),
                cum=-20 * torch.rand((rows,), generator=g, device=DEV),
                done=torch.rand((rows,), generator=g, device=DEV) < case["done"],
                scale=0.5 + torch.rand((rows,), generator=g, device=DEV), eos=2,
                parent=torch.zeros(rows, dtype=torch.int32, device=DEV),
                token=torch.zeros(rows, dtype=torch.int32, device=DEV),
                cum_out=torch.zeros(rows, device=DEV),
                done_out=torch.zeros(rows, dtype=torch.bool, device=DEV))


def _step_inputs(case, seed):
    lens = _spread(case["lo"], case["hi"], case["groups"])
    each = [a for a in lens for _ in range(case["beams"])]
    full = {**case, "batch": len(each)}
    s, _ = _pool_inputs(full, seed, each, [1] * len(each), case["beams"])
    s.update(_beam_inputs(case, seed))
    s["rows"] = torch.ones(len(each), dtype=torch.int32, device=DEV)
    return s


def prepare(case, seed):
    make = dict(attn=_attn_inputs, grow=_grow_inputs, compact=_compact_inputs, fork=_fork_inputs,
                beam=_beam_inputs, step=_step_inputs)[case["kind"]]
    s = make(case, seed)
    s["case"] = case
    if case["kind"] == "attn":
        s["out"] = torch.zeros(s["q"].shape, dtype=torch.float32 if case["fp32"] else BF, device=DEV)
    if own:
        _handles(s)
    return s


# ----------------------------------------------------------------- the framework's own calls

def _handles(s):
    """The descriptors and workspaces that a user's program keeps."""
    import sparse_long_context_sfi_gb300 as sfi
    case = s["case"]
    s["err"] = torch.zeros(4, dtype=torch.int32, device=DEV)
    if "k" in s:
        paged = s["table"] is not None
        cap = s["table"].shape[1] * PAGE if paged else s["k"].shape[3]
        hkv = case["hkv"]
        s["kv"] = sfi.SfiKvCache(
            n_layers=s["k"].shape[0], batch=s["seq_len"].numel(), n_q_heads=case.get("hq", hkv),
            n_kv_heads=hkv, head_dim=D, capacity=cap, page_size=PAGE if paged else 0,
            n_pages=s["k"].shape[1] if paged else 0,
            max_pages_per_seq=s["table"].shape[1] if paged else 0,
            max_len=int(s["seq_len"].max()), k=s["k"].data_ptr(), v=s["v"].data_ptr(),
            page_table=s["table"].data_ptr() if paged else None,
            seq_len=s["seq_len"].data_ptr(), err=s["err"].data_ptr())
    if "refs" in s:
        s["pool"] = sfi.SfiPagePool(page_table=s["table"].data_ptr(), refs=s["refs"].data_ptr())
        s["ws_bytes"] = sfi.sfi_pages_workspace_bytes(s["kv"])
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=DEV)
        sfi.sfi_workspace_init(s["ws"], s["ws_bytes"])
    if case["kind"] == "attn":
        s["max_rows"] = max(s["rows"])
        s["ws_bytes"] = sfi.sfi_window_workspace_bytes(s["kv"], s["n_rows"], s["max_rows"],
                                                       case["sink"], case["window"])
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=DEV)
        sfi.sfi_workspace_init(s["ws"], s["ws_bytes"])
    if case["kind"] == "grow":
        s["max_rows"] = int(s["rows"].max())
    if case["kind"] == "fork":
        s["budget"] = sfi.SfiBudget(n_sink=case["sink"], n_window=64, n_select=case["select"],
                                    prior_tau=64, lambda_=0.1)
        s["mem"] = sfi.SfiSparseMem(kc=s["kc"].data_ptr(), vc=s["vc"].data_ptr(),
                                    sel_idx=s["sel"].data_ptr(), sel_cnt=s["cnt"].data_ptr(),
                                    rows=s["have"].data_ptr())
    if "logits" in s:
        s["beam"] = sfi.SfiBeam(
            n_groups=case["groups"], n_beams=case["beams"], vocab=case["vocab"],
            logits_fp32=1 if case["fp32"] else 0, row_stride=case["vocab"], eos=s["eos"],
            logits=s["logits"].data_ptr(), cum=s["cum"].data_ptr(), done=s["done"].data_ptr(),
            rank_scale=s["scale"].data_ptr(), parent=s["parent"].data_ptr(),
            token=s["token"].data_ptr(), cum_out=s["cum_out"].data_ptr(),
            done_out=s["done_out"].data_ptr())
        s["beam_bytes"] = sfi.sfi_beam_workspace_bytes(s["beam"])
        s["beam_ws"] = torch.empty(s["beam_bytes"], dtype=torch.uint8, device=DEV)
        sfi.sfi_workspace_init(s["beam_ws"], s["beam_bytes"])


def _own_run(s):
    import sparse_long_context_sfi_gb300 as sfi
    case, kind = s["case"], s["case"]["kind"]
    if kind == "attn":
        one = case["rows_hi"] == 1
        sfi.sfi_window_attn(s["kv"], s["q"], s["out"], case["fp32"], None if one else s["start"],
                            s["n_rows"], s["max_rows"], case["sink"], case["window"], s["ws"],
                            s["ws_bytes"])
        return s["out"]
    if kind == "beam":
        sfi.sfi_beam_select(s["beam"], s["beam_ws"], s["beam_bytes"])
        return _beam_out(s)
    s["ints"].copy_(s["saved"])
    if kind == "grow":
        if case["evict"]:
            sfi.sfi_pages_evict(s["kv"], s["pool"], 4, case["evict"])
        sfi.sfi_pages_reserve(s["kv"], s["pool"], s["rows"], s["ws"], s["ws_bytes"])
        sfi.sfi_append_chunk(s["kv"], s["k_new"], s["v_new"], s["start"], s["n_rows"],
                             s["max_rows"])
    elif kind == "compact":
        sfi.sfi_pages_compact(s["kv"], s["pool"], s["n_used"], s["ws"], s["ws_bytes"])
    elif kind == "fork":
        sfi.sfi_reorder(s["kv"], s["src"], pool=s["pool"], budget=s["budget"], mem=s["mem"])
    else:
        sfi.sfi_beam_select(s["beam"], s["beam_ws"], s["beam_bytes"])
        sfi.sfi_reorder(s["kv"], s["parent"], pool=s["pool"])
        sfi.sfi_pages_reserve(s["kv"], s["pool"], None, s["ws"], s["ws_bytes"])
    return _pool_out(s)


def _beam_out(s):
    return dict(parent=s["parent"], token=s["token"], cum=s["cum_out"], done=s["done_out"])


def _pool_out(s):
    kind = s["case"]["kind"]
    out = dict(table=s["table"], refs=s["refs"], seq_len=s["seq_len"])
    if kind == "fork":
        out.update(kc=s["kc"], vc=s["vc"], sel=s["sel"], cnt=s["cnt"], have=s["have"])
    else:
        out.update(k=s["k"], v=s["v"])
    if kind == "compact":
        out["n_used"] = s["n_used"]
    if kind == "step":
        out.update(_beam_out(s))
    return out


# ------------------------------------------------------------------------- the plain forms

def _cache_rows(s, b, at):
    """K and V rows of sequence b at the positions `at`: fp32 [hkv][n][D]."""
    if s["table"] is None:
        return s["k"][0, b][:, at].float(), s["v"][0, b][:, at].float()
    page, row = s["table"][b].long()[at // PAGE], at % PAGE
    return (s["k"][0][page, :, row].transpose(0, 1).float(),
            s["v"][0][page, :, row].transpose(0, 1).float())


def _plain_block(s, b, i0, i1):
    """Attention of the query positions [i0, i1) of sequence b, over the sinks and the union of
    their windows."""
    case = s["case"]
    hkv, group = case["hkv"], case["hq"] // case["hkv"]
    low = max(0, i0 - case["window"] + 1)
    at = torch.cat([torch.arange(min(case["sink"], low), device=DEV),
                    torch.arange(low, i1, device=DEV)])
    k, v = _cache_rows(s, b, at)
    row = sum(s["rows"][:b]) + i0 - (s["lens"][b] - s["rows"][b])
    q = s["q"][0, row:row + i1 - i0].float().view(i1 - i0, hkv, group, D).permute(1, 2, 0, 3)
    z = torch.matmul(q.reshape(hkv, -1, D), k.transpose(1, 2)) / math.sqrt(D)
    i = torch.arange(i0, i1, device=DEV)[:, None]
    seen = (at <= i) & ((at < case["sink"]) | (at > i - case["window"]))
    z = z.view(hkv, group, i1 - i0, -1).masked_fill(~seen, -math.inf)
    p = torch.exp(z - z.amax(-1, keepdim=True))
    o = torch.matmul((p / p.sum(-1, keepdim=True)).view(hkv, -1, at.numel()), v)
    s["out"][0, row:row + i1 - i0] = o.view(hkv, group, i1 - i0, D).permute(2, 0, 1, 3).reshape(
        i1 - i0, case["hq"], D).to(s["out"].dtype)


def _plain_attn(s):
    step = max(128, min(1024, s["case"]["window"] // 2))
    for b, (length, rows) in enumerate(zip(s["lens"], s["rows"])):
        for i0 in range(length - rows, length, step):
            _plain_block(s, b, i0, min(length, i0 + step))
    return s["out"]


def _plain_evict(s, sink, window):
    cols = torch.arange(s["cols"], device=DEV)
    dead = (cols >= _columns(sink)) & (cols < ((s["seq_len"] - window) // PAGE)[:, None])
    dead &= s["table"] >= 0
    s["refs"].sub_(torch.bincount(s["table"][dead], minlength=s["pages"]))
    s["table"][dead] = -1


def _plain_reserve(s, rows):
    """Pages for the next rows[b] positions of each sequence: missing ones and copies of shared
    ones, from the lowest free pages in order of sequence and position."""
    table, refs, length = s["table"], s["refs"], s["seq_len"]
    cols = torch.arange(s["cols"], device=DEV)
    first = length // PAGE
    last = (length + rows + PAGE - 1) // PAGE
    span = (cols >= first[:, None]) & (cols < last[:, None]) & (rows > 0)[:, None]
    b, c = (span & (table >= 0)).nonzero(as_tuple=True)
    old = table[b, c].long()
    order = torch.sort(old, stable=True).indices
    same = torch.arange(len(old), device=DEV) - torch.searchsorted(old[order], old[order])
    rank = torch.empty_like(same).scatter_(0, order, same)
    leave = refs[old] - rank > 1  # all but the last of those that share a page copy it
    need = span & (table < 0)
    need[b[leave], c[leave]] = True
    nb, nc = need.nonzero(as_tuple=True)
    new = (refs == 0).nonzero().flatten()[:len(nb)]
    was = table[nb, nc].long()
    table[nb, nc] = new.to(torch.int32)
    refs[new] = 1
    refs.sub_(torch.bincount(was[was >= 0], minlength=s["pages"]))
    keep = (was >= 0) & (nc == first[nb]) & (length[nb] % PAGE > 0)
    to, of = new[keep], was[keep]
    live = (torch.arange(PAGE, device=DEV) < (length[nb] % PAGE)[keep][:, None])[None, :, None, :, None]
    s["k"][:, to] = torch.where(live, s["k"][:, of], s["k"][:, to])
    s["v"][:, to] = torch.where(live, s["v"][:, of], s["v"][:, to])


def _plain_append(s):
    row = torch.arange(s["n_rows"], device=DEV)
    b = torch.searchsorted(s["start"], row.to(torch.int32), right=True) - 1
    at = s["seq_len"][b] + row - s["start"][b]
    page, slot = s["table"][b, at // PAGE].long(), (at % PAGE).long()
    s["k"][:, page, :, slot] = s["k_new"].transpose(0, 1)
    s["v"][:, page, :, slot] = s["v_new"].transpose(0, 1)
    s["seq_len"].add_(s["rows"])


def _plain_compact(s):
    used = s["refs"] > 0
    n_used = used.sum()
    ids = torch.arange(s["pages"], device=DEV)
    holes = (~used & (ids < n_used)).nonzero().flatten()
    movers = (used & (ids >= n_used)).nonzero().flatten()
    ids[movers] = holes
    s["table"].copy_(torch.where(s["table"] >= 0, ids[s["table"].clamp(min=0).long()], -1))
    s["refs"][holes] = s["refs"][movers]
    s["refs"][movers] = 0
    s["k"][:, holes] = s["k"][:, movers]
    s["v"][:, holes] = s["v"][:, movers]
    s["n_used"].fill_(0).add_(n_used)


def _plain_reorder(s, src):
    before = torch.bincount(s["table"][s["table"] >= 0], minlength=s["pages"])
    src = src.long()
    s["table"].copy_(s["table"][src])
    after = torch.bincount(s["table"][s["table"] >= 0], minlength=s["pages"])
    s["refs"].add_(after).sub_(before)
    s["seq_len"].copy_(s["seq_len"][src])
    if "kc" in s:
        for name in ("kc", "vc", "sel", "cnt", "have"):
            s[name].copy_(s[name][:, src])


def _plain_select(s):
    """Scores in 64 bits (two candidates of different beams may be close), the best n_beams of
    each group with ties to the lowest flat index."""
    case = s["case"]
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    score = x - top - torch.log(torch.exp(x - top).sum(-1, keepdim=True)) + s["cum"].double()[:, None]
    score = torch.where(torch.isnan(score), -math.inf, score)
    alone = torch.arange(case["vocab"], device=DEV) == s["eos"]
    rest = torch.where(alone, s["cum"].double()[:, None], -math.inf)
    score = torch.where(s["done"][:, None], rest, score)
    ranked = torch.where(s["done"][:, None] & ~alone, math.nan, score * s["scale"].double()[:, None])
    # what a finished beam does not offer sorts below -inf
    shape = (case["groups"], case["beams"] * case["vocab"])
    ranked = torch.where(torch.isnan(ranked), -math.inf, ranked).view(shape)
    best = torch.sort(ranked, dim=1, descending=True, stable=True).indices[:, :case["beams"]]
    base = torch.arange(case["groups"], device=DEV)[:, None] * case["beams"]
    parent = (base + best // case["vocab"]).flatten()
    token = (best % case["vocab"]).flatten()
    s["parent"].copy_(parent)
    s["token"].copy_(token)
    s["cum_out"].copy_(score.view(shape).gather(1, best).flatten())
    s["done_out"].copy_(s["done"][parent] | (token == s["eos"]))


def _plain_run(s):
    case, kind = s["case"], s["case"]["kind"]
    if kind == "attn":
        return _plain_attn(s)
    if kind == "beam":
        _plain_select(s)
        return _beam_out(s)
    s["ints"].copy_(s["saved"])
    if kind == "grow":
        if case["evict"]:
            _plain_evict(s, 4, case["evict"])
        _plain_reserve(s, s["rows"])
        _plain_append(s)
    elif kind == "compact":
        _plain_compact(s)
    elif kind == "fork":
        _plain_reorder(s, s["src"])
    else:
        _plain_select(s)
        _plain_reorder(s, s["parent"])
        _plain_reserve(s, s["rows"])
    return _pool_out(s)


def run(state):
    return _own_run(state) if own else _plain_run(state)


# ------------------------------------------------------- the definitions, in 64 bits

def _exact_attn(case, seed):
    s = _attn_inputs(case, seed)
    group, done = case["hq"] // case["hkv"], 0
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, (length, rows) in enumerate(zip(s["lens"], s["rows"])):
        pos = torch.arange(length, device=DEV)
        if s["table"] is None:
            kb, vb = s["k"][0, b, :, :length], s["v"][0, b, :, :length]
        else:
            pages = s["table"][b].long()
            kb, vb = (t[0, pages].transpose(0, 1).reshape(case["hkv"], -1, D)[:, :length]
                      for t in (s["k"], s["v"]))
        for lo in range(0, rows, 512):
            n = min(512, rows - lo)
            i = length - rows + lo + torch.arange(n, device=DEV)
            reach = (pos < case["sink"]) | (pos > i[0] - case["window"])
            at = pos[reach & (pos <= i[-1])]
            q = s["q"][0, done + lo:done + lo + n].double()
            k, v = (t[:, at].double().repeat_interleave(group, 0) for t in (kb, vb))
            z = torch.einsum("nhd,hmd->hnm", q, k) * D ** -0.5
            hidden = (at > i[:, None]) | ((at >= case["sink"]) & (i[:, None] - at >= case["window"]))
            w = torch.softmax(torch.where(hidden, -math.inf, z), -1)
            out[0, done + lo:done + lo + n] = torch.einsum("hnm,hmd->nhd", w, v)
        done += rows
    return out


def _exact_select(case, seed):
    s = _beam_inputs(case, seed)
    beams, vocab = case["beams"], case["vocab"]
    lp = torch.log_softmax(s["logits"].double(), -1) + s["cum"].double()[:, None]
    picked = []
    for g in range(case["groups"]):
        pairs = []
        for r in range(g * beams, (g + 1) * beams):
            w = float(s["scale"][r].double())
            if bool(s["done"][r]):
                c = float(s["cum"][r].double())
                pairs.append((-c * w, r, s["eos"], c, True))
                continue
            row, keep = lp[r], min(beams, vocab)
            last = torch.topk(row, keep).values[-1]
            at = (row >= last).nonzero().flatten()
            pairs += [(-c * w, r, v, c, v == s["eos"]) for v, c in zip(at.tolist(), row[at].tolist())]
        picked += sorted(pairs)[:beams]
    def whole(k):
        return torch.tensor([p[k] for p in picked], dtype=torch.int32, device=DEV)
    return dict(parent=whole(1), token=whole(2),
                cum=torch.tensor([p[3] for p in picked], dtype=torch.float64, device=DEV),
                done=torch.tensor([p[4] for p in picked], device=DEV))


def exact(case, seed):
    if case["kind"] == "attn":
        return _exact_attn(case, seed)
    if case["kind"] == "beam":
        return _exact_select(case, seed)
    if case["kind"] == "step":  # the pages are moved, not computed
        none = dict.fromkeys(("table", "refs", "seq_len", "k", "v"))
        return {**none, **_exact_select(case, seed)}
    return None
