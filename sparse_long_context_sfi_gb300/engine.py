"""Device state of one SFI decode workload and the calls that step it.

`SfiState` owns (through PyTorch allocations) the KV cache, the packed sparse memory, the
evidence buffer and the workspace, and builds the C descriptors. Stepping goes through the
C ABI only: `step()` issues the per-step calls, `run()` hands a whole decode run to the
native driver `sfi_decode_run` (capturable in a CUDA graph).
"""
from __future__ import annotations

import ctypes as C

import numpy as np
import torch

from . import (SfiBeam, SfiBudget, SfiDecodePlan, SfiKvCache, SfiPagePool, SfiRope, SfiRopeRows,
               SfiScoring, SfiSparseMem, sfi_append_chunk, sfi_append_kv, sfi_beam_select,
               sfi_beam_workspace_bytes, sfi_compact, sfi_cross_attn, sfi_cross_workspace_bytes,
               sfi_decode_run, sfi_dense_decode_attn, sfi_fast_decode_step, sfi_pages_compact,
               sfi_pages_evict, sfi_pages_release, sfi_pages_reserve, sfi_pages_workspace_bytes,
               sfi_reorder, sfi_rope_append, sfi_rope_apply, sfi_rope_turns, sfi_schedule,
               sfi_schedule_tokens, sfi_score_tokens, sfi_scoring_workspace_bytes, sfi_select,
               sfi_sparse_decode_attn, sfi_window_attn, sfi_window_workspace_bytes,
               sfi_workspace_bytes, sfi_workspace_init)


def _torch_stream(stream):
    """The torch stream behind a `stream` argument (None: the current one). Tensors made for a call
    are allocated on the stream that uses them, so that their memory is reused in its order."""
    if stream is None:
        return torch.cuda.current_stream()
    return torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream


def _want(name, t, dtypes, shape, device):
    """Refuses a tensor that the kernels, which get its address alone, would read or write wrongly."""
    dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
    if (not isinstance(t, torch.Tensor) or t.dtype not in dtypes or tuple(t.shape) != tuple(shape) or
            not t.is_contiguous() or t.device != device):
        have = (f"{t.dtype} {tuple(t.shape)} on {t.device}" if isinstance(t, torch.Tensor) else type(t).__name__)
        raise ValueError(f"{name}: contiguous {' or '.join(map(str, dtypes))} {tuple(shape)} on {device}"
                         f" wanted, not {have}")


def _want_rows(name, t, shape, device):
    """Rows of heads that a rope call reads: packed heads, rows anywhere, as in a fused projection."""
    if (not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or tuple(t.shape) != tuple(shape) or
            t.device != device):
        have = (f"{t.dtype} {tuple(t.shape)} on {t.device}" if isinstance(t, torch.Tensor) else type(t).__name__)
        raise ValueError(f"{name}: torch.bfloat16 {tuple(shape)} on {device} wanted, not {have}")
    layers, rows, heads, dim = shape
    if t.numel() == 0:
        return heads * dim      # (nothing is read, whatever the strides say)
    # (of a single row the layers' distance counts, its own stride says nothing)
    step = t.stride(1) if rows > 1 else t.stride(0) if layers > 1 else heads * dim
    if (t.stride(3) != 1 or (heads > 1 and t.stride(2) != dim) or step < heads * dim or step % 8 or
            (layers > 1 and t.stride(0) != rows * step) or t.data_ptr() % 16):
        raise ValueError(f"{name}: heads lie packed, rows a multiple of 8 elements apart and layers the rows apart,"
                         f" on 16 bytes; not strides {t.stride()}")
    return step


_MASK = (torch.uint8, torch.bool)


def _at(device):
    """`device` with its number: a kernel runs on the current device, whatever its arrays are on."""
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


def _here(device):
    if device.type == "cuda" and device.index != torch.cuda.current_device():
        raise ValueError(f"the state is on {device}, which is not the current device")


def _capturing(stream):
    """Whether the call is being captured into a graph."""
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(_torch_stream(stream)):
        return torch.cuda.is_current_stream_capturing()


class _Workspace:
    """A workspace that calls of any shape share, one after the other. What a larger one replaces is
    kept: a captured graph goes on using it. A capture that finds none has one to itself, for its
    clearing is part of the graph and not done yet for anybody else."""

    def __init__(self, device):
        self.device, self.now, self.kept = device, None, []

    def get(self, need, stream):
        if self.now is not None and self.now.numel() >= need:
            return self.now
        size = need if self.now is None else max(need, 2 * self.now.numel())
        with torch.cuda.stream(_torch_stream(stream)):
            ws = torch.empty(size, dtype=torch.uint8, device=self.device)
        sfi_workspace_init(ws, size, stream=stream)
        self.kept.append(ws)
        if not _capturing(stream):
            self.now = ws
        return ws


class Rope:
    """Rotary positions for the calls that take `rope`: frequencies on the device and what goes with
    them. scaling, factor, original_len, low, high: as for sfi_rope_turns; q_norm, k_norm: weights
    (bf16 [128]) of the norm that every head goes through first."""

    def __init__(self, rot_dim=128, interleaved=False, base=10000.0, scaling="none", factor=1.0,
                 original_len=0.0, low=1.0, high=32.0, q_norm=None, k_norm=None, norm_eps=1e-6, device="cuda"):
        turns, self.amplitude = sfi_rope_turns(rot_dim, base, scaling, factor, original_len, low, high)
        self.device = _at(device)
        for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
            if w is not None:
                _want(name, w, torch.bfloat16, (128,), self.device)
                if w.data_ptr() % 16:
                    raise ValueError(f"{name}: lies on 16 bytes")
        if (q_norm is not None or k_norm is not None) and not 0 < norm_eps < float("inf"):
            raise ValueError("norm_eps is above zero and finite")
        self.turns = torch.from_numpy(turns.view(np.int64)).to(self.device)
        self.q_norm, self.k_norm = q_norm, k_norm
        self.desc = SfiRope(rot_dim=rot_dim, interleaved=1 if interleaved else 0, amplitude=self.amplitude,
                            norm_eps=norm_eps, turns=self.turns.data_ptr(),
                            q_norm=None if q_norm is None else q_norm.data_ptr(),
                            k_norm=None if k_norm is None else k_norm.data_ptr())


class SfiState:
    def __init__(self, cfg, len0, device="cuda", page_table=None, n_pages=0, capacity=None):
        self.cfg = cfg
        self.device = _at(device)
        B, Ly, Hkv, Hq, D = cfg.batch, cfg.n_layers, cfg.n_kv_heads, cfg.n_q_heads, cfg.head_dim
        self.len0 = np.asarray(len0, dtype=np.int64)
        self.capacity = capacity or int(self.len0.max()) + cfg.steps
        bf = torch.bfloat16
        if cfg.page_size:
            pt = np.asarray(page_table, dtype=np.int32)
            self.page_table = torch.from_numpy(pt).to(self.device)
            self.n_pages = int(n_pages)
            self.max_pages = int(pt.shape[1])
            self.capacity = self.max_pages * cfg.page_size
            shape = (Ly, self.n_pages, Hkv, cfg.page_size, D)
        else:
            self.page_table = None
            self.n_pages = 0
            self.max_pages = 0
            shape = (Ly, B, Hkv, self.capacity, D)
        self.k = torch.zeros(shape, dtype=bf, device=self.device)
        self.v = torch.zeros(shape, dtype=bf, device=self.device)
        self.seq_len = torch.from_numpy(self.len0.astype(np.int32)).to(self.device)
        self.err = torch.zeros(4, dtype=torch.int32, device=self.device)
        U = Ly * B * Hkv
        self.n_units = U
        comp = cfg.n_sink + cfg.n_select
        self.kc = torch.zeros((Ly, B, Hkv, comp, D), dtype=bf, device=self.device)
        self.vc = torch.zeros((Ly, B, Hkv, comp, D), dtype=bf, device=self.device)
        self.sel_idx = torch.zeros((U, max(1, cfg.n_select)), dtype=torch.int32, device=self.device)
        self.sel_cnt = torch.zeros(U, dtype=torch.int32, device=self.device)
        self.rows = torch.zeros(U, dtype=torch.int32, device=self.device)
        self.scores = torch.zeros((U, self.capacity), dtype=torch.float32, device=self.device)
        self.kv = SfiKvCache(
            n_layers=Ly, batch=B, n_q_heads=Hq, n_kv_heads=Hkv, head_dim=D, capacity=self.capacity,
            page_size=cfg.page_size, n_pages=self.n_pages, max_pages_per_seq=self.max_pages,
            max_len=int(self.len0.max()), k=self.k.data_ptr(), v=self.v.data_ptr(),
            page_table=None if self.page_table is None else self.page_table.data_ptr(),
            seq_len=self.seq_len.data_ptr(), err=self.err.data_ptr())
        self.budget = SfiBudget(n_sink=cfg.n_sink, n_window=cfg.n_window, n_select=cfg.n_select,
                                prior_tau=cfg.prior_tau, lambda_=cfg.lam)
        self.mem = SfiSparseMem(kc=self.kc.data_ptr(), vc=self.vc.data_ptr(),
                                sel_idx=self.sel_idx.data_ptr(), sel_cnt=self.sel_cnt.data_ptr(),
                                rows=self.rows.data_ptr())
        self.ws_bytes = sfi_workspace_bytes(self.kv, self.budget)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        sfi_workspace_init(self.ws, self.ws_bytes)
        self.t = 0
        self._upto = self.len0.copy()   # host bound of every length (len0: the lengths at the start)
        self._window_ws = _Workspace(self.device)
        self._off_course = False    # lengths that are no longer len0 and the steps since
        self._replayed = False      # a captured call may have changed the lengths unseen

    # -- host bookkeeping -------------------------------------------------------------------
    def reset_lengths(self):
        """Every sequence at its length of the start again."""
        self.seq_len.copy_(torch.from_numpy(self.len0.astype(np.int32)))
        self._upto = self.len0.copy()
        self._off_course = False
        self.t = 0

    def _grown(self, rows):
        """The host's bounds after `rows` further rows (of each sequence, or of all)."""
        self._upto = np.minimum(self._upto + rows, self.capacity)

    def _longest(self, more, stream):
        """Host bound of every length before `more` further rows each. Where it would leave no room
        for them the lengths themselves are read: which sequences a mask released, a reserve
        refused or a map reordered is known to the device alone."""
        capturing = _capturing(stream)
        if self._off_course:
            self._replayed = self._replayed or capturing
        if self._replayed:
            return self.capacity - more
        if int(self._upto.max()) + more > self.capacity and not capturing:
            with torch.cuda.stream(_torch_stream(stream)):
                self._upto = self.seq_len.cpu().numpy().astype(np.int64)
        return int(self._upto.max())

    def schedule(self, masks: np.ndarray) -> np.ndarray:
        """Slow flags [steps][B] from per-sequence boundary masks [B][steps]."""
        return np.stack([sfi_schedule(masks[b], self.cfg.t_max) for b in range(self.cfg.batch)], 1)

    def schedule_tokens(self, tokens: np.ndarray, trigger_ids) -> np.ndarray:
        """Slow flags [steps][B] from per-sequence generated token ids [B][steps]: a slow step
        follows a trigger token (or T_max steps without one)."""
        return np.stack([sfi_schedule_tokens(tokens[b], trigger_ids, self.cfg.t_max)
                         for b in range(self.cfg.batch)], 1)

    # -- one decode step through the individual calls -----------------------------------------
    def step(self, q, k_new, v_new, slow_b: np.ndarray, out, out_fp32=True, stream=None,
             fused=True, active=None, rope=None, pos=None):
        """q [Ly][B][Hq][D] bf16, k_new/v_new [Ly][B][Hkv][D] bf16 (device); slow_b [B] bool.
        fused: the fast sequences' append runs inside sfi_fast_decode_step (as in the native
        driver); otherwise every row is appended first and the fast step is
        sfi_sparse_decode_attn. active: device uint8 [B], e.g. from reserve: the others are left as
        they are (their rows of out, too). rope: q and k_new are turned to their positions first
        (pos: device int32 [B], None: the lengths); their rows, and v_new's, which are packed then,
        may be a fused projection's."""
        if rope is not None:
            q, k_new, v_new = self._turned(rope, q, k_new, v_new, out, out_fp32, pos, active, stream)
        elif pos is not None:
            raise ValueError("pos goes with rope")
        return self._step(q, k_new, v_new, slow_b, None, active, out, out_fp32, stream, fused)

    def _turned(self, rope, q, k_new, v_new, out, out_fp32, pos, active, stream):
        """q and k_new of single tokens, turned, and v_new, all packed: the calls that append on their own
        take their addresses alone."""
        _here(self.device)
        c, n = self.cfg, self.cfg.batch
        self._masked(active)
        io = self._chunk(n, q, k_new, v_new, out, out_fp32, rope, pos)
        with torch.cuda.stream(_torch_stream(stream)):
            v_new = v_new.contiguous()
            q_out, k_out = (torch.empty((c.n_layers, n, h, c.head_dim), dtype=torch.bfloat16, device=self.device)
                            for h in (c.n_q_heads, c.n_kv_heads))
        io.q_out, io.k_out = q_out.data_ptr(), k_out.data_ptr()
        sfi_rope_apply(self._whole(), rope.desc, io, None, n, 1, active=active, stream=stream)
        return q_out, k_out, v_new

    def _rope_rows(self, rope, q, k_new, v_new, pos, n):
        """The rows that a rope call reads."""
        c, dev = self.cfg, self.device
        if rope.device != dev:
            raise ValueError(f"the rope is on {rope.device}, the state on {dev}")
        io = SfiRopeRows()
        io.q_stride = _want_rows("q", q, (c.n_layers, n, c.n_q_heads, c.head_dim), dev)
        io.k_stride = _want_rows("k_new", k_new, (c.n_layers, n, c.n_kv_heads, c.head_dim), dev)
        io.v_stride = _want_rows("v_new", v_new, (c.n_layers, n, c.n_kv_heads, c.head_dim), dev)
        io.q, io.k, io.v = q.data_ptr(), k_new.data_ptr(), v_new.data_ptr()
        if pos is not None:
            _want("pos", pos, torch.int32, (n,), dev)
            io.pos = pos.data_ptr()
        return io

    def _step(self, q, k_new, v_new, slow_b, masks, active, out, out_fp32, stream, fused):
        """masks: slow_b and its complement on the device, if they are there already."""
        _here(self.device)
        kv = self.kv
        bound = self._longest(1, stream)
        slow_b = np.asarray(slow_b, bool)
        mixed = slow_b.any() and not slow_b.all()
        a_slow = a_fast = active
        self._masked(active)
        if active is not None:
            bound = min(bound, self.capacity - 1)       # (what is full is not active)
        if mixed:
            m = masks
            if m is None:
                m = torch.from_numpy(np.stack([slow_b, ~slow_b]).astype(np.uint8)).to(self.device)
            if active is not None:
                with torch.cuda.stream(_torch_stream(stream)):
                    m = ((m != 0) & (active != 0)).view(torch.uint8)
            a_slow, a_fast = m[0], m[1]
        kv.max_len = bound
        if not fused:
            sfi_append_kv(kv, k_new, v_new, active=active, stream=stream)
        elif slow_b.any():
            sfi_append_kv(kv, k_new, v_new, active=a_slow, stream=stream)
        kv.max_len = bound + 1
        if slow_b.any():
            sfi_dense_decode_attn(kv, q, out, out_fp32, self.scores, self.ws, self.ws_bytes,
                                  active=a_slow, stream=stream)
            sfi_select(kv, self.scores, self.budget, self.mem, active=a_slow, stream=stream)
            sfi_compact(kv, self.budget, self.mem, active=a_slow, stream=stream)
        if not slow_b.all():
            if fused:
                kv.max_len = bound
                sfi_fast_decode_step(kv, self.mem, self.budget, k_new, v_new, q, out, out_fp32,
                                     self.ws, self.ws_bytes, active=a_fast, stream=stream)
                kv.max_len = bound + 1
            else:
                sfi_sparse_decode_attn(kv, self.mem, self.budget, q, out, out_fp32, self.ws,
                                       self.ws_bytes, active=a_fast, stream=stream)
        self._stepped(stream)
        return mixed and (a_slow, a_fast)

    def _stepped(self, stream):
        self._grown(1)
        self._replayed = self._replayed or _capturing(stream)
        self.t += 1

    # -- a whole run through the native driver --------------------------------------------------
    def side_stream(self, priority=0):
        """The layer-wise pipeline's side stream and its fork and join events (created once;
        the events are recorded once here so that their driver objects exist before any
        stream capture)."""
        if getattr(self, "_side", None) is None:
            side = torch.cuda.Stream(device=self.device, priority=priority)
            fork, join = torch.cuda.Event(), torch.cuda.Event()
            fork.record()
            join.record()
            torch.cuda.synchronize(self.device)
            self._side = (side, fork, join)
        return self._side

    def make_plan(self, slow: np.ndarray, q, k_new, v_new, out, out_fp32=True, out_per_step=True,
                  dense_only=False, events=None, t0=0, t1=None, pipeline=False, pipeline_group=0,
                  concurrent=None):
        """slow: uint8 [steps][B]; q/k_new/v_new/out: device tensors with a leading step axis.
        events: optional list of 2 * (t1 - t0) torch.cuda.Event(enable_timing=True) or None,
        recorded before (2 t) and after (2 t + 1) step t's attention kernel (None: not
        recorded). [t0, t1): the steps this plan covers (a run can be issued as several
        consecutive plans). pipeline: run slow steps group of layers by group, with the
        Selector and compaction of each group on a side stream beside the next group's
        attention; pipeline_group: layers per group (0: about a quarter of the layers).
        concurrent: on steps that mix slow and fast sequences, the fast sequences' fused fast
        step runs on a side stream beside the slow sequences' chain (not with pipeline; the
        results are the same bits); None: on when the plan has such a step."""
        t1 = slow.shape[0] if t1 is None else t1
        q, k_new, v_new = q[t0:t1], k_new[t0:t1], v_new[t0:t1]
        if out_per_step:
            out = out[t0:t1]
        slow = np.ascontiguousarray(slow[t0:t1], dtype=np.uint8)
        steps = slow.shape[0]
        mixed = np.array([(r.any() and not r.all()) for r in slow])
        masks = None
        if concurrent is None:
            concurrent = bool(mixed.any()) and not pipeline and not dense_only
        if mixed.any():
            m = np.stack([slow, 1 - slow], axis=1).astype(np.uint8)
            masks = torch.from_numpy(m).to(self.device)
        plan = SfiDecodePlan(
            n_steps=steps, slow=slow.ctypes.data, q=q.data_ptr(), k_new=k_new.data_ptr(),
            v_new=v_new.data_ptr(), out=out.data_ptr(), out_fp32=1 if out_fp32 else 0,
            out_per_step=1 if out_per_step else 0, scores_f=self.scores.data_ptr(),
            masks=None if masks is None else masks.data_ptr(),
            len_start=int(self._upto.max() if self._off_course else self.len0.max() + t0), dense_only=1 if dense_only else 0)
        if pipeline or concurrent:
            side, fork, join = self.side_stream()
            plan.side_stream, plan.fork_event, plan.join_event = (side.cuda_stream, fork.cuda_event,
                                                                  join.cuda_event)
            plan.pipeline_group = int(pipeline_group)
            plan.concurrent_fast = 1 if concurrent and not pipeline else 0
        ev_arr = None
        if events is not None:
            assert len(events) == 2 * steps
            for e in events:          # make sure the driver-level event objects exist
                if e is not None:
                    e.record()
            torch.cuda.synchronize()
            ev_arr = (C.c_void_p * (2 * steps))(*[None if e is None else e.cuda_event
                                                  for e in events])
            plan.events = C.cast(ev_arr, C.c_void_p)
        plan._keep = (slow, masks, q, k_new, v_new, out, ev_arr, events)
        return plan

    def run(self, plan: SfiDecodePlan, stream=None, active=None):
        """Issue a plan. Steps [t0, t1) start at the lengths of the start and t0 rows, or where
        prompts, windowed steps and reordering have left the lengths since. active (device uint8
        [B], for all steps; not with events): the other sequences are left as they are; the steps
        are then issued one by one, on `stream` alone."""
        if active is not None:
            return self._run_active(plan, active, stream)
        _here(self.device)
        steps = plan.n_steps
        if self._off_course:
            plan = SfiDecodePlan.from_buffer_copy(plan)     # (its arrays are the caller's)
            plan.len_start = self._longest(steps, stream)
        sfi_decode_run(self.kv, self.budget, self.mem, plan, self.ws, self.ws_bytes, stream=stream)
        if self._off_course:
            self._grown(steps)
        else:
            at = self.len0 - self.len0.max() + plan.len_start + steps
            self._upto = np.minimum(np.maximum(self._upto, at), self.capacity)

    def _run_active(self, plan, active, stream):
        _here(self.device)
        slow, masks, q, k_new, v_new, out, _, events = plan._keep
        if events is not None:
            raise ValueError("a plan with events runs with all sequences")
        self._masked(active)
        out_fp32 = bool(plan.out_fp32)
        for t in range(plan.n_steps):
            o = out[t] if plan.out_per_step else out
            if not plan.dense_only:
                self._step(q[t], k_new[t], v_new[t], slow[t], None if masks is None else masks[t], active,
                           o, out_fp32, stream, True)
                continue
            self.kv.max_len = min(self._longest(1, stream), self.capacity - 1)
            sfi_append_kv(self.kv, k_new[t], v_new[t], active=active, stream=stream)
            self.kv.max_len += 1
            sfi_dense_decode_attn(self.kv, q[t], o, out_fp32, None, self.ws, self.ws_bytes, active=active,
                                  stream=stream)
            self._stepped(stream)

    # -- prompts, pages and beams ------------------------------------------------------------
    def pool(self, stream=None) -> SfiPagePool:
        """The page pool behind the table (made on first use: every entry the table holds then
        counts as one reference; not in a capture, as the entries are counted on the way)."""
        _here(self.device)
        if getattr(self, "_pool", None) is None:
            if self.page_table is None:
                raise ValueError("a contiguous cache has no pages")
            if _capturing(stream):
                raise ValueError("the page pool is made by a first call outside the capture")
            with torch.cuda.stream(_torch_stream(stream)):
                held = self.page_table[self.page_table >= 0]
                self.page_refs = torch.bincount(held.long(), minlength=self.n_pages).to(torch.int32)
                self._pool = SfiPagePool(page_table=self.page_table.data_ptr(),
                                         refs=self.page_refs.data_ptr())
                self._pages_bytes = sfi_pages_workspace_bytes(self.kv)
                self._pages_ws = torch.empty(self._pages_bytes, dtype=torch.uint8, device=self.device)
                self._pages_ok = torch.empty(self.cfg.batch, dtype=torch.uint8, device=self.device)
        return self._pool

    def _whole(self):
        """The descriptor for calls that launch the same whatever the lengths are."""
        _here(self.device)
        self.kv.max_len = self.capacity
        return self.kv

    def _bound(self, stream):
        """The descriptor with the host's bound of every length, by which a call is sized. A graph
        is replayed at lengths that the host does not see: its calls, and all after it, are
        sized by the capacity."""
        self._replayed = self._replayed or _capturing(stream)
        self.kv.max_len = self.capacity if self._replayed else int(self._upto.max())
        return self.kv

    def reserve(self, n_new=None, active=None, ok=None, stream=None):
        """Pages for the next n_new[b] positions (device int32 [B]; None: one each). Returns `ok`
        (device uint8 [B], its own unless given): 1 for the active sequences that may write
        them, to be given as `active` to the calls that do."""
        self._masked(active)
        if n_new is not None:
            _want("n_new", n_new, torch.int32, (self.cfg.batch,), self.device)
        if ok is not None:
            _want("ok", ok, torch.uint8, (self.cfg.batch,), self.device)
        pool = self.pool(stream)
        ok = self._pages_ok if ok is None else ok
        sfi_pages_reserve(self._whole(), pool, n_new, self._pages_ws, self._pages_bytes,
                          active=active, ok=ok, stream=stream)
        return ok

    def evict(self, n_window=None, active=None, stream=None):
        """Give up the pages outside the sinks and the recent window."""
        self._masked(active)
        sfi_pages_evict(self._whole(), self.pool(stream), self.cfg.n_sink,
                        self.cfg.n_window if n_window is None else n_window, active=active,
                        stream=stream)

    def release(self, active=None, stream=None):
        """Give up all pages of the active sequences; their lengths become 0."""
        self._masked(active)
        sfi_pages_release(self._whole(), self.pool(stream), active=active, stream=stream)
        if active is None and not _capturing(stream):
            self._upto = np.zeros_like(self._upto)
        self._off_course = True

    def compact_pages(self, stream=None):
        """Move the pages in use to the front of the pool; returns their number (device int32)."""
        pool = self.pool(stream)
        with torch.cuda.stream(_torch_stream(stream)):
            used = torch.empty(1, dtype=torch.int32, device=self.device)
        sfi_pages_compact(self._whole(), pool, used, self._pages_ws, self._pages_bytes, stream=stream)
        return used

    def prefill(self, q, k_new, v_new, rows, out, out_fp32=False, n_window=None, stream=None, rope=None,
                pos=None):
        """One chunk of a prompt: rows[b] (host) new tokens of every sequence, packed in order of
        sequence. Reserves their pages (paged cache), appends k_new/v_new [Ly][n][Hkv][D] and
        attends q [Ly][n][Hq][D] under the sinks and a window of n_window (default: the
        budget's) into out [Ly][n][Hq][D]. A sequence that does not fit its capacity, or whose
        pages the pool does not cover, is left out (its rows of out, too), and the error word
        says so. rope: q and k_new are turned to their positions on the way (pos: device int32 [n],
        None: the cache's); their rows, and v_new's, may then be a fused projection's. Copies rows
        to the device, so it cannot be captured."""
        rows = np.asarray(rows, dtype=np.int32)
        if rows.shape != (self.cfg.batch,) or (rows < 0).any() or q.dim() != 4:
            raise ValueError("rows: a count for every sequence; q: [Ly][n][Hq][D]")
        start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        n, most = int(q.shape[1]), int(rows.max())
        if n < start[-1] or tuple(out.shape) != tuple(q.shape):
            raise ValueError("q and out hold the rows of every sequence")
        io = self._chunk(n, q, k_new, v_new, out, out_fp32, rope, pos)
        window = self.cfg.n_window if n_window is None else n_window
        with torch.cuda.stream(_torch_stream(stream)):
            dev = torch.from_numpy(start).to(self.device)
            if self.page_table is not None:
                active = served = self.reserve(torch.from_numpy(rows).to(self.device), stream=stream)
            else:
                active, served = None, self._fitting(rows, None, stream)
        q = self._append(q, k_new, v_new, dev, n, most, active, stream, rope, io)
        self._grown(rows)
        self._off_course = True
        self._window(q, out, out_fp32, dev, n, most, window, stream, served)

    def window_step(self, q, k_new, v_new, out, out_fp32=True, n_window=None, active=None,
                    stream=None, rope=None, pos=None):
        """One new token each, attended under the sinks and a window straight from the cache (no
        packed memory): q/out [Ly][B][Hq][D], k_new/v_new [Ly][B][Hkv][D]. A sequence without
        room is left out, as by prefill. rope, pos: as for prefill."""
        window = self.cfg.n_window if n_window is None else n_window
        self._masked(active)
        io = self._chunk(self.cfg.batch, q, k_new, v_new, out, out_fp32, rope, pos)
        if self.page_table is not None:
            active = served = self.reserve(active=active, stream=stream)
        else:
            served = self._fitting(1, active, stream)
        q = self._append(q, k_new, v_new, None, self.cfg.batch, 1, active, stream, rope, io)
        self._grown(1)
        self.t += 1
        self._off_course = True
        self._window(q, out, out_fp32, None, self.cfg.batch, 1, window, stream, served)

    def _masked(self, active):
        if active is not None:
            _want("active", active, _MASK, (self.cfg.batch,), self.device)

    def _chunk(self, n, q, k_new, v_new, out, out_fp32, rope=None, pos=None):
        """The arrays of a chunk of n rows; those of a rope call are returned."""
        c, dev = self.cfg, self.device
        io = None
        if rope is not None:
            io = self._rope_rows(rope, q, k_new, v_new, pos, n)
        else:
            if pos is not None:
                raise ValueError("pos goes with rope")
            _want("q", q, torch.bfloat16, (c.n_layers, n, c.n_q_heads, c.head_dim), dev)
            _want("k_new", k_new, torch.bfloat16, (c.n_layers, n, c.n_kv_heads, c.head_dim), dev)
            _want("v_new", v_new, torch.bfloat16, (c.n_layers, n, c.n_kv_heads, c.head_dim), dev)
        _want("out", out, torch.float32 if out_fp32 else torch.bfloat16, q.shape, dev)
        return io

    def _append(self, q, k_new, v_new, start, n, most, active, stream, rope, io):
        """The chunk's keys and values into the cache; returns the queries, turned where there is rope."""
        if rope is None:
            sfi_append_chunk(self._whole(), k_new, v_new, start, n, most, active=active, stream=stream)
            return q
        with torch.cuda.stream(_torch_stream(stream)):
            turned = torch.empty(q.shape, dtype=torch.bfloat16, device=self.device)
        io.q_out = turned.data_ptr()
        sfi_rope_append(self._whole(), rope.desc, io, start, n, most, active=active, stream=stream)
        return turned

    def _fitting(self, rows, active, stream):
        """Which of the active sequences of a contiguous cache have room for `rows` more (host int or
        [B]): what the append takes and the attention may look at. `active` itself where the
        host's bounds say that all have."""
        if not (self._replayed or _capturing(stream)) and (self._upto + rows).max() <= self.capacity:
            return active
        with torch.cuda.stream(_torch_stream(stream)):
            more = rows if isinstance(rows, int) else torch.from_numpy(rows).to(self.device)
            fits = self.seq_len + more <= self.capacity
            if active is not None:
                fits &= active != 0
            return fits.view(torch.uint8)

    def _window(self, q, out, out_fp32, start, n, most, window, stream, active=None):
        kv = self._bound(stream)
        ws = self._window_ws.get(sfi_window_workspace_bytes(kv, n, most, self.cfg.n_sink, window), stream)
        sfi_window_attn(kv, q, out, out_fp32, start, n, most, self.cfg.n_sink, window, ws, ws.numel(),
                        active=active, stream=stream)

    def reorder(self, src, stream=None):
        """Every sequence b takes over the state of sequence src[b] (device int32 [B]): table,
        length, packed memory. Forked sequences share their pages until they are reserved."""
        _want("src", src, torch.int32, (self.cfg.batch,), self.device)
        pool = self.pool(stream) if self.page_table is not None else None
        sfi_reorder(self._whole(), src, pool=pool, budget=self.budget, mem=self.mem, stream=stream)
        self._upto = np.full_like(self._upto, self._upto.max())     # (src stays on the device)
        self._replayed = self._replayed or _capturing(stream)
        self._off_course = True


class BeamSearch:
    """Beams of n_groups prompts on the device: scores, finished flags and the selection, whose
    `parent` is the src of SfiState.reorder. The first selection expands beam 0 of each group."""

    def __init__(self, n_groups, n_beams, vocab, eos=-1, device="cuda"):
        self.n_groups, self.n_beams, self.vocab, self.eos = n_groups, n_beams, vocab, eos
        rows = n_groups * n_beams
        dev = dict(device=_at(device))
        self.cum = torch.full((rows,), -float("inf"), dtype=torch.float32, **dev)
        self.cum[::n_beams] = 0.0
        self.done = torch.zeros(rows, dtype=torch.uint8, **dev)
        self.parent = torch.zeros(rows, dtype=torch.int32, **dev)
        self.token = torch.zeros(rows, dtype=torch.int32, **dev)
        self._ws = _Workspace(self.cum.device)

    def select(self, logits, rank_scale=None, stream=None):
        """logits [rows][vocab] (bf16 or fp32, rows may be strided): keeps the best beams; returns
        (parent, token); cum and done are updated in place, so that a captured selection can
        be replayed."""
        if logits.shape != (self.n_groups * self.n_beams, self.vocab) or logits.stride(1) != 1:
            raise ValueError("logits are [rows][vocab] with contiguous rows")
        if logits.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("logits are bf16 or fp32")
        if logits.device != self.cum.device:
            raise ValueError(f"logits are on {logits.device}, the beams on {self.cum.device}")
        _here(self.cum.device)
        if rank_scale is not None:
            _want("rank_scale", rank_scale, torch.float32, self.cum.shape, self.cum.device)
        beam = SfiBeam(
            n_groups=self.n_groups, n_beams=self.n_beams, vocab=self.vocab,
            logits_fp32=1 if logits.dtype == torch.float32 else 0, row_stride=logits.stride(0),
            eos=self.eos, logits=logits.data_ptr(), cum=self.cum.data_ptr(),
            done=self.done.data_ptr() if self.eos >= 0 else None,
            rank_scale=None if rank_scale is None else rank_scale.data_ptr(),
            parent=self.parent.data_ptr(), token=self.token.data_ptr(),
            cum_out=self.cum.data_ptr(), done_out=self.done.data_ptr())
        ws = self._ws.get(sfi_beam_workspace_bytes(beam), stream)
        sfi_beam_select(beam, ws, ws.numel(), stream=stream)
        return self.parent, self.token


class EncoderStates:
    """Keys and values of encoder inputs on the device, one sequence each, and the attention of a
    decoder's rows to them. Rows of one input lie together: of a prompt's chunk, of its beams. The
    calls of one object share its workspace: they follow each other, also in captured graphs, and what
    runs at once is called on objects of its own."""

    def __init__(self, n_layers, batch, n_q_heads, n_kv_heads, capacity, device="cuda"):
        self.n_layers, self.batch, self.n_q_heads, self.n_kv_heads = n_layers, batch, n_q_heads, n_kv_heads
        self.capacity, self.device = capacity, _at(device)
        dev = dict(device=self.device)
        self.k, self.v = (torch.zeros((n_layers, batch, n_kv_heads, capacity, 128), dtype=torch.bfloat16, **dev)
                          for _ in "kv")
        self.seq_len = torch.zeros(batch, dtype=torch.int32, **dev)
        self.err = torch.zeros(4, dtype=torch.int32, **dev)
        self.lens = np.zeros(batch, dtype=np.int64)
        self.kv = SfiKvCache(
            n_layers=n_layers, batch=batch, n_q_heads=n_q_heads, n_kv_heads=n_kv_heads, head_dim=128,
            capacity=capacity, page_size=0, n_pages=0, max_pages_per_seq=0, max_len=0, k=self.k.data_ptr(),
            v=self.v.data_ptr(), page_table=None, seq_len=self.seq_len.data_ptr(), err=self.err.data_ptr())
        self._ws = _Workspace(self.device)

    def clear(self, which=None, stream=None):
        """Empty the inputs of `which` (indices on the host; None: all)."""
        _here(self.device)
        which = list(range(self.batch)) if which is None else sorted({int(i) for i in which})
        if any(i < 0 or i >= self.batch for i in which):
            raise ValueError(f"inputs are numbered from 0 to {self.batch - 1}")
        if _capturing(stream):
            raise ValueError("the host keeps the lengths: no changes in a capture")
        with torch.cuda.stream(_torch_stream(stream)):
            if len(which) == self.batch:
                self.seq_len.zero_()
            elif which:
                self.seq_len[torch.tensor(which).to(self.device)] = 0
        self.lens[which] = 0

    def write(self, k_new, v_new, rows, stream=None):
        """rows[e] (host) further states of every input, packed: k_new, v_new [Ly][n][Hkv][128]."""
        _here(self.device)
        rows = np.asarray(rows, dtype=np.int32)
        if rows.shape != (self.batch,) or (rows < 0).any():
            raise ValueError("rows: a count for every input")
        if (self.lens + rows).max() > self.capacity:
            raise ValueError(f"an input of more than {self.capacity} states")
        n = int(rows.sum())
        for name, t in (("k_new", k_new), ("v_new", v_new)):
            _want(name, t, torch.bfloat16, (self.n_layers, n, self.n_kv_heads, 128), self.device)
        if _capturing(stream):
            raise ValueError("the host keeps the lengths: no changes in a capture")
        start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        with torch.cuda.stream(_torch_stream(stream)):
            dev = torch.from_numpy(start).to(self.device)
        self.kv.max_len = int(self.lens.max())
        sfi_append_chunk(self.kv, k_new, v_new, dev, n, int(rows.max()), stream=stream)
        self.lens += rows

    def attend(self, q, out, rows=1, out_fp32=False, active=None, stream=None):
        """q [Ly][n][Hq][128] to all states of their input, into out [Ly][n][Hq][128]: rows[e] rows of
        every input (host; an int: as many of each, which can be captured). active: device uint8
        [inputs]. Rows behind the last, and of inputs that are not active, are left as they are."""
        _here(self.device)
        each = isinstance(rows, (int, np.integer))
        counts = np.full(self.batch, rows, dtype=np.int64) if each else np.asarray(rows, dtype=np.int64)
        if counts.shape != (self.batch,) or (counts < 0).any() or not isinstance(q, torch.Tensor) or q.dim() != 4:
            raise ValueError("rows: a count for every input; q: [Ly][n][Hq][128]")
        n, most = int(q.shape[1]), int(counts.max())
        if counts.sum() > n:
            raise ValueError("q holds the rows of every input")
        _want("q", q, torch.bfloat16, (self.n_layers, n, self.n_q_heads, 128), self.device)
        _want("out", out, torch.float32 if out_fp32 else torch.bfloat16, q.shape, self.device)
        if active is not None:
            _want("active", active, _MASK, (self.batch,), self.device)
        if most == 0:
            return
        start = None
        if not (each and rows == 1 and n == self.batch):
            with torch.cuda.stream(_torch_stream(stream)):
                if each:
                    start = torch.arange(0, (self.batch + 1) * most, most, dtype=torch.int32, device=self.device)
                else:
                    start = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(self.device)
        # (a captured call is replayed when other inputs may have been written)
        self.kv.max_len = self.capacity if _capturing(stream) else int(self.lens.max())
        ws = self._ws.get(sfi_cross_workspace_bytes(self.kv, n, most), stream)
        sfi_cross_attn(self.kv, q, out, out_fp32, start, n, most, ws, ws.numel(), active=active, stream=stream)


class TokenScores:
    """Log probabilities of tokens under rows of logits. The calls of one object share its workspace: they
    follow each other, also in captured graphs; what runs at once has an object of its own."""

    def __init__(self, device="cuda"):
        self.device = _at(device)
        self._ws = _Workspace(self.device)

    def score(self, logits, token=None, n_top=0, rank=False, entropy=False, stream=None):
        """logits [rows][vocab] (bf16 or fp32, rows may be strided), token: device int32 [rows] (below 0:
        none). Returns a dict of what was asked for: logprob [rows] (with token), rank [rows], entropy
        [rows], top_token and top_logprob [rows][n_top], as sfi_score_tokens defines them."""
        if not isinstance(logits, torch.Tensor) or logits.dim() != 2 or logits.shape[1] < 1 or logits.stride(1) != 1:
            raise ValueError("logits are [rows][vocab] with contiguous rows")
        if logits.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("logits are bf16 or fp32")
        if logits.device != self.device:
            raise ValueError(f"logits are on {logits.device}, the scores on {self.device}")
        _here(self.device)
        rows, vocab = logits.shape
        stride = logits.stride(0) if rows > 1 else vocab
        if stride < vocab:
            raise ValueError("rows of logits do not overlap")
        if token is not None:
            _want("token", token, torch.int32, (rows,), self.device)
        elif rank:
            raise ValueError("a rank goes with a token")
        if not 0 <= n_top <= min(32, vocab):
            raise ValueError("n_top is at most 32 and the vocabulary")
        if token is None and not entropy and not n_top:
            raise ValueError("nothing is asked for")
        with torch.cuda.stream(_torch_stream(stream)):
            new = lambda kind, *shape: torch.empty(shape, dtype=kind, device=self.device)
            out = {}
            if token is not None:
                out["logprob"] = new(torch.float32, rows)
            if rank:
                out["rank"] = new(torch.int32, rows)
            if entropy:
                out["entropy"] = new(torch.float32, rows)
            if n_top:
                out["top_token"], out["top_logprob"] = new(torch.int32, rows, n_top), new(torch.float32, rows, n_top)
        if rows == 0:
            return out
        sc = SfiScoring(n_rows=rows, vocab=vocab, logits_fp32=1 if logits.dtype == torch.float32 else 0, n_top=n_top,
                        row_stride=stride, logits=logits.data_ptr(),
                        token=None if token is None else token.data_ptr(),
                        **{name: t.data_ptr() for name, t in out.items()})
        ws = self._ws.get(sfi_scoring_workspace_bytes(sc), stream)
        sfi_score_tokens(sc, ws, ws.numel(), stream=stream)
        return out
