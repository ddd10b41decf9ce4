"""One compression event as a user runs it: buffers plus the C-ABI calls.

``MeanKEvent``   score (Mean-K) → select → pack + re-RoPE
``SlotMapEvent`` score (QueryMemory) → select → redirect + free
``PagedEvent``   LSE-recovery score → LRFU keep score → select → tail plan →
                 in-place compaction
``TieredMeanKEvent`` the Mean-K event with the index and the raw history in
                 host memory: score in bounded layer tiles, select, tiered pack
``TreeDecodeEvent`` a decoding step with drafted trees on a paged cache: tree
                 attention per layer → commit of the accepted path →
                 accumulated weight → eviction to a budget
``HistoryEvent`` prompts and decoding on a paged cache whose older blocks are
                 held in 8 bits: norms, rotation and storing per layer →
                 attention over the prompt, or over history and cache → full
                 blocks packed to 8 bits

All only allocate caller-side buffers with torch and call the library's
entry points; an event can be captured in a CUDA graph (``capture()``) so
that its launches replay without host overhead.

``MeanKEvent.run`` pipelines over groups of layers: the score of group g+1
(tensor-core and exponential heavy) runs on the caller's stream while the
select and pack of group g (latency-bound, then HBM-bound streaming) run on a
second stream, so the two kinds of work share the SMs instead of taking
turns.  Every call
covers whole layers, which is possible because every tensor is laid out
layer-major.
"""
from __future__ import annotations

from typing import Optional, Sequence

import numpy as np
import torch

from . import (BLOCK_TOKENS, kvc_pack_rerope, kvc_pack_tiered, kvc_pack_tiered_slots,
               kvc_repo_plan, kvc_recover_score_ex,
               kvc_recover_score_workspace_size, kvc_score_ex, kvc_score_qmem_ex,
               kvc_redirect_free,
               kvc_redirect_free_workspace_size, kvc_rope_table, kvc_score,
               kvc_lrfu_update, kvc_score_qmem, kvc_score_qmem_workspace_size,
               kvc_score_workspace_size, kvc_select, kvc_tail_compact, kvc_tail_plan,
               TREE_MAX_NODES, kvc_prompt_attn, kvc_q8_attn, kvc_q8_attn_workspace_size,
               kvc_q8_pack, kvc_qkv_rope,
               kvc_attn_mass, kvc_attn_mass_workspace_size, kvc_mass_evict,
               kvc_mass_evict_workspace_size, kvc_tree_attn, kvc_tree_attn_workspace_size,
               kvc_tree_commit)


def _dev_i64(x, device) -> torch.Tensor:
    return torch.as_tensor(np.asarray(x, dtype=np.int64), device=device)


def _ws(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _on(stream, device):
    """The context that sends torch's own calls to `stream` as the library takes it: None (the
    current stream), a Stream, or a raw handle (0: the default stream)."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return torch.cuda.stream(stream)
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return torch.cuda.stream(torch.cuda.ExternalStream(handle, device=device) if handle
                             else torch.cuda.default_stream(device))


def groups_hint(L: int) -> int:
    """Layer groups of the event.  One group (score all layers, then select,
    then pack) measures fastest on GB300 for the 8B-class event: the
    tensor-core scorer fills every SM's registers, so a concurrent pack could
    not share the SMs anyway, and a single persistent score launch balances
    its units best.  More groups remain available for experiments."""
    return 1


class MeanKEvent:
    """Buffers and calls of a Mean-K-mode event over ragged sessions.

    Layouts (see include/kvc.h): q [L][n_sess][Hq][W][D], meank
    [L][H][nb_total][D], kraw/vraw [L_pack][H][n_tok][D]; outputs scores
    [L][H][nb_total], kept [L][H][n_sess][budget], kview/vview
    [L_pack][H][n_sess][32·budget][D].  Pack runs on the first L_pack layers.
    """

    def __init__(self, L: int, H: int, Hq: int, D: int, W: int,
                 hist: Sequence[int], budget: int, n_sink: int, n_recent: int,
                 L_pack: Optional[int] = None, theta: float = 1e6,
                 pos0: int = 0, keepmask: bool = False, device="cuda",
                 groups: Optional[int] = None):
        self.L, self.H, self.Hq, self.D, self.W = L, H, Hq, D, W
        self.hist = [int(n) for n in hist]
        if any(n % BLOCK_TOKENS for n in self.hist):
            raise ValueError("history lengths must be multiples of 32 tokens")
        self.n_sess = len(self.hist)
        self.budget, self.n_sink, self.n_recent = budget, n_sink, n_recent
        self.L_pack = L if L_pack is None else L_pack
        self.device = torch.device(device)
        tok_off = np.concatenate([[0], np.cumsum(self.hist)]).astype(np.int64)
        blk_off = tok_off // BLOCK_TOKENS
        self.n_tok = int(tok_off[-1])
        self.nb_total = int(blk_off[-1])
        self.nb_max = max(n // BLOCK_TOKENS for n in self.hist)
        seg = [0]
        for l in range(L):
            for h in range(H):
                base = (l * H + h) * self.nb_total
                for r in range(self.n_sess):
                    seg.append(base + int(blk_off[r + 1]))
        self.n_seg = L * H * self.n_sess
        dev = self.device
        self.tok_off = _dev_i64(tok_off, dev)
        self.blk_off = _dev_i64(blk_off, dev)
        self.seg_off = _dev_i64(seg, dev)
        self.scores = torch.empty(L, H, self.nb_total, dtype=torch.float32, device=dev)
        self.kept = torch.empty(L, H, self.n_sess, budget, dtype=torch.int32, device=dev)
        self.kept_count = torch.empty(L, H, self.n_sess, dtype=torch.int32, device=dev)
        words = (self.nb_max + 31) // 32
        self.keepmask = (torch.empty(self.n_seg, words, dtype=torch.int32, device=dev)
                         if keepmask else None)
        self.ws = _ws(kvc_score_workspace_size(L, H, Hq, W, self.n_sess, self.nb_max,
                                               self.nb_total), dev)
        self.view_tokens = BLOCK_TOKENS * budget
        self.rope_tab = torch.empty(self.view_tokens, D // 2, 2, dtype=torch.float32,
                                    device=dev)
        kvc_rope_table(self.rope_tab, self.view_tokens, pos0, D, theta)
        shape = (self.L_pack, H, self.n_sess, self.view_tokens, D)
        self.kview = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        self.vview = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.graph = None
        self.side = torch.cuda.Stream(device=dev)
        self.groups = self._layer_groups(groups_hint(L) if groups is None else groups)
        self.score_kernel = "auto"  # the scorer run() uses (a kvc_kernel name)

    @staticmethod
    def _split(L: int, n: int):
        n = max(1, min(n, L))
        edges = [round(i * L / n) for i in range(n + 1)]
        return [(edges[i], edges[i + 1]) for i in range(n) if edges[i + 1] > edges[i]]

    def _layer_groups(self, n: int):
        return self._split(self.L, n)

    # -- the three steps, on a range of layers [l0, l1) ------------------
    def score(self, q, meank, stream=None, l0=0, l1=None, kernel=None):
        """Scores of layers [l0, l1); `kernel` names one scorer (kvc_score_ex);
        by default the event's `score_kernel` ("auto": the library's choice)."""
        l1 = self.L if l1 is None else l1
        kernel = self.score_kernel if kernel is None else kernel
        kvc_score_ex(q[l0:l1], meank[l0:l1], self.scores[l0:l1], l1 - l0, self.H, self.Hq,
                     self.D, self.W, self.blk_off, self.n_sess, self.nb_total, self.nb_max,
                     self.ws, kernel, self.dev_status, stream)

    def select(self, scores=None, stream=None, l0=0, l1=None):
        l1 = self.L if l1 is None else l1
        per = self.H * self.n_sess
        kvc_select(self.scores if scores is None else scores,
                   self.seg_off[l0 * per:l1 * per + 1], (l1 - l0) * per, self.nb_max,
                   self.budget, self.n_sink, self.n_recent, self.kept[l0:l1],
                   self.kept_count[l0:l1],
                   None if self.keepmask is None else self.keepmask[l0 * per:l1 * per],
                   self.dev_status, stream)

    def pack(self, kraw, vraw, kept=None, kept_count=None, stream=None, l0=0, l1=None):
        l1 = self.L_pack if l1 is None else min(l1, self.L_pack)
        if l1 <= l0:
            return
        kept = self.kept if kept is None else kept
        kept_count = self.kept_count if kept_count is None else kept_count
        kvc_pack_rerope(kraw[l0:l1], vraw[l0:l1], kept[l0:l1], kept_count[l0:l1],
                        l1 - l0, self.H, self.D, self.tok_off, self.n_sess, self.n_tok,
                        self.budget, self.rope_tab, self.kview[l0:l1], self.vview[l0:l1],
                        self.dev_status, stream)

    def run_serial(self, q, meank, kraw, vraw, stream=None):
        """score → select → pack over all layers, one stream."""
        self.score(q, meank, stream)
        self.select(stream=stream)
        self.pack(kraw, vraw, stream=stream)

    def run(self, q, meank, kraw, vraw, timers=None):
        """The event, layer groups pipelined over two streams (asynchronous
        with respect to the host; ordered after prior work on the current
        stream, and the current stream waits for all of it).  With one layer
        group every launch stays on the current stream.  `timers`, if
        given, is a list that receives (stage, start, end) CUDA events around
        every launch, recorded on the launching stream."""
        main = torch.cuda.current_stream(self.device)
        side = self.side if len(self.groups) > 1 else main
        if side is not main:
            side.wait_stream(main)

        def timed(stage, stream, fn):
            if timers is None:
                fn()
                return
            a = torch.cuda.Event(enable_timing=True)
            b = torch.cuda.Event(enable_timing=True)
            a.record(stream)
            fn()
            b.record(stream)
            timers.append((stage, a, b))

        for (l0, l1) in self.groups:
            timed("score", main, lambda: self.score(q, meank, main, l0, l1))
            if side is not main:
                done = torch.cuda.Event()
                done.record(main)
                side.wait_event(done)
            with torch.cuda.stream(side):
                timed("select", side, lambda: self.select(None, side, l0, l1))
                if l0 < self.L_pack:
                    timed("pack", side, lambda: self.pack(kraw, vraw, stream=side, l0=l0, l1=l1))
        if side is not main:
            main.wait_stream(side)

    # -- CUDA graph ----------------------------------------------------
    def capture(self, q, meank, kraw, vraw):
        """Capture run() on these input tensors; replay() re-runs it."""
        s = torch.cuda.Stream(device=self.device)
        s.wait_stream(torch.cuda.current_stream(self.device))
        with torch.cuda.stream(s):
            self.run(q, meank, kraw, vraw)  # warm-up (sets kernel attributes)
        torch.cuda.current_stream(self.device).wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.run(q, meank, kraw, vraw)
        self.graph = g
        return g

    def replay(self):
        self.graph.replay()


class TieredMeanKEvent(MeanKEvent):
    """KVMem's tiered execution view ("Tiered movement"): the Mean-K index and
    the raw K/V history stay in pinned host memory; only the execution view,
    the scores and this event's scratch live on the GPU.

    score   the index is scored in bounded tiles of `stage_layers` layers:
            each tile is copied host → device into one of two staging
            buffers on a copy stream while the previous tile is scored on
            the current stream (the scorer is the device-resident one, and
            a unit's partial sums merge in one order whatever else a launch
            holds, so the scores are the same bit for bit);
    select  as MeanKEvent;
    pack    kvc_pack_tiered: blocks that the previous step also kept come
            from the previous view (raw K from a raw-K cache, V from the V
            view), the others are read by the kernel from host memory.
    Two sets of (kept lists, raw-K cache, V view) alternate between steps.
    """

    def __init__(self, *args, stage_layers: int = 4, **kw):
        super().__init__(*args, **kw)
        dev = self.device
        self.stage_layers = max(1, min(stage_layers, self.L))
        self.stage = [torch.empty(self.stage_layers, self.H, self.nb_total, self.D,
                                  dtype=torch.bfloat16, device=dev) for _ in range(2)]
        self.copy_stream = torch.cuda.Stream(device=dev)
        self.kept_sets = [self.kept, torch.empty_like(self.kept)]
        self.count_sets = [self.kept_count, torch.empty_like(self.kept_count)]
        self.kcaches = [torch.empty_like(self.kview), torch.empty_like(self.kview)]
        self.vviews = [self.vview, torch.empty_like(self.vview)]
        self.n_hits = torch.zeros(1, dtype=torch.int32, device=dev)
        self.cur, self.steps = 0, 0
        # per staging buffer: an event after the last score that read it
        # (kept across calls, so the next step's first copies need wait only
        # for that, not for the previous step's select and pack)
        self.stage_free = [None, None]

    def score_tiered(self, q, meank_host, after_tile=None):
        """Scores of every layer from the host-resident index [L][H][nb][D].
        `after_tile(l0, l1)`, if given, is called after each tile's score is
        queued (on the current stream, while the copy stream brings in the
        next tiles)."""
        main = torch.cuda.current_stream(self.device)
        cs = self.copy_stream
        free = self.stage_free
        for gi, (l0, l1) in enumerate(self._split(self.L, -(-self.L // self.stage_layers))):
            b = gi % 2
            n = l1 - l0
            with torch.cuda.stream(cs):
                if free[b] is not None:
                    cs.wait_event(free[b])
                self.stage[b][:n].copy_(meank_host[l0:l1], non_blocking=True)
                ready = torch.cuda.Event()
                ready.record(cs)
            main.wait_event(ready)
            kvc_score(q[l0:l1], self.stage[b][:n], self.scores[l0:l1], n, self.H, self.Hq,
                      self.D, self.W, self.blk_off, self.n_sess, self.nb_total, self.nb_max,
                      self.ws, self.dev_status, main)
            free[b] = torch.cuda.Event()
            free[b].record(main)
            if after_tile is not None:
                after_tile(l0, l1)

    def pack_tiered(self, kraw_host, vraw_host, l0=0, l1=None):
        """The tiered pack of packed layers [l0, l1) (all of them by default)."""
        l1 = self.L_pack if l1 is None else min(l1, self.L_pack)
        if l1 <= l0:
            return
        cur, prev = self.cur, 1 - self.cur
        first = self.steps == 0
        sl = slice(l0, l1)
        kvc_pack_tiered(kraw_host[sl], vraw_host[sl],
                        None if first else self.kept_sets[prev][sl],
                        None if first else self.count_sets[prev][sl],
                        None if first else self.kcaches[prev][sl],
                        None if first else self.vviews[prev][sl],
                        self.kept_sets[cur][sl], self.count_sets[cur][sl],
                        l1 - l0, self.H, self.D, self.tok_off, self.n_sess, self.n_tok,
                        self.budget, self.rope_tab, self.kcaches[cur][sl], self.kview[sl],
                        self.vviews[cur][sl], self.n_hits, self.dev_status)

    def step(self, q, meank_host, kraw_host, vraw_host, pipelined=True):
        """One agent step; afterwards kview / vview hold this step's view.
        Pipelined (the default): each index tile's select and pack are queued
        right after its score, so they run while the copy stream brings in
        the next tiles (layers are independent: the same outputs bit for bit
        as score, select, pack one after another)."""
        cur = self.cur
        self.kept, self.kept_count = self.kept_sets[cur], self.count_sets[cur]
        self.vview = self.vviews[cur]
        if pipelined:
            main = torch.cuda.current_stream(self.device)

            def tile(l0, l1):
                self.select(stream=main, l0=l0, l1=l1)
                self.pack_tiered(kraw_host, vraw_host, l0, l1)

            self.score_tiered(q, meank_host, after_tile=tile)
        else:
            self.score_tiered(q, meank_host)
            self.select()
            self.pack_tiered(kraw_host, vraw_host)
        self.cur, self.steps = 1 - cur, self.steps + 1


class RepoTieredEvent(TieredMeanKEvent):
    """KVMem's tiered view with its repository view ("Tiered movement": the
    repository view tracks where each block lives, blocks recalled often
    prefer host RAM over NVMe).  The raw history lives in a KvcRepo: every
    block in its backing file, the most-used ones in host slots.  A step
    scores and selects as TieredMeanKEvent, copies the packed layers' kept
    lists to the host, plans the blocks the step uses and the ones it misses
    (kvc_repo_plan), brings the misses into host slots (kvc_repo_step: one
    vectored read per run of consecutive blocks), applies the slots that
    changed to the slot table it keeps on the GPU, and packs with
    kvc_pack_tiered_slots, which reuses the previous view on the GPU and reads
    only the misses from the slots.  The repository holds the L_pack packed
    layers: repo.L == L_pack, repo.n_blocks == n_tok / 32."""

    def __init__(self, *args, repo, **kw):
        super().__init__(*args, **kw)
        if repo.L != self.L_pack or repo.H != self.H or repo.D != self.D or \
                repo.n_blocks * BLOCK_TOKENS != self.n_tok:
            raise ValueError("the repository must hold the packed layers of this history")
        self.repo = repo
        # the slot table stays on the GPU; each step applies only its changes
        self.host_slot = torch.from_numpy(repo.slot_table().copy()).to(self.device)
        self.tok_off_host = self.tok_off.cpu().numpy()
        self.prev_host = None
        self.last_plan = (0, 0)  # (blocks used, blocks missed) of the last step

    def pack_repo(self):
        cur, prev = self.cur, 1 - self.cur
        first = self.steps == 0
        Lp = self.L_pack
        kept = self.kept_sets[cur][:Lp].cpu().numpy().reshape(-1)
        cnt = self.count_sets[cur][:Lp].cpu().numpy().reshape(-1)
        kp, cp = (None, None) if first else self.prev_host
        used, need = kvc_repo_plan(kept, cnt, kp, cp, Lp, self.H, self.n_sess, self.budget,
                                   self.tok_off_host, self.repo.n_blocks)
        self.repo.step(used, need, table=False)
        units, slots = self.repo.changes()
        if len(units):
            self.host_slot[torch.from_numpy(units).to(self.device)] = \
                torch.from_numpy(slots).to(self.device)
        ks, vs = self.repo.slots()
        kvc_pack_tiered_slots(ks, vs, self.repo.slot_elems, self.repo.n_slots, self.host_slot,
                              None if first else self.kept_sets[prev][:Lp],
                              None if first else self.count_sets[prev][:Lp],
                              None if first else self.kcaches[prev],
                              None if first else self.vviews[prev],
                              self.kept_sets[cur][:Lp], self.count_sets[cur][:Lp], Lp, self.H,
                              self.D, self.tok_off, self.n_sess, self.n_tok, self.budget,
                              self.rope_tab, self.kcaches[cur], self.kview, self.vviews[cur],
                              self.n_hits, self.dev_status)
        self.prev_host = (kept, cnt)
        self.last_plan = (len(used), len(need))

    def step(self, q, meank_host):
        """One agent step; afterwards kview / vview hold this step's view."""
        cur = self.cur
        self.kept, self.kept_count = self.kept_sets[cur], self.count_sets[cur]
        self.vview = self.vviews[cur]
        self.score_tiered(q, meank_host)
        self.select()
        self.pack_repo()
        self.cur, self.steps = 1 - cur, self.steps + 1


def event_bytes(L: int, H: int, Hq: int, D: int, W: int, nb_total: int, n_sess: int,
                L_pack: int, view_tokens: int, budget: int) -> dict:
    """Bytes a Mean-K event must move through HBM, by stage: the Mean-K index
    and the query windows read once (score); the kept K and V rows read once
    and the execution views written once, plus the kept indices (pack).
    Select reads only the scores, which the score stage has just written."""
    meank = L * H * nb_total * D * 2
    q = n_sess * L * Hq * W * D * 2
    view = L_pack * H * n_sess * view_tokens * D
    pack = 2 * 2 * view * 2 + L * H * n_sess * budget * 4
    return {"score": meank + q, "select": 0, "pack": pack, "event": meank + q + pack}


class SlotMapEvent:
    """Buffers and calls of a QueryMemory-mode event: rule score over the
    paged K pool, token-level select (no forced set), redirect + free."""

    def __init__(self, n_sess: int, N: int, L: int, H: int, Hq: int, D: int,
                 n_slots: int, budget: int, prefix_len: int, sentinel: int = 0,
                 freed_cap: Optional[int] = None, device="cuda"):
        self.n_sess, self.N, self.L, self.H, self.Hq, self.D = n_sess, N, L, H, Hq, D
        self.n_slots, self.budget = n_slots, budget
        self.prefix_len, self.sentinel = prefix_len, sentinel
        dev = self.device = torch.device(device)
        self.rule = torch.empty(n_sess, N, dtype=torch.float32, device=dev)
        self.seg_off = _dev_i64(np.arange(n_sess + 1) * N, dev)
        self.kept = torch.empty(n_sess, budget, dtype=torch.int32, device=dev)
        self.kept_count = torch.empty(n_sess, dtype=torch.int32, device=dev)
        self.words = (N + 31) // 32
        self.keepmask = torch.empty(n_sess, self.words, dtype=torch.int32, device=dev)
        self.ws_score = _ws(kvc_score_qmem_workspace_size(n_sess, L, Hq, N), dev)
        self.ws_free = _ws(kvc_redirect_free_workspace_size(n_sess, N, n_slots), dev)
        self.freed_cap = n_slots if freed_cap is None else freed_cap
        self.freed = torch.empty(max(self.freed_cap, 1), dtype=torch.int32, device=dev)
        self.n_freed = torch.zeros(1, dtype=torch.int32, device=dev)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=dev)

    def score(self, M, kpool, slot_map, stream=None, kernel="auto"):
        kvc_score_qmem_ex(M, kpool, slot_map, self.sentinel, self.rule, self.n_sess,
                          self.L, self.H, self.Hq, self.D, self.N, self.n_slots,
                          self.ws_score, kernel, self.dev_status, stream)

    def select(self, rule=None, stream=None):
        kvc_select(self.rule if rule is None else rule, self.seg_off, self.n_sess,
                   self.N, self.budget, 0, 0, self.kept, self.kept_count,
                   self.keepmask, self.dev_status, stream)

    def redirect(self, slot_map, refcnt, keepmask=None, stream=None):
        kvc_redirect_free(slot_map, self.keepmask if keepmask is None else keepmask,
                          self.n_sess, self.N, refcnt, self.n_slots, self.prefix_len,
                          self.sentinel, self.freed, self.freed_cap, self.n_freed,
                          self.ws_free, self.dev_status, stream)

    def run(self, M, kpool, slot_map, refcnt, stream=None):
        self.score(M, kpool, slot_map, stream)
        self.select(stream=stream)
        self.redirect(slot_map, refcnt, stream=stream)


class PagedEvent:
    """Buffers and calls of an ActKV compression operation on a paged KV
    cache (ActKV §3.3 on the §2 layout): LSE-recovery score of the current
    action token (§7.1), the LRFU keep score at the end of the action region
    (§5.2), token-level select of `keep` tokens per request by keep score (no
    forced set), conflict-free tail plan and one-shot in-place compaction
    (§7.2).  All requests have max_blocks·block_size positions; select takes
    each request's whole row as its segment."""

    def __init__(self, n_req: int, max_blocks: int, block_size: int, L: int, H: int,
                 Hq: int, D: int, n_slots: int, keep: int, device="cuda"):
        self.n_req, self.max_blocks, self.BS = n_req, max_blocks, block_size
        self.L, self.H, self.Hq, self.D = L, H, Hq, D
        self.n_slots, self.keep = n_slots, keep
        self.cap = max_blocks * block_size
        dev = self.device = torch.device(device)
        self.state = torch.zeros(n_req, self.cap, dtype=torch.float32, device=dev)
        self.keep_score = torch.zeros(n_req, self.cap, dtype=torch.float32, device=dev)
        wsb = kvc_recover_score_workspace_size(n_req, max_blocks, L, H, Hq, D, block_size)
        self.ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
        self.seg_off = _dev_i64(np.arange(n_req + 1) * self.cap, dev)
        self.kept = torch.empty(n_req, keep, dtype=torch.int32, device=dev)
        self.kept_count = torch.empty(n_req, dtype=torch.int32, device=dev)
        self.words = (self.cap + 31) // 32
        self.keepmask = torch.empty(n_req, self.words, dtype=torch.int32, device=dev)
        i32 = dict(dtype=torch.int32, device=dev)
        self.src = torch.empty(n_req, self.cap, **i32)
        self.dst = torch.empty(n_req, self.cap, **i32)
        self.n_pairs = torch.empty(n_req, **i32)
        self.n_tail = torch.empty(n_req, **i32)
        self.freed = torch.empty(n_req, max_blocks, **i32)
        self.n_freed = torch.empty(n_req, **i32)
        self.new_table = torch.empty(n_req, max_blocks, **i32)
        self.tail_mask = torch.empty(n_req, self.words, **i32)
        self.dev_status = torch.zeros(1, **i32)

    def score(self, q, lse, kpool, block_table, seqused, count, stream=None, kernel="auto"):
        kvc_recover_score_ex(q, lse, kpool, self.n_slots, block_table, self.max_blocks,
                             seqused, count, self.n_req, self.L, self.H, self.Hq, self.D,
                             self.BS, self.state, self.ws, kernel, self.dev_status, stream)

    def lrfu(self, top_p: float = 0.9, lam: float = 0.5, stream=None):
        kvc_lrfu_update(self.state, self.seg_off, self.n_req, self.cap, top_p, lam,
                        self.keep_score, None, self.dev_status, stream)

    def select(self, stream=None, source=None):
        kvc_select(self.state if source is None else source, self.seg_off, self.n_req,
                   self.cap, self.keep, 0, 0, self.kept, self.kept_count, self.keepmask,
                   self.dev_status, stream)

    def plan(self, seqused, block_table, stream=None):
        kvc_tail_plan(self.keepmask, self.words, seqused, block_table, self.max_blocks,
                      self.n_req, self.BS, self.n_slots, self.src, self.dst, self.n_pairs,
                      self.n_tail, self.freed, self.n_freed, self.new_table, self.tail_mask,
                      self.dev_status, stream)

    def compact(self, kpool, vpool, stream=None):
        kvc_tail_compact(kpool, vpool, self.n_slots, self.L, self.H, self.D, self.src,
                         self.dst, self.n_pairs, self.cap, self.n_req, self.dev_status, stream)

    def run(self, q, lse, kpool, vpool, block_table, seqused, count, stream=None, lrfu=True):
        self.score(q, lse, kpool, block_table, seqused, count, stream)
        if lrfu:
            self.lrfu(stream=stream)
        self.select(stream, self.keep_score if lrfu else None)
        self.plan(seqused, block_table, stream)
        self.compact(kpool, vpool, stream)


class TreeDecodeEvent:
    """Buffers and calls of a decoding step with drafted trees on a paged KV
    cache that is held to `budget` rows per (layer, KV head).

    A step: the model writes the nodes' keys and values at the positions after
    each request's cache and calls ``attend`` per layer; once the accepted path
    is known, ``finish`` commits its rows (kvc_tree_commit), adds their attention
    weights to ``mass`` (kvc_attn_mass), evicts what exceeds the budget by it
    (kvc_mass_evict) and carries the lengths over to the next step.  Per request,
    on the device: ``ctx`` rows held, ``t_end`` tokens seen; ``mass`` and ``pos``
    (weight and original position per row) are updated in place.  With max_tree 1
    it is plain decoding.  ``start`` begins with a prefilled cache and ``observe``
    adds the weights of its last queries (a window, or the whole prompt), so that
    the first eviction has something to go by.

    The launches depend on the constructor's sizes only, so a step can be captured
    in a CUDA graph.  ``stream`` is None (the current stream), a Stream or a raw
    handle, as in the library's calls; the buffers belong to the stream they are
    first used on."""

    def __init__(self, n_req: int, max_blocks: int, block_size: int, L: int, H: int, Hq: int,
                 D: int, n_slots: int, n_q: int, max_tree: int, budget: int, n_sink: int = 0,
                 n_recent: int = 0, max_path: Optional[int] = None, max_observe: int = 0,
                 decay: float = 1.0, scale: Optional[float] = None, device="cuda"):
        self.n_req, self.max_blocks, self.BS = n_req, max_blocks, block_size
        self.L, self.H, self.Hq, self.D = L, H, Hq, D
        self.n_slots, self.n_q, self.max_tree = n_slots, n_q, max_tree
        self.max_path = max_tree if max_path is None else max_path
        self.budget, self.n_sink, self.n_recent = budget, n_sink, n_recent
        self.max_observe, self.decay = max_observe, decay
        self.scale = D ** -0.5 if scale is None else scale
        dev = self.device = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        cap = max_blocks * block_size
        self.out = torch.empty(L, n_q, Hq, D, dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty(L, n_q, Hq, dtype=torch.float32, device=dev)
        self.mass = torch.zeros(L, n_req, H, cap, dtype=torch.float32, device=dev)
        self.pos = torch.zeros(L, n_req, H, cap, **i32)
        self.ctx = torch.zeros(n_req, **i32)
        self.t_end = torch.zeros(n_req, **i32)
        self.n_mass = torch.zeros(n_req, **i32)
        self.n_pos = torch.zeros(n_req, **i32)
        self.seq = torch.zeros(n_req, **i32)
        self.n_out = torch.zeros(n_req, **i32)
        self.row_idx = torch.zeros(n_req, self.max_path, **i32)
        self.row_vis = torch.zeros(n_req, self.max_path, **i32)
        self.row_off = torch.arange(n_req + 1, **i32) * self.max_path
        rows = max(self.max_path, max_observe)
        self.ws = _ws(max(
            kvc_tree_attn_workspace_size(n_req, max_blocks, max_tree, H, Hq, D, block_size),
            kvc_attn_mass_workspace_size(n_req, max_blocks, rows, L, H, Hq, D, block_size),
            kvc_mass_evict_workspace_size(n_req, max_blocks, L, H, block_size, budget)), dev)
        self.dev_status = torch.zeros(1, **i32)

    def start(self, ctx):
        """A cache of ctx[r] rows per request, the first tokens of its request."""
        self.ctx.copy_(ctx)
        self.t_end.copy_(ctx)
        self.n_mass.zero_()
        self.n_pos.zero_()

    def observe(self, q, lse, row_vis, row_off, kpool, block_table, stream=None):
        """Adds the weights of queries q [L][n][Hq][D] with the given LSE (requests
        one after another, row_off) to the cached rows they see."""
        n = q.shape[1]
        kvc_attn_mass(q, lse, n, None, row_vis, row_off, n, self.max_observe, kpool,
                      self.n_slots, block_table, self.max_blocks, self.ctx, self.n_mass,
                      self.n_req, self.L, self.H, self.Hq, self.D, self.BS, self.scale,
                      self.decay, self.mass, self.ws, self.dev_status, stream)
        with _on(stream, self.device):
            self.n_mass.copy_(self.ctx)

    def attend(self, layer, q, kpool, vpool, block_table, q_off, tree_mask=None, stream=None):
        """One layer's attention: q [n_q][Hq][D], the layer's pools; out[layer] and
        lse[layer] are written.  tree_mask None: chains."""
        words = 0 if tree_mask is None else tree_mask.shape[1]
        kvc_tree_attn(q, kpool, vpool, self.n_slots, block_table, self.max_blocks, self.ctx,
                      q_off, tree_mask, words, self.n_req, self.n_q, self.max_tree, self.H,
                      self.Hq, self.D, self.BS, self.scale, self.out[layer], self.lse[layer],
                      self.ws, self.dev_status, stream)
        return self.out[layer]

    def commit(self, kpool, vpool, block_table, q_off, path, n_path, stream=None):
        kvc_tree_commit(kpool, vpool, self.n_slots, block_table, self.max_blocks, self.ctx,
                        q_off, path, n_path, self.max_path, self.n_req, self.L, self.H, self.D,
                        self.BS, self.seq, self.row_idx, self.row_vis, self.dev_status, stream)

    def accumulate(self, q, kpool, block_table, stream=None):
        """Weights of the committed rows; q [L][n_q][Hq][D] are the step's queries."""
        kvc_attn_mass(q, self.lse, self.n_q, self.row_idx, self.row_vis, self.row_off,
                      self.n_req * self.max_path, self.max_path, kpool, self.n_slots,
                      block_table, self.max_blocks, self.seq, self.n_mass, self.n_req, self.L,
                      self.H, self.Hq, self.D, self.BS, self.scale, self.decay, self.mass,
                      self.ws, self.dev_status, stream)

    def evict(self, kpool, vpool, block_table, stream=None):
        kvc_mass_evict(kpool, vpool, self.n_slots, block_table, self.max_blocks, self.seq,
                       self.n_pos, self.t_end, self.mass, self.pos, self.mass, self.pos,
                       self.n_out, self.n_req, self.L, self.H, self.D, self.BS, self.budget,
                       self.n_sink, self.n_recent, self.ws, self.dev_status, stream)

    def finish(self, q, kpool, vpool, block_table, q_off, path, n_path, stream=None):
        """The step after the last layer, on the path accepted from its outputs."""
        self.commit(kpool, vpool, block_table, q_off, path, n_path, stream)
        self.accumulate(q, kpool, block_table, stream)
        with _on(stream, self.device):
            self.t_end.add_(self.seq).sub_(self.ctx)
        self.evict(kpool, vpool, block_table, stream)
        with _on(stream, self.device):
            for n in (self.ctx, self.n_mass, self.n_pos):
                n.copy_(self.n_out)


class HistoryEvent:
    """Buffers and calls of prompts and decoding on a paged KV cache whose older blocks
    are held in 8 bits.

    A step, of prompts or of few rows per request: per layer ``write`` (the new tokens'
    queries and keys are normed and rotated, keys and values stored behind the cache;
    kvc_qkv_rope), then ``prompt`` (kvc_prompt_attn: many rows, requests without a history)
    or ``attend`` (kvc_q8_attn: few rows, or a drafted tree, over history and cache);
    after the last layer ``finish``, which takes the rows into the cache and moves every
    full block that is older than the last `recent` rows to 8 bits (kvc_q8_pack).

    Per request, on the device: ``ctx`` rows in bf16, ``len8`` positions in 8 bits,
    ``t_end`` tokens seen (the rotation goes by it).  The caller owns the pools, the
    8-bit pools (``k8``, ``v8`` [L][n_blocks8][H][block_size][D] uint8, ``kscale``,
    ``vscale`` [L][n_blocks8][H] fp32), ``block_table`` and ``table8``; a request's pages
    are its own.  ``finish`` turns its row of block_table so that the pages of packed
    blocks come last and are written again, and uses table8's entries in order.  One
    step moves at most `max_move` blocks of a request (the rest follow in later steps);
    `max_blocks` has room for the recent rows, a block, and what one step adds beyond
    what it moves.

    The constructor's n_q and max_rows are the largest step's; ``begin`` takes those of the
    step at hand, which its launches are planned by (one event serves long prompts and
    single tokens).  The launches depend on these host sizes only, so a step can be captured
    in a CUDA graph.  ``stream`` is None (the current stream), a Stream or a raw handle, as
    in the library's calls; the buffers belong to the stream they are first used on."""

    def __init__(self, n_req: int, max_blocks: int, max_blocks8: int, block_size: int, L: int,
                 H: int, Hq: int, D: int, n_slots: int, n_blocks8: int, n_q: int, max_rows: int,
                 n_pos: int, recent: int = 0, max_move: Optional[int] = None,
                 theta: float = 1e6, eps: float = 1e-6, scale: Optional[float] = None,
                 device="cuda"):
        self.n_req, self.max_blocks, self.max_blocks8, self.BS = n_req, max_blocks, max_blocks8, block_size
        self.L, self.H, self.Hq, self.D = L, H, Hq, D
        self.n_slots, self.n_blocks8, self.n_q, self.max_rows = n_slots, n_blocks8, n_q, max_rows
        if recent < 0 or (max_move is not None and max_move < 1):
            raise ValueError(f"HistoryEvent: recent {recent}, max_move {max_move}")
        self.n_pos, self.recent, self.eps = n_pos, recent, eps
        self.max_move = max_blocks if max_move is None else min(max_move, max_blocks)
        self.scale = D ** -0.5 if scale is None else scale
        dev = self.device = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.q = torch.empty(L, n_q, Hq, D, dtype=torch.bfloat16, device=dev)
        self.out = torch.empty(L, n_q, Hq, D, dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty(L, n_q, Hq, dtype=torch.float32, device=dev)
        self.ctx = torch.zeros(n_req, **i32)
        self.len8 = torch.zeros(n_req, **i32)
        self.t_end = torch.zeros(n_req, **i32)
        self.src = torch.empty(n_req, self.max_move, **i32)
        self.dst = torch.empty(n_req, self.max_move, **i32)
        self._page = torch.arange(max_blocks, dtype=torch.int64, device=dev)
        self.rope = torch.empty(n_pos, D // 2, 2, dtype=torch.float32, device=dev)
        with torch.cuda.device(dev):
            kvc_rope_table(self.rope, n_pos, 0, D, theta)
        self.pos = torch.empty(n_q, **i32)
        # (steps of fewer rows need no more)
        self.ws = _ws(kvc_q8_attn_workspace_size(n_req, max_blocks8, max_blocks,
                                                 min(max_rows, TREE_MAX_NODES), H, Hq, D, block_size), dev)
        self.dev_status = torch.zeros(1, **i32)
        self.step_q, self.step_rows = n_q, max_rows
        # ctx as prompt takes it: −1, which no call accepts, where new rows have a history before them
        self._prompt_ctx = torch.zeros(n_req, **i32)
        self._refused = torch.full((n_req,), -1, **i32)

    def begin(self, q_off, pos=None, stream=None, n_q: Optional[int] = None,
              max_rows: Optional[int] = None):
        """A step whose requests' new tokens are q_off's: at the positions that follow t_end,
        or pos [n_q] behind it (a drafted tree's depths: 0 for the next position).  n_q: the
        rows of the step's buffers, max_rows: the most that a request brings (None: the
        constructor's); a request that brings more is recorded as KVC_ERR_BOUNDS and gets no
        attention."""
        n = self.n_q if n_q is None else n_q
        most = min(self.max_rows, n) if max_rows is None else max_rows
        if not (1 <= n <= self.n_q and 1 <= most <= self.max_rows):
            raise ValueError(f"HistoryEvent.begin: a step of {n} rows, {most} of a request, in an event made "
                             f"for {self.n_q} and {self.max_rows}")
        self.q_off, self.step_q, self.step_rows = q_off, n, most
        with _on(stream, self.device):
            x = torch.arange(n, dtype=torch.int32, device=self.device)
            r = torch.bucketize(x, q_off[1:], right=True, out_int32=True).clamp_(max=self.n_req - 1)
            self.pos[:n].copy_(x - q_off[r] if pos is None else pos)
            self.pos[:n].add_(self.t_end[r])
            held = (self.len8 > 0) & (q_off[1:] > q_off[:-1])
            torch.where(held, self._refused, self.ctx, out=self._prompt_ctx)

    def write(self, layer, q, k, v, kpool, vpool, block_table, wq=None, wk=None, k_raw=None,
              stream=None):
        """One layer's projections q, k, v ([the step's n_q][heads·D], any row stride); the
        layer's pools.  The rotated queries are in self.q[layer]."""
        kvc_qkv_rope(q, k, v, self.step_q, wq, wk, self.eps, self.rope, self.n_pos, self.pos,
                     self.q_off, self.ctx, self.n_req, block_table, self.max_blocks, kpool, vpool,
                     self.n_slots, self.H, self.Hq, self.D, self.BS, self.q[layer], k_raw,
                     self.dev_status, stream)

    def prompt(self, layer, kpool, vpool, block_table, stream=None):
        """Causal attention of the new rows over cache and new rows, of requests that hold
        nothing in 8 bits.  A request with new rows behind a history is recorded as
        KVC_ERR_BOUNDS and its rows are left alone (attend takes it)."""
        kvc_prompt_attn(self.q[layer], kpool, vpool, self.n_slots, block_table, self.max_blocks,
                        self._prompt_ctx, self.q_off, self.n_req, self.step_q, self.step_rows, self.H,
                        self.Hq, self.D, self.BS, self.scale, self.out[layer], self.lse[layer],
                        self.dev_status, stream)
        return self.out[layer, :self.step_q]

    def attend(self, layer, kpool, vpool, block_table, k8, v8, kscale, vscale, table8,
               tree_mask=None, stream=None):
        """Attention of the new rows (at most 1024 of a request) over history, cache and new
        rows; tree_mask None: chains."""
        words = 0 if tree_mask is None else tree_mask.shape[1]
        kvc_q8_attn(self.q[layer], k8, v8, kscale, vscale, self.n_blocks8, table8,
                    self.max_blocks8, self.len8, kpool, vpool, self.n_slots, block_table,
                    self.max_blocks, self.ctx, self.q_off, tree_mask, words, self.n_req,
                    self.step_q, min(self.step_rows, TREE_MAX_NODES), self.H, self.Hq, self.D,
                    self.BS, self.scale, self.out[layer], self.lse[layer], self.ws,
                    self.dev_status, stream)
        return self.out[layer, :self.step_q]

    def finish(self, kpool, vpool, block_table, k8, v8, kscale, vscale, table8, n_rows=None,
               stream=None):
        """The step after the last layer: the first n_rows [n_req] of a request's new rows (None:
        all) join the cache, full blocks move to 8 bits, all layers.  The accepted nodes of
        a drafted tree are brought to the front before (kvc_tree_commit, ctx_len = ctx)."""
        BS = self.BS
        with _on(stream, self.device):
            n = self.q_off[1:] - self.q_off[:-1] if n_rows is None else n_rows
            self.ctx.add_(n)
            self.t_end.add_(n)
            room = self.max_blocks8 - self.len8 // BS
            move = ((self.ctx - self.recent).clamp(min=0) // BS).clamp(max=self.max_move)
            move = torch.minimum(move, room)
            i = self._page[:self.max_move]
            some = i < move[:, None]
            at = ((self.len8 // BS)[:, None] + i).clamp(max=self.max_blocks8 - 1)
            self.src.copy_(torch.where(some, block_table[:, :self.max_move], -1))
            self.dst.copy_(torch.where(some, table8.gather(1, at), -1))
        kvc_q8_pack(kpool, vpool, self.n_slots, k8, v8, kscale, vscale, self.n_blocks8, self.src,
                    self.dst, self.n_req * self.max_move, self.L, self.H, self.D, BS,
                    self.dev_status, stream)
        with _on(stream, self.device):
            block_table.copy_(block_table.gather(1, (self._page + move[:, None]) % self.max_blocks))
            self.ctx.sub_(move * BS)
            self.len8.add_(move * BS)


def paged_bytes(n_req: int, seq: int, L: int, H: int, Hq: int, D: int, n_pairs: int) -> dict:
    """Bytes an ActKV operation must move through HBM, by stage: every
    visible key row read once, the query token, LSE and the state read and
    written (score); the state read and the keep score read and written
    (lrfu); the keep scores read (select); the keep mask and block table
    (plan); K and V rows of every planned pair read and written once per
    layer (compact)."""
    score = n_req * seq * L * H * D * 2 + n_req * L * Hq * (D * 2 + 4) + n_req * seq * 8
    lrfu = n_req * seq * 12
    select = n_req * seq * 4
    plan = n_req * (seq // 8 + seq // 4)
    compact = n_pairs * L * 2 * H * D * 2 * 2
    return {"score": score, "lrfu": lrfu, "select": select, "plan": plan, "compact": compact,
            "event": score + lrfu + select + plan + compact}
