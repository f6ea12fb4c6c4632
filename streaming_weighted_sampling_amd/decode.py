"""Decoding over an 8-bit cache between eviction events: one layer, several sequences.

[Nexus] ("Forget Without Compromise: Nexus Sampling for Streaming KV-Cache
Eviction Under Fixed Budgets", section 2.1) decodes over the kept rows and evicts
again whenever the budget is hit.  This driver holds the kept rows in the paged
8-bit cache: step() norms and rotates one new token per sequence, appends it and
attends; evict() reads the cache back, runs one nx_evict_batch event over all
sequences with the last W queries as the window, and refills the cache with the
kept rows.  Nothing synchronises: row counts, also the heads' different ones under
per-head budgets, stay on the device (but for an event at full capacity whose head_cap
is the capacity too: the next steps then need the counts).  Marshalling only; every byte of a step
moves inside libnexus.so.
"""

import ctypes
import functools
import weakref
from dataclasses import replace

import torch

from ._lib import NX_CACHE_BLOCK, NX_HEADS_ALLOC, NX_HEADS_GIVEN, NX_HEADS_UNIFORM, NexusError, NxUnit
from .api import NexusConfig, make_units, new_workspace, nx_evict_batch, nx_read_device_status
from .paged import (new_paged_cache, new_paged_workspace, nx_paged_append, nx_paged_attn, nx_paged_gather,
                    nx_qk_norm_rope)


def _not_captured(what):
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"DecodeCache.{what} cannot be captured into a graph: the row bound, the query ring's place "
                           "and the event number are the host's, a replay would not move them")


def _on_own_device(method):
    """The eviction calls work on the current GPU's current stream: make the cache's GPU the current one."""
    @functools.wraps(method)
    def call(self):
        with torch.cuda.device(self.device):
            return method(self)
    return call


class EventBuffers:
    """What an event uses only while it runs: the rows read back from the cache, the kept ones as
    [heads][seqs * cap_rows][D], and the event's workspace.  DecodeCaches of one configuration and size
    (the layers of a model) can share one, as long as their events are ordered on one stream."""

    def __init__(self, cfg, n_seqs, capacity, cap_rows, walk_iters, device):
        hk, d = cfg.n_kv_heads, cfg.head_dim
        self.shape = replace(cfg), n_seqs, capacity, cap_rows, walk_iters, device
        self.k = torch.zeros(n_seqs, hk, capacity, d, dtype=cfg.dtype, device=device)
        self.v = torch.zeros_like(self.k)
        self.kept_k = torch.zeros(hk, n_seqs * cap_rows, d, dtype=cfg.dtype, device=device)
        self.kept_v = torch.zeros_like(self.kept_k)
        self.ws = new_workspace(cfg, capacity, n_seqs, walk_iters, device=device)
        self.users = weakref.WeakSet()      # whose events report in this workspace


class DecodeCache:
    """`n_seqs` sequences of one layer, up to `capacity` rows per head.

    rope: Rope or None; q_weight / k_weight: [head_dim] norm weights or None.
    head_budget: with head_alloc = NX_HEADS_GIVEN the units that each head keeps, [n_seqs, n_kv_heads]
    or what expands to it, at most head_cap (0: budget); the attribute, int32 on the device, may be
    rewritten in place between events.
    Keys are rotated (and normed) once, when they arrive; evicted positions
    leave holes that nothing refers to again, so a kept row is stored as it was.
    event_buffers: another DecodeCache's, to share them (by default each has its own, which are larger than
    an unquantised cache would be).
    seed, layer and (with per-head budgets) budget may be changed between events; what sizes the buffers
    is fixed.  load, step and evict run eagerly (RuntimeError in a graph's capture; the nx_* calls they make can
    be captured).  Evicting re-quantises the kept rows in their new blocks.  With cfg.block > 1 an
    event needs a row count that is a multiple of the block.
    """

    def __init__(self, cfg: NexusConfig, n_seqs, capacity, budget, walk_iters, *, fmt="e4m3", page_blocks=4,
                 rope=None, q_weight=None, k_weight=None, eps=1e-6, seed=0, layer=0, head_cap=0, head_budget=None,
                 event_buffers=None, device="cuda"):
        if cfg.compact:
            raise ValueError("the kept rows are copied into new blocks: compact must be 0")
        if (cfg.head_alloc == NX_HEADS_GIVEN) != (head_budget is not None):
            raise ValueError("head_budget goes with head_alloc = NX_HEADS_GIVEN")
        self.cfg, self.n_seqs, self.capacity = cfg, n_seqs, capacity
        self.budget, self.walk_iters, self.seed, self.layer = budget, walk_iters, seed, layer
        self.rope, self.q_weight, self.k_weight, self.eps = rope, q_weight, k_weight, eps
        hk, d, page = cfg.n_kv_heads, cfg.head_dim, page_blocks * NX_CACHE_BLOCK
        pages = -(-capacity // page)
        self.cache = new_paged_cache(cfg, n_seqs, n_seqs * hk * pages, pages, fmt=fmt, page_blocks=page_blocks,
                                     device=device)
        self.device = self.cache.device
        self.cache.table.copy_(torch.arange(n_seqs * hk * pages, dtype=torch.int32).view(n_seqs, hk, pages))
        self.ws = new_paged_workspace(cfg, self.cache, capacity)
        self.out = torch.empty(n_seqs, cfg.n_q_heads, d, dtype=cfg.dtype, device=self.device)
        # The last W rotated queries of every sequence, a ring over dimension 2; one place more, so that
        # a step that is refused half-way has not overwritten the oldest of them.
        self.ring = torch.zeros(n_seqs, cfg.n_q_heads, cfg.window + 1, d, dtype=cfg.dtype, device=self.device)
        self._places = [self.ring[:, :, i] for i in range(cfg.window + 1)]
        self.queries = 0      # queries seen since load()
        self.rows = 0         # the host's bound on the heads' row counts
        self.step_no = 0      # eviction events
        cap = head_cap if head_cap and cfg.head_alloc != NX_HEADS_UNIFORM else budget
        self.cap_rows = min(cap * cfg.block, capacity)
        if event_buffers is None:
            event_buffers = EventBuffers(cfg, n_seqs, capacity, self.cap_rows, walk_iters, self.device)
        elif event_buffers.shape != (cfg, n_seqs, capacity, self.cap_rows, walk_iters, self.device):
            raise ValueError("event_buffers were made for a cache of another configuration or size")
        self._bufs = event_buffers
        event_buffers.users.add(self)
        self.k, self.v, self.evict_ws = event_buffers.k, event_buffers.v, event_buffers.ws
        self.kept_k, self.kept_v = event_buffers.kept_k, event_buffers.kept_v
        self.keep = torch.zeros(n_seqs, hk, cap, dtype=torch.int32, device=self.device)
        self.head_budget = torch.zeros(n_seqs, hk, dtype=torch.int32, device=self.device)
        if head_budget is not None:
            given = torch.as_tensor(head_budget).expand(n_seqs, hk)
            if given.is_floating_point() or int(given.min()) < max(1, cfg.n_sink + cfg.n_recent) or \
                    int(given.max()) > cap:
                raise ValueError(f"head_budget: whole numbers from {max(1, cfg.n_sink + cfg.n_recent)} (the forced "
                                 f"units) to {cap} expected")
            self.head_budget.copy_(given)
        self.counts = torch.zeros(n_seqs, hk, dtype=torch.int32, device=self.device)
        self.window = torch.zeros(n_seqs, cfg.n_q_heads, cfg.window, d, dtype=cfg.dtype, device=self.device)
        self.head_cap = cap
        self._units = torch.zeros(n_seqs * ctypes.sizeof(NxUnit), dtype=torch.uint8, device=self.device)
        self._units_of = None

    @property
    def event_buffers(self):
        return self._bufs

    def load(self, k, v):
        """Replaces the rows: k, v [n_seqs, n_kv_heads, rows, D], keys already rotated (a prompt's
        rows, or the out_k / out_v of a first event)."""
        n, hk, rows, d = k.shape
        if n != self.n_seqs or v.shape != k.shape or (hk, d) != (self.cfg.n_kv_heads, self.cfg.head_dim):
            raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)}: rows of {self.n_seqs} sequences with "
                             f"{self.cfg.n_kv_heads} heads of {self.cfg.head_dim} expected")
        for x, name in ((k, "k"), (v, "v")):
            if x.dtype != self.cfg.dtype:
                raise TypeError(f"{name}: dtype {x.dtype}, expected {self.cfg.dtype}")
            if x.device != self.device:
                raise ValueError(f"{name} is on {x.device}, the cache on {self.device}")
        if rows > self.capacity:
            raise ValueError(f"{rows} rows, capacity {self.capacity}")
        _not_captured("load")
        flat = [x.permute(0, 2, 1, 3).reshape(n * rows, hk, d) for x in (k, v)]
        self.cache.lens.zero_()
        if rows:
            nx_paged_append(self.cfg, self.cache, *flat, workspace=self.ws)
        self.rows, self.queries = rows, 0

    def step(self, q, k, v, positions=None):
        """One new token per sequence: q [n_seqs, n_q_heads, D], k, v [n_seqs, n_kv_heads, D] as
        projected, positions int32 [n_seqs] (with rope).  Returns out [n_seqs, n_q_heads, D], which the next
        step overwrites."""
        if self.rows + 1 > self.capacity:
            raise ValueError("the cache is full: evict first")
        if (self.rope is None) != (positions is None):
            raise ValueError("positions go with rope")
        _not_captured("step")
        cfg = self.cfg
        q_rot = self._places[self.queries % len(self._places)]
        normed = self.k_weight is not None
        _, k_new = nx_qk_norm_rope(cfg, q, k if normed else None, workspace=self.ws, q_weight=self.q_weight,
                                   k_weight=self.k_weight, eps=self.eps, rope=self.rope, positions=positions,
                                   out_q=q_rot)
        if normed:       # normed keys come rotated; others are rotated on their way into the cache
            nx_paged_append(cfg, self.cache, k_new, v, workspace=self.ws)
        else:
            nx_paged_append(cfg, self.cache, k, v, workspace=self.ws, rope=self.rope, positions=positions)
        self.queries += 1
        self.rows += 1
        return nx_paged_attn(cfg, self.cache, q_rot, workspace=self.ws, max_tokens=self.rows, out=self.out)

    @_on_own_device
    def evict(self):
        """One eviction event over all sequences, back to the budget.  A head that the device rejects
        (check() raises) keeps all its rows.  A budget of the whole capacity is refused once the cache is
        full: nothing could follow."""
        cfg, w, bufs = self.cfg, self.cfg.window, self.event_buffers
        if self.queries < w:
            raise ValueError(f"an event needs {w} queries, {self.queries} were seen")
        if self.rows % cfg.block:     # a short last block would be counted as a whole one
            raise ValueError(f"{self.rows} rows are not whole blocks of {cfg.block}")
        uniform = cfg.head_alloc == NX_HEADS_UNIFORM
        if (self.budget if uniform else self.head_cap) != self.keep.shape[2]:
            raise ValueError(f"the event's buffers hold {self.keep.shape[2]} units a head: another "
                             f"{'budget' if uniform else 'head_cap'} needs another DecodeCache")
        kept = min(cfg.kept_rows(self.rows, self.head_cap), self.cap_rows)
        if kept == self.capacity and uniform:
            raise ValueError(f"an event makes no room: its budget holds all {self.capacity} rows of the capacity")
        _not_captured("evict")
        first = (self.queries + 1) % (w + 1)     # the oldest query's place in the ring
        head = min(w, w + 1 - first)
        self.window[:, :, :head].copy_(self.ring[:, :, first:first + head])
        self.window[:, :, head:].copy_(self.ring[:, :, :w - head])
        nx_paged_gather(cfg, self.cache, workspace=self.ws, max_tokens=self.rows, out_k=bufs.k, out_v=bufs.v)
        now = self.rows, self.budget, self.layer
        if self._units_of != now:              # the event's records, rewritten in place
            d, r = cfg.head_dim, self.cap_rows
            self._units.copy_(make_units(
                [dict(q=self.window[s], k=bufs.k[s], v=bufs.v[s], keep=self.keep[s],
                      out_k=bufs.kept_k[0, s * r:], out_v=bufs.kept_v[0, s * r:],
                      kv_head_stride=self.capacity * d, out_head_stride=self.n_seqs * r * d,
                      n_tokens=self.rows, budget=self.budget, layer=self.layer, seq_id=s,
                      head_cap=self.head_cap, head_budget=self.head_budget[s],
                      head_tokens=self.cache.lens[s], head_tokens_out=self.counts[s])
                 for s in range(self.n_seqs)], device="cpu"))
            self._units_of = now
        # The event writes the count of every head that it serves; one that the device rejects keeps -1
        # here, and its rows as they were.
        self.counts.fill_(-1)
        if cfg.head_alloc == NX_HEADS_ALLOC:
            self.head_budget.fill_(-1)
        nx_evict_batch(cfg, self._units, self.n_seqs, self.rows, self.walk_iters, self.seed, workspace=bufs.ws,
                       step=self.step_no, max_out_rows=kept)
        if cfg.head_alloc == NX_HEADS_ALLOC and cfg.n_sink + cfg.n_recent == 0:
            # An allocation of no rows is not rejected (no row is forced): such a head keeps none.
            self.counts.masked_fill_((self.counts < 0) & (self.head_budget == 0) & (self.cache.lens <= self.rows), 0)
        self.cache.lens.masked_fill_(self.counts >= 0, 0)      # (the append leaves a head whose count is -1)
        nx_paged_append(cfg, self.cache, bufs.kept_k.permute(1, 0, 2), bufs.kept_v.permute(1, 0, 2),
                        workspace=self.ws, max_new=self.cap_rows, head_new=self.counts)
        # Where a head may keep as many rows as the cache holds, only the counts say how long the longest is.
        self.rows = kept if kept < self.capacity else max(0, int(self.cache.lens.max()))
        self.step_no += 1

    @_on_own_device
    def check(self):
        """Synchronises and raises NexusError on an error that a step or an event recorded (both are
        cleared; with shared event_buffers also an event of another cache).  The cache can be used on:
        what was rejected is as it was before."""
        errors = []
        for ws in (self.ws, self.event_buffers.ws):
            try:
                nx_read_device_status(self.cfg, ws)
            except NexusError as e:
                errors.append(e)
        if errors:
            for user in self.event_buffers.users:      # a rejected head may be longer than the bound
                user.rows = max(0, int(user.cache.lens.max()))
            raise errors[0]
