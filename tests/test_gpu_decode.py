"""DecodeCache: prompt rows, decode steps, eviction events and decoding on, every stage against the
oracle or the single calls it is made of."""

import numpy as np
import pytest
import torch

import streaming_weighted_sampling_amd as nx
from oracle import paged
from tests.test_gpu_paged import DT, Cache, _check_attn, _np, _randn

pytestmark = pytest.mark.gpu
DEV = "cuda"


class View(Cache):
    """The array readers of Cache on a DecodeCache's cache."""

    def __init__(self, d, dtype, fmt):
        self.cfg, self.c, self.d, self.hkv = d.cfg, d.cache, d.cfg.head_dim, d.cfg.n_kv_heads
        self.n_seqs, self.group = d.n_seqs, d.cfg.n_q_heads // d.cfg.n_kv_heads
        self.fmt, self.dtype, self.pb = fmt, dtype, d.cache.k_codes.shape[1]


@pytest.mark.parametrize("dtype,fmt,d,normed,alloc,block", [
    ("bf16", "e4m3", 128, True, 0, 1), ("bf16", "int8", 64, False, 0, 1), ("f32", "int8", 64, False, 2, 1),
    ("bf16", "e4m3", 64, True, 2, 1), ("bf16", "e4m3", 128, False, 0, 32)])
def test_decode_evict_decode(dtype, fmt, d, normed, alloc, block):
    S, hk, grp, W = 2, 2, 4, 8
    budget = 90 if block == 1 else 3
    cfg = nx.NexusConfig(hk * grp, hk, d, W, DT[dtype], head_alloc=alloc, head_floor=20 if alloc else 0, block=block)
    rope = nx.Rope(nx.rope_table(400, d // 2, device=DEV), pairs=True)
    wq = _randn(1, d, dtype=dtype) if normed else None
    wk = _randn(2, d, dtype=dtype) if normed else None
    dec = nx.DecodeCache(cfg, S, 256, budget, 3, fmt=fmt, page_blocks=2, rope=rope, q_weight=wq, k_weight=wk,
                         seed=7, layer=3, head_cap=150 if alloc else 0, device=DEV)
    view = View(dec, dtype, fmt)
    k0, v0 = _randn(3, S, hk, 140, d, dtype=dtype), _randn(4, S, hk, 140, d, dtype=dtype)
    with pytest.raises(ValueError, match="queries"):
        dec.evict()
    dec.load(k0, v0)
    ws = nx.new_workspace(cfg, 1, 1, 0, device=DEV)
    pos, seen = 140, []

    def steps(n):
        nonlocal pos
        for i in range(n):
            qkv = _randn(1000 + pos, S, (grp + 2) * hk, d, dtype=dtype)
            q, k, v = qkv.split((hk * grp, hk, hk), 1)
            p = torch.full((S,), pos, dtype=torch.int32, device=DEV)
            out = dec.step(q, k, v, p)
            want, _ = nx.nx_qk_norm_rope(cfg, q, workspace=ws, q_weight=wq, rope=rope, positions=p)
            seen.append(want)
            pos += 1
            if i % 7 == 0:
                _check_attn(view, want, [1] * S, out)
        dec.check()

    steps(20)
    if block == 1:
        steps(1)
    assert dec.cache.lens.flatten().tolist() == [160 + (block == 1)] * (S * hk)
    for event in range(2):
        lens = dec.cache.lens.cpu().numpy()
        gk, gv = nx.nx_paged_gather(cfg, dec.cache, workspace=dec.ws, max_tokens=dec.rows)
        dec.evict()
        dec.check()
        assert torch.equal(dec.window, torch.stack(seen[-W:], 2))
        counts = dec.counts.cpu().numpy()
        for s in range(S):
            for h in range(hk):
                keep = dec.keep[s, h].cpu().numpy()
                if block > 1:
                    keep = np.concatenate([np.arange(b * block, min((b + 1) * block, lens[s, h]))
                                           for b in keep[:-(-counts[s, h] // block)]])
                keep = keep[:counts[s, h]]
                ref = paged.Head(d, dtype, fmt)
                ref.append(_np(gk[s, h])[keep], _np(gv[s, h])[keep])
                assert int(dec.cache.lens[s, h]) == len(ref) == counts[s, h]
                for b, want in enumerate(ref.blocks):
                    for (codes, scale), (wc, wsc) in zip(view.block(s, h, b), want):
                        assert scale == wsc and np.array_equal(codes, wc), (s, h, b)
                for got, want in zip(view.tail(s, h, len(ref) % 32), ref.tail):
                    assert not want or np.array_equal(got, np.stack(want))
            if not alloc and event == 0:
                # the same event by nx_evict_step on the gathered rows
                n = int(lens[s, 0])
                ews = nx.new_workspace(cfg, n, 1, 3, device=DEV)
                keep, _, _ = nx.nx_evict_step(cfg, dec.window[s], gk[s, :, :n].contiguous(),
                                              gv[s, :, :n].contiguous(), n, budget, 3, 7, workspace=ews, layer=3,
                                              step=0, seq_id=s)
                assert torch.equal(keep, dec.keep[s])
        if alloc:
            assert counts.sum() == S * hk * budget and len(set(counts.flatten())) > 1
        steps(40)
        if block > 1:
            with pytest.raises(ValueError, match="whole blocks"):
                dec.evict()
            steps(24)


def test_decode_cache_refuses_what_it_cannot_hold():
    cfg = nx.NexusConfig(4, 2, 64, 4)
    with pytest.raises(ValueError, match="compact"):
        nx.DecodeCache(nx.NexusConfig(4, 2, 64, 4, compact=1), 1, 64, 32, 1, device=DEV)
    dec = nx.DecodeCache(cfg, 1, 64, 32, 1, page_blocks=1, device=DEV)
    with pytest.raises(ValueError, match="capacity"):
        dec.load(*[torch.zeros(1, 2, 65, 64, dtype=torch.bfloat16, device=DEV)] * 2)
    dec.load(*[torch.zeros(1, 2, 64, 64, dtype=torch.bfloat16, device=DEV)] * 2)
    q, k = _randn(1, 1, 4, 64, dtype="bf16"), _randn(2, 1, 2, 64, dtype="bf16")
    with pytest.raises(ValueError, match="full"):
        dec.step(q, k, k)
    dec.load(*[torch.zeros(1, 2, 0, 64, dtype=torch.bfloat16, device=DEV)] * 2)
    out = dec.step(q, k, k)              # the first row of an empty cache: attention is that row
    dec.check()
    assert torch.equal(out, k.repeat_interleave(2, 1))
    with pytest.raises(ValueError, match="sequences"):
        dec.load(*[torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16, device=DEV)] * 2)
    with pytest.raises(ValueError, match="positions"):
        dec.step(q, k, k, torch.zeros(1, dtype=torch.int32, device=DEV))
    turned = nx.DecodeCache(cfg, 1, 64, 32, 1, page_blocks=1, rope=nx.Rope(nx.rope_table(9, 64, device=DEV)),
                            device=DEV)
    with pytest.raises(ValueError, match="positions"):
        turned.step(q, k, k)


def _held(dec, s, h):
    """What the cache holds of one head: the rows it stands for and the unquantised ones."""
    k, v = nx.nx_paged_gather(dec.cfg, dec.cache, workspace=dec.ws, max_tokens=dec.capacity)
    n = int(dec.cache.lens[s, h])
    return n, k[s, h, :n].clone(), v[s, h, :n].clone()


def _fill(dec, rows, steps, seed=200):
    S, hk, hq, d = dec.n_seqs, dec.cfg.n_kv_heads, dec.cfg.n_q_heads, dec.cfg.head_dim
    dec.load(_randn(seed, S, hk, rows, d, dtype="bf16"), _randn(seed + 1, S, hk, rows, d, dtype="bf16"))
    for i in range(steps):
        qkv = _randn(seed + 2 + i, S, hq + 2 * hk, d, dtype="bf16")
        dec.step(*qkv.split((hq, hk, hk), 1))


@pytest.mark.parametrize("events", [0, 1])
def test_a_rejected_head_keeps_its_rows(events):
    """One head's resident count is out of range for the event (in the first event, and in one after
    which the buffers hold an earlier event's rows)."""
    cfg = nx.NexusConfig(4, 2, 64, 4)
    dec = nx.DecodeCache(cfg, 2, 256, 50, 2, page_blocks=2, device=DEV)
    _fill(dec, 90, 10)
    for _ in range(events):
        dec.evict()
        _fill(dec, 120, 7, seed=300)
    dec.check()
    n = dec.rows
    dec.rows -= 3                              # the host's bound is too low for every head ...
    dec.cache.lens[0].sub_(3)                  # ... but those of sequence 0, which now hold three fewer
    before = [_held(dec, s, h) for s in range(2) for h in range(2)]
    dec.evict()
    with pytest.raises(nx.NexusError) as e:
        dec.check()
    assert e.value.code == nx.NX_EINVAL
    assert dec.cache.lens.tolist() == [[50, 50], [n, n]] and dec.rows == n
    for h in range(2):
        got = _held(dec, 1, h)
        assert got[0] == n and all(torch.equal(a, b) for a, b in zip(got[1:], before[2 + h][1:]))
    dec.check()
    _fill_more = _randn(400, 2, 8, 64, dtype="bf16").split((4, 2, 2), 1)
    dec.step(*_fill_more)
    dec.evict()                                # with the bound put right the same heads are served
    dec.check()
    assert dec.cache.lens.tolist() == [[50, 50], [50, 50]]


def test_a_head_that_is_allocated_no_rows_is_empty():
    """Head 0 attends evenly over 100 rows, head 1 over 20 only, whose weights are then the 20 largest
    of both heads: two heads of budget 10 leave nothing for head 0."""
    cfg = nx.NexusConfig(2, 2, 64, 4, head_alloc=2, head_floor=0)
    dec = nx.DecodeCache(cfg, 1, 128, 10, 0, page_blocks=1, head_cap=40, device=DEV)
    k = torch.zeros(1, 2, 96, 64, dtype=torch.bfloat16, device=DEV)
    k[0, 1, :, 0] = -8.0
    k[0, 1, 5:25, 0] = 8.0
    v = _randn(1, 1, 2, 96, 64, dtype="bf16")
    dec.load(k, v)
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 8.0
    new = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    new[0, 1, 0] = -8.0
    for _ in range(4):
        dec.step(q, new, new)
    dec.evict()
    dec.check()
    assert dec.head_budget.tolist() == [[0, 20]] and dec.cache.lens.tolist() == [[0, 20]]
    assert dec.keep[0, 1, :20].tolist() == list(range(5, 25))
    out = dec.step(q, new, new)
    dec.check()
    assert torch.equal(out[0, 0], new[0, 0]) and dec.cache.lens.tolist() == [[1, 21]]


def test_given_head_budgets():
    cfg = nx.NexusConfig(4, 2, 64, 4, head_alloc=nx.NX_HEADS_GIVEN, n_sink=2)
    given = torch.tensor([[30, 61], [7, 2]])
    dec = nx.DecodeCache(cfg, 2, 256, 40, 2, page_blocks=2, head_cap=64, head_budget=given, device=DEV)
    for _ in range(2):
        _fill(dec, 100, 6)
        dec.evict()
        dec.check()
        assert dec.cache.lens.tolist() == given.tolist() and dec.rows == 64
        assert (dec.keep[:, :, :2] == torch.arange(2, device=DEV)).all()       # the forced units
    dec.head_budget[0, 1] = 0                  # a budget that the event refuses
    _fill(dec, 100, 6)
    dec.evict()
    with pytest.raises(nx.NexusError):
        dec.check()
    assert dec.cache.lens.tolist() == [[30, 106], [7, 2]] and dec.rows == 106
    even = nx.DecodeCache(cfg, 2, 256, 40, 2, head_budget=[9, 40], device=DEV)
    assert even.head_budget.tolist() == [[9, 40]] * 2


def test_events_under_a_head_cap_of_the_whole_capacity():
    """The loop "step until full, then evict" goes on: the bound on the rows follows the heads' counts."""
    cfg = nx.NexusConfig(4, 2, 64, 4, head_alloc=2, head_floor=8)
    dec = nx.DecodeCache(cfg, 2, 64, 24, 2, page_blocks=1, head_cap=64, device=DEV)
    _fill(dec, 50, 0)
    for event in range(3):
        while dec.rows < dec.capacity:
            dec.step(*_randn(500 + dec.rows, 2, 8, 64, dtype="bf16").split((4, 2, 2), 1))
        dec.evict()
        dec.check()
        lens = dec.cache.lens
        assert dec.rows == int(lens.max()) < 64 and (lens.sum(1) == 48).all()


def test_an_event_that_makes_no_room_is_refused():
    dec = nx.DecodeCache(nx.NexusConfig(4, 2, 64, 4), 1, 64, 64, 2, page_blocks=1, device=DEV)
    _fill(dec, 50, 10)
    before = _held(dec, 0, 1)
    dec.evict()                                # below the capacity: keeps every row, quantised anew
    dec.check()
    assert dec.rows == 60 and _held(dec, 0, 1)[0] == before[0] == 60
    _fill(dec, 60, 4)
    before = _held(dec, 0, 1)
    with pytest.raises(ValueError, match="room"):
        dec.evict()
    dec.check()
    assert dec.step_no == 1 and all(torch.equal(a, b) for a, b in zip(_held(dec, 0, 1)[1:], before[1:]))


def test_capture_of_the_driver_is_refused():
    """Its host counters would not move with the replays: the ring's place and the row bound go wrong."""
    dec = nx.DecodeCache(nx.NexusConfig(4, 2, 64, 4), 1, 64, 32, 2, page_blocks=1, device=DEV)
    _fill(dec, 40, 5)
    before = _held(dec, 0, 0)
    args = _randn(3, 1, 8, 64, dtype="bf16").split((4, 2, 2), 1)
    rows = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16, device=DEV)
    for call in (lambda: dec.step(*args), dec.evict, lambda: dec.load(rows, rows)):
        with pytest.raises(RuntimeError, match="captured"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                args[0] + 1                    # a graph of something
                call()
    torch.cuda.synchronize()
    assert (dec.rows, dec.queries, dec.step_no) == (45, 5, 0)
    assert all(torch.equal(a, b) for a, b in zip(_held(dec, 0, 0)[1:], before[1:]))
    dec.step(*args)
    dec.evict()
    dec.check()
    assert dec.rows == 32


def _unchanged(dec, rows, queries, before):
    S, hk = dec.n_seqs, dec.cfg.n_kv_heads
    return (dec.rows, dec.queries) == (rows, queries) and dec.cache.lens.tolist() == [[rows] * hk] * S and \
        all(torch.equal(a, b) for a, b in zip(_held(dec, 0, 0)[1:], before[1:]))


def test_a_refused_load_leaves_the_rows():
    dec = nx.DecodeCache(nx.NexusConfig(4, 2, 64, 4), 1, 128, 32, 1, page_blocks=1, device=DEV)
    _fill(dec, 40, 9)
    before = _held(dec, 0, 0)
    rows = _randn(601, 1, 2, 20, 64, dtype="bf16")
    for a, b in ((rows, rows.float()), (rows.float(), rows), (rows, rows.cpu()), (rows, rows[..., :32]),
                 (rows[:, :1], rows[:, :1]), (rows[..., :32], rows[..., :32])):
        with pytest.raises((ValueError, TypeError)):
            dec.load(a, b)
        assert _unchanged(dec, 49, 9, before)


@pytest.mark.parametrize("window", [1, 4, 5])
def test_a_refused_step_leaves_the_query_window(window):
    dec = nx.DecodeCache(nx.NexusConfig(4, 2, 64, window), 1, 128, 32, 1, page_blocks=1, device=DEV)
    _fill(dec, 40, 9)
    qs = [_randn(202 + i, 1, 8, 64, dtype="bf16")[:, :4] for i in range(9)]
    q, k, v = _randn(600, 1, 8, 64, dtype="bf16").split((4, 2, 2), 1)
    before = _held(dec, 0, 0)
    wide = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device=DEV)
    for bad in (v[:, :1], v.float(), wide[..., ::2], wide[..., 4:68], v.cpu()):
        with pytest.raises((ValueError, TypeError, nx.NexusError)):
            dec.step(q, k, bad)                # the query has taken its place by then
        assert _unchanged(dec, 49, 9, before)
    dec.evict()
    dec.check()
    assert torch.equal(dec.window, torch.stack(qs[-window:], 2))


def test_events_at_many_row_counts_hold_no_more_memory():
    """One set of event records, rewritten as the row count changes; each event as nx_evict_step has it."""
    cfg = nx.NexusConfig(4, 2, 64, 4)
    dec = nx.DecodeCache(cfg, 1, 128, 32, 1, page_blocks=1, seed=5, device=DEV)
    ews = nx.new_workspace(cfg, 128, 1, 1, device=DEV)
    held = None
    for event, rows in enumerate((40, 41, 90, 40, 77, 78, 90, 41)):
        _fill(dec, rows, 6, seed=700 + event)
        n = dec.rows
        k, v = nx.nx_paged_gather(cfg, dec.cache, workspace=dec.ws, max_tokens=n)
        dec.evict()
        dec.check()
        want, _, _ = nx.nx_evict_step(cfg, dec.window[0], k[0], v[0], n, 32, 1, 5, workspace=ews, step=event)
        assert torch.equal(want, dec.keep[0])
        del k, v, want
        torch.cuda.synchronize()
        if event:
            assert held is None or torch.cuda.memory_allocated() == held
            held = torch.cuda.memory_allocated()


def test_layers_that_share_event_buffers():
    """Each as with buffers of its own; an error is found by whichever is asked, for all of them."""
    cfg = nx.NexusConfig(4, 2, 64, 4)

    def layers(share):
        made = []
        for i in range(3):
            made.append(nx.DecodeCache(cfg, 2, 128, 40, 2, page_blocks=1, seed=9, layer=i,
                                       event_buffers=made[0].event_buffers if share and made else None, device=DEV))
        return made
    shared, own = layers(True), layers(False)
    assert len({d.k.data_ptr() for d in shared}) == 1 and len({d.k.data_ptr() for d in own}) == 3
    for event in range(2):
        for both in (shared, own):
            for i, dec in enumerate(both):
                _fill(dec, 60 + 5 * i, 6, seed=800 + 40 * i + event)
            for dec in both:
                dec.evict()
            for dec in both:
                dec.check()
        for a, b in zip(shared, own):
            assert torch.equal(a.keep, b.keep) and a.rows == b.rows == 40
            for s in range(2):
                for h in range(2):
                    x, y = _held(a, s, h), _held(b, s, h)
                    assert x[0] == y[0] == 40 and all(torch.equal(p, q) for p, q in zip(x[1:], y[1:]))
    for i, dec in enumerate(shared):
        _fill(dec, 60 + 5 * i, 6, seed=900)
    shared[1].rows -= 2                        # that layer's event rejects all heads
    for dec in shared:
        dec.evict()
    with pytest.raises(nx.NexusError):
        shared[2].check()
    assert [d.rows for d in shared] == [40, 71, 40] and (shared[1].cache.lens == 71).all()
    shared[0].check()                          # read once, then clear


def test_the_whole_loop_on_a_side_stream():
    """Load, steps and events under another current stream, while the default stream is busy."""
    cfg = nx.NexusConfig(4, 2, 64, 4)

    def loop():
        dec = nx.DecodeCache(cfg, 2, 96, 32, 2, page_blocks=1, seed=3, device=DEV)
        _fill(dec, 60, 36)
        outs = []
        for event in range(2):
            dec.evict()
            for i in range(64):
                outs.append(dec.step(*_randn(1000 + i + 64 * event, 2, 8, 64, dtype="bf16").split((4, 2, 2), 1)).clone())
        dec.check()
        return torch.stack(outs), dec.cache.lens.clone(), dec.keep.clone()
    want = loop()
    torch.cuda.synchronize()
    big, side = torch.randn(4096, 4096, device=DEV), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        big @ big
    with torch.cuda.stream(side):
        got = loop()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
