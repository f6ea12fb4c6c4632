"""The decode-step operators on the GPU against the fp64 oracle (oracle/paged.py).

Stored codes, scales and tails are compared bit for bit: the rotation is formed in
fp64 on both sides and every rounding is defined.  Attention is compared within a
bound derived per output element (see _attn_bound)."""

import numpy as np
import pytest
import torch

import streaming_weighted_sampling_amd as nx
from oracle import paged

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}      # half a rounding step, relative


def _np(t):
    return t.detach().double().cpu().numpy()


def _randn(seed, *shape, dtype="f32"):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(DT[dtype])


class Cache:
    """A GPU cache with shuffled pages, and helpers to read its arrays back."""

    def __init__(self, n_seqs, hkv, group, d, dtype, fmt, page_blocks, max_pages, seed=0, max_q=1, spare=3):
        self.cfg = nx.NexusConfig(hkv * group, hkv, d, 1, DT[dtype])
        n = n_seqs * hkv * max_pages
        self.c = nx.new_paged_cache(self.cfg, n_seqs, n + spare, max_pages, fmt=fmt, page_blocks=page_blocks,
                                    device=DEV)
        g = torch.Generator().manual_seed(seed)
        self.c.table.copy_(torch.randperm(n + spare, generator=g)[:n].view(n_seqs, hkv, max_pages))
        self.d, self.hkv, self.n_seqs, self.group, self.fmt, self.dtype = d, hkv, n_seqs, group, fmt, dtype
        self.pb = page_blocks
        self.ws = nx.new_paged_workspace(self.cfg, self.c, max(1, self.c.capacity), max_q)

    def check(self):
        nx.nx_read_device_status(self.cfg, self.ws)

    def fill(self, lens, seed=1, garbage=True):
        """Random codes, scales and tails for the given lengths; whatever lies outside them holds
        the worst the types have (NaN, infinities), which no result may show."""
        c, rng = self.c, np.random.default_rng(seed)
        lens = torch.as_tensor(lens, dtype=torch.int32).view(self.n_seqs, self.hkv)
        c.lens.copy_(lens)
        if garbage:
            for t in (c.k_codes, c.v_codes):
                t.view(torch.uint8).fill_(0x7F)          # e4m3 NaN, int8 127
            for t in (c.k_scale, c.v_scale, c.k_tail, c.v_tail):
                t.fill_(float("nan"))
            c.v_tail[..., ::2, :] = float("inf")
        for s in range(self.n_seqs):
            for h in range(self.hkv):
                n = int(lens[s, h])
                for b in range(n // 32):
                    page = int(c.table[s, h, b // self.pb])
                    for codes, scale in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale)):
                        x = torch.from_numpy(rng.standard_normal((32, self.d)).astype(np.float32))
                        top = x.abs().max() / paged.TOP[self.fmt]
                        y = (x / top)
                        y = y.round().to(torch.int8) if self.fmt == "int8" else y.to(torch.float8_e4m3fn)
                        if codes is c.v_codes:
                            y = y.view(torch.uint8).view(4, 8, self.d).transpose(1, 2).contiguous()
                        codes.view(torch.uint8)[page, b % self.pb] = y.view(torch.uint8).to(DEV)
                        scale[page, b % self.pb] = top * float(2.0 ** rng.integers(-3, 4))
                r = n % 32
                x = torch.from_numpy(rng.standard_normal((2, 32, self.d))).to(DT[self.dtype]).to(DEV)
                c.k_tail[s, h, :r] = x[0, :r]
                v = c.v_tail[s, h].transpose(1, 2).reshape(32, self.d)
                v[:r] = x[1, :r]
                c.v_tail[s, h] = v.view(4, 8, self.d).transpose(1, 2)

    def block(self, s, h, b):
        """((K codes, scale), (V codes, scale)) of a whole block, as values."""
        c, page = self.c, int(self.c.table[s, h, b // self.pb])
        k, v = _np(c.k_codes[page, b % self.pb].float()), _np(c.v_codes[page, b % self.pb].float())
        return ((k, float(c.k_scale[page, b % self.pb])),
                (v.transpose(0, 2, 1).reshape(32, self.d), float(c.v_scale[page, b % self.pb])))

    def tail(self, s, h, n):
        return (_np(self.c.k_tail[s, h, :n]),
                _np(self.c.v_tail[s, h]).transpose(0, 2, 1).reshape(32, self.d)[:n])

    def rows(self, s, h):
        n = int(self.c.lens[s, h])
        out = []
        for i in range(2):
            parts = [x[i][0] * x[i][1] for x in (self.block(s, h, b) for b in range(n // 32))]
            out.append(np.concatenate(parts + [self.tail(s, h, n % 32)[i]]))
        return out


def _attn_bound(dtype, d, out, mag, size, v):
    """Error of one output element o = sum p v / sum p, with A = sum p |v| / sum p (mag) and
    S = max_t scale sum_d |q_d k_td| (size):
      result rounded once                                       HALF[dtype] |o|
      p rounded to f16 (relative 2^-11), two terms for fp32 2^-22, bf16 tail 2^-17
      logits: fp32 sums of d products and a scale, (d + 8) 2^-24 S; q's two f16 terms for
      fp32 rows 2^-22 S; the largest |q| is at least 2^13 in f16, whose smallest step then
      moves a logit by less than 2^-36 S d; the exponent argument (|z| < 2^8) and exp2: 2^-15
      where z is large costs p nothing in relative terms beyond 2^-24 |z| <= 2^-16
      a relative error e of p moves o by at most 2 e A (numerator and denominator)
      sums over at most 64 + 32 + 4 + 2048 / 4 terms in a row: 2^-24 * 700 < 2^-14 A
      p's smallest f16 step: p is held times 2^7 and times the ratio r of its block's V scale to
      the reference, which is at most twice the largest scale (r is 1 where it would be below
      2^-12).  Half of f16's smallest step is 2^-25, so p is off by up to 2^-32 / r and its term
      by 2^-32 |v| / r <= 2^-31 max |v| (a block's largest code is M, so M times its scale is a
      |v|), for each of the n rows, over a sum of p that is at least 1"""
    p = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -22
    logit = (d + 8) * 2.0 ** -24 * size + (2.0 ** -22 * size if dtype == "f32" else 0.0)
    e = p + logit + 2.0 ** -16
    return HALF[dtype] * np.abs(out) + (2 * e[..., None] + 2.0 ** -14) * mag + \
        len(v) * 2.0 ** -31 * np.abs(v).max(initial=0.0) + 1e-30


def _check_attn(cache, q, counts, out, lse=None, scale=None):
    """out rows of every sequence against the oracle on the arrays read back."""
    at, grp, got = 0, cache.group, _np(out)
    for s, m in enumerate(counts):
        for h in range(cache.hkv):
            k, v = cache.rows(s, h)
            x = _np(q[at:at + m, h * grp:(h + 1) * grp])
            o, l, mag, size = paged.attend(x, k, v, scale)
            y = got[at:at + m, h * grp:(h + 1) * grp]
            err = np.abs(y - o)
            bad = ~(err <= _attn_bound(cache.dtype, cache.d, o, mag, size, v))
            assert not bad.any(), (s, h, m, len(k), float(np.nanmax(err)), int(bad.sum()))
            if lse is not None:
                z = _np(lse[at:at + m, h * grp:(h + 1) * grp])
                assert np.array_equal(np.isneginf(z), np.isneginf(l))
                f = np.isfinite(l)
                # p's rounding does not enter the sum; logits, exp2, sums as above
                z, l = np.where(f, z, 0.0), np.where(f, l, 0.0)
                lim = (cache.d + 8) * 2.0 ** -24 * size + 2.0 ** -14 + 2.0 ** -22 * (np.abs(l) + size)
                assert (np.abs(z - l)[f] <= lim[f]).all(), (s, h, np.abs(z - l)[f].max())
        at += m


# ---------------------------------------------------------------- norm and rotation

@pytest.mark.parametrize("rows", [1, 7, 130])
@pytest.mark.parametrize("d,dtype,rot,pairs", [
    (128, "bf16", 128, False), (128, "bf16", 64, True), (128, "f32", 48, False), (64, "bf16", 64, True),
    (64, "f32", 16, False), (64, "f32", 16, True), (128, "bf16", 0, False), (64, "bf16", 32, False)])
def test_norm_rope(rows, d, dtype, rot, pairs):
    hq, hk = 6, 2
    cfg = nx.NexusConfig(hq, hk, d, 1, DT[dtype])
    ws = nx.new_workspace(cfg, 1, 1, 0, device=DEV)
    qkv = _randn(rows, rows, hq + 2 * hk, d, dtype=dtype) * 3
    qkv[0, 0] = 0                                    # a row of zeros stays zero
    q, k, _ = qkv.split((hq, hk, hk), 1)
    wq, wk = _randn(2, d, dtype=dtype), _randn(3, d, dtype=dtype)
    rope = pos = cs = None
    if rot:
        rope = nx.Rope(nx.rope_table(300, rot, 100.0, device=DEV), pairs)
        pos = torch.randint(0, 300, (rows,), device=DEV, dtype=torch.int32)
        cs = _np(rope.cos_sin[pos.long()])
    out_q = torch.zeros(hq, rows + 2, d, dtype=DT[dtype], device=DEV)     # a query window's layout
    oq, ok = nx.nx_qk_norm_rope(cfg, q, k, workspace=ws, q_weight=wq, k_weight=wk, eps=1e-5, rope=rope,
                                positions=pos, out_q=out_q[:, 1:-1].permute(1, 0, 2))
    nx.nx_read_device_status(cfg, ws)
    assert not out_q[:, 0].any() and not out_q[:, -1].any()
    for x, w, y in ((q, wq, oq), (k, wk, ok)):
        want = paged.norm_rope(_np(x), _np(w), 1e-5, cs, pairs)
        plain = np.abs(paged.norm_rope(_np(x), _np(w), 1e-5))
        # fp32: d squares summed, a square root, a quotient, three products, a sum: the square sum's
        # relative error d 2^-24 counts half, so (d / 2 + 8) 2^-24 <= 2^-17 of each rotated term
        mag = plain if cs is None else plain + np.abs(paged.rotate(plain, np.abs(cs), pairs)) + \
            np.abs(paged.rotate(plain, np.concatenate([np.abs(cs[:, :rot // 2]), -np.abs(cs[:, rot // 2:])], 1), pairs))
        assert (np.abs(_np(y) - want) <= HALF[dtype] * np.abs(want) + 2.0 ** -17 * mag + 1e-30).all()
    # in place on slices of the projection, rotation only on the keys
    q0, k0 = q.clone(), k.clone()
    nx.nx_qk_norm_rope(cfg, q, k, workspace=ws, q_weight=wq, eps=1e-5, rope=rope, positions=pos, out_q=q, out_k=k)
    assert torch.equal(q, oq)
    want = paged.norm_rope(_np(k0), None, 0, cs, pairs)
    mag = np.abs(_np(k0)).max(-1, keepdims=True) * 2
    assert (np.abs(_np(k) - want) <= HALF[dtype] * np.abs(want) + 2.0 ** -22 * mag).all()
    only, none = nx.nx_qk_norm_rope(cfg, q0, workspace=ws, q_weight=wq, eps=1e-5, rope=rope, positions=pos)
    assert none is None and torch.equal(only, oq)
    nx.nx_read_device_status(cfg, ws)


def test_norm_rope_reports_a_position_outside_the_table():
    cfg = nx.NexusConfig(2, 1, 64, 1)
    ws = nx.new_workspace(cfg, 1, 1, 0, device=DEV)
    rope = nx.Rope(nx.rope_table(4, 64, device=DEV))
    q = _randn(1, 3, 2, 64, dtype="bf16")
    for bad in (4, -1):
        pos = torch.tensor([0, bad, 3], dtype=torch.int32, device=DEV)
        nx.nx_qk_norm_rope(cfg, q, workspace=ws, rope=rope, positions=pos)
        with pytest.raises(nx.NexusError) as e:
            nx.nx_read_device_status(cfg, ws)
        assert e.value.code == nx.NX_EINVAL
    nx.nx_qk_norm_rope(cfg, q, workspace=ws, rope=rope)
    nx.nx_read_device_status(cfg, ws)


# ---------------------------------------------------------------- append

def _append_all(cache, steps, rot, pairs, seed, in_place=True):
    """Runs `steps` (row counts per sequence) through the kernel and the oracle."""
    c, cfg = cache.c, cache.cfg
    heads = [[paged.Head(cache.d, cache.dtype, cache.fmt) for _ in range(cache.hkv)] for _ in range(cache.n_seqs)]
    rope = nx.Rope(nx.rope_table(5000, rot, 1000.0, device=DEV), pairs) if rot else None
    for step, counts in enumerate(steps):
        n = sum(counts)
        kv = _randn(seed + step, n, 2 * cache.hkv + 1, cache.d, dtype=cache.dtype)
        kv[..., 1::32] *= 8
        k, v = kv[:, :cache.hkv], kv[:, cache.hkv:2 * cache.hkv]
        pos = torch.randint(0, 5000, (n,), device=DEV, dtype=torch.int32) if rot else None
        start = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)
        out = None if in_place else torch.empty_like(c.lens)
        nx.nx_paged_append(cfg, c, k, v, workspace=cache.ws, max_new=max(counts), new_start=start, rope=rope,
                           positions=pos, lens_out=out)
        if out is not None:
            c.lens.copy_(out)
        turned = paged.rotate(_np(k), _np(rope.cos_sin[pos.long()]), pairs) if rot else _np(k)
        at = 0
        for s, m in enumerate(counts):
            for h in range(cache.hkv):
                heads[s][h].append(turned[at:at + m, h], _np(v)[at:at + m, h])
            at += m
    cache.check()
    return heads


def _compare(cache, heads):
    for s in range(cache.n_seqs):
        for h in range(cache.hkv):
            ref = heads[s][h]
            assert int(cache.c.lens[s, h]) == len(ref), (s, h)
            for b, want in enumerate(ref.blocks):
                for (codes, scale), (wc, wsc) in zip(cache.block(s, h, b), want):
                    assert scale == wsc, (s, h, b)
                    assert np.array_equal(codes, wc), (s, h, b, np.abs(codes - wc).max())
            for got, want in zip(cache.tail(s, h, len(ref) % 32), ref.tail):
                if want:
                    assert np.array_equal(got, np.stack(want)), (s, h)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,dtype,rot,pairs,page_blocks", [
    (128, "bf16", 128, False, 4), (128, "f32", 64, True, 1), (64, "bf16", 32, True, 2),
    (64, "f32", 64, False, 8), (128, "bf16", 0, False, 2)])
def test_append(d, dtype, rot, pairs, page_blocks, fmt):
    cache = Cache(3, 2, 2, d, dtype, fmt, page_blocks, -(-16 // page_blocks))
    # single tokens, none, mid-block to mid-block, exactly full, several blocks at once
    steps = [(1, 1, 1), (30, 0, 31), (1, 0, 1), (65, 1, 64), (0, 33, 95), (1, 1, 1), (190, 200, 0), (1, 1, 1)]
    _compare(cache, _append_all(cache, steps, rot, pairs, 10))


def test_append_writes_only_what_it_must():
    cache = Cache(2, 2, 1, 128, "bf16", "e4m3", 2, 4, spare=9)
    c = cache.c
    for t in (c.k_codes, c.v_codes):
        t.view(torch.uint8).fill_(0xA5)
    for t in (c.k_scale, c.v_scale, c.k_tail, c.v_tail):
        t.fill_(7.0)
    before = [t.clone() for t in (c.k_codes.view(torch.uint8), c.v_codes.view(torch.uint8), c.k_scale, c.v_scale)]
    tails = [t.clone() for t in (c.k_tail, c.v_tail)]
    _append_all(cache, [(70, 5)], 0, False, 3)
    used = {(int(c.table[0, h, 0]), b) for h in range(2) for b in range(2)}
    for t, old in zip((c.k_codes.view(torch.uint8), c.v_codes.view(torch.uint8), c.k_scale, c.v_scale), before):
        for p in range(t.shape[0]):
            for b in range(t.shape[1]):
                if (p, b) not in used:
                    assert torch.equal(t[p, b], old[p, b]), (p, b)
    for s, n in ((0, 6), (1, 5)):
        assert torch.equal(c.k_tail[s, :, n:], tails[0][s, :, n:])
        v = c.v_tail[s].transpose(2, 3).reshape(2, 32, 128)
        assert (v[:, n:] == 7.0).all() and not (v[:, :n] == 7.0).all()


def test_append_per_head_counts_and_separate_lens():
    cache = Cache(2, 3, 1, 64, "bf16", "int8", 4, 2)
    k, v = _randn(5, 2 * 40, 3, 64, dtype="bf16"), _randn(6, 2 * 40, 3, 64, dtype="bf16")
    counts = torch.tensor([[40, 0, 33], [1, 32, 31]], dtype=torch.int32, device=DEV)
    out = torch.full_like(cache.c.lens, -5)
    nx.nx_paged_append(cache.cfg, cache.c, k, v, workspace=cache.ws, head_new=counts, lens_out=out)
    cache.check()
    assert not cache.c.lens.any() and torch.equal(out, counts)
    cache.c.lens.copy_(out)
    heads = []
    for s in range(2):
        heads.append([])
        for h in range(3):
            heads[s].append(paged.Head(64, "bf16", "int8"))
            m = int(counts[s, h])
            heads[s][h].append(_np(k)[s * 40:s * 40 + m, h], _np(v)[s * 40:s * 40 + m, h])
    _compare(cache, heads)


def test_append_head_major_rows_and_broadcast_heads():
    """Rows as an eviction event leaves them ([heads][rows][D]), and one head's rows for all."""
    cache = Cache(1, 3, 1, 64, "bf16", "e4m3", 1, 4)
    k, v = _randn(7, 3, 50, 64, dtype="bf16"), _randn(8, 1, 50, 64, dtype="bf16")
    nx.nx_paged_append(cache.cfg, cache.c, k.permute(1, 0, 2), v.expand(3, 50, 64).permute(1, 0, 2),
                       workspace=cache.ws)
    cache.check()
    heads = [[paged.Head(64, "bf16", "e4m3") for _ in range(3)]]
    for h in range(3):
        heads[0][h].append(_np(k)[h], _np(v)[0])
    _compare(cache, heads)


def test_append_zero_and_tiny_blocks_and_non_finite_elements():
    cache = Cache(1, 1, 1, 64, "f32", "int8", 1, 8)
    x = _randn(9, 128, 1, 64)
    x[:32] = 0
    x[32:64] *= 2.0 ** -110
    x[70, 0, 3], x[71, 0, 5], x[72, 0, 7] = float("nan"), float("inf"), -float("inf")
    nx.nx_paged_append(cache.cfg, cache.c, x, x, workspace=cache.ws)
    with pytest.raises(nx.NexusError) as e:
        cache.check()
    assert e.value.code == nx.NX_ENONFINITE
    cache.check()                                    # read once, then clear
    heads = [[paged.Head(64, "f32", "int8")]]
    heads[0][0].append(_np(x)[:, 0], _np(x)[:, 0])
    _compare(cache, heads)
    assert [s for (_, s), _ in heads[0][0].blocks[:2]] == [0.0, 0.0]


def test_append_leaves_bad_sequences_and_reports_them():
    cache = Cache(4, 1, 1, 64, "bf16", "e4m3", 1, 2)
    k = _randn(11, 8, 1, 64, dtype="bf16")
    cache.c.lens.copy_(torch.tensor([[62], [63], [-1], [0]], dtype=torch.int32))
    tails = cache.c.k_tail.clone()
    start = torch.tensor([0, 2, 4, 6, 8], dtype=torch.int32, device=DEV)
    nx.nx_paged_append(cache.cfg, cache.c, k, k, workspace=cache.ws, max_new=2, new_start=start)
    with pytest.raises(nx.NexusError) as e:
        cache.check()
    assert e.value.code == nx.NX_EINVAL
    assert cache.c.lens.flatten().tolist() == [64, 63, -1, 2]     # 63 + 2 rows do not fit 64
    assert torch.equal(cache.c.k_tail[1:3], tails[1:3])
    for bad in ([0, 2, 1, 6, 8], [0, 2, 4, 6, 9], [-1, 1, 2, 3, 4], [0, 3, 4, 5, 6]):
        cache.c.lens.zero_()
        out = torch.full_like(cache.c.lens, -7)
        nx.nx_paged_append(cache.cfg, cache.c, k, k, workspace=cache.ws, max_new=2, lens_out=out,
                           new_start=torch.tensor(bad, dtype=torch.int32, device=DEV))
        with pytest.raises(nx.NexusError):
            cache.check()
        for s in range(4):
            m = bad[s + 1] - bad[s]
            ok = bad[s] >= 0 and 0 <= m <= 2 and bad[s + 1] <= 8
            assert int(out[s]) == (m if ok else 0), bad
    # a page number outside the pool: reported, nothing written there
    cache.c.lens.zero_()
    cache.c.table[0, 0, 0] = cache.c.k_codes.shape[0]
    cache.c.table[1, 0, 0] = -1
    k = _randn(12, 4 * 32, 1, 64, dtype="bf16")
    nx.nx_paged_append(cache.cfg, cache.c, k, k, workspace=cache.ws)
    with pytest.raises(nx.NexusError):
        cache.check()


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,dtype,hkv,group,page_blocks", [
    (128, "bf16", 2, 4, 4), (64, "bf16", 1, 1, 1), (128, "f32", 1, 5, 2), (64, "f32", 2, 8, 8)])
@pytest.mark.parametrize("lens", [
    (0, 1, 31), (32, 33, 64), (95, 700, 1500)], ids=["short", "edges", "long"])
def test_attention_of_single_tokens(lens, d, dtype, hkv, group, page_blocks, fmt):
    cache = Cache(3, hkv, group, d, dtype, fmt, page_blocks, -(-48 // page_blocks))
    cache.fill([n if h == 0 else max(0, n - 17) for n in lens for h in range(hkv)])
    q = _randn(21, 3, hkv * group, d, dtype=dtype) * 2
    lse = torch.empty(3, hkv * group, device=DEV)
    out = nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=cache.ws, max_tokens=max(lens), out_lse=lse)
    cache.check()
    _check_attn(cache, q, [1, 1, 1], out, lse)
    # the bound only sizes the grid; the same call twice is the same bits
    for most in (0, 40, 100000):
        ws = nx.new_paged_workspace(cache.cfg, cache.c, most)
        o = nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=ws, max_tokens=most)
        nx.nx_read_device_status(cache.cfg, ws)
        _check_attn(cache, q, [1, 1, 1], o)
        assert torch.equal(o, nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=ws, max_tokens=most))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,dtype,hkv,group", [(128, "bf16", 2, 4), (64, "bf16", 1, 3), (128, "f32", 1, 2),
                                               (64, "f32", 1, 7)])
@pytest.mark.parametrize("counts", [(3, 0, 5), (17, 1, 40), (2, 64, 9)])
def test_attention_of_several_queries(counts, d, dtype, hkv, group, fmt):
    """Ragged queries, causal among the newest rows; in the last sequence some queries are older
    than every row (a head shorter than the query count) and see nothing."""
    cache = Cache(3, hkv, group, d, dtype, fmt, 2, 8, max_q=64)
    cache.fill([n for m in ((200, 190), (77, 64), (4, 33)) for n in m[:hkv]])
    n = sum(counts)
    q = _randn(22, n + 2, hkv * group, d, dtype=dtype)
    start = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 9.0)
    lse = torch.full((n + 2, hkv * group), 9.0, device=DEV)
    nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=cache.ws, max_tokens=200, max_q=max(counts), q_start=start,
                     out=out, out_lse=lse, scale=0.3)
    cache.check()
    _check_attn(cache, q, counts, out, lse, scale=0.3)
    assert (out[n:] == 9.0).all() and (lse[n:] == 9.0).all()      # rows of no sequence


def test_attention_large_query_windows_and_strided_rows():
    cache = Cache(1, 2, 8, 128, "bf16", "e4m3", 4, 9, max_q=64)
    cache.fill([1100, 1057])
    q = _randn(23, 64, 40, 128, dtype="bf16")[:, 3:19]            # heads of a wider projection
    out = torch.zeros(16, 64, 128, dtype=torch.bfloat16, device=DEV)
    nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=cache.ws, max_tokens=1100, out=out.permute(1, 0, 2))
    cache.check()
    _check_attn(cache, q, [64], out.permute(1, 0, 2))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_extreme_logits_and_scales(dtype):
    """Logits far apart (one row takes all, late and early), rising maxima, uniform rows, and V
    blocks whose scales differ by 2^60."""
    cache = Cache(1, 1, 4, 64, dtype, "int8", 1, 40)
    cache.fill([1279], seed=4)
    for b in range(39):
        page = int(cache.c.table[0, 0, b])
        cache.c.k_scale[page] = 2.0 ** (b % 13 - 9)
        cache.c.v_scale[page] = 2.0 ** (40 - 60 * (b % 2) - b)
    q = _randn(24, 1, 4, 64, dtype=dtype)
    q[0, 1] *= 100
    q[0, 2] = 0
    q[0, 3] *= 2.0 ** -60
    out = nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=cache.ws, max_tokens=1279)
    cache.check()
    _check_attn(cache, q, [1], out)


def test_non_finite_queries_stay_in_their_rows():
    cache = Cache(1, 1, 4, 64, "bf16", "e4m3", 1, 8, max_q=2)
    cache.fill([200])
    q = _randn(25, 2, 4, 64, dtype="bf16")
    ref = nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=cache.ws, max_tokens=200)
    q[0, 1, 5], q[1, 2, 0] = float("nan"), float("inf")
    out = nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=cache.ws, max_tokens=200)
    assert not torch.isfinite(out[0, 1]).any() and not torch.isfinite(out[1, 2]).any()
    keep = torch.ones(2, 4, dtype=torch.bool)
    keep[0, 1] = keep[1, 2] = False
    assert torch.equal(out[keep], ref[keep])


def test_attention_reports_bad_sequences_and_serves_the_others():
    cache = Cache(3, 1, 2, 64, "bf16", "e4m3", 1, 4)
    cache.fill([100, 50, 64])
    q = _randn(26, 3, 2, 64, dtype="bf16")
    cache.c.lens[0, 0] = 129                                       # past the table
    out = nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=cache.ws, max_tokens=128)
    with pytest.raises(nx.NexusError) as e:
        cache.check()
    assert e.value.code == nx.NX_EINVAL
    cache.c.lens[0, 0] = 0
    good = nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=cache.ws, max_tokens=128)
    cache.check()
    assert torch.equal(out[1:], good[1:]) and not good[0].any()
    cache.c.table[1, 0, 0] = 10 ** 6
    out = nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=cache.ws, max_tokens=128)
    with pytest.raises(nx.NexusError):
        cache.check()
    assert torch.equal(out[2], good[2])


def test_shared_pages_may_be_read_by_several_heads():
    cache = Cache(2, 1, 2, 64, "bf16", "int8", 2, 4)
    cache.fill([150, 64])
    cache.c.table[1] = cache.c.table[0]                            # a common prefix
    q = _randn(27, 2, 2, 64, dtype="bf16")
    out = nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=cache.ws, max_tokens=150)
    cache.check()
    _check_attn(cache, q, [1, 1], out)


# ---------------------------------------------------------------- gather

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,dtype,page_blocks", [(128, "bf16", 4), (64, "f32", 1), (128, "f32", 2), (64, "bf16", 8)])
def test_gather(d, dtype, page_blocks, fmt):
    cache = Cache(2, 3, 1, d, dtype, fmt, page_blocks, -(-8 // page_blocks))
    cache.fill([0, 1, 31, 32, 63, 200])
    room = torch.full((2, 2, 3, 210, d), 5.0, dtype=DT[dtype], device=DEV)
    nx.nx_paged_gather(cache.cfg, cache.c, workspace=cache.ws, max_tokens=200, out_k=room[0], out_v=room[1])
    cache.check()
    for s in range(2):
        for h in range(3):
            n = int(cache.c.lens[s, h])
            for i, want in enumerate(cache.rows(s, h)):
                # one product in fp32 (rounded once more to bf16)
                lim = (HALF[dtype] + 2.0 ** -24) * np.abs(want)
                assert (np.abs(_np(room[i, s, h, :n]) - want) <= lim).all()
                assert (room[i, s, h, n:] == 5.0).all()
    k, v = nx.nx_paged_gather(cache.cfg, cache.c, workspace=cache.ws, max_tokens=200)
    assert torch.equal(k[1, 2], room[0, 1, 2, :200]) and not k[0, 0].any()
    nx.nx_paged_gather(cache.cfg, cache.c, workspace=cache.ws, max_tokens=199)
    with pytest.raises(nx.NexusError):
        cache.check()                                              # a head longer than the bound


# ---------------------------------------------------------------- together

def test_pages_past_four_gigabytes():
    """A pool of over 2^32 bytes whose last pages are in use."""
    cfg = nx.NexusConfig(4, 1, 128, 1)
    n = (1 << 32) // (4 * 32 * 128) + 64
    c = nx.new_paged_cache(cfg, 1, n, 8, page_blocks=4, device=DEV)
    c.table.copy_(torch.arange(n - 8, n, dtype=torch.int32).view(1, 1, 8))
    ws = nx.new_paged_workspace(cfg, c, 1000)
    k, v = _randn(31, 1000, 1, 128, dtype="bf16"), _randn(32, 1000, 1, 128, dtype="bf16")
    nx.nx_paged_append(cfg, c, k, v, workspace=ws)
    q = _randn(33, 1, 4, 128, dtype="bf16")
    out = nx.nx_paged_attn(cfg, c, q, workspace=ws, max_tokens=1000)
    gk, _ = nx.nx_paged_gather(cfg, c, workspace=ws, max_tokens=1000)
    nx.nx_read_device_status(cfg, ws)
    small = nx.new_paged_cache(cfg, 1, 8, 8, page_blocks=4, device=DEV)
    small.table.copy_(torch.arange(8, dtype=torch.int32).view(1, 1, 8))
    nx.nx_paged_append(cfg, small, k, v, workspace=ws)
    assert torch.equal(out, nx.nx_paged_attn(cfg, small, q, workspace=ws, max_tokens=1000))
    assert torch.equal(gk, nx.nx_paged_gather(cfg, small, workspace=ws, max_tokens=1000)[0])


def test_a_captured_step_replays_like_eager_steps():
    """Norm, append (lengths advance on the device) and attention in one graph; eager work on the
    same workspace and synchronisation between replays."""
    def world():
        cache = Cache(2, 2, 2, 64, "bf16", "e4m3", 1, 8)
        cache.c.lens.copy_(torch.tensor([[0, 30], [31, 60]], dtype=torch.int32))
        for t, seed in ((cache.c.k_tail, 41), (cache.c.v_tail, 42)):
            t.copy_(_randn(seed, *t.shape, dtype="bf16"))
        for codes in (cache.c.k_codes, cache.c.v_codes):
            codes.view(torch.uint8).fill_(0x31)
        cache.c.k_scale.fill_(0.25)
        cache.c.v_scale.fill_(0.5)
        return cache
    rope = nx.Rope(nx.rope_table(100, 64, device=DEV))
    qkv = torch.empty(2, 8, 64, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    w = _randn(43, 64, dtype="bf16")

    def step(cache, q2, out):
        q, k, v = qkv.split((4, 2, 2), 1)
        nx.nx_qk_norm_rope(cache.cfg, q, workspace=cache.ws, q_weight=w, rope=rope, positions=pos, out_q=q2)
        nx.nx_paged_append(cache.cfg, cache.c, k, v, workspace=cache.ws, rope=rope, positions=pos)
        nx.nx_paged_attn(cache.cfg, cache.c, q2, workspace=cache.ws, max_tokens=200, out=out)

    eager, graph = world(), world()
    q2 = [torch.empty(2, 4, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    out = [torch.empty_like(q2[0]) for _ in range(2)]
    warm = world()
    step(warm, q2[1], out[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            step(graph, q2[1], out[1])
    torch.cuda.current_stream().wait_stream(s)
    for r in range(40):
        qkv.copy_(_randn(100 + r, 2, 8, 64, dtype="bf16"))
        pos.fill_(r)
        step(eager, q2[0], out[0])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], out[1]), r
        if r % 9 == 0:      # eager work between replays, on the graph's own workspace
            nx.nx_paged_attn(graph.cfg, graph.c, q2[1], workspace=graph.ws, max_tokens=200)
    for a, b in ((eager.c.lens, graph.c.lens), (eager.c.k_scale, graph.c.k_scale), (eager.c.v_tail, graph.c.v_tail)):
        assert torch.equal(a, b)
    assert eager.c.lens.flatten().tolist() == [40, 70, 71, 100]
    eager.check()
    graph.check()


def test_two_streams_with_their_own_workspaces():
    cache = Cache(1, 2, 4, 128, "bf16", "int8", 4, 8)
    cache.fill([1000, 900])
    q = _randn(51, 1, 8, 128, dtype="bf16")
    ref = nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=cache.ws, max_tokens=1000)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [nx.new_paged_workspace(cache.cfg, cache.c, 1000) for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for r in range(20):
        for i in range(2):
            o = torch.empty_like(ref) if r else torch.zeros_like(ref)
            streams[i].wait_stream(torch.cuda.current_stream())
            outs[i].append(nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=spaces[i], max_tokens=1000, out=o,
                                            stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for side in outs for o in side)


def test_calls_without_rows_do_nothing():
    cache = Cache(2, 1, 2, 64, "bf16", "e4m3", 1, 2)
    cache.fill([40, 3])
    none = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    before = cache.c.lens.clone()
    nx.nx_paged_append(cache.cfg, cache.c, none, none, workspace=cache.ws)
    assert nx.nx_paged_attn(cache.cfg, cache.c, none.expand(0, 2, 64), workspace=cache.ws, max_tokens=40).numel() == 0
    nx.nx_qk_norm_rope(cache.cfg, none.expand(0, 2, 64), none, workspace=cache.ws)
    start = torch.zeros(3, dtype=torch.int32, device=DEV)
    q = torch.full((3, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, 3.0)
    nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=cache.ws, max_tokens=40, max_q=1, q_start=start, out=out)
    cache.check()
    assert torch.equal(cache.c.lens, before) and (out == 3.0).all()


def test_many_heads_of_uneven_lengths():
    """More heads than workgroups wanted, and more than stay in registers, some empty; the bound on the
    lengths forces pieces."""
    cache = Cache(150, 2, 1, 64, "bf16", "int8", 1, 6, max_q=1)
    lens = [(37 * i) % 190 if i % 7 else 0 for i in range(300)]
    cache.fill(lens, garbage=False)
    q = _randn(61, 150, 2, 64, dtype="bf16")
    for most in (190, 6000):
        ws = nx.new_paged_workspace(cache.cfg, cache.c, most)
        out = nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=ws, max_tokens=most)
        nx.nx_read_device_status(cache.cfg, ws)
        _check_attn(cache, q, [1] * 150, out)


def test_one_workspace_serves_calls_of_different_shapes():
    """A workspace made for the largest call, used by others in between: partials and the notes on
    the cut belong to one call."""
    big = Cache(1, 2, 8, 128, "bf16", "e4m3", 4, 20, max_q=16)
    big.fill([2500, 2431])
    small = Cache(3, 2, 1, 64, "bf16", "int8", 1, 50)
    small.fill([1500, 0, 33, 1111, 1499, 64])
    qb, qs = _randn(71, 16, 16, 128, dtype="bf16"), _randn(72, 3, 2, 64, dtype="bf16")
    for _ in range(3):
        for cache, q, most, counts in ((big, qb, 2500, [16]), (small, qs, 1500, [1, 1, 1]), (big, qb[:1], 2500, [1])):
            out = nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=big.ws, max_tokens=most)
            _check_attn(cache, q, counts, out)
    nx.nx_read_device_status(big.cfg, big.ws)


def test_two_graphs_share_a_workspace():
    """Captured attention calls of different cuts, replayed in turn with eager calls between."""
    long = Cache(1, 2, 4, 128, "bf16", "int8", 4, 20)
    long.fill([2500, 1601])
    many = Cache(9, 2, 2, 64, "bf16", "e4m3", 2, 25)
    many.fill([(97 * i) % 1500 for i in range(18)])
    q = [_randn(81, 1, 8, 128, dtype="bf16"), _randn(82, 9, 4, 64, dtype="bf16")]
    outs, graphs = [torch.empty_like(x) for x in q], []

    def call(i):
        cache = (long, many)[i]
        nx.nx_paged_attn(cache.cfg, cache.c, q[i], workspace=long.ws, max_tokens=(2500, 1500)[i], out=outs[i])

    need = nx.paged_workspace_bytes(many.cfg, many.c, 1500)
    if long.ws.nbytes < need:
        long.ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    for i in range(2):
        call(i)
    torch.cuda.synchronize()
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            call(i)
    for turn in range(3):
        for i in (0, 1, 1, 0):
            outs[i].fill_(9.0)
            graphs[i].replay()
            _check_attn((long, many)[i], q[i], [1] * len(q[i]), outs[i])
        call(turn % 2)
        torch.cuda.synchronize()
    long.check()


def test_debug_mode_raises_at_the_call(monkeypatch):
    monkeypatch.setenv("NX_DEBUG", "1")
    cache = Cache(1, 1, 2, 64, "bf16", "int8", 1, 2)
    rows = _randn(91, 3, 1, 64, dtype="bf16")
    nx.nx_paged_append(cache.cfg, cache.c, rows, rows, workspace=cache.ws)
    assert nx.nx_paged_attn(cache.cfg, cache.c, rows[:1].expand(1, 2, 64), workspace=cache.ws,
                            max_tokens=3).isfinite().all()
    nx.nx_paged_gather(cache.cfg, cache.c, workspace=cache.ws, max_tokens=3)
    nx.nx_qk_norm_rope(cache.cfg, rows.repeat(1, 2, 1), workspace=cache.ws)
    rows[1, 0, 5] = float("inf")
    with pytest.raises(nx.NexusError, match="NONFINITE"):
        nx.nx_paged_append(cache.cfg, cache.c, rows, rows, workspace=cache.ws)
    with pytest.raises(nx.NexusError, match="NONFINITE"):
        cache.check()                    # still recorded; reading it clears it
    cache.c.lens.fill_(65)
    with pytest.raises(nx.NexusError, match="EINVAL"):
        nx.nx_paged_attn(cache.cfg, cache.c, rows[:1].expand(1, 2, 64), workspace=cache.ws, max_tokens=64)
    with pytest.raises(nx.NexusError, match="EINVAL"):
        nx.nx_paged_gather(cache.cfg, cache.c, workspace=cache.ws, max_tokens=64)


def test_a_long_prompt_equals_its_parts():
    """One append of 67 MB of codes (written past the caches) against three smaller ones."""
    n, hk, d = 66001, 8, 64
    rows = _randn(95, 2, n, hk, d, dtype="bf16")
    got = []
    for cuts in ((0, n), (0, 20000, 40007, n)):
        cache = Cache(1, hk, 1, d, "bf16", "int8", 8, -(-n // 256))
        for lo, hi in zip(cuts, cuts[1:]):
            nx.nx_paged_append(cache.cfg, cache.c, rows[0, lo:hi], rows[1, lo:hi], workspace=cache.ws)
        cache.check()
        got.append(nx.nx_paged_gather(cache.cfg, cache.c, workspace=cache.ws, max_tokens=n))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    for x, y in zip(rows, got[0]):       # off by at most half a code and the result's rounding
        x = x.permute(1, 0, 2).float()
        amax = torch.nn.functional.pad(x, (0, 0, 0, -n % 32)).view(hk, -1, 32 * d).abs().amax(-1)
        bound = (amax / 254 * (1 + 2.0 ** -20)).repeat_interleave(32, 1)[:, :n, None] + x.abs() * 2.0 ** -7
        assert ((y[0].float() - x).abs() <= bound).all()


@pytest.mark.parametrize("m", [1, 20])
def test_a_thousand_heads(m):
    """Whole heads by the number of heads, at a bound on the lengths that would cut fewer into pieces."""
    S, most = 520, 2000
    cache = Cache(S, 2, 2, 64, "bf16", "int8", 2, 4, max_q=m)
    cache.fill([(53 * i) % 201 if i % 9 else 0 for i in range(2 * S)], garbage=False)
    q = _randn(97, S * m, 4, 64, dtype="bf16")
    ws = nx.new_paged_workspace(cache.cfg, cache.c, most, m)
    lse = torch.empty(S * m, 4, device=DEV)
    out = nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=ws, max_tokens=most, max_q=m, out_lse=lse)
    nx.nx_read_device_status(cache.cfg, ws)
    _check_attn(cache, q, [m] * S, out, lse)
    longer = nx.new_paged_workspace(cache.cfg, cache.c, 40000, m)      # in pieces
    out = nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=longer, max_tokens=40000, max_q=m)
    _check_attn(cache, q, [m] * S, out)


def test_default_outputs_on_a_side_stream():
    """The current stream is kept busy while another stream's calls make their own outputs."""
    cache = Cache(2, 2, 2, 128, "bf16", "e4m3", 4, 8)
    cache.fill([1000, 33, 0, 640])
    q, k = _randn(101, 2, 4, 128, dtype="bf16"), _randn(102, 2, 2, 128, dtype="bf16")
    want = (nx.nx_qk_norm_rope(cache.cfg, q, k, workspace=cache.ws, q_weight=q[0, 0])[0],
            nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=cache.ws, max_tokens=1000),
            *nx.nx_paged_gather(cache.cfg, cache.c, workspace=cache.ws, max_tokens=1000))
    side, big = torch.cuda.Stream(), torch.randn(4096, 4096, device=DEV)
    for _ in range(3):
        torch.cuda.synchronize()
        for _ in range(20):
            big @ big
        got = (nx.nx_qk_norm_rope(cache.cfg, q, k, workspace=cache.ws, q_weight=q[0, 0], stream=side)[0],
               nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=cache.ws, max_tokens=1000, stream=side),
               *nx.nx_paged_gather(cache.cfg, cache.c, workspace=cache.ws, max_tokens=1000, stream=side))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del got
    cache.check()


# V's scale by block, in powers of two, of 25 blocks and a head whose scales reach up to 2^k
V_SCALES = {
    "alternate": lambda b, k: k * (b % 2), "small_first": lambda b, k: k * (b % 8 > 3),
    "large_first": lambda b, k: k * (b % 8 < 4), "stairs": lambda b, k: k * (b % 5) / 4,
    "one_large": lambda b, k: k * (b == 11)}


def _far_scales_cache(dtype, fmt, d, k, order, max_q):
    """Keys of +-1 in element 0 (+1 where V's scale is the small one, and in the tail), so that a query's
    element 0 alone says how the weights split between blocks of small and of large V."""
    cache = Cache(1, 1, 4, d, dtype, fmt, 2, 14, max_q=max_q)
    cache.fill([25 * 32 + 9], seed=6)
    c, top = cache.c, float(paged.TOP[fmt])
    c.k_codes.view(torch.uint8).zero_()
    c.k_tail.zero_()
    c.k_tail[..., 0] = 1.0
    rng = np.random.default_rng(5)
    for b in range(25):
        page, at = int(c.table[0, 0, b // 2]), b % 2
        e = V_SCALES[order](b, k)
        c.k_codes[page, at, :, 0] = torch.full((32,), top if e == 0 else -top).to(c.k_codes.dtype)
        c.k_scale[page, at] = 1.0 / top
        c.v_scale[page, at] = 2.0 ** e * (1.0 + rng.random()) / 2 / top
    c.v_scale[int(c.table[0, 0, 3]), 0] = 0.0          # codes that stand for zeros
    return cache


@pytest.mark.parametrize("order", list(V_SCALES))
@pytest.mark.parametrize("dtype,fmt,d", [("f32", "int8", 64), ("f32", "e4m3", 128), ("bf16", "e4m3", 64),
                                         ("bf16", "int8", 128)])
@pytest.mark.parametrize("k", [0, 10, 20, 30, 60])
def test_attention_over_v_scales_far_apart(k, dtype, fmt, d, order):
    """Each output against the bound of _attn_bound with its last term (p's smallest f16 step, against the
    head's largest |v|) replaced: where a wavefront's V scales lie within 2^w of each other (w = 8 for fp32
    rows, 14 for bf16 ones), p's half step 2^-25 times the reference scale is, against the sum of p of at
    least 2^7, n 2^(w - 32) of the weighted mean of each block's largest |v|; where they do not, p's rest
    enters as well, and a p is exact to 2^-11 and 2^-22 but for 2^-97 against a largest p of 2^(7 - 73) at
    this test's ratios (2^61 and the tail's) and more, far below the former."""
    w = 8 if dtype == "f32" else 14
    for m in (1, 6):
        cache = _far_scales_cache(dtype, fmt, d, k, order, 6)
        q = torch.zeros(m, 4, d, dtype=DT[dtype], device=DEV)
        # log2 of the weight of a small-V row over that of a large-V one: even, all small, balanced, all large
        lg = torch.tensor([0.0, 100.0, float(k), -100.0])
        q[:, :, 0] = (lg * 0.34657359).to(DEV) * torch.linspace(1, 0.9, m, device=DEV)[:, None]
        kk, v = cache.rows(0, 0)
        largest = np.abs(v).max(-1)
        for b in range(25):
            largest[32 * b:32 * b + 32] = np.abs(v[32 * b:32 * b + 32]).max()
        o, _, mag, size = paged.attend(_np(q), kk, v, 1.0)
        mean = paged.attend(_np(q), kk, largest[:, None], 1.0)[0]
        bound = _attn_bound(dtype, d, o, mag, size, v[:0]) + len(v) * 2.0 ** (w - 32) * mean
        for most in (809, 100000):
            ws = nx.new_paged_workspace(cache.cfg, cache.c, most, m)
            out = nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=ws, max_tokens=most, max_q=m, scale=1.0)
            nx.nx_read_device_status(cache.cfg, ws)
            err = np.abs(_np(out) - o)
            assert (err <= bound).all(), (m, most, float((err / bound).max()),
                                          [float((err / (mag + 1e-30)).max(axis=(0, 2))[i]) for i in range(4)])


def test_one_row_with_any_row_stride():
    c = [Cache(1, 2, 2, 64, "bf16", "e4m3", 1, 4) for _ in range(2)]
    x = _randn(7, 4, 64, dtype="bf16")
    got = []
    for row, other in zip((256, 1 << 40), c):
        other.fill([31, 40])
        k, q = (torch.as_strided(x, (1, n, 64), (row, 64, 1)) for n in (2, 4))
        nx.nx_paged_append(other.cfg, other.c, k, k, workspace=other.ws)
        n = nx.nx_qk_norm_rope(other.cfg, q, k, workspace=other.ws, q_weight=x[0], k_weight=x[1])
        o = torch.as_strided(torch.empty(256, dtype=torch.bfloat16, device=DEV), (1, 4, 64), (row, 64, 1))
        got.append((*n, nx.nx_paged_attn(other.cfg, other.c, q, workspace=other.ws, max_tokens=41, out=o),
                    *nx.nx_paged_gather(other.cfg, other.c, workspace=other.ws, max_tokens=41)))
        other.check()
    assert all(torch.equal(a, b) for a, b in zip(*got)) and other.c.lens.tolist() == [[32, 41]]
    _check_attn(other, q, [1], got[1][2])


@pytest.mark.parametrize("dtype,d,hkv,group,fmt", [("bf16", 128, 2, 4, "e4m3"), ("bf16", 64, 1, 8, "int8"),
                                                   ("f32", 128, 1, 2, "int8"), ("f32", 64, 2, 5, "e4m3")])
@pytest.mark.parametrize("m", [17, 65, 500])
def test_attention_of_long_query_windows(m, dtype, d, hkv, group, fmt):
    """Prompts and their last pieces, in 32-row tiles, whole heads and pieces: sequences that hold exactly the
    queries' rows, more, and fewer (the oldest queries see nothing); causal borders inside blocks, tiles and
    pieces."""
    cache = Cache(3, hkv, group, d, dtype, fmt, 2, 24, max_q=m)
    cache.fill([n - (7 * h if n > 7 else 0) for n in (m, 1500, max(1, m // 3)) for h in range(hkv)], seed=m)
    counts = [m, m, m - 1]
    q = _randn(110 + m, sum(counts), hkv * group, d, dtype=dtype)
    start = torch.tensor([0, m, 2 * m, 3 * m - 1], dtype=torch.int32, device=DEV)
    lse = torch.empty(len(q), hkv * group, device=DEV)
    for most in (1000, 1500, 60000):           # whole heads, pieces of the listed lengths, many small ones
        ws = nx.new_paged_workspace(cache.cfg, cache.c, most, m)
        out = nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=ws, max_tokens=most, max_q=m, q_start=start,
                               out_lse=lse)
        nx.nx_read_device_status(cache.cfg, ws)
        _check_attn(cache, q, counts, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_a_whole_prompt(dtype):
    """2048 queries over their own rows and 512 older ones."""
    cache = Cache(1, 1, 1, 64, dtype, "int8", 8, 10, max_q=2048)
    cache.fill([2560])
    q = _randn(120, 2048, 1, 64, dtype=dtype)
    out = nx.nx_paged_attn(cache.cfg, cache.c, q, workspace=cache.ws, max_tokens=2560)
    cache.check()
    _check_attn(cache, q, [2048], out)


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("f32", 128), ("bf16", 128)])
def test_a_tiny_v_scale_under_the_largest_logit(dtype, d):
    """One block holds nearly all of a row's weight and has a V scale far below (and zero, whose codes stand
    for zeros), in the first, a middle and the last block, in one wavefront and across pieces."""
    for at in (0, 20, 38):
        for scale in (2.0 ** -50, 0.0):
            cache = Cache(1, 1, 4, d, dtype, "int8", 1, 41, max_q=5)
            cache.fill([39 * 32 + 5], seed=8)
            page = int(cache.c.table[0, 0, at])
            cache.c.k_scale[page] *= 8
            cache.c.v_scale[page] = scale
            q = _randn(130, 5, 4, d, dtype=dtype)
            for m, most in ((1, 1253), (1, 50000), (5, 1000), (5, 50000)):
                ws = nx.new_paged_workspace(cache.cfg, cache.c, most, m)
                out = nx.nx_paged_attn(cache.cfg, cache.c, q[:m], workspace=ws, max_tokens=most, max_q=m)
                nx.nx_read_device_status(cache.cfg, ws)
                _check_attn(cache, q[:m], [m], out)


def test_one_workspace_serves_windows_of_every_size():
    """Made for the largest call; the calls of fewer queries cut their work otherwise."""
    cache = Cache(1, 2, 8, 64, "bf16", "e4m3", 4, 12, max_q=64)
    cache.fill([1500, 1333])
    q = _randn(140, 64, 16, 64, dtype="bf16")
    for m in (64, 57, 33, 16, 12, 9, 7, 2, 1, 64):
        out = nx.nx_paged_attn(cache.cfg, cache.c, q[:m], workspace=cache.ws, max_tokens=1500)
        cache.check()
        _check_attn(cache, q[:m], [m], out)


def test_gather_into_views_of_one_head_or_sequence():
    for s, h in ((1, 3), (3, 1), (1, 1)):
        cache = Cache(s, h, 1, 64, "bf16", "e4m3", 1, 4)
        cache.fill([40 + i for i in range(s * h)])
        k, v = nx.nx_paged_gather(cache.cfg, cache.c, workspace=cache.ws, max_tokens=44)
        a = [torch.zeros(s * h * 44 * 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        strides = (5 if s == 1 else 44 * 64, 7 if h == 1 else 44 * 64, 64, 1)
        o = [torch.as_strided(x, (s, h, 44, 64), strides) for x in a]
        nx.nx_paged_gather(cache.cfg, cache.c, workspace=cache.ws, max_tokens=44, out_k=o[0], out_v=o[1])
        cache.check()
        assert torch.equal(a[0], k.flatten()) and torch.equal(a[1], v.flatten())
