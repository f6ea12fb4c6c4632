"""Plain fp64 oracle of the decode-step operators (numpy; test infrastructure only).

The cache is kept the simple way: per (sequence, KV head) a list of whole blocks,
each (codes as values, scale) for K and V, and the list of rows past them.  The
definitions:

  norm    y = x w / sqrt(mean(x^2) + eps)
  rotate  (a, b) -> (a cos - b sin, b cos + a sin)
  append  rotate, round to the element type; a full block of 32 rows has
          scale amax * (1 / M) and codes rne(x * ((1 / amax) * M)), each
          operation rounded to fp32, M = 448 (e4m3) or 127 (int8)
  attend  softmax(scale q K^T) V over the rows t <= n - m + i of query i of m

Pins (tests/test_oracle_paged.py): torch's bf16 and e4m3 conversions, half a step
per quantised element, rotation invariants and a pair by hand, torch's softmax,
empty rows, appends in pieces.
"""

import math

import numpy as np

BLOCK = 32
TOP = {"e4m3": np.float32(448.0), "int8": np.float32(127.0)}


def round_to(x, dtype):
    """Rows as the element type holds them ("bf16" or "f32"), nearest even, as float64."""
    x = np.asarray(x, dtype=np.float64).astype(np.float32)
    if dtype == "f32":
        return x.astype(np.float64)
    b = x.view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def _e4m3_values():
    code = np.arange(127)
    e, m = code >> 3, code & 7
    return np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))


E4M3 = _e4m3_values()          # magnitudes of codes 0 .. 126, ascending


def to_codes(x, fmt):
    """The 8-bit values nearest to x (ties to the even code), as float64."""
    x = np.asarray(x, dtype=np.float64)
    if fmt == "int8":
        return np.rint(x)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(E4M3, a), 1, 126)
    lo = hi - 1
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    pick = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return np.copysign(E4M3[pick], x)


def quantise(block, fmt):
    """(code values, fp32 scale) of one block [32, D]."""
    top = np.float32(np.abs(block).max())
    if not top > np.float32(2.0 ** -100):
        return np.zeros_like(block), 0.0
    one = np.float32(1.0)
    inv = (one / top) * TOP[fmt]
    y = (block.astype(np.float32) * inv).astype(np.float64)
    return to_codes(y, fmt), float(top * (one / TOP[fmt]))


def rotate(x, cos_sin, pairs):
    """Rows x [rows, heads, D] turned by cos_sin [rows, rot]."""
    x = np.array(x, dtype=np.float64)
    rot = cos_sin.shape[1]
    c = cos_sin[:, None, :rot // 2].astype(np.float64)
    s = cos_sin[:, None, rot // 2:].astype(np.float64)
    ia = np.arange(0, rot, 2) if pairs else np.arange(rot // 2)
    ib = ia + 1 if pairs else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x


def norm_rope(x, weight, eps, cos_sin=None, pairs=False):
    """Unrounded norm (weight None: none) and rotation of rows [rows, heads, D]."""
    x = np.asarray(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    return x if cos_sin is None else rotate(x, cos_sin, pairs)


class Head:
    """One (sequence, KV head) of the cache."""

    def __init__(self, head_dim, dtype, fmt):
        self.d, self.dtype, self.fmt = head_dim, dtype, fmt
        self.blocks = []                 # ((k codes, k scale), (v codes, v scale))
        self.tail = [], []               # K rows, V rows

    def __len__(self):
        return BLOCK * len(self.blocks) + len(self.tail[0])

    def append(self, k, v):
        """Rows k, v [rows, D], already rotated; a non-finite element becomes 0."""
        for row in zip(*(round_to(x, self.dtype) for x in (k, v))):
            for side, x in zip(self.tail, row):
                side.append(np.where(np.isfinite(x), x, 0.0))
            if len(self.tail[0]) == BLOCK:
                self.blocks.append(tuple(quantise(np.stack(t), self.fmt) for t in self.tail))
                self.tail = [], []

    def rows(self):
        """(K, V) [rows, D] as the cache stands for them."""
        out = []
        for i in range(2):
            parts = [b[i][0] * b[i][1] for b in self.blocks]
            if self.tail[i]:
                parts.append(np.stack(self.tail[i]))
            out.append(np.concatenate(parts) if parts else np.zeros((0, self.d)))
        return out

    def attend(self, q, scale=None):
        """q [queries, group, D] -> (out, lse, sum p |v| / sum p, the largest sum |q||k| scale)."""
        k, v = self.rows()
        return attend(q, k, v, scale)


def attend(q, k, v, scale=None):
    q = np.asarray(q, dtype=np.float64)
    m, grp, d = q.shape
    n = len(k)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out, mag = np.zeros((m, grp, d)), np.zeros((m, grp, d))
    lse, size = np.full((m, grp), -np.inf), np.zeros((m, grp))
    for i in range(m):
        e = n - m + i + 1
        if e <= 0:
            continue
        x = q[i] @ k[:e].T * scale
        top = x.max(-1, keepdims=True)
        p = np.exp(x - top)
        s = p.sum(-1, keepdims=True)
        out[i] = p @ v[:e] / s
        mag[i] = p @ np.abs(v[:e]) / s
        lse[i] = (top + np.log(s))[:, 0]
        size[i] = (np.abs(q[i]) @ np.abs(k[:e]).T).max(-1) * abs(scale)
    return out, lse, mag, size
