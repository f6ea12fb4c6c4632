"""Torch-facing binding of the decode-step operators: checks and marshalling, no arithmetic.

Between two eviction events each new token is normed and rotated
(nx_qk_norm_rope), appended to a paged 8-bit cache (nx_paged_append) and attended
over it (nx_paged_attn); nx_paged_gather reads the rows back for the next event.
The functions mirror include/nexus.h; shapes and the element type come from the
NexusConfig of the eviction calls.  Work is enqueued on the current stream of
the tensors' device (or the given stream, on which outputs that are not given are
made too; ordering that stream behind the inputs is the caller's).
"""

import ctypes
from dataclasses import dataclass, field, replace

import torch

from ._lib import (NX_CACHE_BLOCK, NX_CACHE_E4M3, NX_CACHE_I8, NX_ROPE_HALF, NX_ROPE_PAIRS, NxDesc,
                   NxPaged, NxRope, NxRows, check, load)
from .api import _DTYPES, NexusConfig

_FORMATS = {torch.float8_e4m3fn: NX_CACHE_E4M3, torch.int8: NX_CACHE_I8}
_NAMES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
_FIXED = frozenset(("cfg", "k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail", "table", "lens"))


# The checks run on every call of a decode step, whose kernels take a few
# microseconds: one comparison of each property, the message made only on failure.

def _bad(t, name, shape, dtype, index):
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the cache or the queries are not")
    raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}, contiguous")


def _tensor(t, name, shape, dtype, index):
    """Address of a whole contiguous tensor."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _bad(t, name, shape, dtype, index)
    return t.data_ptr()


def _opt(t, name, shape, dtype, index):
    return None if t is None else _tensor(t, name, shape, dtype, index)


def _rows(cfg, t, name, heads, index, n):
    """NxRows of an [n, heads, head_dim] tensor with any row and head strides."""
    if t.dtype is not cfg.dtype or t.shape != (n, heads, cfg.head_dim) or t.get_device() != index:
        _bad(t, name, (n, heads, cfg.head_dim), cfg.dtype, index)
    row, head, elem = t.stride()
    if elem != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    return NxRows(t.data_ptr(), row, head)


def _stream(stream, index):
    """Handle of the given stream, or of the current one of GPU `index`."""
    if index < 0:
        raise ValueError("the tensors must be on a GPU")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors on GPU {index}")
    return stream.cuda_stream


def _new(make, stream):
    """A default output, made on the stream that the call runs on: its memory (and its fill)
    belongs to that stream's order."""
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        return make()


def _run(index, fn, *args):
    """fn with GPU `index` current."""
    if torch._C._cuda_getDevice() == index:
        return fn(*args)
    with torch.cuda.device(index):
        return fn(*args)


@dataclass
class Rope:
    """Rotation table: cos_sin [n_pos, rot_dim] float32 (rot_dim / 2 cosines, then the
    sines); pairs=False turns elements (i, i + rot_dim / 2), pairs=True (2 i, 2 i + 1)."""
    cos_sin: torch.Tensor
    pairs: bool = False

    def __setattr__(self, name, t):       # also where the table is replaced later
        if name == "cos_sin" and (t.dim() != 2 or t.dtype != torch.float32 or not t.is_contiguous()):
            raise ValueError("cos_sin must be a contiguous float32 [n_pos, rot_dim] tensor")
        object.__setattr__(self, name, t)

    def _struct(self, positions, n_rows, index):
        t = self.cos_sin
        if t.get_device() != index:
            raise ValueError(f"cos_sin is on {t.device}, the rows are not")
        n_pos, rot = t.shape
        return NxRope(t.data_ptr(), _opt(positions, "positions", (n_rows,), torch.int32, index), n_pos, rot,
                      NX_ROPE_PAIRS if self.pairs else NX_ROPE_HALF)


def rope_table(n_pos, rot_dim, base=10000.0, *, inv_freq=None, first=0, device="cuda"):
    """cos_sin table of positions first .. first + n_pos - 1, angles in float64.

    inv_freq: the rot_dim / 2 frequencies (default base ** (-2 i / rot_dim))."""
    if inv_freq is None:
        i = torch.arange(rot_dim // 2, dtype=torch.float64, device=device)
        inv_freq = float(base) ** (-2.0 * i / rot_dim)
    inv_freq = torch.as_tensor(inv_freq, dtype=torch.float64, device=device)
    pos = torch.arange(first, first + n_pos, dtype=torch.float64, device=device)
    angle = pos[:, None] * inv_freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


@dataclass
class PagedCache:
    """The arrays of one paged 8-bit cache (layouts in include/nexus.h, nx_paged).

    The format is the dtype of the codes (float8_e4m3fn or int8).  table and
    lens may be rewritten between calls (in place); the arrays themselves stay
    (assigning another raises AttributeError: make another PagedCache)."""
    cfg: NexusConfig
    k_codes: torch.Tensor      # [n_pages, page_blocks, 32, D]
    v_codes: torch.Tensor      # [n_pages, page_blocks, 4, D, 8]
    k_scale: torch.Tensor      # [n_pages, page_blocks] float32
    v_scale: torch.Tensor
    k_tail: torch.Tensor       # [n_seqs, n_kv_heads, 32, D] of cfg.dtype
    v_tail: torch.Tensor       # [n_seqs, n_kv_heads, 4, D, 8]
    table: torch.Tensor        # [n_seqs, n_kv_heads, max_pages] int32
    lens: torch.Tensor         # [n_seqs, n_kv_heads] int32
    _c: NxPaged = field(init=False, repr=False, compare=False, default=None)

    def __post_init__(self):
        cfg, d, hk = self.cfg, self.cfg.head_dim, self.cfg.n_kv_heads
        if self.k_codes.dtype not in _FORMATS:
            raise TypeError(f"k_codes: dtype {self.k_codes.dtype}, expected one of {list(_FORMATS)}")
        if self.k_codes.dim() != 4 or self.table.dim() != 3:
            raise ValueError("k_codes must be [n_pages, page_blocks, 32, head_dim], table "
                             "[n_seqs, n_kv_heads, max_pages]")
        n_pages, blocks = self.k_codes.shape[:2]
        n_seqs, _, max_pages = self.table.shape
        dev, f8 = self.k_codes.get_device(), self.k_codes.dtype
        self.device, self.n_seqs, self._index = self.k_codes.device, n_seqs, dev
        self.capacity = max_pages * blocks * NX_CACHE_BLOCK      # rows that a head's table can hold
        c = NxPaged()
        c.n_seqs, c.n_q_heads, c.n_kv_heads, c.head_dim = n_seqs, cfg.n_q_heads, hk, d
        c.dtype, c.format = _DTYPES.get(cfg.dtype, 99), _FORMATS[f8]
        c.page_blocks, c.n_pages, c.max_pages = blocks, n_pages, max_pages
        c.k_codes = _tensor(self.k_codes, "k_codes", (n_pages, blocks, NX_CACHE_BLOCK, d), f8, dev)
        c.v_codes = _tensor(self.v_codes, "v_codes", (n_pages, blocks, 4, d, 8), f8, dev)
        c.k_scale = _tensor(self.k_scale, "k_scale", (n_pages, blocks), torch.float32, dev)
        c.v_scale = _tensor(self.v_scale, "v_scale", (n_pages, blocks), torch.float32, dev)
        c.k_tail = _tensor(self.k_tail, "k_tail", (n_seqs, hk, NX_CACHE_BLOCK, d), cfg.dtype, dev)
        c.v_tail = _tensor(self.v_tail, "v_tail", (n_seqs, hk, 4, d, 8), cfg.dtype, dev)
        c.table = _tensor(self.table, "table", (n_seqs, hk, max_pages), torch.int32, dev)
        c.lens = _tensor(self.lens, "lens", (n_seqs, hk), torch.int32, dev)
        # The shape that _c holds, whatever becomes of the caller's object.
        self._cfg = replace(cfg)
        self._c = c

    def __setattr__(self, name, value):
        # The calls pass the addresses that _c took.
        if name in _FIXED and self._c is not None and value is not getattr(self, name):
            raise AttributeError(f"PagedCache.{name} cannot be replaced: write into it, or make another cache")
        object.__setattr__(self, name, value)

    def _same(self, cfg):
        if cfg != self.cfg:
            raise ValueError("the cache was made for another configuration")

    def _struct(self, cfg, workspace, stream):
        if cfg is not self.cfg:
            self._same(cfg)
        if workspace.get_device() != self._index or not workspace.is_contiguous():
            raise ValueError(f"the workspace must be contiguous on {self.device}")
        # A copy: calls from several threads share the cache object.
        c = NxPaged.from_buffer_copy(self._c)
        c.workspace = workspace.data_ptr()
        c.workspace_bytes = workspace.nbytes
        c.stream = _stream(stream, self._index)
        return c


def new_paged_cache(cfg, n_seqs, n_pages, max_pages, *, fmt="e4m3", page_blocks=4, device="cuda"):
    """An empty cache: zero lengths, and a table whose entries are -1 (no page) until the
    caller hands pages out."""
    if fmt not in _NAMES:
        raise ValueError(f"fmt {fmt!r}, expected one of {sorted(_NAMES)}")
    d, hk = cfg.head_dim, cfg.n_kv_heads

    def zeros(*shape, dtype):
        return torch.zeros(shape, dtype=dtype, device=device)

    codes = [zeros(n_pages, page_blocks, NX_CACHE_BLOCK * d, dtype=torch.uint8).view(_NAMES[fmt])
             for _ in range(2)]
    return PagedCache(
        cfg, codes[0].view(n_pages, page_blocks, NX_CACHE_BLOCK, d),
        codes[1].view(n_pages, page_blocks, 4, d, 8),
        zeros(n_pages, page_blocks, dtype=torch.float32), zeros(n_pages, page_blocks, dtype=torch.float32),
        zeros(n_seqs, hk, NX_CACHE_BLOCK, d, dtype=cfg.dtype), zeros(n_seqs, hk, 4, d, 8, dtype=cfg.dtype),
        zeros(n_seqs, hk, max_pages, dtype=torch.int32) - 1, zeros(n_seqs, hk, dtype=torch.int32))


def paged_workspace_bytes(cfg, cache, max_tokens, max_q=1):
    """Bytes for calls on `cache` of up to max_tokens rows a head and max_q queries a sequence."""
    cache._same(cfg)
    c = NxPaged.from_buffer_copy(cache._c)
    n = load().nx_paged_workspace_bytes(ctypes.byref(c), max_tokens, max_q)
    if n == 0:
        raise ValueError("invalid shape for the workspace query")
    return n


def new_paged_workspace(cfg, cache, max_tokens, max_q=1):
    """Zero-filled workspace of the nx_paged_* calls (nx_read_device_status reads its status)."""
    return torch.zeros(paged_workspace_bytes(cfg, cache, max_tokens, max_q), dtype=torch.uint8,
                       device=cache.device)


def nx_qk_norm_rope(cfg, q, k=None, *, workspace, q_weight=None, k_weight=None, eps=1e-6, rope=None,
                    positions=None, out_q=None, out_k=None, stream=None):
    """Root-mean-square norm of every head of q [rows, n_q_heads, D] and k
    [rows, n_kv_heads, D], then the rotation; returns (out_q, out_k).

    A side without a weight is rotated only; rope None: no rotation.  Outputs
    may be views with other strides (a query window, a cache's append rows) or
    the inputs themselves."""
    dev, n, hq, hk, d = q.get_device(), q.shape[0], cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim
    rq = _rows(cfg, q, "q", hq, dev, n)
    if out_q is None:
        out_q = _new(lambda: torch.empty(n, hq, d, dtype=cfg.dtype, device=q.device), stream)
    roq = _rows(cfg, out_q, "out_q", hq, dev, n)
    rk = rok = None
    if k is not None:
        rk = _rows(cfg, k, "k", hk, dev, n)
        if out_k is None:
            out_k = _new(lambda: torch.empty(n, hk, d, dtype=cfg.dtype, device=q.device), stream)
        rok = _rows(cfg, out_k, "out_k", hk, dev, n)
    elif out_k is not None:
        raise ValueError("out_k without k")
    wq = _opt(q_weight, "q_weight", (d,), cfg.dtype, dev)
    wk = _opt(k_weight, "k_weight", (d,), cfg.dtype, dev)
    if rope is None and positions is not None:
        raise ValueError("positions without rope")
    r = None if rope is None else rope._struct(positions, n, dev)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be contiguous on {q.device}")
    c = NxDesc()
    c.n_q_heads, c.n_kv_heads, c.head_dim, c.dtype = hq, hk, d, _DTYPES.get(cfg.dtype, 99)
    c.workspace, c.workspace_bytes, c.stream = workspace.data_ptr(), workspace.nbytes, _stream(stream, dev)
    check(_run(dev, load().nx_qk_norm_rope, c, r, n, rq, roq, wq, rk, rok, wk, eps), "nx_qk_norm_rope")
    return out_q, out_k


def _per_seq(cache, n, most, starts, most_name, starts_name):
    """The given bound on a sequence's rows, or the even division of n rows."""
    if most is not None:
        return most
    if starts is not None:
        raise ValueError(f"{starts_name} needs {most_name}")
    if n % cache.n_seqs:
        raise ValueError(f"{n} rows do not divide into {cache.n_seqs} sequences")
    return n // cache.n_seqs


def nx_paged_append(cfg, cache, k, v, *, workspace, max_new=None, new_start=None, head_new=None,
                    rope=None, positions=None, lens_out=None, stream=None):
    """Appends rows k, v [rows, n_kv_heads, D] (K rotated by `rope`) to every sequence.

    new_start: int32 [n_seqs + 1] first rows of the sequences (None: max_new rows each,
    default rows // n_seqs); head_new: int32 [n_seqs, n_kv_heads] rows each head takes of
    its sequence's; lens_out: int32 [n_seqs, n_kv_heads] (None: cache.lens is advanced)."""
    own, dev, n, s = cache._cfg, cache._index, k.shape[0], cache.n_seqs
    hk = own.n_kv_heads
    rk = _rows(own, k, "k", hk, dev, n)
    rv = _rows(own, v, "v", hk, dev, n)
    max_new = _per_seq(cache, n, max_new, new_start, "max_new", "new_start")
    ns = _opt(new_start, "new_start", (s + 1,), torch.int32, dev)
    hn = _opt(head_new, "head_new", (s, hk), torch.int32, dev)
    lo = _opt(lens_out, "lens_out", (s, hk), torch.int32, dev)
    if rope is None and positions is not None:
        raise ValueError("positions without rope")
    r = None if rope is None else rope._struct(positions, n, dev)
    c = cache._struct(cfg, workspace, stream)
    check(_run(dev, load().nx_paged_append, c, r, rk, rv, n, ns, hn, max_new, lo), "nx_paged_append")


def nx_paged_attn(cfg, cache, q, *, workspace, max_tokens, max_q=None, q_start=None, scale=None,
                  out=None, out_lse=None, stream=None):
    """Attention of q [rows, n_q_heads, D] over the cache; returns out of q's shape.

    q_start: int32 [n_seqs + 1] first query rows of the sequences (None: max_q each, default
    rows // n_seqs); max_tokens: the expected longest head (any value is correct, and the
    workspace must have been made for at least it); out_lse: float32 [rows, n_q_heads]."""
    own, dev, n = cache._cfg, cache._index, q.shape[0]
    hq = own.n_q_heads
    rq = _rows(own, q, "q", hq, dev, n)
    if out is None:
        out = _new(lambda: torch.empty(n, hq, own.head_dim, dtype=own.dtype, device=q.device), stream)
    ro = _rows(own, out, "out", hq, dev, n)
    max_q = _per_seq(cache, n, max_q, q_start, "max_q", "q_start") if n else 1      # no rows: nothing is done
    if scale is not None and not scale > 0:
        raise ValueError("scale must be positive")
    qs = _opt(q_start, "q_start", (cache.n_seqs + 1,), torch.int32, dev)
    lse = _opt(out_lse, "out_lse", (n, hq), torch.float32, dev)
    c = cache._struct(cfg, workspace, stream)
    check(_run(dev, load().nx_paged_attn, c, rq, ro, n, qs, max_tokens, max_q, scale or 0.0, lse),
          "nx_paged_attn")
    return out


def nx_paged_gather(cfg, cache, *, workspace, max_tokens, out_k=None, out_v=None, stream=None):
    """The cached rows as [n_seqs, n_kv_heads, >= max_tokens, D] tensors (rows past a head's
    length are left as they were; new outputs are zero-filled); returns (out_k, out_v)."""
    own, d = cache._cfg, cache._cfg.head_dim
    shape = cache.n_seqs, own.n_kv_heads, max_tokens, d
    if out_k is None:
        out_k = _new(lambda: torch.zeros(shape, dtype=own.dtype, device=cache.device), stream)
    if out_v is None:
        out_v = _new(lambda: torch.zeros_like(out_k), stream)
    for t, name in ((out_k, "out_k"), (out_v, "out_v")):
        got, st = t.shape, t.stride()
        if t.dtype is not own.dtype or len(got) != 4 or got[:2] != shape[:2] or got[2] < max_tokens or \
                got[3] != d or t.get_device() != cache._index:
            _bad(t, name, shape, own.dtype, cache._index)
        if st[3] != 1 or st[2] != d:
            raise ValueError(f"{name}: rows must be contiguous")
    if out_k.stride() != out_v.stride():
        raise ValueError("out_k and out_v must share their strides")
    c = cache._struct(cfg, workspace, stream)
    check(_run(cache._index, load().nx_paged_gather, c, max_tokens, out_k.data_ptr(), out_v.data_ptr(),
               st[0], st[1]), "nx_paged_gather")
    return out_k, out_v
