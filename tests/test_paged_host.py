"""Host-side validation of the decode-step entry points: bad arguments are refused
before anything reaches a GPU (no launch is made here)."""

import ctypes
import os
import subprocess

import pytest
import torch

import streaming_weighted_sampling_amd as nx
from streaming_weighted_sampling_amd import _lib
from streaming_weighted_sampling_amd._lib import NxDesc, NxPaged, NxRope, NxRows

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 40          # never dereferenced
GB = 1 << 32
EINVAL, EALIAS, EWORK, EUNSUP = (_lib.NX_EINVAL, _lib.NX_EALIAS, _lib.NX_EWORKSPACE,
                                 _lib.NX_EUNSUPPORTED)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libnexus.so not built")
    return _lib.load()


def _cache(**kw):
    c = NxPaged()
    c.n_seqs, c.n_q_heads, c.n_kv_heads, c.head_dim = 4, 32, 8, 128
    c.dtype, c.format, c.page_blocks, c.n_pages, c.max_pages = _lib.NX_BF16, _lib.NX_CACHE_E4M3, 4, 1024, 16
    for i, name in enumerate(("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail", "table", "lens",
                              "workspace")):
        setattr(c, name, FAKE + i * GB)
    c.workspace_bytes = 0        # below 256: every valid call ends with NX_EWORKSPACE, unlaunched
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _r(slot, row=8 * 128, head=128):
    return NxRows(FAKE + slot * GB, row, head)


def test_struct_layouts_match_c(tmp_path):
    src = tmp_path / "layout.c"
    names = {"nx_paged": NxPaged, "nx_rope": NxRope, "nx_rows": NxRows}
    lines = [f'printf("{n} %zu\\n", sizeof({n}));' for n in names]
    lines += [f'printf("{n}.{f} %zu\\n", offsetof({n}, {f}));' for n, t in names.items() for f, _ in t._fields_]
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"nexus.h\"\nint main(void) {\n"
                   + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    for line in out.splitlines():
        name, n = line.rsplit(" ", 1)
        t, _, f = name.partition(".")
        assert int(n) == (getattr(names[t], f).offset if f else ctypes.sizeof(names[t])), name


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=0), EINVAL), (dict(n_q_heads=30), EINVAL), (dict(n_kv_heads=0), EINVAL),
    (dict(n_pages=0), EINVAL), (dict(max_pages=0), EINVAL), (dict(page_blocks=0), EINVAL),
    (dict(page_blocks=3), EUNSUP), (dict(page_blocks=2048), EUNSUP), (dict(head_dim=96), EUNSUP),
    (dict(dtype=2), EUNSUP), (dict(format=2), EUNSUP), (dict(n_seqs=9000), EUNSUP),
    (dict(n_pages=1 << 30, page_blocks=4), EUNSUP), (dict(n_q_heads=8 * 257), EUNSUP),
    (dict(k_codes=None), EINVAL), (dict(v_codes=None), EINVAL), (dict(k_scale=None), EINVAL),
    (dict(v_tail=None), EINVAL), (dict(table=None), EINVAL), (dict(lens=None), EINVAL),
    (dict(k_codes=FAKE + 8), EUNSUP), (dict(v_tail=FAKE + 2), EUNSUP), (dict(workspace=None), EWORK),
    (dict(), EWORK)])
def test_cache_descriptions(lib, kw, code):
    c = _cache(**kw)
    assert lib.nx_paged_append(c, None, _r(20), _r(21), 4, None, None, 1, None) == code
    assert lib.nx_paged_attn(c, _r(20, 4096), _r(21, 4096), 4, None, 100, 1, 0.0, None) == code
    assert lib.nx_paged_gather(c, 100, FAKE + 30 * GB, FAKE + 31 * GB, 8 * 12800, 12800) == code
    assert lib.nx_paged_append(None, None, _r(20), _r(21), 4, None, None, 1, None) == EINVAL


def _ws(**kw):
    return _cache(workspace_bytes=256, **kw)


def test_append_arguments(lib):
    def call(c=None, rope=None, k=_r(20), v=_r(21), n=4, start=None, head_new=None, most=1, out=None):
        return lib.nx_paged_append(c or _ws(), rope, k, v, n, start, head_new, most, out)
    assert call(k=None) == EINVAL
    assert call(k=NxRows(None, 1024, 128)) == EINVAL
    assert call(n=-1) == EINVAL
    assert call(most=-1) == EINVAL
    assert call(most=2) == EINVAL                         # 4 sequences x 2 rows > 4 rows
    assert call(k=_r(20, row=1028)) == EUNSUP             # not a multiple of 16 bytes
    assert call(v=_r(20, head=-128)) == EINVAL
    assert call(k=NxRows(FAKE + 20 * GB + 8, 1024, 128)) == EUNSUP
    assert call(k=_r(0)) == EALIAS                        # new rows inside the codes
    assert call(v=_r(5)) == EALIAS
    assert call(c=_ws(v_codes=FAKE + 4096)) == EALIAS     # codes overlap each other
    assert call(c=_ws(k_scale=FAKE + 4096)) == EALIAS
    assert call(out=FAKE + 7 * GB + 4) == EALIAS          # shifted against lens
    assert call(out=FAKE + 6 * GB) == EALIAS              # the table
    assert call(head_new=FAKE + 7 * GB) == EALIAS         # lens, advanced in place, as the counts to add
    assert call(start=FAKE + 41 * GB, out=FAKE + 41 * GB + 16) == EALIAS
    assert call(out=FAKE + 8 * GB) == EALIAS              # the status word
    assert call(k=_r(20, row=1 << 25)) == EUNSUP          # a row stride of 64 MB
    inside = NxRope(FAKE + 4096, None, 10, 64, 0)         # a table inside the codes
    assert call(rope=inside) == EALIAS
    for kw, code in ((dict(rot_dim=24), EUNSUP), (dict(rot_dim=144), EINVAL), (dict(rot_dim=-16), EINVAL),
                     (dict(n_pos=0), EINVAL), (dict(style=2), EINVAL), (dict(cos_sin=None), EINVAL),
                     (dict(cos_sin=FAKE + 4), EUNSUP)):
        f = dict(cos_sin=FAKE + 40 * GB, positions=None, n_pos=10, rot_dim=64, style=0) | kw
        rope = NxRope(f["cos_sin"], f["positions"], f["n_pos"], f["rot_dim"], f["style"])
        assert call(rope=rope) == code, kw


def test_attention_arguments(lib):
    def call(c=None, q=_r(20, 4096), o=_r(21, 4096), n=4, start=None, t=100, m=1, scale=0.0, lse=None):
        return lib.nx_paged_attn(c or _ws(), q, o, n, start, t, m, scale, lse)
    assert call(m=0) == EINVAL
    assert call(m=2) == EINVAL                            # more rows than there are
    assert call(t=-1) == EINVAL
    assert call(t=1 << 25) == EUNSUP
    assert call(scale=-1.0) == EINVAL
    assert call(scale=float("nan")) == EINVAL
    assert call(o=_r(20, 4096)) == EALIAS
    assert call(o=_r(21, 128)) == EINVAL                  # output rows on top of each other
    assert call(o=_r(21, 4096, 0)) == EINVAL
    assert call(o=_r(4, 4096)) == EALIAS                  # into the tail
    assert call(lse=FAKE + 21 * GB) == EALIAS
    for lo in (6, 7, 8):                                  # table, lens, workspace
        assert call(lse=FAKE + lo * GB) == EALIAS
        assert call(o=_r(lo, 4096)) == EALIAS
    assert call(start=FAKE + 21 * GB + 8192) == EALIAS
    assert call() == EWORK                                # 256 bytes hold no partials
    assert call(n=0, m=0) == EINVAL
    assert call(n=1 << 30, m=1 << 20, start=FAKE + 40 * GB) == EUNSUP      # rows of one head: 2^22
    # slices of one projection do not overlap: the call gets as far as the workspace
    one = NxRows(FAKE + 20 * GB, 3 * 4096, 128)
    two = NxRows(FAKE + 20 * GB + 2 * 4096, 3 * 4096, 128)
    assert call(q=one, o=two) == EWORK
    assert call(q=one, o=NxRows(FAKE + 20 * GB + 4096, 3 * 4096, 128)) == EALIAS


def test_gather_arguments(lib):
    def call(c=None, t=100, k=FAKE + 30 * GB, v=FAKE + 31 * GB, ss=8 * 12800, hs=12800):
        return lib.nx_paged_gather(c or _ws(), t, k, v, ss, hs)
    assert call(k=None) == EINVAL
    assert call(t=-1) == EINVAL
    assert call(t=101) == EINVAL                          # head stride below max_tokens rows
    assert call(ss=12800) == EINVAL
    assert call(v=FAKE + 30 * GB + 4096) == EALIAS
    assert call(k=FAKE) == EALIAS
    assert call(k=FAKE + 30 * GB + 8) == EUNSUP
    assert call(v=FAKE + 7 * GB) == EALIAS                # the row counts
    assert call(t=0, hs=0, ss=0) == _lib.NX_OK            # nothing to do


def test_norm_rope_arguments(lib):
    def desc(**kw):
        d = NxDesc()
        d.n_q_heads, d.n_kv_heads, d.head_dim, d.window, d.dtype = 32, 8, 128, 1, _lib.NX_BF16
        d.workspace, d.workspace_bytes = FAKE, 256
        for k, v in kw.items():
            setattr(d, k, v)
        return d

    def call(d=None, n=4, q=_r(20, 4096), oq=_r(21, 4096), wq=None, k=None, ok=None, wk=None, eps=1e-6):
        return lib.nx_qk_norm_rope(d or desc(), None, n, q, oq, wq, k, ok, wk, eps)
    assert lib.nx_qk_norm_rope(None, None, 4, _r(20), _r(21), None, None, None, None, 1e-6) == EINVAL
    assert call(n=-1) == EINVAL
    assert call(n=0) == _lib.NX_OK
    assert call(q=None) == EINVAL
    assert call(eps=-1.0) == EINVAL
    assert call(eps=float("inf")) == EINVAL
    assert call(d=desc(dtype=5)) == EUNSUP
    assert call(d=desc(head_dim=80)) == EUNSUP
    assert call(d=desc(workspace=None)) == EWORK
    assert call(k=_r(22)) == EINVAL                       # k without out_k
    assert call(wk=FAKE) == EINVAL                        # a weight without k
    assert call(wq=FAKE + 4) == EUNSUP
    assert call(oq=NxRows(FAKE + 20 * GB + 256, 4096, 128)) == EALIAS
    assert call(oq=_r(0, 4096)) == EALIAS                 # the workspace
    assert call(oq=_r(21, 128)) == EINVAL
    assert call(k=_r(22), ok=_r(21)) == EALIAS            # out_k on out_q


def test_workspace_query(lib):
    c = _cache()
    small = lib.nx_paged_workspace_bytes(c, 819, 1)
    assert 256 < small <= lib.nx_paged_workspace_bytes(c, 32768, 1)
    assert lib.nx_paged_workspace_bytes(c, 32768, 1) <= lib.nx_paged_workspace_bytes(c, 32768, 64)
    assert lib.nx_paged_workspace_bytes(None, 100, 1) == 0
    assert lib.nx_paged_workspace_bytes(c, -1, 1) == 0
    assert lib.nx_paged_workspace_bytes(c, 100, 0) == 0
    assert lib.nx_paged_workspace_bytes(_cache(head_dim=32), 100, 1) == 0


def test_the_binding_checks_tensors():
    cfg = nx.NexusConfig(4, 2, 64, 1, torch.bfloat16)
    c = nx.new_paged_cache(cfg, 3, 8, 2, device="cpu")
    assert c.capacity == 2 * 4 * 32 and (c.table == -1).all() and c.n_seqs == 3
    ws = torch.zeros(256, dtype=torch.uint8)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        nx.nx_paged_append(cfg, c, k, k, workspace=ws)
    with pytest.raises(TypeError):
        nx.nx_paged_append(cfg, c, k.float(), k, workspace=ws)
    with pytest.raises(ValueError, match="shape"):
        nx.nx_paged_append(cfg, c, k[:, :1], k, workspace=ws)
    with pytest.raises(ValueError, match="divide"):
        nx.nx_paged_append(cfg, c, k[:2], k[:2], workspace=ws)
    with pytest.raises(ValueError, match="contiguous"):
        nx.nx_paged_append(cfg, c, torch.zeros(3, 2, 128, dtype=torch.bfloat16)[..., ::2], k, workspace=ws)
    with pytest.raises(ValueError, match="max_new"):
        nx.nx_paged_append(cfg, c, k, k, workspace=ws, new_start=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(TypeError):
        nx.nx_paged_append(cfg, c, k, k, workspace=ws, lens_out=torch.zeros(3, 2))
    with pytest.raises(ValueError, match="configuration"):
        nx.nx_paged_append(nx.NexusConfig(8, 2, 64, 1), c, k, k, workspace=ws)
    with pytest.raises(ValueError, match="positions"):
        nx.nx_paged_append(cfg, c, k, k, workspace=ws, positions=torch.zeros(3, dtype=torch.int32))
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="scale"):
        nx.nx_paged_attn(cfg, c, q, workspace=ws, max_tokens=5, scale=0.0)
    with pytest.raises(ValueError, match="out"):
        nx.nx_paged_attn(cfg, c, q, workspace=ws, max_tokens=5, out=q[:2])
    with pytest.raises(ValueError, match="strides"):
        nx.nx_paged_gather(cfg, c, workspace=ws, max_tokens=5,
                           out_k=torch.zeros(3, 2, 5, 64, dtype=torch.bfloat16),
                           out_v=torch.zeros(3, 2, 9, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="out_k"):
        nx.nx_qk_norm_rope(cfg, q, workspace=ws, out_k=q)
    with pytest.raises(ValueError):
        nx.new_paged_cache(cfg, 3, 8, 2, fmt="e5m2", device="cpu")
    with pytest.raises(ValueError, match="cos_sin"):
        nx.Rope(torch.zeros(4, 16, dtype=torch.float64))
    with pytest.raises(ValueError, match="v_codes"):
        nx.PagedCache(cfg, c.k_codes, c.k_codes, c.k_scale, c.v_scale, c.k_tail, c.v_tail, c.table, c.lens)


def test_rope_table_holds_fp64_angles():
    t = nx.rope_table(5, 8, 100.0, first=100000, device="cpu").double()
    i = torch.arange(4, dtype=torch.float64)
    a = torch.arange(100000, 100005, dtype=torch.float64)[:, None] * 100.0 ** (-i / 4)
    assert torch.allclose(t[:, :4], a.cos(), atol=1e-7) and torch.allclose(t[:, 4:], a.sin(), atol=1e-7)


@pytest.mark.parametrize("hq,hkv", [(64, 8), (40, 8), (8, 8), (5, 1), (32, 1), (256, 1)])
@pytest.mark.parametrize("tokens", [0, 100, 1500, 32768])
def test_a_workspace_serves_every_smaller_call(lib, hq, hkv, tokens):
    """The size never falls with max_q or max_tokens, and a call of fewer queries passes the check
    (it has no rows, so nothing is launched)."""
    for n_seqs in (1, 4, 200):
        c = _cache(n_seqs=n_seqs, n_q_heads=hq, n_kv_heads=hkv)
        sizes = [lib.nx_paged_workspace_bytes(c, tokens, m) for m in range(1, 200)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:]))
        assert sizes[-1] <= lib.nx_paged_workspace_bytes(c, tokens, 4096)
        assert all(lib.nx_paged_workspace_bytes(c, t, 17) <= sizes[16] for t in (0, tokens // 3, tokens))
        for most in (16, 64, 150):
            c.workspace_bytes = sizes[most - 1]
            for m in range(1, most + 1):
                for t in (tokens // 2, tokens):
                    assert lib.nx_paged_attn(c, _r(20, 1 << 16), _r(21, 1 << 16), 0, None, t, m, 0.0,
                                             None) == _lib.NX_OK, (most, m, t)


def test_default_outputs_are_made_on_the_given_stream(monkeypatch):
    """Memory made on one stream and written on another could still be in use there, and a fill on
    the one could land on top of the other's result."""
    import contextlib

    from streaming_weighted_sampling_amd import paged
    cfg = nx.NexusConfig(4, 2, 64, 1, torch.bfloat16)
    c = nx.new_paged_cache(cfg, 3, 8, 2, device="cpu")
    ws, q, k = torch.zeros(4096, dtype=torch.uint8), torch.zeros(3, 4, 64).bfloat16(), torch.zeros(3, 2, 64).bfloat16()
    current, made = [None], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def noting(make):
        def f(*a, **kw):
            made.append(current[-1])
            return make(*a, **kw)
        return f

    monkeypatch.setattr(paged, "_run", lambda *a: 0)
    monkeypatch.setattr(paged, "_stream", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "stream", on)
    for name in ("empty", "zeros", "zeros_like"):
        monkeypatch.setattr(torch, name, noting(getattr(torch, name)))
    for stream in (None, "side"):
        nx.nx_qk_norm_rope(cfg, q, k, workspace=ws, stream=stream)
        nx.nx_paged_attn(cfg, c, q, workspace=ws, max_tokens=4, stream=stream)
        nx.nx_paged_gather(cfg, c, workspace=ws, max_tokens=4, stream=stream)
        assert made == [stream] * 5
        made.clear()


def test_given_head_budgets_are_asked_for_and_checked(lib):
    def dec(alloc=nx.NX_HEADS_GIVEN, n_sink=0, **kw):
        cfg = nx.NexusConfig(4, 2, 64, 4, head_alloc=alloc, n_sink=n_sink)
        return nx.DecodeCache(cfg, 3, 256, 40, 2, device="cpu", **kw)
    with pytest.raises(ValueError, match="head_budget"):
        dec()
    with pytest.raises(ValueError, match="head_budget"):
        dec(nx.NX_HEADS_UNIFORM, head_budget=[9, 9])
    for bad in ([0, 9], [9, 41], [-1, 9], [9.5, 9.0]):
        with pytest.raises(ValueError, match="head_budget"):
            dec(head_budget=bad)
    with pytest.raises(ValueError, match="from 3 "):
        dec(n_sink=3, head_budget=[2, 9])
    assert dec(head_budget=[9, 60], head_cap=64).head_budget.tolist() == [[9, 60]] * 3


def test_events_run_on_the_caches_own_gpu(lib, monkeypatch):
    """Whatever GPU is current: the eviction calls take the current one's stream."""
    from streaming_weighted_sampling_amd import decode
    inside, ran = [None], []

    class On:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            inside.append(self.device)

        def __exit__(self, *a):
            inside.pop()

    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    for name in ("nx_paged_append", "nx_paged_gather", "nx_evict_batch", "nx_read_device_status"):
        monkeypatch.setattr(decode, name, lambda *a, name=name, **kw: ran.append((name, inside[-1])))
    dec = nx.DecodeCache(nx.NexusConfig(4, 2, 64, 4), 2, 64, 32, 2, device="cpu")
    dec.rows = dec.queries = 40
    dec.evict()
    dec.check()
    own = torch.device("cpu")
    assert ("nx_evict_batch", own) in ran and ran.count(("nx_read_device_status", own)) == 2
    assert all(device == own for _, device in ran)


def test_the_status_is_read_on_the_workspaces_gpu(monkeypatch):
    """The paged calls run on the GPU of their tensors; the status read waits for that GPU's stream."""
    from streaming_weighted_sampling_amd import api
    current, seen = [0], []

    class On:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            current.append(self.device)

        def __exit__(self, *a):
            current.pop()

    class Workspace:
        is_cuda = True

        def __init__(self, device):
            self.get_device = lambda: device
            self.data_ptr, self.numel, self.element_size = (lambda: 4096), (lambda: 256), (lambda: 1)

    class Library:
        def nx_read_device_status(self, d):
            seen.append(current[-1])
            return 0

    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[-1])
    monkeypatch.setattr(api, "_stream_handle", lambda s: current[-1])
    monkeypatch.setattr(api, "load", Library)
    cfg = nx.NexusConfig(4, 2, 64, 4)
    for device in (0, 3):
        nx.nx_read_device_status(cfg, Workspace(device))
    assert seen == [0, 3] and current == [0]


def test_arrays_of_no_rows_meet_nothing(lib):
    """Wherever an empty slice points: into the cache, the workspace, another array of the call."""
    c = _cache(workspace_bytes=1 << 28)
    for at in (4096, 7 * GB + 16, 8 * GB + 128, 20 * GB + 64):
        assert lib.nx_paged_attn(c, _r(20, 4096), NxRows(FAKE + at, 4096, 128), 0, None, 100, 1, 0.0, None) == 0
        assert lib.nx_paged_attn(c, _r(20, 4096), _r(21, 4096), 0, None, 100, 1, 0.0, FAKE + at) == 0
        assert lib.nx_paged_gather(c, 0, FAKE + at, FAKE + at, 8 * 12800, 12800) == 0
    d = NxDesc()
    d.n_q_heads, d.n_kv_heads, d.head_dim, d.dtype = 32, 8, 128, _lib.NX_BF16
    d.workspace, d.workspace_bytes = FAKE, 256
    assert lib.nx_qk_norm_rope(d, None, 0, _r(20, 4096), NxRows(FAKE + 128, 4096, 128), None, None, None, None,
                               1e-6) == 0


def test_strides_of_a_single_row_or_head_do_not_matter(lib):
    one = _ws(n_seqs=1, n_q_heads=1, n_kv_heads=1)
    c = _ws()
    start = FAKE + 40 * GB
    for row in (3, 0, -8, 1 << 40):
        q, o = NxRows(FAKE + 20 * GB, row, 128), NxRows(FAKE + 21 * GB, row, 128)
        assert lib.nx_paged_attn(c, q, o, 1, start, 100, 1, 0.0, None) == EWORK       # as far as the workspace
        assert lib.nx_paged_attn(c, q, q, 1, start, 100, 1, 0.0, None) == EALIAS
        q, o = NxRows(FAKE + 20 * GB, 128, row), NxRows(FAKE + 21 * GB, 256, row)
        assert lib.nx_paged_attn(one, q, o, 4, start, 100, 4, 0.0, None) == EWORK
        d = NxDesc()
        d.n_q_heads, d.n_kv_heads, d.head_dim, d.dtype = 4, 1, 128, _lib.NX_BF16
        q, o = NxRows(FAKE + 20 * GB, row, 128), NxRows(FAKE + 20 * GB, 5, 128)
        assert lib.nx_qk_norm_rope(d, None, 1, q, o, None, None, None, None, 1e-6) == EWORK     # in place
        assert lib.nx_qk_norm_rope(d, None, 2, q, o, None, None, None, None, 1e-6) != EWORK


def test_the_workspace_must_not_lie_over_the_inputs(lib):
    """The status word and the attention's partials are written into it."""
    arrays = {name: FAKE + i * GB for i, name in enumerate(
        ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail", "table", "lens"))}
    n = lib.nx_paged_workspace_bytes(_cache(), 100, 1)
    for name, at in arrays.items():
        c = _ws(workspace=at)
        assert lib.nx_paged_append(c, None, _r(20), _r(21), 4, None, None, 1, None) == EALIAS, name
        assert lib.nx_paged_attn(c, _r(20, 4096), _r(21, 4096), 4, None, 100, 1, 0.0, None) == EALIAS, name
        assert lib.nx_paged_gather(c, 100, FAKE + 30 * GB, FAKE + 31 * GB, 8 * 12800, 12800) == EALIAS, name
        c = _cache(workspace=at - n + 16, workspace_bytes=n)          # the partials only
        assert lib.nx_paged_attn(c, _r(20, 4096), _r(21, 4096), 4, None, 100, 1, 0.0, None) == EALIAS, name
        # too small a workspace is that, whatever follows it
        c = _cache(workspace=at - 512, workspace_bytes=512)
        assert lib.nx_paged_attn(c, _r(20, 4096), _r(21, 4096), 4, None, 100, 1, 0.0, None) == EWORK, name
    rope = NxRope(FAKE + 41 * GB, FAKE + 42 * GB, 10, 64, 0)
    for slot in (20, 21, 40, 41, 42, 43):
        c = _ws(workspace=FAKE + slot * GB)
        assert lib.nx_paged_append(c, rope, _r(20), _r(21), 4, FAKE + 40 * GB, FAKE + 43 * GB, 1, None) == EALIAS
    for slot in (20, 40):
        c = _ws(workspace=FAKE + slot * GB)
        assert lib.nx_paged_attn(c, _r(20, 4096), _r(21, 4096), 4, FAKE + 40 * GB, 100, 1, 0.0, None) == EALIAS
    for slot in (20, 22, 24, 25, 41, 42):
        d = NxDesc()
        d.n_q_heads, d.n_kv_heads, d.head_dim, d.dtype = 32, 8, 128, _lib.NX_BF16
        d.workspace, d.workspace_bytes = FAKE + slot * GB, 256
        assert lib.nx_qk_norm_rope(d, rope, 4, _r(20, 4096), _r(21, 4096), FAKE + 24 * GB, _r(22), _r(23),
                                   FAKE + 25 * GB, 1e-6) == EALIAS, slot


def test_misaligned_arrays_are_refused(lib):
    q, o, k, v = _r(20, 4096), _r(21, 4096), _r(22), _r(23)

    def calls(c, start=None, head_new=None, lens_out=None, lse=None, rope=None):
        return (lib.nx_paged_append(c, rope, k, v, 4, start, head_new, 1, lens_out),
                lib.nx_paged_attn(c, q, o, 4, start, 100, 1, 0.0, lse))
    for name in ("k_scale", "v_scale", "table", "lens"):
        c = _ws()
        setattr(c, name, getattr(c, name) + 2)
        assert calls(c) == (EUNSUP, EUNSUP), name
        assert lib.nx_paged_gather(c, 100, FAKE + 30 * GB, FAKE + 31 * GB, 8 * 12800, 12800) == EUNSUP
    for off in (1, 4, 8):
        c = _ws(workspace=FAKE + 8 * GB + off)
        assert calls(c) == (EUNSUP, EUNSUP)
        assert lib.nx_paged_gather(c, 100, FAKE + 30 * GB, FAKE + 31 * GB, 8 * 12800, 12800) == EUNSUP
        d = NxDesc()
        d.n_q_heads, d.n_kv_heads, d.head_dim, d.dtype = 32, 8, 128, _lib.NX_BF16
        d.workspace, d.workspace_bytes = FAKE + off, 256
        assert lib.nx_qk_norm_rope(d, None, 4, q, o, None, None, None, None, 1e-6) == EUNSUP
    odd = FAKE + 40 * GB + 2
    assert calls(_ws(), start=odd) == (EUNSUP, EUNSUP)
    assert calls(_ws(), head_new=odd)[0] == calls(_ws(), lens_out=odd)[0] == calls(_ws(), lse=odd)[1] == EUNSUP
    assert calls(_ws(), rope=NxRope(FAKE + 41 * GB, odd, 10, 64, 0))[0] == EUNSUP


def test_a_caches_arrays_cannot_be_replaced():
    """The calls would go on with the addresses of the old ones, whose memory may be gone."""
    import dataclasses
    cfg = nx.NexusConfig(4, 2, 64, 1, torch.bfloat16)
    c = nx.new_paged_cache(cfg, 3, 8, 2, device="cpu")
    for name in ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail", "table", "lens", "cfg"):
        old = getattr(c, name)
        with pytest.raises(AttributeError, match=name):
            setattr(c, name, dataclasses.replace(old) if name == "cfg" else old.clone())
        assert getattr(c, name) is old
    c.lens.fill_(5)
    c.table += 1
    other = dataclasses.replace(c, lens=c.lens.clone())
    assert other._c.lens == other.lens.data_ptr() != c.lens.data_ptr() == c._c.lens


def test_a_changed_configuration_does_not_change_a_caches_shape():
    """Rows are checked against the shape that the cache passes on, not against what its caller's
    configuration has become."""
    cfg = nx.NexusConfig(4, 2, 64, 1, torch.bfloat16)
    c = nx.new_paged_cache(cfg, 3, 8, 2, device="cpu")
    ws = torch.zeros(256, dtype=torch.uint8)
    cfg.n_q_heads, cfg.n_kv_heads = 2, 1
    q, k = torch.zeros(3, 2, 64).bfloat16(), torch.zeros(3, 1, 64).bfloat16()
    with pytest.raises(ValueError, match="shape"):
        nx.nx_paged_attn(cfg, c, q, workspace=ws, max_tokens=5)
    with pytest.raises(ValueError, match="shape"):
        nx.nx_paged_append(cfg, c, k, k, workspace=ws)
    with pytest.raises(ValueError, match="shape"):
        nx.nx_paged_gather(cfg, c, workspace=ws, max_tokens=5, out_k=torch.zeros(3, 1, 5, 64).bfloat16())


def test_the_workspace_query_refuses_another_configuration(lib):
    cfg = nx.NexusConfig(4, 2, 64, 1, torch.bfloat16)
    c = nx.new_paged_cache(cfg, 3, 8, 2, device="cpu")
    assert nx.paged_workspace_bytes(cfg, c, 100, 4) > 0
    for make in (nx.paged_workspace_bytes, nx.new_paged_workspace):
        with pytest.raises(ValueError, match="configuration"):
            make(nx.NexusConfig(64, 2, 64, 1, torch.bfloat16), c, 100, 4)


def test_an_event_reads_the_settings_of_its_time(lib, monkeypatch):
    """Settings changed between events reach the event's records; those that the buffers were sized by
    are refused."""
    import contextlib

    from streaming_weighted_sampling_amd import decode
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    seen = []
    for name in ("nx_paged_append", "nx_paged_gather"):
        monkeypatch.setattr(decode, name, lambda *a, **kw: None)
    monkeypatch.setattr(decode, "nx_evict_batch", lambda cfg, units, n, rows, iters, seed, **kw: seen.append(
        [(u.n_tokens, u.budget, u.layer, u.head_cap)
         for u in (_lib.NxUnit * n).from_buffer_copy(bytes(units.numpy()))]))

    def event(dec, rows):
        dec.rows = dec.queries = rows
        dec.evict()
        return seen.pop()
    dec = nx.DecodeCache(nx.NexusConfig(4, 2, 64, 4), 2, 64, 32, 2, layer=3, device="cpu")
    assert event(dec, 40) == [(40, 32, 3, 32)] * 2 and event(dec, 41) == [(41, 32, 3, 32)] * 2
    dec.layer = 5
    assert event(dec, 40) == [(40, 32, 5, 32)] * 2
    for budget in (33, 16):
        dec.budget = budget
        with pytest.raises(ValueError, match="budget"):
            event(dec, 40)
    per_head = nx.DecodeCache(nx.NexusConfig(4, 2, 64, 4, head_alloc=2), 2, 64, 20, 2, head_cap=30, device="cpu")
    assert event(per_head, 40) == [(40, 20, 0, 30)] * 2
    per_head.budget = 12
    assert event(per_head, 40) == [(40, 12, 0, 30)] * 2
    per_head.head_cap = 31
    with pytest.raises(ValueError, match="head_cap"):
        event(per_head, 40)


def test_event_buffers_are_shared_by_caches_of_one_shape_only(lib):
    cfg = nx.NexusConfig(4, 2, 64, 4)
    first = nx.DecodeCache(cfg, 2, 64, 32, 2, device="cpu")
    for kw in (dict(n_seqs=1), dict(capacity=96), dict(budget=30), dict(walk_iters=1),
               dict(cfg=nx.NexusConfig(8, 2, 64, 4))):
        with pytest.raises(ValueError, match="event_buffers"):
            nx.DecodeCache(**(dict(cfg=cfg, n_seqs=2, capacity=64, budget=32, walk_iters=2) | kw),
                           event_buffers=first.event_buffers, device="cpu")
    second = nx.DecodeCache(cfg, 2, 64, 32, 2, layer=1, event_buffers=first.event_buffers, device="cpu")
    alone = nx.DecodeCache(cfg, 2, 64, 32, 2, layer=1, device="cpu")
    assert second.k is first.k and second.evict_ws is first.evict_ws and alone.k is not first.k
    assert second.keep is not first.keep and second.cache is not first.cache
    assert set(first.event_buffers.users) == {first, second}
    with pytest.raises(AttributeError):
        first.event_buffers = alone.event_buffers
    del second
    assert set(first.event_buffers.users) == {first}


def test_tables_of_more_rows_than_are_counted_in_32_bits(lib):
    """64 heads of 2^31 rows are 2^32 blocks, which the attention's cut would add up in 32 bits."""
    for pages, blocks, code in ((1 << 14, 1024, EWORK), ((1 << 14) + 1, 1024, EUNSUP), (1 << 16, 1024, EUNSUP),
                                (1 << 24, 1, EWORK), (1 << 30, 1, EUNSUP), ((1 << 31) - 1, 64, EUNSUP)):
        c = _cache(max_pages=pages, page_blocks=blocks, n_seqs=1, n_kv_heads=1, n_q_heads=1)
        assert lib.nx_paged_attn(c, _r(20, 4096), _r(21, 4096), 4, None, 100, 1, 0.0, None) == code, (pages, blocks)
        assert (lib.nx_paged_workspace_bytes(c, 100, 1) > 0) == (code == EWORK)


def test_gather_strides_of_a_single_head_or_sequence_do_not_matter(lib):
    def call(seqs, heads, ss, hs):
        c = _ws(n_seqs=seqs, n_kv_heads=heads, n_q_heads=heads, k_tail=FAKE + 30 * GB)     # under out_k
        return lib.nx_paged_gather(c, 100, FAKE + 30 * GB, FAKE + 31 * GB, ss, hs)
    for odd in (0, 3, -8, 1 << 40):
        assert call(1, 8, odd, 12800) == EALIAS            # as far as the last check
        assert call(4, 1, 12800, odd) == EALIAS
        assert call(1, 1, odd, odd) == EALIAS
    assert call(2, 1, 12799, 12800) == EINVAL and call(1, 2, 0, 12799) == EINVAL
    assert call(2, 2, 25600 - 1, 12800) == EINVAL


def test_a_replaced_rotation_table_is_checked():
    """A table of another type or shape would be read as float32 rows, past its end."""
    rope = nx.Rope(torch.zeros(4, 16))
    for bad in (torch.zeros(4, 16, dtype=torch.float16), torch.zeros(64), torch.zeros(4, 32)[:, ::2]):
        with pytest.raises(ValueError, match="cos_sin"):
            rope.cos_sin = bad
    rope.cos_sin = longer = torch.zeros(9, 16)
    rope.pairs = True
    assert rope.cos_sin is longer and rope.pairs
