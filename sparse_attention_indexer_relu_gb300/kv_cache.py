"""Paged key/value cache in 8 bits: the binding of `include/mqakv.h`.

A `KVCache` holds the cache's tensors (the caller's) and passes them to the C
entries: `kv_reserve` makes room, `kv_append` writes new keys and values,
`kv_attention` reads them (all visible keys, or the ones `mqa_topk_prefill`
selected), and `kv_fork`, `kv_free`, `kv_compact` and `kv_copy_pages` manage
the pages.  As in the rest of the package only arguments are marshalled here.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional, Sequence

KV_EXPORTS = ("mqa_kv_scratch_bytes", "mqa_kv_append", "mqa_kv_attention_workspace_bytes", "mqa_kv_attention",
              "mqa_kv_attention_debug",
              "mqa_kv_reserve", "mqa_kv_fork", "mqa_kv_free", "mqa_kv_compact", "mqa_kv_copy_pages",
              "mqa_kv_get_status")
KV_STATUS_BITS = {1: "out_of_pages", 2: "bad_index", 4: "bad_list", 8: "bad_length", 16: "wait_timeout"}
KV_PAGE_SIZES = (16, 32, 64, 128)
KV_HEAD_DIMS = (64, 128)
_MAX_EXTRA = 4


class _Pool(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("page_bytes", ctypes.c_size_t)]


class _Cache(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_exps", "v_exps", "page_table", "seq_lens", "refcounts",
                                                "scratch")] + [("scratch_bytes", ctypes.c_size_t)] +
                [(n, ctypes.c_int) for n in ("num_pages", "page_size", "kv_heads", "head_dim", "max_seqs",
                                             "max_pages", "n_extra")] + [("extra", _Pool * _MAX_EXTRA)])


class KVDebugOptions(ctypes.Structure):
    _fields_ = [("stall", ctypes.c_int), ("wait_timeout_ms", ctypes.c_int)]


def declare(L):
    """Argument types of the cache's entries (called when the library is loaded)."""
    P, I, S, Q, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong, ctypes.c_float
    C = ctypes.POINTER(_Cache)
    L.mqa_kv_scratch_bytes.argtypes = [I, I, ctypes.POINTER(S)]
    L.mqa_kv_append.argtypes = [C, P, P, Q, Q, I, P, I, P]
    L.mqa_kv_attention_workspace_bytes.argtypes = [I, C, I, I, ctypes.POINTER(S)]
    L.mqa_kv_attention.argtypes = [C, P, Q, I, I, P, I, I, P, I, I, F, P, P, P, S, P]
    L.mqa_kv_attention_debug.argtypes = L.mqa_kv_attention.argtypes + [ctypes.POINTER(KVDebugOptions)]
    L.mqa_kv_reserve.argtypes = [C, P, P]
    L.mqa_kv_fork.argtypes = [C, P, P, I, P]
    L.mqa_kv_free.argtypes = [C, P, I, P]
    L.mqa_kv_compact.argtypes = [C, P]
    L.mqa_kv_copy_pages.argtypes = [C, P, P, I, P]
    L.mqa_kv_get_status.argtypes = [C, ctypes.POINTER(ctypes.c_int32), P]
    for name in KV_EXPORTS:
        getattr(L, name).restype = I


def _api():
    import sparse_attention_indexer_relu_gb300 as m
    return m


_TYPES = {}


def _types():
    if not _TYPES:
        import torch
        _TYPES.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    return _TYPES


def _dense(t, dtypes, dim, name, device=None):
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got shape {tuple(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    return t


def _alike(a, b):
    return (a is not None and b is not None and a.dtype == b.dtype and a.shape == b.shape and a.device == b.device and
            a.is_contiguous())


class KVCache:
    """The tensors of a paged cache (include/mqakv.h):

    k, v            uint8 (or float8_e4m3fn) [num_pages, kv_heads, page_size, head_dim] codes
    k_exps, v_exps  uint8 [num_pages, kv_heads] UE8M0
    page_table      int32 [max_seqs, max_pages];  seq_lens int32 [max_seqs]
    refcounts       int32 [num_pages], needed by the page operations only
    scratch         uint8, `kv_scratch_bytes` long and zeroed (made here if None)
    extra           up to 4 further tensors [num_pages, ...] whose pages move along

    The object keeps references and changes nothing by itself; its calls use
    the addresses taken here, so its tensors are not exchanged but by
    `replace`.  Calls that change the cache, and calls that overlap such a
    call, are the caller's to order; handles that share a scratch (those of
    `replace`) count as one cache there."""

    def _fixed(self, name):
        if name in self.__dict__.get("_held", ()):
            raise AttributeError(f"{name} of a KVCache is fixed: its calls use the address of the tensor that it was made "
                                 "of; replace() makes a handle over another one")

    def __setattr__(self, name, value):
        self._fixed(name)
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        self._fixed(name)
        object.__delattr__(self, name)

    def __init__(self, k, v, k_exps, v_exps, page_table, seq_lens, refcounts=None, scratch=None, extra: Sequence = ()):
        import torch
        codes = (torch.uint8, torch.float8_e4m3fn)
        _dense(k, codes, 4, "k")
        dev = k.device
        pages, heads, page, dim = map(int, k.shape)
        _dense(v, codes, 4, "v", dev)
        _dense(k_exps, (torch.uint8,), 2, "k_exps", dev)
        _dense(v_exps, (torch.uint8,), 2, "v_exps", dev)
        _dense(page_table, (torch.int32,), 2, "page_table", dev)
        _dense(seq_lens, (torch.int32,), 1, "seq_lens", dev)
        if v.shape != k.shape or tuple(k_exps.shape) != (pages, heads) or tuple(v_exps.shape) != (pages, heads):
            raise ValueError("k, v, k_exps and v_exps differ in pages, heads or sizes")
        if page not in KV_PAGE_SIZES or dim not in KV_HEAD_DIMS:
            raise ValueError(f"page size {page} or head dimension {dim} is not supported")
        if page_table.shape[0] != seq_lens.shape[0]:
            raise ValueError("page_table and seq_lens differ in sequences")
        if refcounts is not None and tuple(_dense(refcounts, (torch.int32,), 1, "refcounts", dev).shape) != (pages,):
            raise ValueError("refcounts needs one count per page")
        if len(extra) > _MAX_EXTRA:
            raise ValueError(f"at most {_MAX_EXTRA} extra pools")
        for t in extra:
            if not t.is_cuda or not t.is_contiguous() or t.device != dev or t.dim() < 1 or t.shape[0] != pages:
                raise ValueError("an extra pool must be a contiguous CUDA tensor [num_pages, ...] on the cache's device")
        if scratch is None:
            scratch = torch.zeros(kv_scratch_bytes(pages, int(seq_lens.shape[0])), dtype=torch.uint8, device=dev)
        _dense(scratch, (torch.uint8,), 1, "scratch", dev)
        self.k, self.v, self.k_exps, self.v_exps = k, v, k_exps, v_exps
        self.page_table, self.seq_lens, self.refcounts = page_table, seq_lens, refcounts
        self.scratch, self.extra, self.device = scratch, tuple(extra), dev
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page, dim
        self.max_seqs, self.max_pages = map(int, page_table.shape)
        c = _Cache(k=k.data_ptr(), v=v.data_ptr(), k_exps=k_exps.data_ptr(), v_exps=v_exps.data_ptr(),
                   page_table=page_table.data_ptr(), seq_lens=seq_lens.data_ptr(),
                   refcounts=None if refcounts is None else refcounts.data_ptr(), scratch=scratch.data_ptr(),
                   scratch_bytes=scratch.numel(), num_pages=pages, page_size=page, kv_heads=heads, head_dim=dim,
                   max_seqs=self.max_seqs, max_pages=self.max_pages, n_extra=len(extra))
        for i, t in enumerate(extra):
            c.extra[i] = _Pool(t.data_ptr(), t.numel() * t.element_size() // pages)
        self._c = c
        self._ref = ctypes.byref(c)
        self._index = dev.index
        self._held = frozenset(self.__dict__)

    def replace(self, **changes):
        """A cache over the same tensors (the scratch included) but for the given ones."""
        if all(n in ("page_table", "seq_lens", "refcounts") and _alike(t, getattr(self, n)) for n, t in changes.items()):
            other = object.__new__(KVCache)
            other.__dict__.update(self.__dict__, **changes)
            other.__dict__["_c"] = _Cache.from_buffer_copy(self._c)
            for n, t in changes.items():
                setattr(other._c, n, t.data_ptr())
            other.__dict__["_ref"] = ctypes.byref(other._c)
            return other
        now = {n: getattr(self, n) for n in ("k", "v", "k_exps", "v_exps", "page_table", "seq_lens", "refcounts",
                                             "scratch", "extra")}
        now.update(changes)
        return KVCache(**now)


def kv_scratch_bytes(num_pages: int, max_seqs: int) -> int:
    m = _api()
    n = ctypes.c_size_t(0)
    m._check(m.lib().mqa_kv_scratch_bytes(int(num_pages), int(max_seqs), ctypes.byref(n)), "mqa_kv_scratch_bytes")
    return int(n.value)


def alloc_kv_cache(num_pages: int, page_size: int, kv_heads: int, head_dim: int, max_seqs: int, max_pages: int,
                   device=None, extra: Sequence = ()) -> KVCache:
    """An empty cache: no sequence holds a page, every page is free."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    z = lambda *s, dtype=torch.uint8: torch.zeros(s, dtype=dtype, device=dev)  # noqa: E731
    codes = (num_pages, kv_heads, page_size, head_dim)
    return KVCache(z(*codes), z(*codes), z(num_pages, kv_heads) + 127, z(num_pages, kv_heads) + 127,
                   torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device=dev),
                   z(max_seqs, dtype=torch.int32), z(num_pages, dtype=torch.int32), extra=extra)


class _Here:
    """The usual case of `_on`: the cache's device is current and its current stream is used."""

    __slots__ = ("raw",)

    def __init__(self, raw):
        self.raw = raw

    def __enter__(self):
        return self.raw

    def __exit__(self, *_):
        return False


def _on(cache, stream):
    """The cache's device current, `stream` (default: its current stream) as the stream of what is allocated."""
    import torch
    if stream is None and torch._C._cuda_getDevice() == cache._index:
        return _Here(torch._C._cuda_getCurrentRawStream(cache._index))
    return _on_other(cache, stream)


@contextlib.contextmanager
def _on_other(cache, stream):
    import torch
    with torch.cuda.device(cache.device):
        s = torch.cuda.current_stream() if stream is None else stream
        if s.device != cache.device:
            raise ValueError(f"the stream is on {s.device}, the cache on {cache.device}")
        with torch.cuda.stream(s):
            yield s.cuda_stream


def _list(t, cache, name, n=None):
    import torch
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
    if t.dim() != 1 or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({'n' if n is None else n},)")
    if t.device != cache.device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on {cache.device}")
    return t.data_ptr()


def _rows(t, cache, dtypes, heads, name):
    """A [rows, heads, head_dim] tensor whose rows may be strided (a slice of a wider projection)."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.requires_grad and _api()._torch().is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, which the cache's operators do not have: detach it, or call "
                         "them under torch.no_grad()")
    d = cache.head_dim
    if t.dim() != 3 or t.shape[2] != d or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected (rows, {heads or 'heads'}, {d})")
    if t.device != cache.device or (t.shape[0] and (t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != d))):
        raise ValueError(f"{name} must be on {cache.device} with its heads contiguous in a row")
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else t.shape[1] * d


def alloc_kv_workspace(cache: KVCache, rows: int, q_heads: int):
    """Workspace for `kv_attention` calls over up to `rows` rows of `q_heads` heads (caller owns it; calls that
    overlap in time need one each)."""
    import torch
    m = _api()
    n = ctypes.c_size_t(0)
    m._check(m.lib().mqa_kv_attention_workspace_bytes(cache.device.index, cache._ref, int(rows), int(q_heads),
                                                      ctypes.byref(n)), "mqa_kv_attention_workspace_bytes")
    return torch.empty(n.value, dtype=torch.uint8, device=cache.device)


def kv_append(cache: KVCache, k, v, row_starts, stream=None):
    """Write rows k, v [rows, kv_heads, head_dim] (bf16, fp16 or fp32) to their sequences' last positions:
    sequence s has rows [row_starts[s], row_starts[s + 1]) and seq_lens counts them already (`kv_reserve`)."""
    m, types = _api(), _types()
    kp, ks = _rows(k, cache, tuple(types), cache.kv_heads, "k")
    vp, vs = _rows(v, cache, (k.dtype,), cache.kv_heads, "v")
    if v.shape != k.shape:
        raise ValueError("k and v differ in shape")
    rs = _list(row_starts, cache, "row_starts", cache.max_seqs + 1)
    with _on(cache, stream) as s:
        m._check(m.lib().mqa_kv_append(cache._ref, kp, vp, ks, vs, types[k.dtype], rs, int(k.shape[0]), s),
                 "mqa_kv_append")


def kv_attention(q, cache: KVCache, row_starts, selected=None, causal: bool = True, scale: Optional[float] = None,
                 max_rows: Optional[int] = None, workspace=None, out=None, lse=None, stream=None,
                 debug: Optional[dict] = None):
    """Attention of rows q [rows, q_heads, head_dim] (bf16 or fp16) over the cache; returns out, of q's shape.

    Row i of the n rows of a sequence is its position seq_len - n + i and sees the positions up to its own (every
    position of the sequence where not `causal`); with `selected` [rows, k] int32, the listed ones among them (the
    answer of `mqa_topk_prefill`).  scale defaults to head_dim ** -0.5.  max_rows: the most rows of one sequence, if
    known (it only helps to choose the kernels).  lse [rows, q_heads] float32 receives the logarithm of each
    softmax's sum.  Rows before row_starts[0] and at or behind row_starts[-1] are left as they are in `out`
    and `lse`.  debug: test-only knobs (KVDebugOptions)."""
    import torch
    m, types = _api(), _types()
    qp, qs = _rows(q, cache, (torch.bfloat16, torch.float16), None, "q")
    rows, heads = int(q.shape[0]), int(q.shape[1])
    if heads == 0 or heads % cache.kv_heads:
        raise ValueError(f"{heads} query heads do not divide among {cache.kv_heads} key/value heads")
    rs = _list(row_starts, cache, "row_starts", cache.max_seqs + 1)
    sp, n_sel = None, 0
    if selected is not None:
        _dense(selected, (torch.int32,), 2, "selected", cache.device)
        if selected.shape[0] != rows:
            raise ValueError(f"selected has {selected.shape[0]} rows, q {rows}")
        n_sel = int(selected.shape[1])
        sp = selected.data_ptr() or rs  # an empty list still is a list
    with _on(cache, stream) as s:
        if out is None:
            out = torch.empty((rows, heads, cache.head_dim), dtype=q.dtype, device=cache.device)
        _dense(out, (q.dtype,), 3, "out", cache.device)
        if out.shape != q.shape:
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {tuple(q.shape)}")
        if lse is not None and tuple(_dense(lse, (torch.float32,), 2, "lse", cache.device).shape) != (rows, heads):
            raise ValueError(f"lse has shape {tuple(lse.shape)}, expected {(rows, heads)}")
        if workspace is None:
            workspace = alloc_kv_workspace(cache, rows, heads)
        elif workspace.device != cache.device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {cache.device}")
        args = (cache._ref, qp, qs, types[q.dtype], heads, rs, rows, int(max_rows or 0), sp, n_sel, int(bool(causal)),
                cache.head_dim ** -0.5 if scale is None else float(scale), out.data_ptr(),
                None if lse is None else lse.data_ptr(), workspace.data_ptr(),
                workspace.numel() * workspace.element_size(), s)
        if debug is None:
            m._check(m.lib().mqa_kv_attention(*args), "mqa_kv_attention")
        else:
            m._check(m.lib().mqa_kv_attention_debug(*args, ctypes.byref(KVDebugOptions(**debug))),
                     "mqa_kv_attention_debug")
    return out


def kv_reserve(cache: KVCache, counts, stream=None):
    """Extend sequence s by counts[s] positions (int32 [max_seqs]), taking the lowest free pages."""
    m = _api()
    with _on(cache, stream) as s:
        m._check(m.lib().mqa_kv_reserve(cache._ref, _list(counts, cache, "counts", cache.max_seqs), s),
                 "mqa_kv_reserve")


def kv_fork(cache: KVCache, parents, children, stream=None):
    """Each empty sequence children[i] becomes a copy of parents[i]: full pages shared, a partial last page copied."""
    m = _api()
    p = _list(parents, cache, "parents")
    n = int(parents.shape[0])
    with _on(cache, stream) as s:
        m._check(m.lib().mqa_kv_fork(cache._ref, p, _list(children, cache, "children", n), n, s), "mqa_kv_fork")


def kv_free(cache: KVCache, seqs, stream=None):
    """Give back the pages of the listed sequences, which become empty."""
    m = _api()
    with _on(cache, stream) as s:
        m._check(m.lib().mqa_kv_free(cache._ref, _list(seqs, cache, "seqs"), int(seqs.shape[0]), s), "mqa_kv_free")


def kv_compact(cache: KVCache, stream=None):
    """Move the used pages to the front of the pool, tables and refcounts with them."""
    m = _api()
    with _on(cache, stream) as s:
        m._check(m.lib().mqa_kv_compact(cache._ref, s), "mqa_kv_compact")


def kv_copy_pages(cache: KVCache, src, dst, stream=None):
    """Copy the contents of pages src[i] to pages dst[i] (tables and refcounts untouched)."""
    m = _api()
    p = _list(src, cache, "src")
    n = int(src.shape[0])
    with _on(cache, stream) as s:
        m._check(m.lib().mqa_kv_copy_pages(cache._ref, p, _list(dst, cache, "dst", n), n, s), "mqa_kv_copy_pages")


def kv_status(cache: KVCache, stream=None) -> int:
    """The status bits (KV_STATUS_BITS) collected since the last call; clears them (synchronises)."""
    m = _api()
    st = ctypes.c_int32(0)
    with _on(cache, stream) as s:
        m._check(m.lib().mqa_kv_get_status(cache._ref, ctypes.byref(st), s), "mqa_kv_get_status")
    return int(st.value)
