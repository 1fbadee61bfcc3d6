"""Thin ctypes binding of the C ABI in ``include/spgemm_attention.h``: softmax
attention whose mask is the structure of a CSR matrix, its gradients, and
attention of new tokens over a paged key/value cache.

Argument marshalling only, as in ``binding``: outputs and workspaces are torch
tensors, every step runs in the HIP library's kernels. All tensors of a call
are on one device; the call runs on ``stream`` (default: that device's current
stream), which the tensors it allocates then belong to. Nothing here waits for
the GPU, except making and closing a plan.
"""
from __future__ import annotations

import ctypes

from . import binding as _b
from .binding import DeviceCSR, SpgemmError, _check  # noqa: F401  (SpgemmError: what calls raise)

EXPORTS = ["spgemm_attention_plan_create", "spgemm_attention_plan_destroy",
           "spgemm_attention_workspace", "spgemm_attention_forward", "spgemm_attention_backward",
           "spgemm_paged_attention_workspace", "spgemm_paged_attention"]
MAX_HEAD_DIM = 256


class Desc(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("heads_q", ctypes.c_int32),
                ("heads_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("scale", ctypes.c_double)]


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_row", ctypes.c_int64),
                ("stride_head", ctypes.c_int64)]


class PagedCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("npages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("k_stride_page", ctypes.c_int64),
                ("k_stride_slot", ctypes.c_int64), ("k_stride_head", ctypes.c_int64),
                ("v_stride_page", ctypes.c_int64), ("v_stride_slot", ctypes.c_int64),
                ("v_stride_head", ctypes.c_int64)]


class PagedBatch(ctypes.Structure):
    _fields_ = [("pages", ctypes.POINTER(_b.CSRStruct)), ("q_rowptr", ctypes.c_void_p),
                ("lengths", ctypes.c_void_p), ("tokens", ctypes.c_int64),
                ("max_new", ctypes.c_int64), ("max_length", ctypes.c_int64)]


_lib = None


def load():
    """The built library with these entry points declared (raises if it is missing)."""
    global _lib
    if _lib is None:
        lib = _b.load()
        P, I, L = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        D, R = ctypes.POINTER(Desc), ctypes.POINTER(Rows)
        B, C = ctypes.POINTER(PagedBatch), ctypes.POINTER(PagedCache)
        LP = ctypes.POINTER(L)
        sigs = {
            "spgemm_attention_plan_create": [ctypes.POINTER(P), ctypes.POINTER(_b.CSRStruct), I, P],
            "spgemm_attention_workspace": [P, D, I, LP],
            "spgemm_attention_forward": [P, D, R, R, R, R, P, P, L, P],
            "spgemm_attention_backward": [P, D, R, R, R, R, P, R, R, R, R, P, L, P],
            "spgemm_paged_attention_workspace": [D, B, LP],
            "spgemm_paged_attention": [D, R, C, B, R, P, P, L, P],
        }
        for name, args in sigs.items():
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = ctypes.c_int
        lib.spgemm_attention_plan_destroy.argtypes = [P]
        lib.spgemm_attention_plan_destroy.restype = None
        _lib = lib
    return _lib


def _type_code(dtype) -> int:
    import torch
    codes = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
    if dtype not in codes:
        raise ValueError(f"attention takes bfloat16, float16 or float32 tensors, not {dtype}")
    return codes[dtype]


def _on_device(like, stream):
    """A context with the tensor's device and the call's stream current."""
    import torch
    if not like.is_cuda:
        raise ValueError("attention needs tensors on the GPU")
    return torch.cuda.stream(stream) if stream is not None else torch.cuda.device(like.device)


def _heads(name, t, rows, heads, like) -> Rows:
    """A [rows, heads, head_dim] tensor as the library takes it."""
    if t.dim() != 3 or (rows is not None and t.shape[0] != rows) or \
            (heads is not None and t.shape[1] != heads) or t.shape[2] != like.shape[2]:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected "
                         f"({rows if rows is not None else 'rows'}, "
                         f"{heads if heads is not None else 'heads'}, {like.shape[2]})")
    if t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} is {t.dtype} on {t.device}, expected {like.dtype} on "
                         f"{like.device}")
    if t.numel() and t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return Rows(t.data_ptr() if t.numel() else None, t.stride(0), t.stride(1))


def _flat(name, t, shape, dtype, device):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device or \
            not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"{device}")


def _desc(q, hkv: int, scale) -> Desc:
    hq, dim = q.shape[1], q.shape[2]
    return Desc(_type_code(q.dtype), hq, hkv, dim, dim ** -0.5 if scale is None else float(scale))


def _workspace(nbytes: int, device):
    """(tensor, its 256-byte aligned address): the caching allocator's memory is 512-byte aligned."""
    import torch
    if nbytes == 0:
        return None, None
    t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return t, t.data_ptr()


class AttentionPlan:
    """Attention over one mask: query row i sees the key rows that row i of
    the CSR matrix ``mask`` stores (``mask.val`` is not read and may be None).

    The mask is checked and copied; ``backward=True`` prepares its transpose
    too, which ``backward()`` needs. A plan does not change after that: it can
    be used on several streams at once and inside captured graphs, which it
    must outlive. Making one blocks until it is ready.
    """

    def __init__(self, mask: DeviceCSR, backward: bool = False, stream=None):
        import torch
        lib = load()
        for name, t, dtype, n in (("mask.rowptr", mask.rowptr, torch.int64, mask.nrows + 1),
                                  ("mask.col", mask.col, torch.int32, mask.nnz)):
            if not t.is_cuda:
                raise ValueError("attention needs tensors on the GPU")
            _flat(name, t, (n,), dtype, mask.rowptr.device)
        self._lib, self._h = lib, None
        self.nrows, self.ncols, self.nnz = mask.nrows, mask.ncols, mask.nnz
        self.device = mask.rowptr.device
        h = ctypes.c_void_p()
        s = _b.CSRStruct(mask.nrows, mask.ncols, mask.nnz, mask.rowptr.data_ptr(),
                         mask.col.data_ptr() if mask.nnz else None, None)
        with _on_device(mask.rowptr, stream):
            _check(lib.spgemm_attention_plan_create(ctypes.byref(h), ctypes.byref(s),
                                                    1 if backward else 0,
                                                    _b._stream_handle(stream)),
                   "spgemm_attention_plan_create")
        self._h = h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            import torch
            with torch.cuda.device(self.device):
                self._lib.spgemm_attention_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def _ready(self, q):
        if self._h is None:
            raise ValueError("the attention plan is closed")
        if q.dim() != 3:
            raise ValueError(f"q has shape {tuple(q.shape)}, expected (rows, heads, head_dim)")
        if q.device != self.device:
            raise ValueError(f"the plan is on {self.device}, q on {q.device}")

    def _space(self, desc, backward):
        n = ctypes.c_int64(0)
        _check(self._lib.spgemm_attention_workspace(self._h, ctypes.byref(desc), backward,
                                                    ctypes.byref(n)), "spgemm_attention_workspace")
        return (*_workspace(n.value, self.device), n.value)

    def forward(self, q, k, v, scale=None, out=None, lse=None, stream=None):
        """(out, lse) for q [nrows, heads_q, dim] and k, v [ncols, heads_kv, dim].

        out has q's shape and type, lse is [nrows, heads_q] in float32. Either
        may be passed to be written into. scale defaults to dim ** -0.5."""
        import torch
        self._ready(q)
        qs = _heads("q", q, self.nrows, None, q)
        ks = _heads("k", k, self.ncols, None, q)
        vs = _heads("v", v, self.ncols, k.shape[1], q)
        desc = _desc(q, k.shape[1], scale)
        with _on_device(q, stream):
            if out is None:
                out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            if lse is None:
                lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
            os = _heads("out", out, self.nrows, q.shape[1], q)
            _flat("lse", lse, q.shape[:2], torch.float32, q.device)
            _, ws, nbytes = space = self._space(desc, 0)
            _check(self._lib.spgemm_attention_forward(
                self._h, ctypes.byref(desc), ctypes.byref(qs), ctypes.byref(ks), ctypes.byref(vs),
                ctypes.byref(os), _b._ptr(lse), ws, nbytes, _b._stream_handle(stream)),
                "spgemm_attention_forward")
            del space
        return out, lse

    def backward(self, dout, q, k, v, out, lse, scale=None, dq=None, dk=None, dv=None,
                 stream=None):
        """(dq, dk, dv), given dout and what ``forward`` returned. Gradients
        have their tensors' shapes and type, and are written, not added to."""
        import torch
        self._ready(q)
        hq, hkv = q.shape[1], k.shape[1] if k.dim() == 3 else None
        qs = _heads("q", q, self.nrows, None, q)
        ks = _heads("k", k, self.ncols, None, q)
        vs = _heads("v", v, self.ncols, hkv, q)
        os = _heads("out", out, self.nrows, hq, q)
        gs = _heads("dout", dout, self.nrows, hq, q)
        _flat("lse", lse, q.shape[:2], torch.float32, q.device)
        desc = _desc(q, hkv, scale)
        with _on_device(q, stream):
            new = [torch.empty(x.shape, dtype=q.dtype, device=q.device) if g is None else g
                   for g, x in ((dq, q), (dk, k), (dv, v))]
            sinks = [_heads(n, g, x.shape[0], x.shape[1], q)
                     for n, g, x in zip(("dq", "dk", "dv"), new, (q, k, v))]
            _, ws, nbytes = space = self._space(desc, 1)
            _check(self._lib.spgemm_attention_backward(
                self._h, ctypes.byref(desc), ctypes.byref(qs), ctypes.byref(ks), ctypes.byref(vs),
                ctypes.byref(os), _b._ptr(lse), ctypes.byref(gs), *map(ctypes.byref, sinks), ws,
                nbytes, _b._stream_handle(stream)), "spgemm_attention_backward")
            del space
        return tuple(new)


def paged_attention(q, k_cache, v_cache, pages: DeviceCSR, q_rowptr, lengths, max_q: int,
                    max_len: int, scale=None, out=None, lse=None, stream=None):
    """(out, lse) of new tokens over their sequences' paged caches.

    q: [tokens, heads_q, dim]; sequence s's new tokens are its rows
    [q_rowptr[s], q_rowptr[s + 1]). k_cache, v_cache: [pages, slots, heads_kv,
    dim], the new tokens' keys and values already in them. pages: row s of
    this CSR matrix (sequences x cache pages; val may be None) lists sequence
    s's pages in order. lengths: int64, the tokens of each sequence in the
    cache, new ones included. max_q and max_len bound the new tokens and the
    length of any sequence. Each token sees the tokens up to itself. Rows of
    ``out`` and ``lse`` that belong to no sequence are not written.

    The index tensors are read on the GPU, so a captured call follows their
    later values; a sequence that breaks the rules gets NaN."""
    import torch
    lib = load()
    if q.dim() != 3 or k_cache.dim() != 4 or v_cache.shape != k_cache.shape or \
            k_cache.shape[3] != q.shape[2]:
        raise ValueError(f"q {tuple(q.shape)}, k_cache {tuple(k_cache.shape)} and v_cache "
                         f"{tuple(v_cache.shape)} do not fit: expected (tokens, heads, dim) and "
                         "twice (pages, slots, kv heads, dim)")
    tokens, hq, dim = q.shape
    npages, slots, hkv, _ = k_cache.shape
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype != q.dtype or t.device != q.device:
            raise ValueError(f"{name} is {t.dtype} on {t.device}, expected {q.dtype} on {q.device}")
        if t.numel() and dim > 1 and t.stride(3) != 1:
            raise ValueError(f"{name}'s last dimension must be contiguous")
    if pages.ncols != npages:
        raise ValueError(f"the page table names pages of a cache of {pages.ncols}, it has {npages}")
    _flat("pages.rowptr", pages.rowptr, (pages.nrows + 1,), torch.int64, q.device)
    _flat("pages.col", pages.col, (pages.nnz,), torch.int32, q.device)
    _flat("q_rowptr", q_rowptr, (pages.nrows + 1,), torch.int64, q.device)
    _flat("lengths", lengths, (pages.nrows,), torch.int64, q.device)
    qs = _heads("q", q, tokens, None, q)
    desc = _desc(q, hkv, scale)
    table = _b.CSRStruct(pages.nrows, npages, pages.nnz, pages.rowptr.data_ptr(),
                         _b._ptr(pages.col), None)
    cache = PagedCache(_b._ptr(k_cache), _b._ptr(v_cache), npages, slots, *k_cache.stride()[:3],
                       *v_cache.stride()[:3])
    batch = PagedBatch(ctypes.pointer(table), q_rowptr.data_ptr(), _b._ptr(lengths), tokens,
                       int(max_q), int(max_len))
    with _on_device(q, stream):
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if lse is None:
            lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        os = _heads("out", out, tokens, hq, q)
        _flat("lse", lse, q.shape[:2], torch.float32, q.device)
        n = ctypes.c_int64(0)
        _check(lib.spgemm_paged_attention_workspace(ctypes.byref(desc), ctypes.byref(batch),
                                                    ctypes.byref(n)),
               "spgemm_paged_attention_workspace")
        space, ws = _workspace(n.value, q.device)
        _check(lib.spgemm_paged_attention(
            ctypes.byref(desc), ctypes.byref(qs), ctypes.byref(cache), ctypes.byref(batch),
            ctypes.byref(os), _b._ptr(lse), ws, n.value, _b._stream_handle(stream)),
            "spgemm_paged_attention")
        del space
    return out, lse
