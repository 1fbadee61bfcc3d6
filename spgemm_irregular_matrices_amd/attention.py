"""Thin ctypes binding of the C ABI in ``include/spgemm_attention.h``: softmax
attention whose mask is the structure of a CSR matrix, its gradients, and
attention of new tokens over a paged key/value cache.

Argument marshalling only, as in ``binding``: outputs and workspaces are torch
tensors, every step runs in the HIP library's kernels. All tensors of a call
are on one device; the call runs on ``stream`` (default: that device's current
stream), which the tensors it allocates then belong to. Nothing here waits for
the GPU, except making and closing a plan. Calls are not recorded by autograd:
while it records, tensors that require gradients are refused.
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


_codes = {}


def _type_code(dtype) -> int:
    code = _codes.get(dtype)
    if code is None:
        import torch
        _codes.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
        code = _codes.get(dtype)
        if code is None:
            raise ValueError(f"attention takes bfloat16, float16 or float32 tensors, not {dtype}")
    return code


class _Nothing:
    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_NOTHING = _Nothing()


def _on_device(device, stream):
    """A context with the tensors' device and the call's stream current."""
    import torch
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        return torch.cuda.stream(stream)
    if device.type != "cuda":
        raise ValueError("attention needs tensors on the GPU")
    if torch.cuda.current_device() == device.index:
        return _NOTHING
    return torch.cuda.device(device)


def _raw_stream(device) -> int | None:
    """The device's current stream as the library takes it."""
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index) or None


def _heads(name, t, shape, dtype, device) -> Rows:
    """A [rows, heads, dim] tensor of that shape as the library takes it."""
    st = t.stride()
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} is {tuple(t.shape)}, {t.dtype} on {t.device}, expected "
                         f"{tuple(shape)}, {dtype} on {device}")
    if st[2] != 1 and shape[2] > 1 and t.numel():
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return Rows(t.data_ptr(), st[0], st[1])


def _new(like, shape):
    """A new contiguous tensor of `like`'s shape, type and device (the shorter call if it can be)."""
    import torch
    if like.is_contiguous():
        return torch.empty_like(like)
    return torch.empty(shape, dtype=like.dtype, device=like.device)


def _flat(name, t, shape, dtype, device):
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"{device}")


def _dims(q, k):
    """(heads_q, heads_kv, dim) of a call."""
    a, b = q.shape, k.shape
    if len(a) != 3 or len(b) != 3:
        raise ValueError(f"q has shape {tuple(a)} and k {tuple(b)}, expected (rows, heads, dim)")
    return a[1], b[1], a[2]


def _unrecorded():
    """For tensors that require gradients: autograd does not see the library's
    calls, and a result would be cut off from its inputs."""
    import torch
    if torch.is_grad_enabled():
        raise ValueError("attention calls are not recorded by autograd: call them under "
                         "torch.no_grad(), or from a torch.autograd.Function of forward and "
                         "backward, for tensors that require gradients")


def _scale(scale, dim) -> float:
    return max(dim, 1) ** -0.5 if scale is None else float(scale)


def _workspace(nbytes: int, device):
    """A tensor of that many bytes and its address (the caching allocator's
    memory is 512-byte aligned; the library asks for 256), or None twice."""
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
        self._lib, self._h = lib, None
        self.nrows, self.ncols, self.nnz = mask.nrows, mask.ncols, mask.nnz
        self.device = mask.rowptr.device
        self._sizes = {}  # workspace bytes by what they depend on
        with _on_device(self.device, stream):
            _flat("mask.rowptr", mask.rowptr, (mask.nrows + 1,), torch.int64, self.device)
            _flat("mask.col", mask.col, (mask.nnz,), torch.int32, self.device)
            h = ctypes.c_void_p()
            s = _b.CSRStruct(mask.nrows, mask.ncols, mask.nnz, mask.rowptr.data_ptr(),
                             _b._ptr(mask.col), None)
            _check(lib.spgemm_attention_plan_create(ctypes.byref(h), ctypes.byref(s),
                                                    1 if backward else 0, _raw_stream(self.device)),
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

    def _ready(self, device):
        if self._h is None:
            raise ValueError("the attention plan is closed")
        if device != self.device:
            raise ValueError(f"the plan is on {self.device}, q on {device}")

    def _space(self, desc, backward):
        key = (desc.type, desc.heads_q, desc.heads_kv, desc.head_dim, backward)
        n = self._sizes.get(key)
        if n is None:
            n = ctypes.c_int64(0)
            _check(self._lib.spgemm_attention_workspace(self._h, ctypes.byref(desc), backward,
                                                        ctypes.byref(n)),
                   "spgemm_attention_workspace")
            n = self._sizes[key] = n.value
        return (*_workspace(n, self.device), n)

    def forward(self, q, k, v, scale=None, out=None, lse=None, stream=None):
        """(out, lse) for q [nrows, heads_q, dim] and k, v [ncols, heads_kv, dim].

        out has q's shape and type, lse is [nrows, heads_q] in float32. Either
        may be passed to be written into. scale defaults to dim ** -0.5."""
        import torch
        hq, hkv, dim = _dims(q, k)
        if q.requires_grad or k.requires_grad or v.requires_grad:
            _unrecorded()
        dtype, device = q.dtype, q.device
        self._ready(device)
        big, small, line = (self.nrows, hq, dim), (self.ncols, hkv, dim), (self.nrows, hq)
        ref = ctypes.byref
        desc = Desc(_type_code(dtype), hq, hkv, dim, _scale(scale, dim))
        qs = _heads("q", q, big, dtype, device)
        ks = _heads("k", k, small, dtype, device)
        vs = _heads("v", v, small, dtype, device)
        with _on_device(device, stream):
            if out is None:
                out = _new(q, big)
            if lse is None:
                lse = torch.empty(line, dtype=torch.float32, device=device)
            else:
                _flat("lse", lse, line, torch.float32, device)
            os = _heads("out", out, big, dtype, device)
            space, ws, nbytes = self._space(desc, 0)
            _check(self._lib.spgemm_attention_forward(
                self._h, ref(desc), ref(qs), ref(ks), ref(vs), ref(os), lse.data_ptr() or None, ws,
                nbytes, _raw_stream(device)), "spgemm_attention_forward")
        return out, lse

    def backward(self, dout, q, k, v, out, lse, scale=None, dq=None, dk=None, dv=None,
                 stream=None):
        """(dq, dk, dv), given dout and what ``forward`` returned. Gradients
        have their tensors' shapes and type, and are written, not added to."""
        import torch
        hq, hkv, dim = _dims(q, k)
        if (q.requires_grad or k.requires_grad or v.requires_grad or dout.requires_grad
                or out.requires_grad):
            _unrecorded()
        dtype, device = q.dtype, q.device
        self._ready(device)
        big, small = (self.nrows, hq, dim), (self.ncols, hkv, dim)
        ref = ctypes.byref
        desc = Desc(_type_code(dtype), hq, hkv, dim, _scale(scale, dim))
        _flat("lse", lse, (self.nrows, hq), torch.float32, device)
        qs = _heads("q", q, big, dtype, device)
        ks = _heads("k", k, small, dtype, device)
        vs = _heads("v", v, small, dtype, device)
        os = _heads("out", out, big, dtype, device)
        gs = _heads("dout", dout, big, dtype, device)
        with _on_device(device, stream):
            if dq is None:
                dq = _new(q, big)
            if dk is None:
                dk = _new(k, small)
            if dv is None:
                dv = _new(v, small)
            dqs = _heads("dq", dq, big, dtype, device)
            dks = _heads("dk", dk, small, dtype, device)
            dvs = _heads("dv", dv, small, dtype, device)
            space, ws, nbytes = self._space(desc, 1)
            _check(self._lib.spgemm_attention_backward(
                self._h, ref(desc), ref(qs), ref(ks), ref(vs), ref(os), lse.data_ptr() or None,
                ref(gs), ref(dqs), ref(dks), ref(dvs), ws, nbytes, _raw_stream(device)),
                "spgemm_attention_backward")
        return dq, dk, dv


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
    if q.requires_grad or k_cache.requires_grad or v_cache.requires_grad:
        _unrecorded()
    tokens, hq, dim = q.shape
    npages, slots, hkv, _ = k_cache.shape
    dtype, device, seqs = q.dtype, q.device, pages.nrows
    ks, vs = k_cache.stride(), v_cache.stride()
    for name, t, st in (("k_cache", k_cache, ks), ("v_cache", v_cache, vs)):
        if t.dtype != dtype or t.device != device:
            raise ValueError(f"{name} is {t.dtype} on {t.device}, expected {dtype} on {device}")
        if st[3] != 1 and dim > 1 and t.numel():
            raise ValueError(f"{name}'s last dimension must be contiguous")
    if pages.ncols != npages:
        raise ValueError(f"the page table names pages of a cache of {pages.ncols}, it has {npages}")
    desc = Desc(_type_code(dtype), hq, hkv, dim, _scale(scale, dim))
    ref = ctypes.byref
    with _on_device(device, stream):
        nnz = pages.nnz
        _flat("pages.rowptr", pages.rowptr, (seqs + 1,), torch.int64, device)
        _flat("pages.col", pages.col, (nnz,), torch.int32, device)
        _flat("q_rowptr", q_rowptr, (seqs + 1,), torch.int64, device)
        _flat("lengths", lengths, (seqs,), torch.int64, device)
        if out is None:
            out = _new(q, q.shape)
        if lse is None:
            lse = torch.empty((tokens, hq), dtype=torch.float32, device=device)
        else:
            _flat("lse", lse, (tokens, hq), torch.float32, device)
        qs = _heads("q", q, q.shape, dtype, device)
        os = _heads("out", out, q.shape, dtype, device)
        table = _b.CSRStruct(seqs, npages, nnz, pages.rowptr.data_ptr(),
                             pages.col.data_ptr() or None, None)
        cache = PagedCache(k_cache.data_ptr() or None, v_cache.data_ptr() or None, npages, slots,
                           ks[0], ks[1], ks[2], vs[0], vs[1], vs[2])
        batch = PagedBatch(ctypes.pointer(table), q_rowptr.data_ptr(), lengths.data_ptr() or None,
                           tokens, max_q, max_len)
        n = ctypes.c_int64(0)
        _check(lib.spgemm_paged_attention_workspace(ref(desc), ref(batch), ref(n)),
               "spgemm_paged_attention_workspace")
        space, ws = _workspace(n.value, device)
        _check(lib.spgemm_paged_attention(
            ref(desc), ref(qs), ref(cache), ref(batch), ref(os), lse.data_ptr() or None, ws,
            n.value, _raw_stream(device)), "spgemm_paged_attention")
    return out, lse
