"""Thin ctypes binding of ``include/spgemm_cache.h``'s quantised caches: a paged
key/value cache in 8 or 4 bits a value, written, read back and attended to.

Argument marshalling only, as in ``attention``, whose conventions hold here:
one device and stream to a call, outputs and workspaces are torch tensors,
nothing waits for the GPU, and nothing is recorded by autograd.
"""
from __future__ import annotations

import ctypes

from . import attention as _a
from . import binding as _b
from .attention import (_check, _flat, _forward_mode, _given_requires, _heads, _new, _on_device,
                        _raw_stream, _type_code, _unrecorded)
from .binding import DeviceCSR, SpgemmError  # noqa: F401  (SpgemmError: what calls raise)

EXPORTS = ["spgemm_mx_write", "spgemm_mx_read", "spgemm_mx_attention_workspace",
           "spgemm_mx_attention"]
BLOCK = 32  # values that share a scale
FORMATS = {"e4m3": (0, 8), "e2m1": (1, 4)}  # code of the format, bits per value


class MxBytes(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_page", ctypes.c_int64),
                ("stride_slot", ctypes.c_int64), ("stride_head", ctypes.c_int64)]


class MxCache(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("reserved", ctypes.c_int32), ("npages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("k_codes", MxBytes), ("k_scales", MxBytes),
                ("v_codes", MxBytes), ("v_scales", MxBytes)]


_lib = None


def load():
    """The built library with these entry points declared (raises if it is missing)."""
    global _lib
    if _lib is None:
        lib = _a.load()
        P, L = ctypes.c_void_p, ctypes.c_int64
        D, R = ctypes.POINTER(_a.Desc), ctypes.POINTER(_a.Rows)
        B, C = ctypes.POINTER(_a.PagedBatch), ctypes.POINTER(MxCache)
        sigs = {
            "spgemm_mx_write": [D, R, R, C, B, P],
            "spgemm_mx_read": [D, C, B, R, R, P],
            "spgemm_mx_attention_workspace": [D, B, ctypes.POINTER(L)],
            "spgemm_mx_attention": [D, R, C, B, R, P, P, L, P],
        }
        for name, args in sigs.items():
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
    return _lib


def _batch(pages, npages, q_rowptr, lengths, tokens, max_q, max_len, device):
    """The library's batch, and what it points into."""
    import torch
    if pages.ncols != npages:
        raise ValueError(f"the page table names pages of a cache of {pages.ncols}, it has {npages}")
    seqs, nnz = pages.nrows, pages.nnz
    _flat("pages.rowptr", pages.rowptr, (seqs + 1,), torch.int64, device)
    _flat("pages.col", pages.col, (nnz,), torch.int32, device)
    _flat("q_rowptr", q_rowptr, (seqs + 1,), torch.int64, device)
    _flat("lengths", lengths, (seqs,), torch.int64, device)
    table = _b.CSRStruct(seqs, npages, nnz, pages.rowptr.data_ptr(), pages.col.data_ptr() or None,
                         None)
    return _a.PagedBatch(ctypes.pointer(table), q_rowptr.data_ptr(), lengths.data_ptr() or None,
                         tokens, max_q, max_len)


class QuantizedCache:
    """A paged key/value cache of [pages, slots, heads_kv, dim] values in 8
    (``"e4m3"``) or 4 (``"e2m1"``) bits each, with a power of two as scale for
    every 32 values: codes [pages, slots, heads_kv, dim] or [..., dim / 2] and
    scales [..., dim / 32], uint8 (what they stand for: see
    ``include/spgemm_cache.h``). The tensors may be views with any strides whose
    last dimension is contiguous; they are used as they are, not copied (where
    places overlap, of one as in expanded views or of two, they are read but not written). Where they
    lie is looked up in every call: their memory may be given back and taken
    again between calls, and another tensor of the same shape may be put in place
    of one (``k_codes``, ``k_scales``, ``v_codes``, ``v_scales``).

    The index tensors of a call are ``paged_attention``'s: row s of the CSR
    matrix ``pages`` lists sequence s's pages, rows [q_rowptr[s],
    q_rowptr[s + 1]) belong to its last tokens, ``lengths`` counts its tokens,
    these included; ``max_q`` and ``max_len`` bound them. They are read on the
    GPU, so that a captured call follows their later values.
    """

    def __init__(self, k_codes, k_scales, v_codes, v_scales, format: str = "e4m3"):
        import torch
        if format not in FORMATS:
            raise ValueError(f"format is {format!r}, expected one of {tuple(FORMATS)}")
        bits = FORMATS[format][1]
        if k_codes.dim() != 4:
            raise ValueError(f"k_codes has shape {tuple(k_codes.shape)}, expected (pages, slots, kv "
                             "heads, bytes)")
        npages, slots, heads, width = k_codes.shape
        dim = width * 8 // bits
        if dim % BLOCK or dim == 0:
            raise ValueError(f"the cache holds {dim} values a head, expected a multiple of {BLOCK}")
        self.format, self.device, self.dim = format, k_codes.device, dim
        self.npages, self.slots, self.heads = npages, slots, heads
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self._last = None
        self._descs = {}  # of rows, by their type
        self._space = None, 0  # the last call's sizes and the workspace that they ask for
        self._described()

    def __getstate__(self):
        return {**self.__dict__, "_last": None, "_descs": {}}  # (addresses are not a copy's)

    def _described(self) -> MxCache:
        """The cache as the library takes it, from its tensors as they are now. (Where they
        are those of the last call, at the same places, so is the description: 1.5 us
        instead of 6.)"""
        import torch
        kc, ks, vc, vs = self.k_codes, self.k_scales, self.v_codes, self.v_scales
        at = (kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), kc.stride(), ks.stride(),
              vc.stride(), vs.stride())
        if self._last is not None:
            known, a, b, c, d, struct = self._last
            if at == known and a is kc and b is ks and c is vc and d is vs:
                return struct
        code, bits = FORMATS[self.format]
        places = (self.npages, self.slots, self.heads)
        codes, scales = (*places, self.dim * bits // 8), (*places, self.dim // BLOCK)
        parts = []
        for name, t, shape in (("k_codes", kc, codes), ("k_scales", ks, scales),
                               ("v_codes", vc, codes), ("v_scales", vs, scales)):
            if t.shape != shape or t.dtype != torch.uint8 or t.device != self.device:
                raise ValueError(f"{name} is {tuple(t.shape)}, {t.dtype} on {t.device}, expected "
                                 f"{shape}, torch.uint8 on {self.device}")
            st = t.stride()
            if st[3] != 1 and shape[3] > 1 and t.numel():
                raise ValueError(f"{name}'s last dimension must be contiguous")
            if t.numel() and not t.untyped_storage().data_ptr():  # (a view's own is its offset)
                raise ValueError(f"{name}'s memory was given back")
            parts.append(MxBytes(t.data_ptr() or None, st[0], st[1], st[2]))
        struct = MxCache(code, 0, self.npages, self.slots, *parts)
        self._last = at, kc, ks, vc, vs, struct
        return struct

    @classmethod
    def empty(cls, npages: int, slots: int, heads_kv: int, dim: int, format: str = "e4m3",
              device="cuda"):
        """A cache whose values are not set yet, one page after another."""
        import torch
        if format not in FORMATS:
            raise ValueError(f"format is {format!r}, expected one of {tuple(FORMATS)}")
        if dim % BLOCK:
            raise ValueError(f"a quantised cache holds {dim} values a head, expected a multiple of {BLOCK}")
        widths = (dim * FORMATS[format][1] // 8, dim // BLOCK) * 2
        return cls(*(torch.empty(npages, slots, heads_kv, w, dtype=torch.uint8, device=device)
                     for w in widths), format)

    def _rows(self, k, v, what):
        if k.dim() != 3 or k.shape[1:] != (self.heads, self.dim):
            raise ValueError(f"{what} has shape {tuple(k.shape)}, expected (tokens, {self.heads}, "
                             f"{self.dim})")
        dtype = k.dtype
        desc = self._descs.get(dtype)
        if desc is None:
            desc = self._descs[dtype] = _a.Desc(_type_code(dtype), self.heads, self.heads, self.dim, 0.0)
        return desc, _heads("k", k, k.shape, dtype, self.device), _heads("v", v, k.shape, dtype,
                                                                         self.device)

    def write(self, k, v, pages: DeviceCSR, q_rowptr, lengths, max_q: int, max_len: int, stream=None):
        """Quantise the new tokens' k and v [tokens, heads_kv, dim] into their
        places, which end their sequences. Every value is rounded once, to the
        nearest code; a block of 32 with an infinity or a NaN becomes NaN.
        Nothing of a sequence that breaks the rules is written."""
        lib = load()
        if k.requires_grad or v.requires_grad or _forward_mode():
            _unrecorded(k, v)
        desc, ks, vs = self._rows(k, v, "k")
        ref = ctypes.byref
        with _on_device(self.device, stream):
            batch = _batch(pages, self.npages, q_rowptr, lengths, k.shape[0], max_q, max_len,
                           self.device)
            _check(lib.spgemm_mx_write(ref(desc), ref(ks), ref(vs), ref(self._described()), ref(batch),
                                       _raw_stream(self.device)), "spgemm_mx_write")

    def read(self, pages: DeviceCSR, q_rowptr, lengths, max_q: int, max_len: int, tokens: int = None,
             dtype=None, k=None, v=None, stream=None):
        """(k, v) [tokens, heads_kv, dim]: the values of the last q_rowptr[s + 1]
        - q_rowptr[s] tokens of every sequence (whole texts if that is lengths),
        as bfloat16 unless another dtype, or k and v to be written into, say
        otherwise. Rows of no sequence are not written, those of a sequence
        that breaks the rules become NaN."""
        import torch
        lib = load()
        if _given_requires(k, v) or _forward_mode():
            _unrecorded(k, v)
        with _on_device(self.device, stream):
            given = k if k is not None else v
            if given is not None:
                if tokens not in (None, given.shape[0]) or dtype not in (None, given.dtype):
                    raise ValueError("tokens and dtype are those of k and v where they are given")
                tokens, dtype = given.shape[0], given.dtype
            elif tokens is None:
                raise ValueError("read needs the number of tokens, or k and v to write into")
            shape, dtype = (tokens, self.heads, self.dim), dtype or torch.bfloat16
            if k is None:
                k = torch.empty(shape, dtype=dtype, device=self.device)
            if v is None:
                v = torch.empty(shape, dtype=dtype, device=self.device)
            desc, ks, vs = self._rows(k, v, "k")
            batch = _batch(pages, self.npages, q_rowptr, lengths, tokens, max_q, max_len, self.device)
            ref = ctypes.byref
            _check(lib.spgemm_mx_read(ref(desc), ref(self._described()), ref(batch), ref(ks), ref(vs),
                                      _raw_stream(self.device)), "spgemm_mx_read")
        return k, v

    def attention(self, q, pages: DeviceCSR, q_rowptr, lengths, max_q: int, max_len: int, scale=None,
                  out=None, lse=None, stream=None):
        """(out, lse) of new tokens over their sequences, as ``paged_attention``
        with the cache's values for keys and values: q is [tokens, heads_q, dim]
        in bfloat16, float16 or float32."""
        import torch
        lib = load()
        if q.dim() != 3 or q.shape[2] != self.dim:
            raise ValueError(f"q has shape {tuple(q.shape)}, expected (tokens, heads, {self.dim})")
        if q.requires_grad or _given_requires(out, lse) or _forward_mode():
            _unrecorded(q, out, lse)
        tokens, hq, dim = q.shape
        dtype, device = q.dtype, self.device
        desc = _a.Desc(_type_code(dtype), hq, self.heads, dim, _a._scale(scale, dim))
        ref = ctypes.byref
        with _on_device(device, stream):
            if out is None:
                out = _new(q, q.shape)
            if lse is None:
                lse = torch.empty((tokens, hq), dtype=torch.float32, device=device)
            else:
                _flat("lse", lse, (tokens, hq), torch.float32, device)
            qs = _heads("q", q, q.shape, dtype, device)
            os = _heads("out", out, q.shape, dtype, device)
            batch = _batch(pages, self.npages, q_rowptr, lengths, tokens, max_q, max_len, device)
            sizes = dtype, hq, pages.nrows, tokens, max_q, max_len
            known, n = self._space
            if sizes != known:
                size = ctypes.c_int64(0)
                _check(lib.spgemm_mx_attention_workspace(ref(desc), ref(batch), ref(size)),
                       "spgemm_mx_attention_workspace")
                n = size.value
                self._space = sizes, n
            space, ws = _a._workspace(n, device)
            _check(lib.spgemm_mx_attention(
                ref(desc), ref(qs), ref(self._described()), ref(batch), ref(os), lse.data_ptr() or None,
                ws, n, _raw_stream(device)), "spgemm_mx_attention")
        return out, lse
