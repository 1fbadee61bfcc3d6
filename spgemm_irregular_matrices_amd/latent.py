"""Thin ctypes binding of ``include/spgemm_cache.h``'s latent attention: attention
over a paged cache of one latent vector a token, which all heads share.

Argument marshalling only, as in ``attention``, whose conventions hold here:
one device and stream to a call, outputs and workspaces are torch tensors,
nothing waits for the GPU, and nothing is recorded by autograd.
"""
from __future__ import annotations

import ctypes

from . import attention as _a
from .attention import (_check, _flat, _forward_mode, _given_requires, _heads, _on_device,
                        _raw_stream, _unrecorded)
from .binding import DeviceCSR, SpgemmError  # noqa: F401  (SpgemmError: what calls raise)
from .cache import _batch

EXPORTS = ["spgemm_latent_attention_workspace", "spgemm_latent_attention",
           "spgemm_latent_expanded_workspace", "spgemm_latent_expanded"]


class LatentDesc(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("heads", ctypes.c_int32), ("latent_dim", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("key_dim", ctypes.c_int32),
                ("value_dim", ctypes.c_int32), ("scale", ctypes.c_double)]


class LatentCache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("npages", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("stride_page", ctypes.c_int64), ("stride_slot", ctypes.c_int64)]


_lib = None


def load():
    """The built library with these entry points declared (raises if it is missing)."""
    global _lib
    if _lib is None:
        lib = _a.load()
        P, L = ctypes.c_void_p, ctypes.c_int64
        D, R = ctypes.POINTER(LatentDesc), ctypes.POINTER(_a.Rows)
        B, C, LP = ctypes.POINTER(_a.PagedBatch), ctypes.POINTER(LatentCache), ctypes.POINTER(L)
        sigs = {
            "spgemm_latent_attention_workspace": [D, B, LP],
            "spgemm_latent_attention": [D, R, C, B, R, P, P, L, P],
            "spgemm_latent_expanded_workspace": [D, C, B, LP],
            "spgemm_latent_expanded": [D, R, R, R, C, B, R, P, P, L, P],
        }
        for name, args in sigs.items():
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
    return _lib


def _type_code(dtype) -> int:
    code = _a._type_code(dtype)
    if code == 2:
        raise ValueError("latent attention takes bfloat16 or float16 tensors, not float32")
    return code


def _cache_of(cache, dtype, device) -> LatentCache:
    if cache.dtype != dtype or cache.device != device:
        raise ValueError(f"cache is {cache.dtype} on {cache.device}, expected {dtype} on {device}")
    st = cache.stride()
    if st[2] != 1 and cache.shape[2] > 1 and cache.numel():
        raise ValueError("cache's last dimension must be contiguous")
    return LatentCache(cache.data_ptr() or None, cache.shape[0], cache.shape[1], st[0], st[1])


def _outputs(q, shape, out, lse):
    import torch
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty(shape[:2], dtype=torch.float32, device=q.device)
    else:
        _flat("lse", lse, shape[:2], torch.float32, q.device)
    return out, lse, _heads("out", out, shape, q.dtype, q.device)


def latent_attention(q, cache, pages: DeviceCSR, q_rowptr, lengths, max_q: int, max_len: int,
                     value_dim: int, scale: float, out=None, lse=None, stream=None):
    """(out, lse) of new tokens over a paged cache of latent vectors, in their
    space (the absorbed form: for few new tokens, single ones above all).

    q: [tokens, heads, dim]; cache: [pages, slots, dim], of which the first
    ``value_dim`` values of a token are its value and all of them its key, for
    every head. out is [tokens, heads, value_dim]. A model multiplies its key
    weights into q and its value weights into out; ``scale`` is that of the
    heads' own scores, so it has no default. The index arguments are
    ``paged_attention``'s, and so is what a broken batch gets."""
    lib = load()
    if q.dim() != 3 or cache.dim() != 3 or cache.shape[2] != q.shape[2]:
        raise ValueError(f"q {tuple(q.shape)} and cache {tuple(cache.shape)} do not fit: expected "
                         "(tokens, heads, dim) and (pages, slots, dim)")
    if q.requires_grad or cache.requires_grad or _given_requires(out, lse) or _forward_mode():
        _unrecorded(q, cache, out, lse)
    tokens, heads, dim = q.shape
    if not 0 < value_dim <= dim:
        raise ValueError(f"value_dim is {value_dim}, the cache's rows have {dim} values")
    dtype, device = q.dtype, q.device
    desc = LatentDesc(_type_code(dtype), heads, value_dim, dim - value_dim, 0, 0, float(scale))
    cs = _cache_of(cache, dtype, device)
    ref = ctypes.byref
    with _on_device(device, stream):
        out, lse, os = _outputs(q, (tokens, heads, value_dim), out, lse)
        qs = _heads("q", q, q.shape, dtype, device)
        batch = _batch(pages, cache.shape[0], q_rowptr, lengths, tokens, max_q, max_len, device)
        n = ctypes.c_int64(0)
        _check(lib.spgemm_latent_attention_workspace(ref(desc), ref(batch), ref(n)),
               "spgemm_latent_attention_workspace")
        space, ws = _a._workspace(n.value, device)
        _check(lib.spgemm_latent_attention(ref(desc), ref(qs), ref(cs), ref(batch), ref(os),
                                           lse.data_ptr() or None, ws, n.value, _raw_stream(device)),
               "spgemm_latent_attention")
    return out, lse


def latent_attention_expanded(q, cache, w_k, w_v, pages: DeviceCSR, q_rowptr, lengths, max_q: int,
                              max_len: int, scale=None, out=None, lse=None, stream=None):
    """(out, lse) of new tokens over a paged cache of latent vectors, with every
    head's keys and values made from them (the expanded form: for chunks of many
    new tokens).

    w_k: [heads, key_dim, latent_dim] and w_v: [heads, value_dim, latent_dim]
    make a head's key and value from the first latent_dim values of a token's
    row of cache [pages, slots, latent_dim + rope_dim]; the others end every
    head's key as they are. q is [tokens, heads, key_dim + rope_dim], out
    [tokens, heads, value_dim]; scale defaults to (key_dim + rope_dim) ** -0.5.
    The index arguments are ``paged_attention``'s, and so is what a broken
    batch gets. The keys and values are made in a workspace, 4 (key_dim +
    value_dim) bytes for a cached token and head: calls for groups of heads, on
    slices of q, w_k, w_v and out, need a part of it at a time."""
    lib = load()
    if q.dim() != 3 or cache.dim() != 3 or w_k.dim() != 3 or w_v.dim() != 3:
        raise ValueError(f"q {tuple(q.shape)}, cache {tuple(cache.shape)}, w_k {tuple(w_k.shape)} and "
                         f"w_v {tuple(w_v.shape)} must have three dimensions each")
    tokens, heads, dim = q.shape
    key_dim, latent_dim = w_k.shape[1:]
    value_dim, rope_dim = w_v.shape[1], cache.shape[2] - latent_dim
    if w_k.shape[0] != heads or w_v.shape != (heads, value_dim, latent_dim) or \
            dim != key_dim + rope_dim or rope_dim < 0:
        raise ValueError(f"q {tuple(q.shape)}, cache {tuple(cache.shape)}, w_k {tuple(w_k.shape)} and "
                         f"w_v {tuple(w_v.shape)} do not fit: expected (tokens, heads, key_dim + "
                         "rope_dim), (pages, slots, latent_dim + rope_dim), (heads, key_dim, "
                         "latent_dim) and (heads, value_dim, latent_dim)")
    if (q.requires_grad or cache.requires_grad or w_k.requires_grad or w_v.requires_grad
            or _given_requires(out, lse) or _forward_mode()):
        _unrecorded(q, cache, w_k, w_v, out, lse)
    dtype, device = q.dtype, q.device
    desc = LatentDesc(_type_code(dtype), heads, latent_dim, rope_dim, key_dim, value_dim,
                      _a._scale(scale, dim))
    cs = _cache_of(cache, dtype, device)
    ks, vs = _heads("w_k", w_k, w_k.shape, dtype, device), _heads("w_v", w_v, w_v.shape, dtype, device)
    ref = ctypes.byref
    with _on_device(device, stream):
        out, lse, os = _outputs(q, (tokens, heads, value_dim), out, lse)
        qs = _heads("q", q, q.shape, dtype, device)
        batch = _batch(pages, cache.shape[0], q_rowptr, lengths, tokens, max_q, max_len, device)
        n = ctypes.c_int64(0)
        _check(lib.spgemm_latent_expanded_workspace(ref(desc), ref(cs), ref(batch), ref(n)),
               "spgemm_latent_expanded_workspace")
        space, ws = _a._workspace(n.value, device)
        _check(lib.spgemm_latent_expanded(ref(desc), ref(qs), ref(ks), ref(vs), ref(cs), ref(batch),
                                          ref(os), lse.data_ptr() or None, ws, n.value,
                                          _raw_stream(device)), "spgemm_latent_expanded")
    return out, lse
